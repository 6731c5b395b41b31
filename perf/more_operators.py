"""The layer in 8 bits, as measured cases: the root-mean-square norm with the
residual's sum and an output in 8 bits, the experts' products in 8-bit floating
point, and the layer's step with its activation checkpoints in 8 bits.

Each case is one call (or one forward with its backward) as a training or
serving program makes it.  With ``own`` false the operators are computed in
their plain form from elementary torch operations; with ``own`` true by the
framework's entry points.
"""
import math

import torch

own = False

BF16, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
DT = {"bf16": BF16, "f32": F32}
EPS = 1e-5
BLOCK = 128   # columns (and rows, of weights) that share a scale
TOP8 = 448.0  # largest e4m3 value


# --------------------------------------------------------------------- cases

def listed():
    return [
        # norm + residual sum of a decode batch, with the 8-bit rows that the experts read: launch latency counts
        dict(name="rms_fwd_decode", op="rms_fwd", L=4, d=4096, dtype="bf16", residual=True, out8=True),
        # the same of a long prompt of the large-expert layer's width
        dict(name="rms_fwd_prompt", op="rms_fwd", L=32768, d=4096, dtype="bf16", residual=True, out8=True),
        # the norm's backward in training, with the gradient that arrives over the residual stream
        dict(name="rms_bwd_train", op="rms_bwd", L=32768, d=4096, dtype="bf16", residual=True),
        # an odd width in fp32: no row but every fourth starts on 16 bytes
        dict(name="rms_bwd_odd", op="rms_bwd", L=8191, d=1409, dtype="f32", residual=False),
        # 8-bit experts: one token of a decode loop, and a decode batch
        dict(name="fp8_token", op="fp8", L=1, d=4096, h=14336, E=8, K=2, act="swiglu", rows8=True, idle=False),
        dict(name="fp8_batch16", op="fp8", L=16, d=4096, h=14336, E=8, K=2, act="swiglu", rows8=True, idle=False),
        # a decode batch over fine-grained experts, some of its slots without a sequence, rows still in bf16
        dict(name="fp8_fine61", op="fp8", L=61, d=2048, h=1408, E=64, K=6, act="swiglu", rows8=False, idle=True),
        # prompts: the large-expert layer and the fine-grained one
        dict(name="fp8_prompt", op="fp8", L=8192, d=4096, h=14336, E=8, K=2, act="swiglu", rows8=True, idle=False),
        dict(name="fp8_prompt_fine", op="fp8", L=16000, d=2048, h=1408, E=64, K=6, act="swiglu", rows8=False, idle=False),
        # a training step with 8-bit checkpoints: the small SiLU layer, the fine-grained one, the large-expert one
        dict(name="ckpt8_silu", op="ckpt8", L=1500, d=1024, h=4096, E=8, K=2, act="silu"),
        dict(name="ckpt8_fine", op="ckpt8", L=16384, d=2048, h=1408, E=64, K=6, act="swiglu"),
        dict(name="ckpt8_large", op="ckpt8", L=7000, d=4096, h=14336, E=8, K=2, act="swiglu"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _flops(case):
    mats = 3 if case["act"] == "swiglu" else 2
    return (6.0 if case["op"] == "ckpt8" else 2.0) * mats * case["L"] * case["K"] * case["d"] * case["h"]


def _expert_sizes(rng):
    E = _log_int(rng, 2, 64)
    d = 128 * _log_int(rng, 1, 32)
    h = 128 * _log_int(rng, 1, 112)
    while E * d * h > 8 * 4096 * 14336:
        h = 128 * max(1, h // 256)
    return dict(d=d, h=h, E=E, K=rng.randint(1, min(8, E)), act=rng.choice(["swiglu", "swiglu", "silu"]))


def draw(rng):
    op = rng.choice(["rms_fwd", "rms_bwd", "fp8", "fp8", "ckpt8"])
    if op in ("rms_fwd", "rms_bwd"):
        d = _log_int(rng, 64, 8192)
        out8 = op == "rms_fwd" and rng.random() < 0.6
        if out8:
            d = (d + 15) // 16 * 16
        elif rng.random() < 0.4:
            d = (d + 63) // 64 * 64
        L = _log_int(rng, 1, min(65536, 32768 * 4096 // d))
        dtype = rng.choice(["bf16", "bf16", "f32"])
        if dtype == "f32":
            L = max(1, L // 2)
        case = dict(op=op, L=L, d=d, dtype=dtype, residual=rng.random() < 0.6)
        return dict(case, out8=out8) if op == "rms_fwd" else case
    case = dict(_expert_sizes(rng), op=op, L=_log_int(rng, 1, 16384))
    if op == "fp8":
        case.update(rows8=rng.random() < 0.5, idle=rng.random() < 0.3)
        limit = _flops(dict(op="fp8", L=8192, d=4096, h=14336, K=2, act="swiglu"))
    else:
        limit = _flops(dict(op="ckpt8", L=7000, d=4096, h=14336, K=2, act="swiglu"))
    while case["L"] > 1 and (_flops(case) > limit or case["L"] * case["K"] > 131072):
        case["L"] = case["L"] * 2 // 3
    return case


# --------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *size):
    return torch.randn(*size, device="cuda", generator=g)


def _stream_rows(L, d, dtype, g):
    """Rows of a residual stream: unit spread, an offset per column and a few
    columns ten times as large."""
    big = 1.0 + 9.0 * (torch.rand(d, device="cuda", generator=g) < 0.004)
    return (_randn(g, L, d) * big + 0.3 * _randn(g, d)).to(dtype)


def _routing(L, E, K, g):
    """Top-K ids and gates of a router with unequal experts."""
    top = torch.topk(_randn(g, L, E) + _randn(g, E), K, dim=1)
    return top.indices.to(torch.int32).contiguous(), torch.softmax(top.values, dim=1).contiguous()


def _weights8(E, N, R, g):
    """e4m3 weights (E,N,R) and fp32 scales per 128 x 128 of a matrix of variance about 1/R."""
    q = torch.empty(E, N, R, dtype=F8, device="cuda")
    for e in range(E):
        q[e] = (100.0 * _randn(g, N, R)).clamp_(-TOP8, TOP8).to(F8)
    u = torch.rand(E, N // BLOCK, R // BLOCK, device="cuda", generator=g)
    return q, (0.5 + u) / (100.0 * math.sqrt(R))


def prepare(case, seed):
    g = _gen(seed)
    op, L, d = case["op"], case["L"], case["d"]
    st = dict(case)
    if op in ("rms_fwd", "rms_bwd"):
        dt = DT[case["dtype"]]
        st["x"] = _stream_rows(L, d, dt, g)
        st["w"] = 1.0 + 0.1 * _randn(g, d)
        if op == "rms_fwd":
            st["r"] = _randn(g, L, d).to(dt) if case["residual"] else None
        else:
            # what the forward left: the sum that was normed (here x) and its statistic
            st["rstd"] = torch.rsqrt(st["x"].float().square().mean(dim=1) + EPS)
            st["dy"] = _randn(g, L, d).to(dt)
            st["ds"] = _randn(g, L, d).to(dt) if case["residual"] else None
        if own:
            from mixture_experts_atomic_gb300.block import RMSNorm
            st["norm"] = RMSNorm(L, d, dt, eps=EPS, device="cuda")
        return st
    h, E, K, act = (case[k] for k in ("h", "E", "K", "act"))
    st["ids"], st["gates"] = _routing(L, E, K, g)
    if op == "fp8":
        st["x"] = _stream_rows(L, d, BF16, g)
        if case["rows8"]:  # what the norm leaves
            st["x"], st["sx"] = _rows8(st["x"].float())
        if case["idle"]:
            # slots of a decode batch that hold no sequence: id -1 in all K
            st["ids"][torch.rand(L, device="cuda", generator=g) < 0.2] = -1
        st["q1"], st["s1"] = _weights8(E, h, d, g)
        st["q2"], st["s2"] = _weights8(E, h, d, g) if act == "swiglu" else (None, None)
        st["q3"], st["s3"] = _weights8(E, d, h, g)
        if own:
            from mixture_experts_atomic_gb300.fp8 import Fp8Experts
            st["experts"] = Fp8Experts(L, d, h, E, K, act=act, device="cuda")
            st["experts"].load(*(st[n + i] for i in "123" for n in "qs"))
        return st
    st["x"] = _randn(g, L, d).to(BF16)
    st["dY"] = _randn(g, L, d).to(BF16)
    for n, rows, cols in (("W1", d, h), ("W2", d, h), ("W3", h, d)):
        if n == "W2" and act != "swiglu":
            st[n] = None
            continue
        st[n] = torch.empty(E, rows, cols, dtype=BF16, device="cuda")
        for e in range(E):
            st[n][e] = (_randn(g, rows, cols) / math.sqrt(rows)).to(BF16)
    if own:
        from mixture_experts_atomic_gb300.layer import MoELayer
        st["layer"] = MoELayer(L, d, h, E, K, BF16, act, "cuda", with_dgates=False, checkpoint8=True)
    return st


# --------------------------------------------------------------------- one pass

def _blocks(v):
    """The row blocks of v (..., C) as (..., ceil(C / 128), 128), zeros behind the last column."""
    c = v.shape[-1]
    n = (c + BLOCK - 1) // BLOCK
    if n * BLOCK != c:
        v = torch.nn.functional.pad(v, (0, n * BLOCK - c))
    return v.view(*v.shape[:-1], n, BLOCK)


def _rows8(v):
    """e4m3 rows and the scale (a power of two) of each of their blocks of 128 columns."""
    b = _blocks(v)
    m, e = torch.frexp(b.abs().amax(dim=-1))
    s = ((e - 9 + (m > 0.875).int()).clamp(min=-126) + 127 << 23).view(F32)
    q = (b / s[..., None]).reshape(*v.shape[:-1], -1)[..., :v.shape[-1]]
    return q.to(F8).contiguous(), s.contiguous()


def _values8(q, s):
    """What e4m3 rows with their blocks' scales stand for, in 32 bits."""
    return (_blocks(q.float()) * s[..., None]).reshape(*q.shape[:-1], -1)[..., :q.shape[-1]]


def _matrix8(q, s):
    """What an e4m3 matrix (N,R) with scales per 128 x 128 stands for, in 32 bits."""
    N, R = q.shape
    return (q.float().view(N // BLOCK, BLOCK, R // BLOCK, BLOCK) * s[:, None, :, None]).view(N, R)


def _int8(v):
    """What int8 codes of v's row blocks of 128 columns stand for."""
    b = _blocks(v)
    s = b.abs().amax(dim=-1, keepdim=True) / 127.0
    q = torch.round(b / torch.where(s > 0, s, torch.ones_like(s))).clamp(-127, 127)
    return (q * s).reshape(v.shape)


def _rms_fwd(st):
    x, w, r = st["x"], st["w"], st["r"]
    if own:
        if st["out8"]:
            q, qs, y, s, rstd = st["norm"].forward8(x, w, r)
            from mixture_experts_atomic_gb300.fp8 import dequantize_rows
            out = {"y": y, "rstd": rstd, "y8": dequantize_rows(q, qs)}
        else:
            y, s, rstd = st["norm"].forward(x, w, r)
            out = {"y": y, "rstd": rstd}
    else:
        dt = x.dtype
        s32 = x.float() if r is None else x.float() + r.float()
        rstd = torch.rsqrt(s32.square().mean(dim=1) + EPS)
        y32 = s32 * rstd[:, None] * w
        y, s = y32.to(dt), s32.to(dt)
        out = {"y": y, "rstd": rstd}
        if st["out8"]:
            out["y8"] = _values8(*_rows8(y32)).to(BF16)  # four bits of mantissa: exact
    if r is not None:
        out["s"] = s
    return out


def _rms_bwd(st):
    if own:
        dx, dw = st["norm"].backward(st["dy"], st["x"], st["rstd"], st["w"], st["ds"])
    else:
        dy = st["dy"].float()
        xh = st["x"].float() * st["rstd"][:, None]
        gw = dy * st["w"]
        dx = (gw - xh * (gw * xh).mean(dim=1, keepdim=True)) * st["rstd"][:, None]
        if st["ds"] is not None:
            dx = dx + st["ds"].float()
        dx = dx.to(st["x"].dtype)
        dw = (dy * xh).sum(dim=0)
    return {"dx": dx, "dw": dw}


def _fp8(st):
    if own:
        return {"y": st["experts"].forward(st["x"], st["ids"], st["gates"], st.get("sx"))}
    L, d, E = st["L"], st["d"], st["E"]
    x = _values8(st["x"], st["sx"]) if st["rows8"] else _values8(*_rows8(st["x"].float()))
    # a row for every slot, added up slot by slot
    rows = torch.zeros(L, st["K"], d, device=x.device)
    for e in range(E):
        t, k = torch.nonzero(st["ids"] == e, as_tuple=True)
        if t.numel() == 0:
            continue
        xe = x[t]
        hid = xe @ _matrix8(st["q1"][e], st["s1"][e]).t()
        hid = hid * torch.sigmoid(hid)
        if st["act"] == "swiglu":
            hid = hid * (xe @ _matrix8(st["q2"][e], st["s2"][e]).t())
        out = _values8(*_rows8(hid)) @ _matrix8(st["q3"][e], st["s3"][e]).t()
        rows[t, k] = out * st["gates"][t, k][:, None]
    return {"y": rows.sum(dim=1).to(BF16)}


def _ckpt8(st):
    # (without the gates' gradient, as with a router that is not trained: its fp32 digits behind the fourth depend on
    # the side of a border that a code falls on)
    names = ("dX", "dW1", "dW2", "dW3")
    if own:
        layer = st["layer"]
        layer.dispatch(st["ids"])
        y = layer.forward(st["x"], st["gates"], st["W1"], st["W2"], st["W3"])
        grads = layer.backward(st["dY"], st["x"], st["gates"], st["W1"], st["W2"], st["W3"])
        out = dict(zip(names, grads))
        out["y"] = y
        return {k: v for k, v in out.items() if v is not None}
    L, d, E, sw = st["L"], st["d"], st["E"], st["act"] == "swiglu"
    x, dY = st["x"].float(), st["dY"].float()
    y, dX = (torch.zeros(L, d, device=x.device) for _ in range(2))
    dW1, dW3 = torch.empty_like(st["W1"]), torch.empty_like(st["W3"])
    dW2 = torch.empty_like(st["W2"]) if sw else None
    for e in range(E):
        t, k = torch.nonzero(st["ids"] == e, as_tuple=True)
        g = st["gates"][t, k][:, None]
        W1, W3 = st["W1"][e].float(), st["W3"][e].float()
        a = x[t] @ W1
        hid = a * torch.sigmoid(a)
        if sw:
            W2 = st["W2"][e].float()
            b = x[t] @ W2
            hid = hid * b
            b = _int8(b)
        y.index_add_(0, t, g * (hid @ W3))
        a = _int8(a)  # what is kept for the backward pass
        sig = torch.sigmoid(a)
        act = a * sig
        slope = sig * (1.0 + a * (1.0 - sig))
        hid = act * b if sw else act
        dW3[e] = ((g * hid).t() @ dY[t]).to(BF16)
        dh = g * (dY[t] @ W3.t())
        da = dh * b * slope if sw else dh * slope
        dW1[e] = (x[t].t() @ da).to(BF16)
        dx = da @ W1.t()
        if sw:
            db = dh * act
            dW2[e] = (x[t].t() @ db).to(BF16)
            dx = dx + db @ W2.t()
        dX.index_add_(0, t, dx)
    out = {"y": y.to(BF16), "dX": dX.to(BF16), "dW1": dW1, "dW2": dW2, "dW3": dW3}
    return {k: v for k, v in out.items() if v is not None}


_RUN = {"rms_fwd": _rms_fwd, "rms_bwd": _rms_bwd, "fp8": _fp8, "ckpt8": _ckpt8}


def run(state):
    return _RUN[state["op"]](state)


# --------------------------------------------------------------------- work

def work(case):
    op, L, d = case["op"], case["L"], case["d"]
    if op == "rms_fwd":
        e = 2 if case["dtype"] == "bf16" else 4
        # with 8-bit rows: codes and scales, and the values they stand for
        eight = L * d + 4 * L * ((d + BLOCK - 1) // BLOCK) + 2 * L * d if case["out8"] else 0
        return {"bytes": L * d * e * (4 if case["residual"] else 2) + eight + 4 * L + 4 * d, "flops": 6 * L * d}
    if op == "rms_bwd":
        e = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": L * d * e * (4 if case["residual"] else 3) + 4 * L + 8 * d, "flops": 12 * L * d}
    h, E, K = (case[k] for k in ("h", "E", "K"))
    mats = 3 if case["act"] == "swiglu" else 2
    if op == "fp8":
        live = L * (0.8 if case["idle"] else 1.0)
        used = E * (1.0 - (1.0 - K / E) ** live)
        return {"bytes": used * mats * d * h * (1 + 4.0 / BLOCK ** 2) + L * d * (3 if case["rows8"] else 4) + 8 * L * K,
                "flops": 2.0 * mats * live * K * d * h}
    used = E * (1.0 - (1.0 - K / E) ** L)
    # weights in, gradients of all of them out; x and dY in (x by both passes), y and dX out; the codes both ways
    kept = 2.0 * (mats - 1) * L * K * h * (1 + 4.0 / BLOCK)
    return {"bytes": 2.0 * mats * d * h * (2 * used + E) + 10.0 * L * d + kept + 8 * L * K, "flops": _flops(case)}


# --------------------------------------------------------------------- exact

def _two_to(e):
    """2^e in 64 bits, to the bit (a power function need not be)."""
    return (e.long() + 1023 << 52).view(torch.float64)


def _e4m3_64(v):
    """v rounded to the nearest e4m3 value (ties to even), in 64 bits."""
    _, e = torch.frexp(v)
    step = _two_to((e - 4).clamp(min=-9))
    return torch.round(v / step) * step


def _eight64(v):
    """The values of v's blocks of 128 columns in e4m3 with a power-of-two scale, in 64 bits."""
    out = torch.empty_like(v)
    for c in range(0, v.shape[1], BLOCK):
        p = v[:, c:c + BLOCK]
        # the least power of two that brings the largest to 448
        f, e = torch.frexp(p.abs().amax(dim=1, keepdim=True) / TOP8)
        s = _two_to(torch.where(f == 0.5, e - 1, e).clamp(min=-126))
        out[:, c:c + BLOCK] = _e4m3_64(p / s) * s
    return out


def _codes64(v):
    """The values of v's blocks of 128 columns in int8 with a scale of a 127th of the largest, in 64 bits."""
    out = torch.empty_like(v)
    for c in range(0, v.shape[1], BLOCK):
        p = v[:, c:c + BLOCK]
        s = (p.abs().amax(dim=1, keepdim=True) / 127.0).clamp(min=1e-300)
        out[:, c:c + BLOCK] = torch.round(p / s) * s
    return out


def _grown(s, n, dim):
    return s.double().repeat_interleave(BLOCK, dim=dim).narrow(dim, 0, n)


def exact(case, seed):
    """The definitions in 64 bits."""
    global own
    op, L, d = case["op"], case["L"], case["d"]
    if op in ("fp8", "ckpt8") and _flops(case) > 1.8e13:
        return None
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    x = st["x"].double()
    if op == "rms_fwd":
        s = x if st["r"] is None else x + st["r"].double()
        rstd = 1.0 / torch.sqrt(torch.linalg.vecdot(s, s) / d + EPS)
        y = torch.einsum("td,t,d->td", s, rstd, st["w"].double())
        out = {"y": y, "rstd": rstd}
        if case["out8"]:
            out["y8"] = _eight64(y)
        if st["r"] is not None:
            out["s"] = s
        return out
    if op == "rms_bwd":
        # dx = rstd * (g without its part along xh), the columns' scale inside g
        xh = torch.einsum("td,t->td", x, st["rstd"].double())
        g = torch.einsum("td,d->td", st["dy"].double(), st["w"].double())
        dx = st["rstd"].double()[:, None] * (g - xh * (torch.linalg.vecdot(g, xh) / d)[:, None])
        if st["ds"] is not None:
            dx += st["ds"].double()
        return {"dx": dx, "dw": torch.einsum("td,td->d", st["dy"].double(), xh)}
    h, E, K, sw = case["h"], case["E"], case["K"], case["act"] == "swiglu"
    ids, gates = st["ids"], st["gates"].double()
    y = torch.zeros(L, d, dtype=torch.float64, device="cuda")
    if op == "fp8":
        x = x * _grown(st["sx"], d, 1) if case["rows8"] else _eight64(x)

        def matrix(n, e):
            q = st["q" + n][e].double()
            return q * _grown(_grown(st["s" + n][e], q.shape[0], 0), q.shape[1], 1)

        for e in range(E):
            t, k = torch.where(ids == e)
            if t.numel() == 0:
                continue
            a = torch.einsum("td,hd->th", x[t], matrix("1", e))
            hid = a / (1.0 + torch.exp(-a))
            if sw:
                hid = hid * torch.einsum("td,hd->th", x[t], matrix("2", e))
            y.index_add_(0, t, torch.einsum("th,dh,t->td", _eight64(hid), matrix("3", e), gates[t, k]))
        return {"y": y}
    dY = st["dY"].double()
    dX = torch.zeros_like(y)
    dW = {n: torch.zeros(st[n].shape, dtype=torch.float64, device="cuda") for n in ("W1", "W2", "W3")
          if st[n] is not None}
    for e in range(E):
        t, k = torch.where(ids == e)
        if t.numel() == 0:
            continue
        w = {n: st[n][e].double() for n in dW}
        xe, dye, g = x[t], dY[t], gates[t, k]
        a = xe @ w["W1"]
        b = xe @ w["W2"] if sw else torch.ones_like(a)
        y.index_add_(0, t, torch.einsum("th,hd,t->td", a / (1.0 + torch.exp(-a)) * b, w["W3"], g))
        a = _codes64(a)
        b = _codes64(b) if sw else b
        p = 1.0 / (1.0 + torch.exp(-a))
        up = (dye @ w["W3"].t()) * g[:, None]
        dW["W3"][e] = torch.einsum("th,td,t->hd", p * a * b, dye, g)
        da = up * b * (p + a * p * (1.0 - p))
        dW["W1"][e] = xe.t() @ da
        back = da @ w["W1"].t()
        if sw:
            db = up * a * p
            dW["W2"][e] = xe.t() @ db
            back += db @ w["W2"].t()
        dX.index_add_(0, t, back)
    out = {"y": y, "dX": dX}
    out.update({"d" + n: v for n, v in dW.items()})
    return out
