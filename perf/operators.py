"""The operators around and inside the MoE layer, as measured cases: layer
norm with the residual sum, the router's balance and z loss, the router's
gradient from dense logit gradients, and the expert products on 4-bit weights.

Each case is one call (or one forward with its backward) as a training or
serving program makes it.  With ``own`` false the operators are computed in
their plain form from elementary torch operations; with ``own`` true by the
framework's entry points.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
DT = {"bf16": BF16, "f32": F32}
EPS = 1e-5


# --------------------------------------------------------------------- cases

def listed():
    return [
        # layer norm + residual sum of a decode batch: launch latency counts
        dict(name="norm_fwd_decode", op="norm_fwd", L=4, d=4096, dtype="bf16", residual=True),
        # the same of a training batch of the large-expert layer's width
        dict(name="norm_fwd_train", op="norm_fwd", L=32768, d=4096, dtype="bf16", residual=True),
        # its backward, with the gradient that arrives over the residual stream
        dict(name="norm_bwd_train", op="norm_bwd", L=32768, d=4096, dtype="bf16", residual=True),
        # an odd width in fp32: no row but every fourth starts on 16 bytes
        dict(name="norm_bwd_odd", op="norm_bwd", L=8191, d=1409, dtype="f32", residual=False),
        # router losses of a small layer, loss and gradient
        dict(name="balance_small", op="balance", L=512, E=8, K=2, masked=False, gates=True),
        # of the fine-grained layer, with padding tokens masked
        dict(name="balance_e64", op="balance", L=65536, E=64, K=6, masked=True, gates=True),
        # of a long batch of the 8-expert layer, the losses' gradient alone
        dict(name="balance_long", op="balance", L=262144, E=8, K=2, masked=True, gates=False),
        # router gradient of the large-expert layer and of the fine-grained layer
        dict(name="router_grad_e8", op="router_grad", L=32768, d=4096, E=8, dtype="bf16"),
        dict(name="router_grad_e64", op="router_grad", L=65536, d=2048, E=64, dtype="bf16"),
        # 4-bit experts: one token, a decode batch, and a batch over fine-grained experts
        dict(name="int4_token", op="int4", L=1, d=4096, h=14336, E=8, K=2, act="swiglu", group=128, idle=False),
        dict(name="int4_batch16", op="int4", L=16, d=4096, h=14336, E=8, K=2, act="swiglu", group=128, idle=False),
        dict(name="int4_fine64", op="int4", L=61, d=2048, h=1408, E=64, K=6, act="swiglu", group=64, idle=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "balance", "router_grad", "int4"])
    if op in ("norm_fwd", "norm_bwd"):
        d = _log_int(rng, 64, 8192)
        if rng.random() < 0.5:
            d = (d + 63) // 64 * 64
        L = _log_int(rng, 1, min(65536, 32768 * 4096 // d))
        dtype = rng.choice(["bf16", "bf16", "f32"])
        if dtype == "f32":
            L = max(1, L // 2)
        return dict(op=op, L=L, d=d, dtype=dtype, residual=rng.random() < 0.6)
    if op == "balance":
        E = _log_int(rng, 4, 256)
        K = rng.randint(1, min(8, E))
        L = _log_int(rng, 1, min(262144, 52000 * 64 // E))
        return dict(op=op, L=L, E=E, K=K, masked=rng.random() < 0.5, gates=rng.random() < 0.7)
    if op == "router_grad":
        E = _log_int(rng, 4, 128)
        d = 64 * _log_int(rng, 1, 64)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        L = _log_int(rng, 1, min(65536, 60000 * 2048 // d, 60000 * 2048 * 64 // (d * max(E, 8))))
        if dtype == "f32":
            L = max(1, L // 2)
        return dict(op=op, L=L, d=d, E=E, dtype=dtype)
    E = _log_int(rng, 2, 64)
    d = 128 * _log_int(rng, 1, 32)
    h = 128 * _log_int(rng, 1, 112)
    while E * d * h > 0.9 * 8 * 4096 * 14336:
        h = 128 * max(1, h // 256)
    return dict(op=op, L=_log_int(rng, 1, 64), d=d, h=h, E=E, K=rng.randint(1, min(8, E)),
                act=rng.choice(["swiglu", "swiglu", "silu"]), group=rng.choice([32, 64, 128]),
                idle=rng.random() < 0.3)


# --------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _stream_rows(L, d, dtype, g):
    """Rows of a residual stream: unit spread, an offset per column and a few
    columns ten times as large."""
    x = torch.randn(L, d, device="cuda", generator=g)
    col = 0.3 * torch.randn(d, device="cuda", generator=g)
    big = 1.0 + 9.0 * (torch.rand(d, device="cuda", generator=g) < 0.004)
    return (x * big + col).to(dtype)


def _routing(L, E, K, g):
    """Logits of a router with unequal experts, its top-K ids and gates."""
    logits = torch.randn(L, E, device="cuda", generator=g) + torch.randn(E, device="cuda", generator=g)
    top = torch.topk(logits, K, dim=1)
    return logits, top.indices.to(torch.int32).contiguous(), torch.softmax(top.values, dim=1).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = dict(case)
    if op in ("norm_fwd", "norm_bwd"):
        L, d, dt = case["L"], case["d"], DT[case["dtype"]]
        st["x"] = _stream_rows(L, d, dt, g)
        st["w"] = 1.0 + 0.1 * torch.randn(d, device="cuda", generator=g)
        st["b"] = 0.1 * torch.randn(d, device="cuda", generator=g)
        if op == "norm_fwd":
            st["r"] = torch.randn(L, d, device="cuda", generator=g).to(dt) if case["residual"] else None
        else:
            # what the forward left: the normalised sum (here x) and its statistics
            x = st["x"].float()
            st["mean"] = x.mean(dim=1)
            st["rstd"] = torch.rsqrt((x - st["mean"][:, None]).square().mean(dim=1) + EPS)
            del x
            st["dy"] = torch.randn(L, d, device="cuda", generator=g).to(dt)
            st["ds"] = torch.randn(L, d, device="cuda", generator=g).to(dt) if case["residual"] else None
        if own:
            from mixture_experts_atomic_gb300.block import LayerNorm
            st["norm"] = LayerNorm(L, d, dt, eps=EPS, device="cuda")
    elif op == "balance":
        L, E, K = case["L"], case["E"], case["K"]
        st["logits"], st["ids"], st["gates_kept"] = _routing(L, E, K, g)
        st["valid"] = (torch.rand(L, device="cuda", generator=g) < 0.9).to(torch.uint8) if case["masked"] else None
        st["dgates"] = torch.randn(L, K, device="cuda", generator=g) / math.sqrt(L)
        st["dloss"] = torch.tensor([0.01, 0.001], device="cuda")
        if own:
            from mixture_experts_atomic_gb300.block import BalanceLoss
            st["loss"] = BalanceLoss(L, E, K, device="cuda")
    elif op == "router_grad":
        L, d, E, dt = case["L"], case["d"], case["E"], DT[case["dtype"]]
        st["x"] = torch.randn(L, d, device="cuda", generator=g).to(dt)
        st["Wr"] = torch.randn(d, E, device="cuda", generator=g) / math.sqrt(d)
        p = torch.softmax(torch.randn(L, E, device="cuda", generator=g), dim=1)
        st["dl"] = (p * torch.randn(L, E, device="cuda", generator=g)).contiguous()
        if own:
            from mixture_experts_atomic_gb300.block import RouterGrad
            st["grad"] = RouterGrad(L, d, E, dt, device="cuda")
    else:
        L, d, h, E, K, G = (case[k] for k in ("L", "d", "h", "E", "K", "group"))
        st["x"] = torch.randn(L, d, device="cuda", generator=g).to(BF16)
        _, st["ids"], st["gates"] = _routing(L, E, K, g)
        if case["idle"]:
            # slots of a decode batch that hold no sequence: id -1 in all K
            st["ids"][torch.rand(L, device="cuda", generator=g) < 0.2] = -1
        for n, rows, cols in (("1", d, h), ("2", d, h), ("3", h, d)):
            if n == "2" and case["act"] != "swiglu":
                st["q2"] = st["s2"] = None
                continue
            # what a symmetric 4-bit quantiser leaves of normal weights of variance about 1/rows
            q = torch.randn(E, rows, cols, device="cuda", generator=g)
            st["q" + n] = q.mul_(2.7).round_().clamp_(-8, 7).to(torch.int8)
            del q
            u = torch.rand(E, rows // G, cols, device="cuda", generator=g)
            st["s" + n] = ((0.5 + u) / (2.7 * math.sqrt(rows))).to(BF16)
        if own:
            from mixture_experts_atomic_gb300.int4 import Int4Experts
            st["experts"] = Int4Experts(L, d, h, E, K, act=case["act"], group=G, device="cuda")
            st["experts"].load(st["q1"], st["s1"], st["q2"], st["s2"], st["q3"], st["s3"])
            for n in "123":  # the packed weights are what a serving program keeps
                del st["q" + n], st["s" + n]
    return st


# --------------------------------------------------------------------- one pass

def _norm_fwd(st):
    if own:
        y, s, mean, rstd = st["norm"].forward(st["x"], st["w"], st["b"], st["r"])
    else:
        dt = st["x"].dtype
        s32 = st["x"].float() + (st["r"].float() if st["r"] is not None else 0.0)
        mean = s32.mean(dim=1)
        c = s32 - mean[:, None]
        rstd = torch.rsqrt(c.square().mean(dim=1) + EPS)
        y = (c * rstd[:, None] * st["w"] + st["b"]).to(dt)
        s = s32.to(dt)
    out = {"y": y, "mean": mean, "rstd": rstd}
    if st["r"] is not None:
        out["s"] = s
    return out


def _norm_bwd(st):
    if own:
        dx, dw, db = st["norm"].backward(st["dy"], st["x"], st["mean"], st["rstd"], st["w"], st["ds"])
    else:
        dy = st["dy"].float()
        xh = (st["x"].float() - st["mean"][:, None]) * st["rstd"][:, None]
        gw = dy * st["w"]
        dx = (gw - gw.mean(dim=1, keepdim=True) - xh * (gw * xh).mean(dim=1, keepdim=True)) * st["rstd"][:, None]
        if st["ds"] is not None:
            dx = dx + st["ds"].float()
        dx = dx.to(st["x"].dtype)
        dw = (dy * xh).sum(dim=0)
        db = dy.sum(dim=0)
    return {"dx": dx, "dw": dw, "db": db}


def _balance(st):
    L, E, K = st["L"], st["E"], st["K"]
    logits, ids, valid = st["logits"], st["ids"], st["valid"]
    gate_args = (ids, st["gates_kept"], st["dgates"]) if st["gates"] else (None, None, None)
    if own:
        losses, counts = st["loss"].forward(logits, ids, valid)
        dlogits = st["loss"].backward(logits, st["dloss"], valid, *gate_args)
        return {"losses": losses, "counts": counts, "dlogits": dlogits}
    top = logits.max(dim=1).values
    ex = torch.exp(logits - top[:, None])
    norm = ex.sum(dim=1)
    lse = (top + torch.log(norm)).double()
    p = (ex / norm[:, None]).double()
    on = torch.ones(L, dtype=torch.bool, device=logits.device) if valid is None else valid != 0
    counts = torch.zeros(E, dtype=torch.int32, device=logits.device)
    counts.index_add_(0, ids.reshape(-1).long(), on.to(torch.int32)[:, None].expand(L, K).reshape(-1))
    n = on.sum().clamp(min=1).double()
    f = counts.double() / (n * K)
    w = on.double()
    mean_p = (p * w[:, None]).sum(dim=0) / n
    losses = torch.stack([E * (f * mean_p).sum(), (w * lse * lse).sum() / n]).float()
    a, z = st["dloss"][0].double(), st["dloss"][1].double()
    dl = (a * E / n) * p * (f - (p * f).sum(dim=1, keepdim=True)) + (2.0 * z / n) * lse[:, None] * p
    if st["gates"]:
        gk, dg = st["gates_kept"].double(), st["dgates"].double()
        dl = dl.scatter_add(1, ids.long(), gk * (dg - (gk * dg).sum(dim=1, keepdim=True)))
    return {"losses": losses, "counts": counts, "dlogits": (dl * w[:, None]).float()}


def _router_grad(st):
    if own:
        dx, dWr, dbias = st["grad"].backward(st["x"], st["Wr"], st["dl"])
    else:
        dWr = st["x"].float().t() @ st["dl"]
        dbias = st["dl"].sum(dim=0)
        dx = (st["dl"] @ st["Wr"].t()).to(st["x"].dtype)
    return {"dx": dx, "dWr": dWr, "dbias": dbias}


def _weights(q, s, which, G):
    """The weights that q and s stand for, of the experts in `which`, in 32 bits."""
    q, s = q[which].float(), s[which].float()
    n, rows, cols = q.shape
    return (q.view(n, rows // G, G, cols) * s[:, :, None, :]).view(n, rows, cols)


def _int4(st):
    if own:
        return {"y": st["experts"].forward(st["x"], st["ids"], st["gates"])}
    L, E, K, G = st["L"], st["E"], st["K"], st["group"]
    x = st["x"].float()
    ids = st["ids"].long()
    live = ids >= 0
    gates = st["gates"] * live
    if L * K < E:  # fewer slots than experts: each slot's own weights
        which = ids.clamp(min=0).reshape(-1)
        rows = x.repeat_interleave(K, dim=0)[:, None, :]
        hid = torch.matmul(rows, _weights(st["q1"], st["s1"], which, G))
        hid = hid * torch.sigmoid(hid)
        if st["act"] == "swiglu":
            hid = hid * torch.matmul(rows, _weights(st["q2"], st["s2"], which, G))
        out = torch.matmul(hid, _weights(st["q3"], st["s3"], which, G))
        y = (out.view(L, K, -1) * gates[:, :, None]).sum(dim=1)
    else:  # every expert on every token, weighted by the token's gate for it
        which = torch.arange(E, device=x.device)
        mix = torch.zeros(L, E, device=x.device).scatter_add(1, ids.clamp(min=0), gates)
        hid = torch.matmul(x, _weights(st["q1"], st["s1"], which, G))
        hid = hid * torch.sigmoid(hid)
        if st["act"] == "swiglu":
            hid = hid * torch.matmul(x, _weights(st["q2"], st["s2"], which, G))
        out = torch.matmul(hid, _weights(st["q3"], st["s3"], which, G))
        y = (out * mix.t()[:, :, None]).sum(dim=0)
    return {"y": y.to(BF16)}


_RUN = {"norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd, "balance": _balance, "router_grad": _router_grad,
        "int4": _int4}


def run(state):
    return _RUN[state["op"]](state)


# --------------------------------------------------------------------- work

def work(case):
    op, L = case["op"], case["L"]
    if op in ("norm_fwd", "norm_bwd"):
        d, e = case["d"], 2 if case["dtype"] == "bf16" else 4
        if op == "norm_fwd":
            return {"bytes": L * d * e * (4 if case["residual"] else 2) + 8 * L + 8 * d, "flops": 9 * L * d}
        return {"bytes": L * d * e * (4 if case["residual"] else 3) + 8 * L + 12 * d, "flops": 16 * L * d}
    if op == "balance":
        E, K = case["E"], case["K"]
        # forward and backward are two calls: the logits are read by each
        b = 12 * L * E + 4 * L * K + (12 * L * K if case["gates"] else 0) + (2 * L if case["masked"] else 0)
        return {"bytes": b + 8 * E, "flops": 16 * L * E}
    if op == "router_grad":
        d, E, e = case["d"], case["E"], 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * L * d * e + 4 * L * E + 8 * d * E, "flops": 4 * L * d * E}
    d, h, E, K, G = (case[k] for k in ("d", "h", "E", "K", "group"))
    mats = 3 if case["act"] == "swiglu" else 2
    used = E * (1.0 - (1.0 - K / E) ** (L * (0.8 if case["idle"] else 1.0)))
    return {"bytes": used * mats * d * h * (0.5 + 2.0 / G) + 4 * L * d + 8 * L * K, "flops": 2.0 * mats * L * K * d * h}


# --------------------------------------------------------------------- exact

def exact(case, seed):
    """The definitions in 64 bits."""
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    f64 = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() and k[0] not in "qs" else v
           for k, v in st.items()}
    op = case["op"]
    if op == "norm_fwd":
        s = f64["x"] if f64["r"] is None else f64["x"] + f64["r"]
        var, mean = torch.var_mean(s, dim=1, correction=0)
        rstd = 1.0 / torch.sqrt(var + EPS)
        out = {"y": torch.addcmul(f64["b"], (s - mean[:, None]) * rstd[:, None], f64["w"]), "mean": mean, "rstd": rstd}
        if f64["r"] is not None:
            out["s"] = s
        return out
    if op == "norm_bwd":
        # dx = rstd * (g - projection of g on the span of 1 and xh), the columns' scale inside g
        xh = (f64["x"] - f64["mean"][:, None]) * f64["rstd"][:, None]
        g = f64["dy"] * f64["w"]
        d = case["d"]
        dx = f64["rstd"][:, None] * (g - (g.sum(1, keepdim=True) + xh * torch.linalg.vecdot(g, xh)[:, None]) / d)
        if st["ds"] is not None:
            dx = dx + st["ds"].double()
        return {"dx": dx, "dw": torch.einsum("td,td->d", f64["dy"], xh), "db": f64["dy"].sum(0)}
    if op == "balance":
        L, E, K = case["L"], case["E"], case["K"]
        keep = torch.arange(L, device="cuda") if st["valid"] is None else torch.nonzero(st["valid"]).flatten()
        lg = f64["logits"][keep]
        n = max(1, keep.numel())
        lse = torch.logsumexp(lg, dim=1)
        p = torch.exp(lg - lse[:, None])
        hot = torch.zeros(lg.shape[0], E, dtype=torch.float64, device="cuda").scatter_(1, st["ids"][keep].long(), 1.0)
        counts = hot.sum(0)
        f = counts / (n * K)
        losses = torch.stack([E * torch.dot(f, p.sum(0)) / n, lse.square().sum() / n])
        a, z = float(f64["dloss"][0]), float(f64["dloss"][1])
        d = p * ((a * E / n) * (f[None, :] - (p @ f)[:, None]) + (2.0 * z / n) * lse[:, None])
        if case["gates"]:
            gk, dg = f64["gates_kept"][keep], f64["dgates"][keep]
            d.scatter_add_(1, st["ids"][keep].long(), gk * dg - gk * torch.linalg.vecdot(gk, dg)[:, None])
        dl = torch.zeros(L, E, dtype=torch.float64, device="cuda")
        dl[keep] = d
        return {"losses": losses, "counts": counts.to(torch.int32), "dlogits": dl}
    if op == "router_grad":
        dl, wr = f64["dl"], f64["Wr"]
        return {"dx": torch.einsum("te,de->td", dl, wr), "dWr": torch.einsum("td,te->de", f64["x"], dl),
                "dbias": dl.sum(0)}
    y = torch.zeros(case["L"], case["d"], dtype=torch.float64, device="cuda")
    G = case["group"]

    def product(rows, n, e):
        w = st["q" + n][e].double() * st["s" + n][e].double().repeat_interleave(G, dim=0)
        return rows @ w

    for e in range(case["E"]):
        t, k = torch.nonzero(st["ids"] == e, as_tuple=True)
        if t.numel() == 0:
            continue
        xe = f64["x"][t]
        a = product(xe, "1", e)
        hid = a / (1.0 + torch.exp(-a))
        if case["act"] == "swiglu":
            hid = hid * product(xe, "2", e)
        y.index_add_(0, t, product(hid, "3", e) * f64["gates"][t, k][:, None])
    return {"y": y}
