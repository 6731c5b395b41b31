"""Definitions in fp64 of the operators in 8 bits, and bounds on what a kernel
may be off (imported by the tests; shares nothing with the CUDA path).  All of
it runs on whatever device its tensors are on."""
from __future__ import annotations

import torch

U32 = 2.0 ** -24                                    # half a step of fp32, relative
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float8_e4m3fn: 2.0 ** -4}
BF = HALF[torch.bfloat16]


def inside(got, want, tol, what):
    """|got - want| <= tol elementwise (NaN fails), with the worst place in the message."""
    got = got.detach().to(want.device).double()
    bad = ~((got - want).abs() <= tol)
    if bad.any():
        i = tuple(torch.nonzero(bad)[0].tolist())
        over = ((got - want).abs() / tol)[bad].max()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {i}: got {got[i]:.9g}, want "
                             f"{want[i]:.9g}; worst {over:.3g} of the tolerance")


def matmul_err(n):
    """Relative to the sum of the terms' sizes: a sum of n products in fp32, each step off by a step at most (the tensor
    memory truncates), and the products' own factors."""
    return 2.0 * (n + 16) * U32


def silu(a):
    return a / (1.0 + torch.exp(-a))


def layer_forward(x, ids, gates, W1, W2, W3):
    """y of the bf16 layer and a bound on |y - kernel| before y's rounding: the hidden activations are rounded to bf16
    once, everything else is fp32."""
    x, gates = x.double(), gates.double()
    L, K = ids.shape
    E, d, h = W1.shape
    y = torch.zeros(L, d, dtype=torch.float64, device=x.device)
    bound = torch.zeros_like(y)
    for e in range(E):
        t, k = torch.nonzero(ids == e, as_tuple=True)
        if t.numel() == 0:
            continue
        w1, w3 = W1[e].double(), W3[e].double()
        a, aa = x[t] @ w1, x[t].abs() @ w1.abs()
        hid, err = silu(a), 1.1 * aa * matmul_err(d)        # |silu'| <= 1.1
        if W2 is not None:
            w2 = W2[e].double()
            b, ba = x[t] @ w2, x[t].abs() @ w2.abs()
            err = err * b.abs() + hid.abs() * ba * matmul_err(d)
            hid = hid * b
        # (the sigmoid's fast exponential: a few steps of fp32, and |a| of them in the exponent)
        herr = BF * hid.abs() + err + (16 + 4 * a.abs()) * U32 * hid.abs()
        g = gates[t, k][:, None]
        y.index_add_(0, t, g * (hid @ w3))
        bound.index_add_(0, t, g.abs() * (herr @ w3.abs() + matmul_err(h) * (hid.abs() @ w3.abs())))
    return y, bound


def layer_backward(dY, x, ids, gates, W1, W2, W3, A, B):
    """Gradients of the layer evaluated at the checkpoints A, B, per expert lists of (rows of e, h) values in the order
    of torch.nonzero(ids == e), and bounds on what the kernels may be off before the outputs' own rounding: dA, dB and
    g H are rounded to bf16 on their way between products."""
    dY, x, gates = dY.double(), x.double(), gates.double()
    L, K = ids.shape
    E, d, h = W1.shape
    out = {"dX": torch.zeros(L, d, dtype=torch.float64, device=x.device),
           "dgates": torch.zeros(L, K, dtype=torch.float64, device=x.device)}
    for n, w in (("dW1", W1), ("dW2", W2), ("dW3", W3)):
        if w is not None:
            out[n] = torch.zeros(w.shape, dtype=torch.float64, device=x.device)
    tol = {n: torch.zeros_like(v) for n, v in out.items()}
    for e in range(E):
        t, k = torch.nonzero(ids == e, as_tuple=True)
        if t.numel() == 0:
            continue
        w1, w3 = W1[e].double(), W3[e].double()
        xe, dy, g = x[t], dY[t], gates[t, k][:, None]
        a = A[e]
        b = B[e] if W2 is not None else torch.ones_like(a)
        fast = (16 + 4 * a.abs()) * U32                     # relative, of the sigmoid and what is formed from it
        sig = 1.0 / (1.0 + torch.exp(-a))
        act, slope = a * sig, sig * (1.0 + a * (1.0 - sig))
        slope_size = sig * (1.0 + a.abs())
        up, upa = dy @ w3.t(), dy.abs() @ w3.abs().t()
        uerr = upa * matmul_err(d)
        hid = act * b
        out["dgates"][t, k] = (hid * up).sum(1)
        tol["dgates"][t, k] = (hid.abs() * (uerr + (fast + h * U32) * up.abs())).sum(1) + 1e-30
        gh = g * hid
        out["dW3"][e] = gh.t() @ dy
        tol["dW3"][e] = ((BF + fast) * gh.abs()).t() @ dy.abs() + matmul_err(len(t)) * (gh.abs().t() @ dy.abs())
        dh, derr = g * up, g.abs() * uerr
        da = dh * b * slope
        daerr = BF * da.abs() + b.abs() * slope_size * (derr + fast * dh.abs())
        parts = [("dW1", w1, da, daerr)]
        if W2 is not None:
            db = dh * act
            parts.append(("dW2", W2[e].double(), db, BF * db.abs() + act.abs() * (derr + fast * dh.abs())))
        for n, w, v, verr in parts:
            out[n][e] = xe.t() @ v
            tol[n][e] = xe.abs().t() @ verr + matmul_err(len(t)) * (xe.abs().t() @ v.abs())
            out["dX"].index_add_(0, t, v @ w.t())
            tol["dX"].index_add_(0, t, verr @ w.abs().t() + matmul_err(2 * h) * (v.abs() @ w.abs().t()))
    return out, tol


def blocks(v):
    """Row blocks of 128 columns of v (L,d): (L, ceil(d/128), 128), zeros behind the last column."""
    L, d = v.shape
    n = -(-d // 128)
    return torch.nn.functional.pad(v, (0, 128 * n - d)).view(L, n, 128)


def rows8(v):
    """(codes as float64 values, scales) of v's blocks of 128 columns, by the definition: the scale the least power of
    two (2^-126 or more) that brings the largest to at most 448; each value to the nearest e4m3 value, ties to the even
    one; NaN scales for blocks with a NaN or an infinity."""
    b = blocks(v.double())
    top = b.abs().amax(2)
    ok = top.isfinite()
    f, e = torch.frexp(torch.where(ok, top, torch.ones_like(top)) / 448.0)
    k = torch.where(f == 0.5, e - 1, e).clamp(min=-126)
    k = torch.where(f == 0, torch.full_like(k, -126), k)    # (a block of zeros: frexp has no exponent for it)
    s = (k.long() + 1023 << 52).view(torch.float64)
    u = b / s[..., None]
    _, ue = torch.frexp(torch.nan_to_num(u, 0, 0, 0))
    step = ((ue - 4).clamp(min=-9).long() + 1023 << 52).view(torch.float64)
    q = torch.round(u / step) * step
    s = torch.where(ok, s, torch.full_like(s, float("nan")))
    return q.flatten(1)[:, :v.shape[1]], s


def grown(s, d):
    """A scale for every column, (L,d) in fp64, of scales (L, ceil(d/128))."""
    return s.double().repeat_interleave(128, dim=1)[:, :d]


def rms(x, residual, w, eps):
    s = x.double() if residual is None else x.double() + residual.double()
    rstd = 1.0 / torch.sqrt((s * s).mean(1) + eps)
    return s * rstd[:, None] * w.double(), s, rstd


def rms_grad(dy, s, rstd, w, dsum):
    """dx, dweight, and xh and g of the formulas."""
    g, xh = dy.double() * w.double(), s.double() * rstd.double()[:, None]
    dx = rstd.double()[:, None] * (g - xh * (g * xh).mean(1, keepdim=True))
    if dsum is not None:
        dx = dx + dsum.double()
    return dx, (dy.double() * xh).sum(0), xh, g


def matrix8(q, s):
    """What one e4m3 matrix (N,R) with scales (N/128, R/128) stands for, (R,N) in fp64."""
    return (q.double() * s.double().repeat_interleave(128, 0).repeat_interleave(128, 1)).t()


def experts8(x, ids, gates, mats):
    """y (L,d) of 8-bit rows' values x (fp64) through 8-bit experts, and a bound on |y - kernel| before y's rounding.
    mats: (q1, s1, q2, s2, q3, s3).  The hidden activations go to 8-bit rows by the definition; the kernel's are off by
    fp32's roundings, which can push one over a border between two codes: what it may then be is what the bound counts."""
    q1, s1, q2, s2, q3, s3 = mats
    E, h, d = q1.shape
    L, K = ids.shape
    y = torch.zeros(L, d, dtype=torch.float64, device=x.device)
    bound = torch.zeros_like(y)
    for e in range(E):
        t, k = torch.nonzero(ids == e, as_tuple=True)
        if t.numel() == 0:
            continue
        w1, w3 = matrix8(q1[e], s1[e]), matrix8(q3[e], s3[e])
        a, err = x[t] @ w1, 1.1 * (x[t].abs() @ w1.abs()) * matmul_err(d)
        hid = silu(a)
        if q2 is not None:
            w2 = matrix8(q2[e], s2[e])
            b = x[t] @ w2
            err = err * b.abs() + hid.abs() * (x[t].abs() @ w2.abs()) * matmul_err(d)
            hid = hid * b
        err = err + (16 + 4 * a.abs()) * U32 * hid.abs()
        codes, s = rows8(hid)
        sc = grown(s, h)
        val = codes * sc
        off = torch.zeros_like(val)
        for v in (hid - err, hid + err):                # the codes at the ends, at the block's scale
            u = (v / sc).clamp(-448, 448)
            _, ue = torch.frexp(u)
            step = ((ue - 4).clamp(min=-9).long() + 1023 << 52).view(torch.float64)
            off = torch.maximum(off, (torch.round(u / step) * step * sc - val).abs())
        # a block whose largest value is next to a border between scales: subnormals round at twice, or half, the step
        top, terr = blocks(hid).abs().amax(2), blocks(err).amax(2)
        edge = ((top - terr <= 224 * s) | (top + terr > 448 * s)) & (s > 2.0 ** -126)
        off = off + grown(edge.double() * s * 2.0 ** -9, h)
        g = gates[t, k].double()[:, None]
        out = val @ w3
        err = off @ w3.abs() + matmul_err(h) * ((val.abs() + off) @ w3.abs())
        y.index_add_(0, t, g * out)
        # each slot's row waits for the others in fp16 (prompts): half a step of it, 2^-11 of the value.  (At its scale
        # the block's largest is 2^14 or more, and subnormals' half step 2^-25, 2^-39 of the largest: the sum's own
        # bound above is larger.)
        bound.index_add_(0, t, g.abs() * (err + 2.0 ** -11 * (out.abs() + err)))
    return y, bound + matmul_err(K) * y.abs()
