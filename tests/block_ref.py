"""Definitions in fp64 of the layer norm, the router's losses, the dense router
gradient and the 4-bit expert products, on CPU tensors (imported by the
tests; shares nothing with the CUDA path)."""
from __future__ import annotations

import torch

U32 = 2.0 ** -24                                    # half a step of fp32, relative
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def d64(t):
    return None if t is None else t.detach().cpu().double()


def norm(x, residual, w, b, eps):
    s = d64(x) if residual is None else d64(x) + d64(residual)
    mean = s.mean(1, keepdim=True)
    var = ((s - mean) ** 2).mean(1, keepdim=True)
    rstd = 1.0 / torch.sqrt(var + eps)
    y = (s - mean) * rstd * d64(w)
    if b is not None:
        y = y + d64(b)
    return y, s, mean[:, 0], rstd[:, 0]


def norm_grad(dy, s, mean, rstd, w, dsum):
    dy, s, mean, rstd, w = d64(dy), d64(s), d64(mean)[:, None], d64(rstd)[:, None], d64(w)
    xh = (s - mean) * rstd
    g = dy * w
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    if dsum is not None:
        dx = dx + d64(dsum)
    return dx, (dy * xh).sum(0), dy.sum(0), xh, g


def balance(logits, ids, valid):
    """(losses, counts, N, lse, active) by the definition, token by token masks and all."""
    lg = d64(logits)
    L, E = lg.shape
    K = ids.shape[1]
    active = torch.ones(L, dtype=torch.bool) if valid is None else valid.cpu() != 0
    active = active & ~(lg == -float("inf")).all(1)
    safe = torch.where(active[:, None], lg, torch.zeros(()).double())
    lse = torch.logsumexp(safe, 1)
    p = torch.exp(safe - lse[:, None]) * active[:, None]
    n = int(active.sum())
    counts = torch.zeros(E, dtype=torch.int64)
    idc = ids.cpu().long()
    for t in range(L):
        if active[t]:
            for e in idc[t].tolist():
                if 0 <= e < E:
                    counts[e] += 1
    if n == 0:
        return torch.zeros(2).double(), counts, 0, lse, active, p
    f = counts.double() / (n * K)
    bal = E * (f * p.sum(0) / n).sum()
    z = (lse[active] ** 2).sum() / n
    return torch.stack([bal, z]), counts, n, lse, active, p


def balance_grad(logits, ids, valid, dlosses, gates, dgates):
    _, counts, n, lse, active, p = balance(logits, ids, valid)
    L, E = p.shape
    K = ids.shape[1]
    a, z = float(dlosses[0]), float(dlosses[1])
    dl = torch.zeros(L, E, dtype=torch.float64)
    scale = torch.zeros(L, E, dtype=torch.float64)   # size of the terms, for the error bound
    if n:
        f = counts.double() / (n * K)
        f = f - f.mean()
        dot = (p * f).sum(1, keepdim=True)
        dl += a * E / n * p * (f - dot) + 2 * z / n * lse[:, None] * p
        scale += abs(a) * E / n * p * 2 * f.abs().max() + 2 * abs(z) / n * lse.abs()[:, None] * p
    if gates is not None:
        g, dg, idc = d64(gates), d64(dgates), ids.cpu().long()
        sd, sa = (g * dg).sum(1, keepdim=True), (g * dg).abs().sum(1, keepdim=True)
        for k in range(K):
            e = idc[:, k]
            ok = (e >= 0) & (e < E) & active
            r = torch.nonzero(ok).flatten()
            dl[r, e[r]] += (g[:, k:k + 1] * (dg[:, k:k + 1] - sd))[r, 0]
            scale[r, e[r]] += (g[:, k:k + 1].abs() * (dg[:, k:k + 1].abs() + sa))[r, 0]
    return torch.where(active[:, None], dl, torch.zeros(()).double()), scale


def int4_weights(q, s, group):
    return d64(q.float()) * d64(s).repeat_interleave(group, dim=1)


def silu(a):
    return a / (1.0 + torch.exp(-a))


def int4_layer(x, ids, gates, W1, W2, W3):
    """y and a bound on |y - kernel| before the last rounding: the hidden
    activations are rounded to bf16 once, everything else is fp32."""
    x, gates, ids = d64(x), d64(gates), ids.cpu().long()
    L, K = ids.shape
    E, d, h = W1.shape
    y = torch.zeros(L, d, dtype=torch.float64)
    bound = torch.zeros(L, d, dtype=torch.float64)
    for e in range(E):
        t, k = torch.nonzero(ids == e, as_tuple=True)
        if t.numel() == 0:
            continue
        a, ab = x[t] @ W1[e], x[t].abs() @ W1[e].abs()
        hid, err = silu(a), 1.1 * ab        # |silu'| <= 1.1
        if W2 is not None:
            b, bb = x[t] @ W2[e], x[t].abs() @ W2[e].abs()
            err = err * b.abs() + hid.abs() * bb
            hid = hid * b
        g = gates[t, k][:, None]
        # sums of d and of h terms, each step off by at most U32 of the sum of the terms' sizes
        herr = HALF[torch.bfloat16] * hid.abs() + (d + 16) * U32 * err + 8 * U32 * hid.abs()
        y.index_add_(0, t, g * (hid @ W3[e]))
        bound.index_add_(0, t, g.abs() * (herr @ W3[e].abs() + (h + 16) * U32 * (hid.abs() @ W3[e].abs())))
    return y, bound


def inside(got, want, tol, what):
    """|got - want| <= tol elementwise (NaN fails), with the worst place in the message."""
    got = d64(got)
    bad = ~((got - want).abs() <= tol)
    if bad.any():
        i = torch.nonzero(bad)[0].tolist()
        over = ((got - want).abs() / tol).max()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {i}: got "
                             f"{got[tuple(i)]:.9g}, want {want[tuple(i)]:.9g}; worst {over:.3g} of the tolerance")
