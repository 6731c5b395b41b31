"""Layer norm, router losses and dense router gradient on the GPU against their
fp64 definitions (block_ref), at the sizes and masks where they can go wrong.
Tolerances are elementwise: the rounding of the output type plus fp32 error
bounds of the sums involved (number of additions in a row x half a step x the
sum of the terms' sizes)."""
import pytest
import torch

import block_ref as R
from mixture_experts_atomic_gb300 import binding as B
from mixture_experts_atomic_gb300.block import BalanceLoss, LayerNorm, MoEBlock, RouterGrad

pytestmark = pytest.mark.gpu

from gpu_util import ensure_built  # noqa: E402

U = R.U32
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


# ------------------------------------------------------------------ layer norm

NORM_CASES = [(L, d, dt) for dt in (BF16, F32) for L, d in
              [(1, 1), (3, 2), (5, 3), (7, 64), (1, 256), (33, 257), (9, 1000), (130, 1024), (65, 1410), (64, 1409),
               (21, 2048), (17, 4096), (3, 4100), (4, 8192), (2, 16384), (2, 33000), (2, 9001), (700, 1411),
               (3, 8191), (5, 700), (2, 5001)]]


def _norm_inputs(L, d, dt, seed, offset=0.5):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return ((r(L, d) * (1 + 5 * (torch.rand(d, generator=g) < 0.05)) + offset).to(dt).cuda(), r(L, d).to(dt).cuda(),
            (1 + 0.2 * r(d)).cuda(), (0.3 * r(d)).cuda(), r(L, d).to(dt).cuda(), r(L, d).to(dt).cuda())


def _check_fwd(got, x, res, w, b, eps, dt):
    y, s, mean, rstd = got
    yr, sr, mr, rr = R.norm(x, res, w, b, eps)
    d = x.shape[1]
    n = 48 + d / 1024                                      # additions in a row of a thread and of the tree
    smax = sr.abs().amax(1, keepdim=True)
    emu = n * U * smax[:, 0]
    R.inside(mean, mr, emu + 1e-30, "mean")
    # the variance: n steps of the sum of squares, and the mean's error (second order, bounded by its square)
    var = 1 / rr ** 2
    er = rr * (0.5 * (2 * n * U + emu ** 2 * rr ** 2 + 4 * U * smax[:, 0] * rr) + 4 * U)
    R.inside(rstd, rr, er + 1e-30, "rstd")
    del var
    xh = (sr - mr[:, None]).abs() * rr[:, None]
    e = R.d64(w).abs() * ((emu + 2 * U * smax[:, 0])[:, None] * rr[:, None] + xh * (er / rr)[:, None]) \
        + 4 * U * (yr.abs() + xh * R.d64(w).abs())
    R.inside(y, yr, R.HALF[dt] * (yr.abs() + e) + e + 1e-30, "y")
    if res is not None:
        R.inside(s, sr, R.HALF[dt] * sr.abs() + U * sr.abs(), "s")


@pytest.mark.parametrize("residual,bias", [(True, True), (False, False)])
@pytest.mark.parametrize("L,d,dt", NORM_CASES)
def test_norm_forward(L, d, dt, residual, bias):
    x, res, w, b, _, _ = _norm_inputs(L, d, dt, L * 7 + d)
    norm = LayerNorm(L, d, dt, eps=1e-5)
    got = norm.forward(x, w, b if bias else None, res if residual else None)
    torch.cuda.synchronize()
    assert (got[1] is x) == (not residual)
    _check_fwd(got, x, res if residual else None, w, b if bias else None, 1e-5, dt)


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("L,d,dt", NORM_CASES + [(2500, 96, BF16), (2500, 520, F32), (1300, 2048, BF16)])
def test_norm_backward(L, d, dt, residual):
    x, _, w, _, dy, ds = _norm_inputs(L, d, dt, L * 5 + d)
    ds = ds if residual else None
    _, _, mean, rstd = R.norm(x, None, w, None, 1e-5)
    mean, rstd = mean.float().cuda(), rstd.float().cuda()
    norm = LayerNorm(L, d, dt)
    dx, dw, db = norm.backward(dy, x, mean, rstd, w, ds)
    torch.cuda.synchronize()
    dxr, dwr, dbr, xh, g = R.norm_grad(dy, x, mean, rstd, w, ds)
    n = 48 + d / 1024
    rs, mu = R.d64(rstd)[:, None], R.d64(mean)[:, None]
    gm, xm, gx = (v.abs().amax(1, keepdim=True) for v in (g, xh, g * xh))
    exh = 3 * U * (R.d64(x).abs().amax(1, keepdim=True) + mu.abs()) * rs + 3 * U * xm     # error of xh
    mgx = (g * xh).mean(1, keepdim=True).abs()
    e = rs * (n * U * gm + xm * (n * U * gx + gm * exh) + exh * mgx + 8 * U * (gm + xm * mgx))
    tot = dxr.abs() + e
    R.inside(dx, dxr, R.HALF[dt] * tot + e + 4 * U * tot + (4 * U * R.d64(ds).abs() if residual else 0), "dx")
    m = 64 + L / 64                                        # rows of a CTA in a row, then the partial sums
    dya = R.d64(dy).abs()
    R.inside(dw, dwr, m * U * (dya * xh.abs()).sum(0) + (dya * exh).sum(0), "dw")
    R.inside(db, dbr, m * U * dya.sum(0), "db")


@pytest.mark.parametrize("offset", [100.0, 1000.0])
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("L,d,dt", [(300, 64, F32), (300, 96, F32), (300, 133, F32), (300, 1024, F32), (300, 1409, F32),
                                    (40, 8190, F32), (40, 33000, F32), (300, 64, BF16), (300, 138, BF16), (300, 1024, BF16),
                                    (300, 4096, BF16), (300, 5120, BF16), (300, 8191, BF16)])
def test_norm_backward_of_rows_with_an_offset(L, d, dt, residual, offset):
    """Rows whose offset is many times their spread: x - mean keeps what a difference of products would round off."""
    x, _, w, _, dy, ds = _norm_inputs(L, d, dt, L * 5 + d, offset)
    ds = ds if residual else None
    _, _, mean, rstd = R.norm(x, None, w, None, 1e-5)
    mean, rstd = mean.float().cuda(), rstd.float().cuda()
    dx, dw, db = LayerNorm(L, d, dt).backward(dy, x, mean, rstd, w, ds)
    torch.cuda.synchronize()
    dxr, dwr, dbr, xh, g = R.norm_grad(dy, x, mean, rstd, w, ds)
    n = 48 + d / 1024
    rs = R.d64(rstd)[:, None]
    gm, xm, gx = (v.abs().amax(1, keepdim=True) for v in (g, xh, g * xh))
    exh = 2 * U * xm                                       # x - mean, and its product with rstd, rounded once each
    mgx = (g * xh).mean(1, keepdim=True).abs()
    e = rs * (n * U * gm + xm * (n * U * gx + gm * exh) + exh * mgx + 8 * U * (gm + xm * mgx))
    tot = dxr.abs() + e
    R.inside(dx, dxr, R.HALF[dt] * tot + e + 4 * U * tot + (4 * U * R.d64(ds).abs() if residual else 0), "dx")
    m = 64 + L / 64
    dya = R.d64(dy).abs()
    R.inside(dw, dwr, m * U * (dya * xh.abs()).sum(0) + (dya * exh).sum(0), "dw")
    R.inside(db, dbr, m * U * dya.sum(0), "db")


def test_norm_gradient_against_differences():
    L, d = 6, 200
    x, _, w, b, dy, _ = _norm_inputs(L, d, F32, 3)
    norm = LayerNorm(L, d, F32)
    _, s, mean, rstd = norm.forward(x, w, b)
    dx, dw, db = norm.backward(dy, s, mean, rstd, w)
    torch.cuda.synchronize()
    g = torch.Generator().manual_seed(9)
    h = 1e-5
    f = lambda xx, ww, bb: (R.norm(xx, None, ww, bb, 1e-5)[0] * R.d64(dy)).sum()  # noqa: E731
    for grad, at in ((dx, 0), (dw, 1), (db, 2)):
        v = torch.randn(grad.shape, generator=g).double()
        args = [R.d64(x), R.d64(w), R.d64(b)]
        up, dn = list(args), list(args)
        up[at], dn[at] = args[at] + h * v, args[at] - h * v
        want = float((f(*up) - f(*dn)) / (2 * h))
        got = float((R.d64(grad) * v).sum())
        # third-order term of the difference and the kernel's fp32 sums
        assert abs(got - want) <= 1e-5 * (R.d64(grad).abs() * v.abs()).sum(), (at, got, want)


def test_norm_in_place_sum_and_extremes():
    L, d = 9, 1536
    x, res, w, b, _, _ = _norm_inputs(L, d, BF16, 11)
    shape = B.make_shape(L, d, 0, 1, 1, BF16, "identity")
    outs = []
    for place in range(3):  # sum into its own tensor, over the residual, over x
        xx, rr = x.clone(), res.clone()
        s = (torch.empty_like(x), rr, xx)[place]
        y, mean, rstd = torch.empty_like(x), torch.empty(L, device="cuda"), torch.empty(L, device="cuda")
        B.layernorm_forward(shape, xx, rr, w, b, 1e-5, s, y, mean, rstd)
        outs.append((s, y, mean, rstd))
    for o in outs[1:]:
        assert all(torch.equal(a, c) for a, c in zip(o, outs[0]))
    # a constant row: variance 0, y = b;  a row with a large offset keeps its spread
    x32 = torch.randn(3, 4096, device="cuda")
    x32[0] = 7.25
    x32[1] += 1000.0
    wf, bf = torch.ones(4096, device="cuda"), torch.full((4096,), 0.5, device="cuda")
    norm = LayerNorm(3, 4096, F32)
    got = norm.forward(x32, wf, bf)
    assert torch.equal(got[0][0], bf)
    _check_fwd(got, x32, None, wf, bf, 1e-5, F32)
    # NaN and inf stay in their row
    x32[1, 5] = float("nan")
    x32[2, 7] = float("inf")
    y = norm.forward(x32, wf, bf)[0]
    assert y[1].isnan().all() and y[2].isnan().any() and torch.equal(y[0], bf)


@pytest.mark.parametrize("L,d,dt", [(9000, 65, BF16), (9000, 138, BF16), (4000, 1701, BF16), (700, 4100, BF16),
                                    (700, 4700, BF16), (400, 8191, BF16), (9000, 35, F32), (9000, 133, F32),
                                    (700, 4099, F32), (400, 8190, F32)])
def test_norm_rows_that_share_words(L, d, dt):
    """Rows that do not start on 16 bytes, several to a CTA; the sum written over the residual changes nothing else."""
    for residual in (True, False):
        test_norm_forward(L, d, dt, residual, True)
        test_norm_backward(L, d, dt, residual)
    x, res, w, b, _, _ = _norm_inputs(L, d, dt, d)
    norm = LayerNorm(L, d, dt)
    y, s, mean, rstd = (t.clone() for t in norm.forward(x, w, b, res))
    B.layernorm_forward(norm.shape, x, res, w, b, norm.eps, res, norm.y, norm.mean, norm.rstd)
    assert torch.equal(res, s) and torch.equal(norm.y, y)
    assert torch.equal(norm.mean, mean) and torch.equal(norm.rstd, rstd)


def test_norm_no_tokens_and_repeatable():
    norm = LayerNorm(0, 512, BF16)
    e = torch.empty(0, 512, dtype=BF16, device="cuda")
    w = torch.ones(512, device="cuda")
    norm.forward(e, w)
    norm.dw.fill_(3)
    _, dw, db = norm.backward(e, e, norm.mean, norm.rstd, w)
    assert not dw.any() and not db.any()
    x, _, w, _, dy, ds = _norm_inputs(3000, 768, BF16, 5)
    norm = LayerNorm(3000, 768, BF16)
    _, s, mean, rstd = norm.forward(x, w)
    a = [t.clone() for t in norm.backward(dy, s, mean, rstd, w, ds)]
    norm.dw.fill_(float("nan"))
    assert all(torch.equal(u, v) for u, v in zip(a, norm.backward(dy, s, mean, rstd, w, ds)))


# ------------------------------------------------------------------ router losses

BALANCE_CASES = [(1, 1, 1), (1, 8, 2), (5, 3, 2), (200, 5, 3), (1000, 8, 2), (513, 12, 4), (700, 16, 1), (999, 33, 5),
                 (640, 64, 6), (300, 100, 8), (777, 128, 8), (257, 130, 3), (129, 256, 8), (70, 401, 2), (66, 512, 8)]


def _balance_inputs(L, E, K, seed):
    g = torch.Generator().manual_seed(seed)
    lg = 1.5 * torch.randn(L, E, generator=g) + torch.randn(E, generator=g)
    top = torch.topk(lg, K, dim=1)
    return (lg, top.indices.int().contiguous(), torch.softmax(top.values, 1).contiguous(),
            torch.randn(L, K, generator=g), (torch.rand(L, generator=g) < 0.8).to(torch.uint8))


def _check_balance(lg, ids, valid, gates, dg, dlosses=(0.7, -0.3)):
    L, E = lg.shape
    K = ids.shape[1]
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    loss = BalanceLoss(L, E, K)
    losses, counts = loss.forward(c(lg), c(ids), c(valid))
    dl = torch.tensor(dlosses, device="cuda")
    out = loss.backward(c(lg), dl, c(valid), *(map(c, (ids, gates, dg)) if gates is not None else ()))
    torch.cuda.synchronize()
    want, cnt, n, lse, active, p = R.balance(lg, ids, valid)
    assert torch.equal(counts.cpu().long(), cnt) and int(loss.active) == n
    # exp of a difference of numbers up to M: its error is that of the difference, (2 M + 4) half steps
    M = float(lg[active][~torch.isinf(lg[active])].abs().max()) if n else 0.0
    ep = (4 * M + 24 + E / 8) * U
    tol = torch.stack([want[0] * (ep + (64 + L / 64) * U),
                       want[1] * (64 + L / 64) * U + 2 * float(lse[active].abs().max() if n else 0) * (M + 8) * 4 * U])
    R.inside(losses, want, tol + 1e-12, "losses")
    dref, scale = R.balance_grad(lg, ids, valid, dlosses, gates, dg)
    R.inside(out, dref, (2 * ep + 32 * U) * scale + 1e-30, "dlogits")
    return out


@pytest.mark.parametrize("masked,with_gates", [(False, True), (True, True), (True, False)])
@pytest.mark.parametrize("L,E,K", BALANCE_CASES)
def test_balance(L, E, K, masked, with_gates):
    lg, ids, gates, dg, valid = _balance_inputs(L, E, K, 3 * L + E)
    _check_balance(lg, ids, valid if masked else None, gates if with_gates else None, dg if with_gates else None)


def test_balance_long_and_even_load():
    # many tokens per CTA, and a load so even that f - sum f p nearly cancels
    L, E, K = 40000, 8, 1
    g = torch.Generator().manual_seed(1)
    lg = 0.01 * torch.randn(L, E, generator=g)
    ids = (torch.arange(L) % E).int()[:, None].contiguous()
    ids[0] = 3
    _check_balance(lg, ids, None, None, None, (1.0, 0.0))


def test_balance_masked_values():
    """-inf logits (masked experts), rows of nothing but -inf, the type's lowest value, and NaN or inf in tokens
    that are not valid."""
    L, E, K = 64, 8, 2
    lg, ids, gates, dg, _ = _balance_inputs(L, E, K, 77)
    lg[:, 5] = -float("inf")
    lg[3] = -float("inf")
    lg[4, 1:] = torch.finfo(F32).min
    lg[6, :7] = -float("inf")
    ids[9, 1] = -1                      # an empty slot
    ids[10, 0] = E + 3
    valid = torch.ones(L, dtype=torch.uint8)
    valid[20:30] = 0
    ok = lg.clone()
    lg[20] = float("nan")
    lg[21, 2] = float("inf")
    a = _check_balance(ok, ids, valid, gates, dg)
    gates[22], dg[23] = float("nan"), float("inf")
    loss = BalanceLoss(L, E, K)
    losses, counts = loss.forward(lg.cuda(), ids.cuda(), valid.cuda())
    b = loss.backward(lg.cuda(), torch.tensor([0.7, -0.3], device="cuda"), None, ids.cuda(), gates.cuda(), dg.cuda())
    assert torch.equal(a, b) and losses.isfinite().all()
    # NaN in a token that counts reaches the losses
    lg[0, 0] = float("nan")
    losses, _ = loss.forward(lg.cuda(), ids.cuda(), valid.cuda())
    assert losses.isnan().all()


def test_balance_nothing_active():
    L, E, K = 40, 6, 2
    lg, ids, gates, dg, _ = _balance_inputs(L, E, K, 5)
    for L2, valid in ((L, torch.zeros(L, dtype=torch.uint8)), (0, None)):
        loss = BalanceLoss(L2, E, K)
        losses, counts = loss.forward(lg[:L2].cuda(), ids[:L2].cuda(), None if valid is None else valid.cuda())
        out = loss.backward(lg[:L2].cuda(), torch.ones(2, device="cuda"), None, ids[:L2].cuda(), gates[:L2].cuda(),
                            dg[:L2].cuda())
        assert not losses.any() and not counts.any() and int(loss.active) == 0 and not out.any()


def test_balance_gradient_against_differences():
    L, E, K = 12, 6, 2
    lg, ids, _, _, valid = _balance_inputs(L, E, K, 8)
    loss = BalanceLoss(L, E, K)
    loss.forward(lg.cuda(), ids.cuda(), valid.cuda())
    out = R.d64(loss.backward(lg.cuda(), torch.tensor([0.9, 0.4], device="cuda")))
    v = torch.randn(L, E, generator=torch.Generator().manual_seed(2)).double()
    h = 1e-5
    f = lambda z: float((R.balance(z, ids, valid)[0] * torch.tensor([0.9, 0.4]).double()).sum())  # noqa: E731
    want = (f(lg.double() + h * v) - f(lg.double() - h * v)) / (2 * h)
    assert abs(float((out * v).sum()) - want) <= 1e-5 * float((out.abs() * v.abs()).sum())


# ------------------------------------------------------------------ router gradient and logits

@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("L,d,E", [(1, 64, 1), (5, 64, 3), (64, 192, 8), (65, 1024, 8), (1000, 576, 7), (300, 640, 16),
                                   (129, 64, 12), (257, 256, 17), (500, 320, 32), (333, 448, 64), (200, 128, 100),
                                   (130, 192, 128), (70, 64, 200), (100, 128, 256), (4097, 64, 40), (9000, 64, 8)])
def test_router_grad(L, d, E, dt):
    g = torch.Generator().manual_seed(L + d + E)
    x = torch.randn(L, d, generator=g).to(dt).cuda()
    Wr = torch.randn(d, E, generator=g).cuda()
    dl = torch.randn(L, E, generator=g).cuda()
    grad = RouterGrad(L, d, E, dt)
    dx, dWr, db = grad.backward(x, Wr, dl)
    torch.cuda.synchronize()
    X, W, D = R.d64(x), R.d64(Wr), R.d64(dl)
    sx = D.abs() @ W.abs().t()
    # bf16 outputs are formed from two-part products at least: 2^-15 of the terms
    R.inside(dx, D @ W.t(), R.HALF[dt] * (D @ W.t()).abs() + ((E + 16) * U + (2.0 ** -15 if dt == BF16 else 0)) * sx,
             "dx")
    n = 128 + L / 16
    R.inside(dWr, X.t() @ D, n * U * (X.abs().t() @ D.abs()), "dWr")
    R.inside(db, D.sum(0), n * U * D.abs().sum(0), "dbias")
    a = [t.clone() for t in (dx, dWr, db)]
    assert all(torch.equal(u, v) for u, v in zip(a, grad.backward(x, Wr, dl)))


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("L,d,E", [(70, 64, 65), (1000, 576, 100), (4097, 320, 128), (2, 64, 128), (600, 128, 129),
                                   (31, 192, 24), (2500, 1088, 33), (5000, 2048, 90)])
def test_router_grad_groups_of_experts(L, d, E, dt):
    test_router_grad(L, d, E, dt)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("L,d,E", [(70, 64, 8), (333, 448, 64), (300, 320, 100), (1000, 576, 7)])
def test_router_grad_added_to_a_gradient(L, d, E, dt):
    g = torch.Generator().manual_seed(L + d + E)
    x = torch.randn(L, d, generator=g).to(dt).cuda()
    Wr = torch.randn(d, E, generator=g).cuda()
    dl = torch.randn(L, E, generator=g).cuda()
    base = torch.randn(L, d, generator=g).to(dt).cuda()
    grad = RouterGrad(L, d, E, dt)
    into = base.clone()
    dx, dWr, _ = grad.backward(x, Wr, dl, add_to=into)
    assert dx is into
    part = R.d64(dl) @ R.d64(Wr).t()
    want = part + R.d64(base)
    sx = R.d64(dl).abs() @ R.d64(Wr).abs().t()
    h = R.HALF[dt]
    R.inside(dx, want, h * (want.abs() + 2 * part.abs()) + ((E + 16) * U + (2.0 ** -15 if dt == BF16 else 0)) * sx
             + 2 * U * want.abs(), "dx")
    alone, dWr2, _ = grad.backward(x, Wr, dl)
    R.inside(alone, part, h * part.abs() + ((E + 16) * U + (2.0 ** -15 if dt == BF16 else 0)) * sx, "dx alone")


def test_router_grad_without_dx_and_tokens():
    E, d = 20, 128
    shape = B.make_shape(50, d, 0, E, 1, BF16, "identity")
    x, Wr, dl = (torch.randn(*s, device="cuda") for s in ((50, d), (d, E), (50, E)))
    dW, dW2 = torch.empty(d, E, device="cuda"), torch.empty(d, E, device="cuda")
    B.router_backward_logits(shape, x.to(BF16), Wr, dl, dW, None, torch.empty(50, d, dtype=BF16, device="cuda"))
    B.router_backward_logits(shape, x.to(BF16), Wr, dl, dW2, None, None)
    assert torch.equal(dW, dW2)
    grad = RouterGrad(0, d, E, BF16)
    _, dWr, db = grad.backward(x[:0].to(BF16), Wr, dl[:0])
    assert not dWr.any() and not db.any()


@pytest.mark.parametrize("L,d,E,K,dt", [(300, 256, 8, 2, BF16), (300, 512, 64, 6, BF16), (1025, 192, 12, 3, BF16),
                                        (77, 128, 8, 2, BF16), (200, 128, 100, 8, BF16), (150, 64, 5, 2, F32)])
def test_router_logits(L, d, E, K, dt):
    """The logits come with the same ids and gates as without them, from both router calls."""
    g = torch.Generator().manual_seed(4)
    x = torch.randn(L, d, generator=g).to(dt).cuda()
    Wr, b = torch.randn(d, E, generator=g).cuda(), torch.randn(E, generator=g).cuda()
    shape = B.make_shape(L, d, 128, E, K, dt, "identity")
    want = R.d64(x) @ R.d64(Wr) + R.d64(b)
    tol = (d + 16) * U * (R.d64(x).abs() @ R.d64(Wr).abs() + R.d64(b).abs())

    def run(f, logits):
        ids = torch.empty(L, K, dtype=torch.int32, device="cuda")
        gates = torch.empty(L, K, device="cuda")
        f(shape, x, Wr, b, ids, gates, logits=logits)
        return ids, gates

    for f in (B.router_forward, B.router_dispatch_build):
        lg = torch.full((L, E), float("nan"), device="cuda")
        i1, g1 = run(f, lg)
        i0, g0 = run(f, None)
        assert torch.equal(i0, i1) and torch.equal(g0, g1)
        R.inside(lg, want, tol, "logits")
        # the ids are the K largest of these very logits, the lower index first among equals
        order = torch.sort(lg, dim=1, descending=True, stable=True).indices[:, :K]
        assert torch.equal(order.int(), i1)


# ------------------------------------------------------------------ together

def test_block_step_against_differences():
    """One training step of the block in fp32: every parameter's gradient against a difference of the fp64 loss
    <out, dout> + a balance + z z-loss + <s, ds>, with the routing held where the kernels put it."""
    L, d, h, E, K = 48, 64, 64, 4, 2
    g = torch.Generator().manual_seed(6)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    p = {"norm_w": 1 + 0.1 * r(d), "norm_b": 0.1 * r(d), "Wr": r(d, E) / 8, "bias": 0.1 * r(E), "W1": r(E, d, h) / 8,
         "W2": r(E, d, h) / 8, "W3": r(E, h, d) / 8}
    x, res, dout, ds = r(L, d), r(L, d), r(L, d), r(L, d)
    dev = {k: v.cuda() for k, v in p.items()}
    block = MoEBlock(L, d, h, E, K, F32)
    out, s, losses, counts = block.forward(x.cuda(), res.cuda(), dev)
    ids = block._kept[4].cpu().long()
    coef = (0.8, 0.05)
    grads = block.backward(dout.cuda(), torch.tensor(coef, device="cuda"), dev, ds.cuda())
    torch.cuda.synchronize()
    f_e = torch.bincount(ids.flatten(), minlength=E).double() / (L * K)

    def loss(q, xx):
        u, ss, _, _ = R.norm(xx, res, q["norm_w"], q["norm_b"], 1e-5)
        lg = u @ R.d64(q["Wr"]) + R.d64(q["bias"])
        gt = torch.softmax(torch.gather(lg, 1, ids), 1)
        hid = R.silu(torch.einsum("td,edh->teh", u, R.d64(q["W1"]))) * torch.einsum("td,edh->teh", u, R.d64(q["W2"]))
        full = torch.einsum("teh,ehd->ted", hid, R.d64(q["W3"]))
        y = (torch.gather(full, 1, ids[:, :, None].expand(L, K, d)) * gt[:, :, None]).sum(1)
        pr, lse = torch.softmax(lg, 1), torch.logsumexp(lg, 1)
        return float((y * dout.double()).sum() + coef[0] * E * (f_e * pr.mean(0)).sum() + coef[1] * (lse ** 2).mean()
                     + (ss * ds.double()).sum()), y

    q = {k: v.double() for k, v in p.items()}
    y = loss(q, x.double())[1]
    assert (R.d64(out) - y).abs().max() <= 1e-4 * y.abs().max()
    step = 1e-5
    for name, grad in grads.items():
        v = r(*grad.shape).double()
        if name == "x":
            want = (loss(q, x.double() + step * v)[0] - loss(q, x.double() - step * v)[0]) / (2 * step)
        else:
            up, dn = dict(q), dict(q)
            up[name], dn[name] = q[name] + step * v, q[name] - step * v
            want = (loss(up, x.double())[0] - loss(dn, x.double())[0]) / (2 * step)
        got = float((R.d64(grad) * v).sum())
        assert abs(got - want) <= 2e-5 * float((R.d64(grad).abs() * v.abs()).sum()), (name, got, want)


def test_block_bf16_on_another_stream_and_in_a_graph():
    """The bf16 block on a side stream, and captured in a graph while nothing else runs: the same results."""
    L, d, h, E, K = 300, 256, 256, 8, 2
    g = torch.Generator().manual_seed(16)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    p = {"norm_w": 1 + 0.1 * r(d), "norm_b": 0.1 * r(d), "Wr": r(d, E) / 16}
    dev = {k: v.cuda() for k, v in p.items()}
    dev.update({k: (r(E, *s) / 16).to(BF16).cuda() for k, s in (("W1", (d, h)), ("W2", (d, h)), ("W3", (h, d)))})
    x, res, dout = (r(L, d).to(BF16).cuda() for _ in range(3))
    dl = torch.tensor([0.01, 0.001], device="cuda")
    block = MoEBlock(L, d, h, E, K, BF16)

    def step():
        out, s, losses, counts = block.forward(x, res, dev)
        grads = block.backward(dout, dl, dev)
        return [out, s, losses, counts] + [grads[k] for k in ("x", "norm_w", "norm_b", "Wr", "bias", "W1", "W3")]

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = [t.clone() for t in step()]
    side.synchronize()
    # dgates are summed by float atomics: what depends on them agrees to fp32 (bf16 for x) rounding, the rest exactly
    loose = {4: 2.0 ** -7, 5: 1e-4, 6: 1e-4, 7: 1e-4, 8: 1e-4}
    for i, (a, b) in enumerate(zip(got, want)):
        if i in loose:
            assert (a.float() - b.float()).abs().max() <= loose[i] * b.float().abs().max(), i
        else:
            assert torch.equal(a, b), i
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for t in outs:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(zip(outs, want)):
        if i in loose:
            assert (a.float() - b.float()).abs().max() <= loose[i] * b.float().abs().max(), i
        else:
            assert torch.equal(a, b), i
    assert block.layer.device_error() == 0


def test_example_trains_and_serves():
    """The example's training steps lower the error, and its 4-bit batch agrees with the bf16 layer."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")
    spec = importlib.util.spec_from_file_location("moe_block_example", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    p, history = m.train(512, 256, 256, 8, 2, 30)
    assert history[-1][0] < 0.98 * history[0][0], history
    assert all(h[1] == h[1] for h in history)
    y4, y16 = m.serve(p, 7, 2, group=64)
    assert (y4.float() - y16.float()).abs().max() <= 2e-2 * y16.float().abs().max()


def test_block_with_a_loss_mask_against_differences():
    """A token left out of the losses is still routed: with a gradient at its output, its gates' gradient reaches
    every parameter before them."""
    L, d, h, E, K = 48, 64, 64, 4, 2
    g = torch.Generator().manual_seed(26)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    p = {"norm_w": 1 + 0.1 * r(d), "norm_b": 0.1 * r(d), "Wr": r(d, E) / 8, "bias": 0.1 * r(E), "W1": r(E, d, h) / 8,
         "W2": r(E, d, h) / 8, "W3": r(E, h, d) / 8}
    x, res, dout, ds = r(L, d), r(L, d), r(L, d), r(L, d)
    coef = (0.8, 0.05)
    for valid in ((torch.arange(L) % 3 != 0).to(torch.uint8), torch.zeros(L, dtype=torch.uint8)):
        dev = {k: v.cuda() for k, v in p.items()}
        block = MoEBlock(L, d, h, E, K, F32)
        out, s, losses, counts = block.forward(x.cuda(), res.cuda(), dev, valid.cuda())
        ids = block._kept[4].cpu().long()
        grads = block.backward(dout.cuda(), torch.tensor(coef, device="cuda"), dev, ds.cuda())
        torch.cuda.synchronize()
        on = valid.bool()
        n = max(1, int(on.sum()))
        f_e = torch.bincount(ids[on].flatten(), minlength=E).double() / (n * K)
        assert torch.equal(counts.cpu().long(), torch.bincount(ids[on].flatten(), minlength=E))

        def loss(q, xx):
            u, ss, _, _ = R.norm(xx, res, q["norm_w"], q["norm_b"], 1e-5)
            lg = u @ R.d64(q["Wr"]) + R.d64(q["bias"])
            gt = torch.softmax(torch.gather(lg, 1, ids), 1)
            hid = R.silu(torch.einsum("td,edh->teh", u, R.d64(q["W1"]))) * torch.einsum("td,edh->teh", u, R.d64(q["W2"]))
            full = torch.einsum("teh,ehd->ted", hid, R.d64(q["W3"]))
            y = (torch.gather(full, 1, ids[:, :, None].expand(L, K, d)) * gt[:, :, None]).sum(1)
            pr, lse = torch.softmax(lg, 1)[on], torch.logsumexp(lg, 1)[on]
            return float((y * dout.double()).sum() + coef[0] * E * (f_e * pr.sum(0) / n).sum()
                         + coef[1] * (lse ** 2).sum() / n + (ss * ds.double()).sum())

        q = {k: v.double() for k, v in p.items()}
        step = 1e-5
        for name, grad in grads.items():
            v = r(*grad.shape).double()
            if name == "x":
                want = (loss(q, x.double() + step * v) - loss(q, x.double() - step * v)) / (2 * step)
            else:
                up, dn = dict(q), dict(q)
                up[name], dn[name] = q[name] + step * v, q[name] - step * v
                want = (loss(up, x.double()) - loss(dn, x.double())) / (2 * step)
            got = float((R.d64(grad) * v).sum())
            assert abs(got - want) <= 2e-5 * float((R.d64(grad).abs() * v.abs()).sum()), (name, got, want)


def test_balance_gates_of_all():
    """The gates' share of tokens that are out of the losses, with masks of both kinds; the others' rows as without."""
    for L, E, K in ((5, 3, 2), (700, 8, 2), (333, 64, 6), (90, 100, 8), (70, 512, 8)):
        lg, ids, gates, dg, valid = _balance_inputs(L, E, K, 9 * L)
        lg[2] = -float("inf")
        ids[3, 0] = -1
        c = [t.cuda() for t in (lg, ids, gates, dg, valid)]
        loss = BalanceLoss(L, E, K)
        loss.forward(c[0], c[1], c[4])
        dl = torch.tensor([0.7, -0.3], device="cuda")
        some = loss.backward(c[0], dl, None, c[1], c[2], c[3]).clone()
        every = loss.backward(c[0], dl, None, c[1], c[2], c[3], gates_of_all=True).cpu()
        on = valid.bool() & (torch.arange(L) != 2)
        assert torch.equal(every[on], some.cpu()[on]) and not some[~on.cuda()].any()
        g, d = R.d64(gates), R.d64(dg)
        sd, sa = (g * d).sum(1, keepdim=True), (g * d).abs().sum(1, keepdim=True)
        want, scale = torch.zeros(L, E + 1).double(), torch.zeros(L, E + 1).double()
        slot = torch.where(ids >= 0, ids, torch.tensor(E, dtype=torch.int32)).long()
        want.scatter_add_(1, slot, g * (d - sd))
        scale.scatter_add_(1, slot, g.abs() * (d.abs() + sa))
        R.inside(every[~on], want[~on, :E], (K + 4) * U * scale[~on, :E] + 1e-30, "gates' share")
        assert torch.equal(loss.backward(c[0], dl, gates_of_all=True), loss.backward(c[0], dl))


def test_balance_backward_mask():
    """A mask given to backward leaves tokens out besides the forward's; a malformed one is refused."""
    for L, E, K in ((40, 6, 2), (700, 8, 2), (333, 64, 6), (90, 130, 3)):
        lg, ids, gates, dg, valid = _balance_inputs(L, E, K, 4 * L)
        more = torch.ones(L, dtype=torch.uint8)
        more[::3] = 0
        c = [t.cuda() for t in (lg, ids, gates, dg, valid, more)]
        loss = BalanceLoss(L, E, K)
        dl = torch.tensor([0.7, -0.3], device="cuda")
        loss.forward(c[0], c[1], c[4])
        want = loss.backward(c[0], dl, None, *c[1:4]).clone()
        assert torch.equal(loss.backward(c[0], dl, c[4], *c[1:4]), want)
        share = loss.backward(c[0], dl, None, *c[1:4], gates_of_all=True).clone()
        both = loss.backward(c[0], dl, c[5], *c[1:4], gates_of_all=True).clone()
        out = loss.backward(c[0], dl, c[5], *c[1:4])
        assert not out[::3].any() and torch.equal(out[more.bool()], want[more.bool()])
        assert torch.equal(both[more.bool()], share[more.bool()])
        gone = torch.zeros_like(valid).cuda()
        assert torch.equal(both[::3], loss.backward(c[0], dl, gone, *c[1:4], gates_of_all=True)[::3])
    with pytest.raises(ValueError, match="valid: dtype"):
        loss.backward(c[0], dl, c[4].bool())
    with pytest.raises(ValueError, match="valid: shape"):
        loss.backward(c[0], dl, c[4][:-1])


@pytest.mark.parametrize("L,dt", [(300, BF16), (40, F32)])
def test_block_with_tokens_that_are_not_finite(L, dt):
    """Padding tokens that hold NaN or infinities, left out of the losses: the other tokens' rows and the losses are
    those of a batch whose padding is finite."""
    d, h, E, K = 128, 128, 8, 2
    g = torch.Generator().manual_seed(41)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    p = {"norm_w": 1 + 0.1 * r(d), "norm_b": 0.1 * r(d), "Wr": r(d, E) / 8, "bias": 0.1 * r(E)}
    dev = {k: v.cuda() for k, v in p.items()}
    dev.update({k: (r(E, *s) / 11).to(dt).cuda() for k, s in (("W1", (d, h)), ("W2", (d, h)), ("W3", (h, d)))})
    x, res, dout = (r(L, d).to(dt).cuda() for _ in range(3))
    valid = torch.ones(L, dtype=torch.uint8, device="cuda")
    valid[-9:] = 0
    dout[-9:] = 0
    dl = torch.tensor([0.01, 0.001], device="cuda")
    on = valid.bool()
    outs = []
    for bad in (False, True):
        xx = x.clone()
        if bad:
            xx[-1], xx[-2, 3], xx[-3, 5] = float("nan"), float("inf"), -float("inf")
        block = MoEBlock(L, d, h, E, K, dt)
        out, s, losses, counts = block.forward(xx, res, dev, valid)
        grads = block.backward(dout, dl, dev)
        assert block.layer.device_error() == 0
        outs.append([t.clone() for t in (out[on], s[on], losses, counts, grads["x"][on])])
    good, mixed = outs
    assert mixed[0].isfinite().all() and mixed[4].isfinite().all()
    for a, b in zip(good[1:4], mixed[1:4]):
        assert torch.equal(a, b)
    # (sums of two terms, the gate gradients by atomics: fp32 rounding, and bf16's)
    for i in (0, 4):
        assert (good[i].float() - mixed[i].float()).abs().max() <= 2.0 ** -7 * good[i].float().abs().max()
