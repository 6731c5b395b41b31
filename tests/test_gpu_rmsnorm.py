"""The root-mean-square norm, its rows in 8-bit floating point and its backward
on the GPU against their fp64 definitions (eight_ref).  Tolerances are
elementwise: the rounding of the output type plus fp32 error bounds of the sums
involved (number of additions in a row x half a step x the terms' sizes)."""
import pytest
import torch

import eight_ref as R
from mixture_experts_atomic_gb300 import binding as B
from mixture_experts_atomic_gb300 import fp8
from mixture_experts_atomic_gb300.block import MoEBlock, RMSNorm

pytestmark = pytest.mark.gpu

from gpu_util import ensure_built  # noqa: E402

U = R.U32
BF16, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


CASES = [(L, d, dt) for dt in (BF16, F32) for L, d in
         [(1, 1), (3, 2), (5, 3), (7, 64), (1, 256), (33, 257), (9, 1000), (130, 1024), (65, 1410), (64, 1409), (21, 2048),
          (17, 4096), (3, 4100), (4, 8192), (2, 16384), (2, 33000), (2, 9001), (700, 1411), (3, 8191), (5, 700), (2, 5001),
          (4000, 65), (3000, 1409)]]
CASES8 = [(L, d, dt) for dt in (BF16, F32) for L, d in
          [(1, 16), (3, 32), (5, 112), (7, 128), (1, 144), (33, 256), (9, 1008), (130, 1024), (65, 1408), (21, 2048),
           (17, 4096), (3, 4112), (4, 8192), (2, 16384), (2, 33008), (2, 65536), (700, 528), (5, 6160)]]


def _inputs(L, d, dt, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return [t.cuda() for t in ((r(L, d) * (1 + 9 * (torch.rand(d, generator=g) < 0.05)) + 0.5).to(dt), r(L, d).to(dt),
                               1 + 0.2 * r(d), r(L, d).to(dt), r(L, d).to(dt))]


def _rel(d):
    """Relative error of rstd: the additions of squares in a row of a thread and of the tree, and its own operations."""
    return (0.5 * (48 + d / 1024) + 4) * U


def _check_fwd(got, x, res, w, eps, dt):
    y, s, rstd = got
    yr, sr, rr = R.rms(x, res, w, eps)
    e = _rel(x.shape[1]) + U  # (the sum s itself is rounded to fp32 once)
    R.inside(rstd, rr, 2 * e * rr, "rstd")
    if y is not None:
        R.inside(y, yr, (R.HALF[dt] * (1 + 1e-3) + 2 * e + 4 * U) * yr.abs() + 1e-37, "y")
    R.inside(s, sr, (R.HALF[dt] + U) * sr.abs(), "s")
    return yr, 2 * e + 4 * U


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("L,d,dt", CASES)
def test_rms_forward(L, d, dt, residual):
    x, res, w, _, _ = _inputs(L, d, dt, L * 7 + d)
    res = res if residual else None
    got = RMSNorm(L, d, dt, eps=1e-5).forward(x, w, res)
    torch.cuda.synchronize()
    assert (got[1] is x) == (not residual)
    _check_fwd(got, x, res, w, 1e-5, dt)


def _check8(q, scales, want, rel):
    """8-bit rows of fp32 values that are off by rel: each within half a step of what it stands for, and scales that
    bring the block's largest into the top binade."""
    L, d = q.shape
    sc = R.grown(scales, d)
    vals = q.float().double() * sc
    off = rel * want.abs()
    # half a step: 2^-4 of the value (of the upper end of what fp32 may have made of it), or of the subnormals' 2^-9
    tol = torch.maximum(R.HALF[F8] * (want.abs() + off), sc * 2.0 ** -10) + off
    R.inside(vals, want, tol, "8-bit rows")
    top = R.blocks(want).abs().amax(2)
    sd = scales.double()
    assert bool((torch.frexp(sd)[0] == 0.5).all()), "scales are powers of two"
    assert bool((top * (1 - rel) <= 448 * sd).all())
    small = sd <= 2.0 ** -126
    assert bool(((top * (1 + rel) > 224 * sd) | small).all())


@pytest.mark.parametrize("residual,with_y", [(True, True), (False, False), (False, True)])
@pytest.mark.parametrize("L,d,dt", CASES8)
def test_rms_forward_in_8_bits(L, d, dt, residual, with_y):
    x, res, w, _, _ = _inputs(L, d, dt, L * 3 + d)
    res = res if residual else None
    norm = RMSNorm(L, d, dt, eps=1e-5)
    q, scales, y, s, rstd = norm.forward8(x, w, res, with_y)
    torch.cuda.synchronize()
    assert (y is None) == (not with_y) and q.dtype == F8 and scales.shape == (L, B.blocks8(d))
    yr, rel = _check_fwd((y, s, rstd), x, res, w, 1e-5, dt)
    _check8(q, scales, yr, rel)
    a, b, c = q.clone(), scales.clone(), rstd.clone()
    y2, s2, r2 = norm.forward(x, w, res)                    # the same statistics and rows without the 8-bit ones
    assert torch.equal(r2, c) and (y is None or torch.equal(y2, y))
    vals = fp8.dequantize_rows(a, b)
    assert torch.equal(vals.float(), (a.float().double() * R.grown(b, d)).float())


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("L,d,dt", CASES + [(2500, 96, BF16), (2500, 520, F32), (1300, 2048, BF16), (1200, 7168, BF16)])
def test_rms_backward(L, d, dt, residual):
    x, _, w, dy, ds = _inputs(L, d, dt, L * 5 + d)
    ds = ds if residual else None
    rstd = R.rms(x, None, w, 1e-5)[2].float()
    dx, dw = RMSNorm(L, d, dt).backward(dy, x, rstd, w, ds)
    torch.cuda.synchronize()
    dxr, dwr, xh, g = R.rms_grad(dy, x, rstd, w, ds)
    n = 48 + d / 1024
    rs = rstd.double()[:, None]
    gx = (g * xh).abs()
    mgx = (g * xh).mean(1, keepdim=True).abs()
    e = rs * (xh.abs() * (n + 4) * U * gx.mean(1, keepdim=True) + 8 * U * (g.abs() + xh.abs() * mgx))
    tot = dxr.abs() + e
    R.inside(dx, dxr, R.HALF[dt] * tot + e + 4 * U * tot + (4 * U * ds.double().abs() if residual else 0) + 1e-37, "dx")
    m = 64 + L / 64                                        # rows of a CTA in a row, then the partial sums
    R.inside(dw, dwr, (m + 4) * U * (dy.double().abs() * xh.abs()).sum(0) + 1e-37, "dw")
    again = RMSNorm(L, d, dt).backward(dy, x, rstd, w, ds)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


def test_rms_gradient_against_differences():
    L, d = 6, 200
    x, _, w, dy, _ = _inputs(L, d, F32, 3)
    norm = RMSNorm(L, d, F32)
    _, s, rstd = norm.forward(x, w)
    dx, dw = norm.backward(dy, s, rstd, w)
    g = torch.Generator().manual_seed(9)
    h = 1e-5
    f = lambda xx, ww: float((R.rms(xx, None, ww, 1e-5)[0] * dy.double()).sum())  # noqa: E731
    for grad, at in ((dx, 0), (dw, 1)):
        v = torch.randn(grad.shape, generator=g).double().cuda()
        args = [x.double(), w.double()]
        up, dn = list(args), list(args)
        up[at], dn[at] = args[at] + h * v, args[at] - h * v
        want = (f(*up) - f(*dn)) / (2 * h)
        got = float((grad.double() * v).sum())
        # third-order term of the difference and the kernel's fp32 sums
        assert abs(got - want) <= 1e-5 * float((grad.double().abs() * v.abs()).sum()), (at, got, want)


def test_rms_in_place_sum_and_odd_rows():
    L, d = 9, 1536
    x, res, w, _, _ = _inputs(L, d, BF16, 11)
    shape = B.make_shape(L, d, 0, 1, 1, BF16, "identity")
    outs = []
    for place in range(3):  # sum into its own tensor, over the residual, over x
        xx, rr = x.clone(), res.clone()
        s = (torch.empty_like(x), rr, xx)[place]
        y, rstd = torch.empty_like(x), torch.empty(L, device="cuda")
        B.rmsnorm_forward(shape, xx, rr, w, 1e-5, s, y, rstd)
        outs.append((s, y, rstd))
    for o in outs[1:]:
        assert all(torch.equal(a, c) for a, c in zip(o, outs[0]))
    for d in (4096, 33008):
        x32 = torch.randn(6, d, device="cuda")
        x32[0] = 0.0                                       # y = 0 and scales of the least normal number
        x32[1, 5] = float("nan")
        x32[2, 7] = float("inf")
        x32[3] *= 1e-38
        x32[4] *= 1e18
        wf = torch.ones(d, device="cuda")
        q, scales, y, _, rstd = RMSNorm(6, d, F32).forward8(x32, wf)
        v = fp8.dequantize_rows(q, scales, F32)
        assert float(y[0].abs().max()) == 0 and float(v[0].abs().max()) == 0 and bool((scales[0] == 2.0 ** -126).all())
        assert y[1].isnan().all() and v[1].isnan().all() and scales[1].isnan().all()
        assert y[2].isnan().any() and v[2, :128].isnan().all()
        assert bool(y[3:].isfinite().all()) and bool(v[3:].isfinite().all())
        for t in (3, 4, 5):
            yr, _, _ = R.rms(x32[t:t + 1], None, wf, 1e-5)
            _check8(q[t:t + 1], scales[t:t + 1], yr, 2 * (_rel(d) + U) + 4 * U)


@pytest.mark.parametrize("eps", [0.0, 1e-5])
@pytest.mark.parametrize("L,d,dt", [(6, 64, BF16), (6, 65, BF16), (6, 1409, F32), (6, 4096, BF16), (6, 8001, F32),
                                    (6, 33008, F32), (300, 1409, BF16)])
def test_rms_of_rows_far_from_one(L, d, dt, eps):
    """Squares that fp32 does not hold."""
    x, _, w, _, _ = _inputs(L, d, dt, L + d)
    for i, f in enumerate((1e-30, 1e-24, 1.0, 1e18, 1e25, 1e34)):
        x[i] = (x[i].double() * f).to(dt)
    got = RMSNorm(L, d, dt, eps=eps).forward(x, w)
    _check_fwd(got, x, None, w, eps, dt)


def test_rms_empty_batch_and_graph():
    for dt in (BF16, F32):
        norm = RMSNorm(0, 64, dt)
        z = torch.empty(0, 64, dtype=dt, device="cuda")
        w = torch.ones(64, device="cuda")
        q, scales, y, s, rstd = norm.forward8(z, w, z)
        dx, dw = norm.backward(z, z, rstd, w)
        assert q.shape == (0, 64) and scales.shape == (0, 1) and dx.shape == (0, 64) and float(dw.abs().max()) == 0
    L, d = 37, 1024
    x, res, w, dy, ds = _inputs(L, d, BF16, 5)
    x2, res2, _, dy2, ds2 = _inputs(L, d, BF16, 6)
    norm, other = RMSNorm(L, d, BF16), RMSNorm(L, d, BF16)

    def step(n, x, res, dy, ds):
        q, scales, y, s, rstd = n.forward8(x, w, res)
        return (q, scales, y, s, rstd) + tuple(n.backward(dy, s, rstd, w, ds))

    want = [t.clone() for t in step(other, x2, res2, dy2, ds2)]
    step(norm, x, res, dy, ds)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(norm, x, res, dy, ds)
    for a, b in ((x, x2), (res, res2), (dy, dy2), (ds, ds2)):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("L,d", [(1, 16), (3, 112), (5, 128), (2, 144), (100, 1408), (33, 4096), (3, 65536)])
def test_quantize_rows_to_the_bit(L, d, dt):
    """Codes and scales of given values have no rounding of their own before the last: they are the definition's."""
    g = torch.Generator().manual_seed(L + d)
    x = (torch.randn(L, d, generator=g) * torch.exp2(torch.randint(-20, 20, (L, 1), generator=g).float())).to(dt).cuda()
    x[0, 0] = 448.0
    x[0, 1:16] = torch.tensor([17, 19, 21, -17, 0.0009765625, 0.0029296875, -0.0048828125, 1.0625, 1.1875, 0, -0.0, 440,
                               -432, 2.0 ** -10, 2.0 ** -11]).to(dt).cuda()   # ties, subnormals, the ends of the range
    if L > 2:
        x[1] = 0
        x[2] = 2.0 ** -120
        x[2, 0] = 1.75 * 2.0 ** -100                         # 448 times a power of two: the scale is that power
    q, s = fp8.quantize_rows(x)
    qr, sr = R.rows8(x)
    assert torch.equal(s.double(), sr)
    assert torch.equal(q.float().double(), qr)
    assert torch.equal(fp8.dequantize_rows(q, s, F32).double(), (qr * R.grown(sr, d)).float().double())
    s3 = s * 0.3                                             # any scales
    assert torch.equal(fp8.dequantize_rows(q, s3, F32), q.float() * R.grown(s3, d).float())
    x[0, 3], x[L - 1, d - 1] = float("inf"), float("nan")
    q, s = fp8.quantize_rows(x)
    v = fp8.dequantize_rows(q, s, dt)
    assert bool(v[0, :min(128, d)].isnan().all()) and bool(v[L - 1, (d - 1) // 128 * 128:].isnan().all())
    _, sr = R.rows8(x)
    assert torch.equal(s.isnan(), sr.isnan()) and torch.equal(torch.nan_to_num(s), torch.nan_to_num(sr.float()))


def test_block_with_the_rms_norm():
    """One step of the pre-norm block on the RMS norm and 8-bit checkpoints: the norm's outputs feed the layer, and its
    gradient is the norm's backward of the layer's."""
    L, d, h, E, K = 512, 256, 384, 8, 2
    g = torch.Generator(device="cuda").manual_seed(8)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    p = {"norm_w": 1 + 0.1 * r(d), "Wr": r(d, E) / 16, "W1": (r(E, d, h) / 16).to(BF16), "W2": (r(E, d, h) / 16).to(BF16),
         "W3": (r(E, h, d) / 20).to(BF16)}
    x, res, dout, dsum = (r(L, d).to(BF16) for _ in range(4))
    block = MoEBlock(L, d, h, E, K, BF16, checkpoint8=True, norm="rms")
    out, s, losses, counts = block.forward(x, res, p)
    u, s2, rstd = RMSNorm(L, d, BF16).forward(x, p["norm_w"], res)
    assert torch.equal(s, s2)
    ids = block._kept[4].clone()
    want, bound = R.layer_forward(u, ids, block._kept[5], p["W1"], p["W2"], p["W3"])
    R.inside(out, want, bound + R.BF * (want.abs() + bound) + 1e-30, "out")
    grads = block.backward(dout, torch.tensor([0.01, 0.001], device="cuda"), p, dsum)
    assert set(grads) == {"x", "norm_w", "Wr", "bias", "W1", "W2", "W3"}
    dx, dw, _, _ = R.rms_grad(block.layer.dX, s, rstd, p["norm_w"], dsum)
    assert float((grads["x"].double() - dx).norm() / dx.norm()) <= R.BF
    assert float((grads["norm_w"].double() - dw).norm() / dw.norm()) <= 1e-5
    p["norm_b"] = torch.zeros(d, device="cuda")
    with pytest.raises(ValueError, match="norm_b"):
        block.forward(x, res, p)
