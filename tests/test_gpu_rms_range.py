"""The root-mean-square norm on rows whose squares fp32 does not hold, up to the
largest and down to the smallest values of its types: y, rstd, the 8-bit rows
and the backward against fp64 (eight_ref), with tolerances counted as for
ordinary rows (a sum of squares of n additions in a row of a thread, then a tree).
rstd itself is subnormal, half a step 2^-150, for rows of fp32's largest values,
and infinite for rows below 2^-128 without eps."""
import pytest
import torch

import eight_ref as R
from mixture_experts_atomic_gb300 import fp8
from mixture_experts_atomic_gb300.block import RMSNorm

pytestmark = pytest.mark.gpu

from gpu_util import ensure_built  # noqa: E402

U = R.U32
BF16, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _rows(d, dt, seed):
    """Rows of one value and of random signs and sizes, from the largest to the smallest of the type."""
    g = torch.Generator().manual_seed(seed)
    sign = torch.where(torch.rand(d, generator=g) < 0.5, -1.0, 1.0).double()
    size = 0.25 + 0.75 * torch.rand(d, generator=g).double()
    big = 3.38e38                                    # the largest bf16 value is 3.3895e38
    sizes = [big, 3e38, 1e38, 1e37, 1e35, 1e34, 1e25, 1.0, 1e-17, 1e-30, 1e-38, 2e-39]
    sizes += [1e-39, 3e-40] if dt == BF16 else [1e-40, 1e-42, 4e-44]
    rows = [v * sign for v in sizes] + [v * sign * size for v in sizes]
    mixed = 3e38 * sign * size                       # one large value among small ones, and the other way round
    mixed[1:] *= 1e-37
    lone = 1e-30 * sign * size
    lone[0] = 1e30
    return torch.stack(rows + [mixed, lone]).to(dt).cuda()


def _rel(d):
    return 2 * ((0.5 * (48 + d / 1024) + 4) * U + U) + 4 * U


SIZES = [(d, dt) for dt in (BF16, F32) for d in (64, 65, 1408, 1409, 4096, 5001, 8001, 16384, 33008)]


@pytest.mark.parametrize("eps", [0.0, 1e-5])
@pytest.mark.parametrize("d,dt", SIZES)
def test_rms_forward_over_the_whole_range(d, dt, eps):
    x = _rows(d, dt, d)
    L = len(x)
    w = (1 + 0.2 * torch.randn(d, generator=torch.Generator().manual_seed(1))).cuda()
    norm = RMSNorm(L, d, dt, eps=eps)
    y, _, rstd = norm.forward(x, w)
    want, _, rr = R.rms(x, None, w, eps)
    rel = _rel(d)
    y = y.clone()
    # Where y is subnormal: x rstd is rounded to a multiple of 2^-149, by half of it at most, which w then multiplies,
    # and the product is rounded so once more; or, to bf16, to a multiple of 2^-133 (the former 2^-16 of that).
    step = 0.5 * (1 + float(w.abs().max())) * 2.0 ** -149
    least = step + 2.0 ** -134 if dt == BF16 else step
    R.inside(y, want, (R.HALF[dt] * (1 + 1e-3) + rel) * want.abs() + least, "y")
    top = float(torch.finfo(F32).max)
    fits = rr <= top
    R.inside(rstd[fits], rr[fits], rel * rr[fits] + 2.0 ** -149, "rstd")
    assert bool((rstd[~fits] == float("inf")).all())
    if d % 16 == 0:
        q, s, y8, _, rstd8 = norm.forward8(x, w)
        assert torch.equal(y8, y) and torch.equal(rstd8, rstd)
        vals, sc = q.float().double() * R.grown(s, d), R.grown(s, d)
        off = rel * want.abs() + step                # (the fp32 value that is brought to 8 bits, as above)
        R.inside(vals, want, torch.maximum(R.HALF[F8] * (want.abs() + off), sc * 2.0 ** -10) + off, "8-bit rows")
        assert torch.equal(fp8.dequantize_rows(q, s, F32).double(), vals.float().double())


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("d,dt", [(64, BF16), (1409, BF16), (4096, BF16), (1409, F32), (4096, F32), (33008, F32)])
def test_rms_backward_after_the_forward_over_the_whole_range(d, dt, residual):
    """What the forward keeps (its sum and its rstd) gives the gradient of every row whose rstd is a finite number."""
    x = _rows(d, dt, d + 1)
    w = (1 + 0.2 * torch.randn(d, generator=torch.Generator().manual_seed(2))).cuda()
    rr = R.rms(x, None, w, 0.0)[2]
    x = x[rr < 1e36].contiguous()                # (dx is about rstd times dy)
    L = len(x)
    g = torch.Generator().manual_seed(3)
    dy = torch.randn(L, d, generator=g).to(dt).cuda()
    ds = torch.randn(L, d, generator=g).to(dt).cuda() if residual else None
    norm = RMSNorm(L, d, dt, eps=0.0)
    _, s, rstd = norm.forward(x, w)
    rstd = rstd.clone()
    dx, dw = norm.backward(dy, s, rstd, w, ds)
    dxr, dwr, xh, gg = R.rms_grad(dy, x, rstd, w, ds)
    n = 48 + d / 1024
    rs = rstd.double()[:, None]
    mgx = (gg * xh).mean(1, keepdim=True).abs()
    # (the factor of x is rstd mean(g xh) and may be subnormal: half a step 2^-150 of it, times x)
    e = rs * (xh.abs() * (n + 4) * U * (gg * xh).abs().mean(1, keepdim=True) + 8 * U * (gg.abs() + xh.abs() * mgx)
              + 2.0 ** -149 * x.double().abs())
    tot = dxr.abs() + e
    least = 2.0 ** -133 if dt == BF16 else 2.0 ** -149
    R.inside(dx, dxr, R.HALF[dt] * tot + e + 4 * U * tot + (4 * U * ds.double().abs() if residual else 0) + least, "dx")
    m = 64 + L / 64
    R.inside(dw, dwr, (m + 4) * U * (dy.double().abs() * xh.abs()).sum(0) + 1e-37, "dw")
