"""Sizes and refusals of the operators in 8 bits, on the CPU: by the library
(status codes, before anything is enqueued) and by the binding."""
import ctypes

import pytest
import torch

from mixture_experts_atomic_gb300 import binding as B
from mixture_experts_atomic_gb300.block import MoEBlock, RMSNorm
from mixture_experts_atomic_gb300.layer import MoELayer

BF, F = torch.bfloat16, torch.float32
OKP = ctypes.c_void_p(0x100000)      # aligned, never dereferenced: validation fails first
BAD = ctypes.c_void_p(0x100004)


@pytest.fixture(scope="module", autouse=True)
def _built():
    try:
        B.lib()
    except RuntimeError:
        import __graft_entry__
        __graft_entry__.build()


def test_checkpoint8_sizes_and_refusals():
    for act, nb in (("swiglu", 2), ("silu", 1)):
        a = B.make_shape(70000, 256, 384, 16, 2, BF, act)
        c = B.make_shape(70000, 256, 384, 16, 2, BF, act, B.CHECKPOINT_8BIT)
        rows = B.padded_rows(a)
        assert B.moeblaze_saved_bytes(a) == rows * nb * 384 * 2
        assert B.moeblaze_saved_bytes(c) == rows * nb * (384 + 3 * 4)
        assert B.moeblaze_forward_workspace_bytes(a) == B.moeblaze_forward_workspace_bytes(c)
        assert B.moeblaze_backward_workspace_bytes(c) - B.moeblaze_backward_workspace_bytes(a) == rows * nb * 384 * 2
        bufs = B.LayerBuffers(torch.zeros(B.moeblaze_saved_bytes(c), dtype=torch.uint8), None, None)
        qa, sa, qb, sb = B.saved_codes(c, bufs)
        assert qa.shape == (rows, 384) and sa.shape == (rows, 3) and (qb is None) == (act == "silu")
        last = sa if sb is None else sb
        assert last.data_ptr() + last.nbytes == bufs.saved.data_ptr() + bufs.saved.nbytes
    # refused: fp32, both flags; the identity layer keeps nothing either way
    for dt, fl in ((F, B.CHECKPOINT_8BIT), (BF, B.CHECKPOINT_8BIT | B.RECOMPUTE_H)):
        s = B.make_shape(700, 128, 128, 8, 2, dt, "swiglu", fl)
        assert B.moeblaze_saved_bytes(s) == 0 and B.moeblaze_backward_workspace_bytes(s) == 0
        d = B.Dispatch(*[OKP.value] * 5)
        assert B.moeblaze_forward(s, OKP, OKP, d, OKP, OKP, OKP, OKP, OKP, OKP, 1 << 40, None) == B.ERR_UNSUPPORTED
        with pytest.raises(ValueError, match="checkpoint8"):
            MoELayer(700, 128, 128, 8, 2, dt, "swiglu", "cpu", recompute_h=bool(fl & B.RECOMPUTE_H), checkpoint8=True)
    s = B.make_shape(700, 128, 0, 8, 2, BF, "identity", B.CHECKPOINT_8BIT)
    assert B.moeblaze_saved_bytes(s) == 0 and B.moeblaze_dispatch_meta_bytes(s) > 0
    # a workspace of the default mode's size is too small
    s = B.make_shape(700, 128, 128, 8, 2, BF, "swiglu", B.CHECKPOINT_8BIT)
    n = B.moeblaze_backward_workspace_bytes(B.make_shape(700, 128, 128, 8, 2, BF, "swiglu"))
    d = B.Dispatch(*[OKP.value] * 5)
    assert B.moeblaze_backward(s, OKP, OKP, OKP, d, *[OKP] * 3, OKP, *[OKP] * 4, None, OKP, n, None) == B.ERR_WORKSPACE


def _norm(L=8, d=64, dt=B.BF16):
    return B.make_shape(L, d, 0, 1, 1, dt, "identity")


def test_rmsnorm_status():
    def fwd(s, x=OKP, res=None, w=OKP, eps=1e-5, su=None, y=OKP, r=OKP, q=None, qs=None):
        return B.moeblaze_rmsnorm_forward(s, x, res, w, eps, su, y, r, q, qs, None)

    assert fwd(_norm(L=-1)) == B.ERR_INVALID_ARG
    assert fwd(_norm(d=0)) == B.ERR_INVALID_ARG
    assert fwd(_norm(dt=5)) == B.ERR_INVALID_ARG
    assert fwd(_norm(L=1 << 31)) == B.ERR_UNSUPPORTED
    assert fwd(_norm(d=(1 << 24) + 1)) == B.ERR_UNSUPPORTED
    assert fwd(_norm(d=72), q=OKP, qs=OKP) == B.ERR_UNSUPPORTED      # 8-bit rows start on 16 bytes
    for k in ("x", "w", "y", "r"):
        assert fwd(_norm(), **{k: None}) == B.ERR_INVALID_ARG, k
    for k in ("x", "res", "w", "su", "y"):
        assert fwd(_norm(), **{k: BAD}) == B.ERR_INVALID_ARG, k
    assert fwd(_norm(), q=OKP) == B.ERR_INVALID_ARG and fwd(_norm(), qs=OKP) == B.ERR_INVALID_ARG
    assert fwd(_norm(), q=BAD, qs=OKP) == B.ERR_INVALID_ARG
    assert fwd(_norm(), eps=-1.0) == B.ERR_INVALID_ARG and fwd(_norm(), eps=float("nan")) == B.ERR_INVALID_ARG
    assert fwd(_norm(L=0), x=None, y=None, r=None) == B.OK
    need = B.moeblaze_rmsnorm_backward_workspace_bytes(_norm())
    assert need > 0 and B.moeblaze_rmsnorm_backward_workspace_bytes(_norm(d=0)) == 0

    def bwd(s, dy=OKP, su=OKP, r=OKP, w=OKP, ds=None, dx=OKP, dw=OKP, ws=OKP, n=need):
        return B.moeblaze_rmsnorm_backward(s, dy, su, r, w, ds, dx, dw, ws, n, None)

    for k in ("dy", "su", "r", "w", "dx", "dw", "ws"):
        assert bwd(_norm(), **{k: None}) == B.ERR_INVALID_ARG, k
    for k in ("dy", "su", "w", "ds", "dx", "ws"):
        assert bwd(_norm(), **{k: BAD}) == B.ERR_INVALID_ARG, k
    assert bwd(_norm(), n=need - 1) == B.ERR_WORKSPACE


def test_rows8_status():
    for f in (B.moeblaze_fp8_quantize_rows, B.moeblaze_fp8_dequantize_rows):
        assert f(0, 64, B.BF16, None, None, None, None) == B.OK
        assert f(-1, 64, B.BF16, OKP, OKP, OKP, None) == B.ERR_INVALID_ARG
        assert f(8, 0, B.BF16, OKP, OKP, OKP, None) == B.ERR_INVALID_ARG
        assert f(8, 64, 7, OKP, OKP, OKP, None) == B.ERR_INVALID_ARG
        assert f(8, 72, B.BF16, OKP, OKP, OKP, None) == B.ERR_UNSUPPORTED
        assert f(1 << 31, 64, B.BF16, OKP, OKP, OKP, None) == B.ERR_UNSUPPORTED
    # arguments in the order x, q, scales and q, scales, x
    for bad in (None, BAD):
        assert B.moeblaze_fp8_quantize_rows(8, 64, B.F32, bad, OKP, OKP, None) == B.ERR_INVALID_ARG
        assert B.moeblaze_fp8_quantize_rows(8, 64, B.F32, OKP, bad, OKP, None) == B.ERR_INVALID_ARG
        assert B.moeblaze_fp8_dequantize_rows(8, 64, B.F32, bad, OKP, OKP, None) == B.ERR_INVALID_ARG
        assert B.moeblaze_fp8_dequantize_rows(8, 64, B.F32, OKP, OKP, bad, None) == B.ERR_INVALID_ARG
    assert B.moeblaze_fp8_quantize_rows(8, 64, B.F32, OKP, OKP, None, None) == B.ERR_INVALID_ARG
    assert B.moeblaze_fp8_dequantize_rows(8, 64, B.F32, OKP, None, OKP, None) == B.ERR_INVALID_ARG


def test_rms_and_rows8_binding_refusals():
    """By the binding: shapes, types and layout before anything goes to C."""
    sh = _norm(4, 64, BF)
    x, w = torch.zeros(4, 64, dtype=BF), torch.ones(64)
    rstd = torch.empty(4)
    ok = dict(x=x, residual=None, weight=w, eps=1e-5, sum=None, y=x.clone(), rstd=rstd)
    for k, bad in (("x", x.float()), ("x", x[:, :32]), ("x", torch.zeros(64, 4, dtype=BF).t()), ("weight", w.to(BF)),
                   ("rstd", rstd[:3]), ("y", None), ("sum", x[:3]), ("residual", x.float())):
        with pytest.raises(ValueError):
            B.rmsnorm_forward(sh, **{**ok, k: bad})
    q = torch.zeros(4, 64, dtype=torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="q_scales"):
        B.rmsnorm_forward(sh, **ok, q=q)
    with pytest.raises(ValueError, match="q:"):
        B.rmsnorm_forward(sh, **ok, q=q.view(torch.uint8), q_scales=torch.empty(4, 1))
    with pytest.raises(ValueError, match="CUDA"):
        B.rmsnorm_forward(sh, **ok)
    with pytest.raises(ValueError):
        B.fp8_quantize_rows(x.half())
    with pytest.raises(B.MoEBlazeError):
        B.fp8_quantize_rows(x[:, :24].contiguous())
    with pytest.raises(ValueError):
        B.fp8_dequantize_rows(q, torch.empty(4, 2))
    with pytest.raises(ValueError):
        B.fp8_dequantize_rows(q, torch.empty(4, 1), torch.float16)
    norm = RMSNorm(4, 72, BF, device="cpu")
    with pytest.raises(ValueError, match="multiple of 16"):
        norm.forward8(torch.zeros(4, 72, dtype=BF), torch.ones(72))
    with pytest.raises(ValueError, match="norm"):
        MoEBlock(4, 128, 128, 2, 1, BF, device="cpu", norm="batch")
