"""Sizes and refusals of the operators in 8 bits, on the CPU: by the library
(status codes, before anything is enqueued) and by the binding."""
import ctypes

import pytest
import torch

from mixture_experts_atomic_gb300 import binding as B
from mixture_experts_atomic_gb300.block import MoEBlock, RMSNorm
from mixture_experts_atomic_gb300.fp8 import Fp8Experts
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


def _fp8_weights(**over):
    return B.Fp8Weights(**{**{k: OKP.value for k in ("q1", "s1", "q2", "s2", "q3", "s3")}, **over})


def test_fp8_status():
    sh = lambda L=8, d=128, h=256, E=4, K=2, dt=BF, act="swiglu", fl=0: B.make_shape(L, d, h, E, K, dt, act, fl)  # noqa: E731
    need = B.moeblaze_fp8_workspace_bytes
    assert need(sh()) > 0 and need(sh(L=0)) == 0
    sizes = [need(sh(L=L)) for L in (1, 2, 16, 31, 32, 33, 64, 100, 1000, 5000)]
    assert sizes == sorted(sizes)                            # buffers for max_tokens hold every smaller call
    for bad in (sh(dt=F), sh(act="identity"), sh(K=5), sh(L=-1), sh(d=64), sh(h=130), sh(E=513), sh(E=512, h=1 << 22)):
        assert need(bad) == 0

    def fwd(s, x=OKP, xs=None, ids=OKP, g=OKP, w=None, y=OKP, ws=OKP, n=1 << 40):
        return B.moeblaze_fp8_forward(s, x, xs, ids, g, w or _fp8_weights(), y, ws, n, None)

    assert fwd(sh(dt=F)) == B.ERR_UNSUPPORTED and fwd(sh(act="identity")) == B.ERR_UNSUPPORTED
    assert fwd(sh(K=5)) == B.ERR_INVALID_ARG
    for k in ("x", "ids", "g", "y", "ws"):
        assert fwd(sh(), **{k: None}) == B.ERR_INVALID_ARG, k
    for k in ("x", "y", "ws"):
        assert fwd(sh(), **{k: BAD}) == B.ERR_INVALID_ARG, k
    for k in ("q1", "s1", "q2", "s2", "q3", "s3"):
        assert fwd(sh(), w=_fp8_weights(**{k: None})) == B.ERR_INVALID_ARG, k
    for k in ("q1", "q2", "q3"):
        assert fwd(sh(), w=_fp8_weights(**{k: BAD.value})) == B.ERR_INVALID_ARG, k
    assert fwd(sh(), n=need(sh()) - 1) == B.ERR_WORKSPACE
    assert fwd(sh(L=0), x=None, ids=None, g=None, y=None, ws=None) == B.OK
    assert B.moeblaze_fp8_quantize_weights(2, 128, 200, B.BF16, OKP, OKP, OKP, None) == B.ERR_UNSUPPORTED
    assert B.moeblaze_fp8_quantize_weights(0, 128, 128, B.BF16, OKP, OKP, OKP, None) == B.ERR_INVALID_ARG
    assert B.moeblaze_fp8_quantize_weights(2, 128, 128, 5, OKP, OKP, OKP, None) == B.ERR_INVALID_ARG
    assert B.moeblaze_fp8_quantize_weights(2, 128, 128, B.F32, BAD, OKP, OKP, None) == B.ERR_INVALID_ARG
    assert B.moeblaze_fp8_pack(2, 128, 128, OKP, BAD, None) == B.ERR_INVALID_ARG
    assert B.moeblaze_fp8_pack(2, 100, 128, OKP, OKP, None) == B.ERR_UNSUPPORTED
    assert B.moeblaze_fp8_dequantize_weights(2, 128, 128, None, 0, OKP, OKP, None) == B.ERR_INVALID_ARG
    assert B.moeblaze_fp8_dequantize_weights(513, 128, 128, OKP, 1, OKP, OKP, None) == B.ERR_UNSUPPORTED


def test_fp8_binding_refusals():
    f8 = torch.float8_e4m3fn
    with pytest.raises(B.MoEBlazeError):
        Fp8Experts(8, 100, 128, 4, 2, device="cpu")
    ex = Fp8Experts(8, 128, 256, 4, 2, device="cpu")
    z = lambda *s, dt=f8: torch.zeros(*s, dtype=dt)  # noqa: E731
    x, ids, g = z(3, 128, dt=BF), z(3, 2, dt=torch.int32), z(3, 2, dt=F)
    with pytest.raises(RuntimeError, match="load"):
        ex.forward(x, ids, g)
    with pytest.raises(RuntimeError, match="load"):
        ex.dequantize()
    ok = [z(4, 256, 128), z(4, 2, 1, dt=F), z(4, 256, 128), z(4, 2, 1, dt=F), z(4, 128, 256), z(4, 1, 2, dt=F)]
    for i, bad in ((0, z(4, 128, 256)), (1, z(4, 1, 2, dt=F)), (2, None), (3, z(4, 2, 1, dt=BF)), (4, z(4, 128, 256, dt=BF)),
                   (5, z(4, 2, 1, dt=F)), (0, z(4, 128, 256).transpose(1, 2))):
        args = list(ok)
        args[i] = bad
        with pytest.raises(ValueError):
            ex.load(*args)
    with pytest.raises(ValueError, match="CUDA"):
        ex.load(*ok)
    assert ex._weights is None
    ex._weights = _fp8_weights()
    with pytest.raises(ValueError, match="at most 8"):
        ex.forward(z(9, 128, dt=BF), z(9, 2, dt=torch.int32), z(9, 2, dt=F))
    for a in ((x.float(), ids, g), (x, ids.long(), g), (x, ids, g[:2]), (x[:, :64], ids, g), (z(3, 128), ids, g),
              (x, ids, g, z(3, 1, dt=F)), (z(3, 128), ids, g, z(3, 2, dt=F))):
        with pytest.raises(ValueError):
            ex.forward(*a)
    with pytest.raises(ValueError):
        B.fp8_quantize_weights(z(128, 128, dt=BF))
    with pytest.raises(ValueError):
        B.fp8_quantize_weights(z(1, 128, 128, dt=torch.half))
    with pytest.raises(B.MoEBlazeError):
        B.fp8_pack(z(1, 100, 128))


def test_fp8_matrix_limits():
    """Sizes whose blocks would not fit a launch's grid or 32 bits are refused, whichever of the two is long."""
    long = 1 << 23
    for call in (lambda E, R, N: B.moeblaze_fp8_pack(E, R, N, OKP, None, None),
                 lambda E, R, N: B.moeblaze_fp8_quantize_weights(E, R, N, B.BF16, None, OKP, OKP, None),
                 lambda E, R, N: B.moeblaze_fp8_dequantize_weights(E, R, N, None, 1, OKP, OKP, None)):
        assert call(1, long, 128) == B.ERR_UNSUPPORTED and call(1, 128, long) == B.ERR_UNSUPPORTED
        assert call(512, 1 << 15, 1 << 15) == B.ERR_UNSUPPORTED
        assert call(1, long - 128, 128) == B.ERR_INVALID_ARG     # (in range: the missing pointer is what is refused)
