"""Refusals of the norm, router-loss, dense router-gradient and 4-bit calls, on
the CPU: by the library (status codes, before anything is enqueued) and by the
binding (shapes, types, layout)."""
import ctypes

import pytest
import torch

from mixture_experts_atomic_gb300 import binding as B

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


def _norm(L=8, d=64, dt=B.BF16):
    return B.make_shape(L, d, 0, 1, 1, dt, "identity")


def test_layernorm_status():
    def fwd(s, x=OKP, res=None, w=OKP, b=None, eps=1e-5, su=None, y=OKP, m=OKP, r=OKP):
        return B.moeblaze_layernorm_forward(s, x, res, w, b, eps, su, y, m, r, None)

    assert fwd(_norm(L=-1)) == B.ERR_INVALID_ARG
    assert fwd(_norm(d=0)) == B.ERR_INVALID_ARG
    assert fwd(_norm(dt=5)) == B.ERR_INVALID_ARG
    assert fwd(_norm(L=1 << 31)) == B.ERR_UNSUPPORTED
    assert fwd(_norm(d=(1 << 24) + 1)) == B.ERR_UNSUPPORTED
    for k in ("x", "w", "y", "m", "r"):
        assert fwd(_norm(), **{k: None}) == B.ERR_INVALID_ARG, k
    for k in ("x", "res", "w", "b", "su", "y"):
        assert fwd(_norm(), **{k: BAD}) == B.ERR_INVALID_ARG, k
    assert fwd(_norm(), eps=-1.0) == B.ERR_INVALID_ARG
    assert fwd(_norm(), eps=float("nan")) == B.ERR_INVALID_ARG
    # nothing to do for no tokens: NULL is fine
    assert fwd(_norm(L=0), x=None, y=None, m=None, r=None) == B.OK
    need = B.moeblaze_layernorm_backward_workspace_bytes(_norm())
    assert need > 0 and B.moeblaze_layernorm_backward_workspace_bytes(_norm(d=0)) == 0

    def bwd(s, dy=OKP, su=OKP, m=OKP, r=OKP, w=OKP, ds=None, dx=OKP, dw=OKP, db=OKP, ws=OKP, n=need):
        return B.moeblaze_layernorm_backward(s, dy, su, m, r, w, ds, dx, dw, db, ws, n, None)

    for k in ("dy", "su", "m", "r", "w", "dx", "dw", "ws"):
        assert bwd(_norm(), **{k: None}) == B.ERR_INVALID_ARG, k
    for k in ("dy", "su", "w", "ds", "dx", "ws"):
        assert bwd(_norm(), **{k: BAD}) == B.ERR_INVALID_ARG, k
    assert bwd(_norm(), n=need - 1) == B.ERR_WORKSPACE


def test_balance_status():
    sh = lambda L=8, E=8, K=2: B.make_shape(L, 1, 0, E, K, F, "identity")  # noqa: E731
    need = B.moeblaze_balance_workspace_bytes(sh())
    assert need > 0

    def fwd(s, lg=OKP, ids=OKP, v=None, lo=OKP, c=OKP, lse=OKP, ws=OKP, n=need):
        return B.moeblaze_balance_forward(s, lg, ids, v, lo, c, lse, ws, n, None)

    assert fwd(sh(K=9, E=8)) == B.ERR_INVALID_ARG
    assert fwd(sh(K=9, E=16)) == B.ERR_UNSUPPORTED
    assert fwd(sh(E=513)) == B.ERR_UNSUPPORTED
    assert fwd(sh(L=1 << 30)) == B.ERR_UNSUPPORTED
    for k in ("lg", "ids", "lo", "c", "lse", "ws"):
        assert fwd(sh(), **{k: None}) == B.ERR_INVALID_ARG, k
    assert fwd(sh(), lg=BAD) == B.ERR_INVALID_ARG
    assert fwd(sh(), n=need - 1) == B.ERR_WORKSPACE

    def bwd(s, lg=OKP, lse=OKP, c=OKP, dl=OKP, ids=None, g=None, dg=None, out=OKP):
        return B.moeblaze_balance_backward(s, lg, lse, c, dl, ids, g, dg, out, None)

    for k in ("lg", "lse", "c", "dl", "out"):
        assert bwd(sh(), **{k: None}) == B.ERR_INVALID_ARG, k
    for given in ({"ids": OKP}, {"g": OKP}, {"dg": OKP}, {"ids": OKP, "g": OKP}, {"g": OKP, "dg": OKP}):
        assert bwd(sh(), **given) == B.ERR_INVALID_ARG, given
    assert bwd(sh(), out=BAD) == B.ERR_INVALID_ARG
    assert bwd(sh(L=0), lg=None, lse=None, out=None) == B.OK


def test_router_logits_status():
    sh = B.make_shape(8, 64, 128, 8, 2, B.BF16, "identity")
    need = B.moeblaze_router_backward_logits_workspace_bytes(sh)
    assert need > 0
    call = lambda s=sh, x=OKP, W=OKP, dl=OKP, dW=OKP, db=OKP, dx=OKP, ws=OKP, n=need: \
        B.moeblaze_router_backward_logits(s, x, W, dl, dW, db, dx, 0, ws, n, None)  # noqa: E731
    for k in ("x", "W", "dl", "dW", "ws"):
        assert call(**{k: None}) == B.ERR_INVALID_ARG, k
    for k in ("x", "dl", "dx", "ws"):
        assert call(**{k: BAD}) == B.ERR_INVALID_ARG, k
    assert call(n=need - 1) == B.ERR_WORKSPACE
    assert call(s=B.make_shape(8, 63, 128, 8, 2, B.BF16, "identity")) == B.ERR_UNSUPPORTED
    assert call(s=B.make_shape(8, 64, 128, 300, 2, B.BF16, "identity")) == B.ERR_UNSUPPORTED
    assert B.moeblaze_router_forward_logits(sh, OKP, OKP, None, OKP, OKP, None, None) == B.ERR_INVALID_ARG
    d = B.Dispatch(0x100000, 0x100000, 0x100000, 0x100000, 0x100000)
    assert B.moeblaze_router_dispatch_build_logits(sh, OKP, OKP, None, OKP, OKP, BAD, d, OKP, 1 << 30, None) \
        == B.ERR_INVALID_ARG


def test_int4_status():
    assert B.moeblaze_int4_weight_bytes(2, 256, 128) == 2 * 256 * 128 // 2
    assert B.moeblaze_int4_scale_bytes(2, 256, 128, 32) == 2 * 8 * 128 * 2
    for m in ((0, 128, 128), (2, 100, 128), (2, 128, 120), (513, 128, 128), (2, -128, 128)):
        assert B.moeblaze_int4_weight_bytes(*m) == 0
        assert B.moeblaze_int4_pack(*m, 64, OKP, OKP, OKP, OKP, None) in (B.ERR_INVALID_ARG, B.ERR_UNSUPPORTED)
        assert B.moeblaze_int4_dequantize(*m, 64, OKP, OKP, OKP, None) in (B.ERR_INVALID_ARG, B.ERR_UNSUPPORTED)
        assert B.moeblaze_int4_quantize(*m, 64, B.BF16, OKP, OKP, OKP, None) in (B.ERR_INVALID_ARG, B.ERR_UNSUPPORTED)
    assert B.moeblaze_int4_scale_bytes(2, 256, 128, 48) == 0
    assert B.moeblaze_int4_pack(2, 128, 128, 16, OKP, OKP, OKP, OKP, None) == B.ERR_INVALID_ARG
    assert B.moeblaze_int4_pack(2, 128, 128, 32, BAD, OKP, OKP, OKP, None) == B.ERR_INVALID_ARG
    assert B.moeblaze_int4_quantize(2, 128, 128, 32, 9, OKP, OKP, OKP, None) == B.ERR_INVALID_ARG
    sh = B.make_shape(4, 256, 384, 8, 2, B.BF16, "swiglu")
    need = B.moeblaze_int4_workspace_bytes(sh, 64)
    assert need > 0
    P = 0x100000

    def w(**kw):
        a = dict(w1=P, s1=P, w2=P, s2=P, w3=P, s3=P, group=64)
        a.update(kw)
        return B.Int4Weights(*[a[k] for k in ("w1", "s1", "w2", "s2", "w3", "s3", "group")])

    def fwd(s=sh, x=OKP, ids=OKP, g=OKP, wt=None, y=OKP, ws=OKP, n=need):
        return B.moeblaze_int4_forward(s, x, ids, g, wt or w(), y, ws, n, None)

    for k in ("x", "ids", "g", "y", "ws"):
        assert fwd(**{k: None}) == B.ERR_INVALID_ARG, k
    for k in ("w1", "s1", "w2", "s2", "w3", "s3"):
        assert fwd(wt=w(**{k: None})) == B.ERR_INVALID_ARG, k
    assert fwd(wt=w(group=100)) == B.ERR_INVALID_ARG
    assert fwd(n=need - 1) == B.ERR_WORKSPACE
    for bad in (B.make_shape(4, 256, 384, 8, 2, B.F32, "swiglu"), B.make_shape(4, 256, 0, 8, 2, B.BF16, "identity"),
                B.make_shape(4, 192, 384, 8, 2, B.BF16, "swiglu")):
        assert fwd(s=bad) == B.ERR_UNSUPPORTED
        assert B.moeblaze_int4_workspace_bytes(bad, 64) == 0
    assert fwd(s=B.make_shape(0, 256, 384, 8, 2, B.BF16, "silu"), x=None, ids=None, g=None, y=None, ws=None,
               wt=w(w2=None, s2=None)) == B.OK


def test_binding_refuses_malformed_tensors():
    t = lambda *s, dt=F: torch.zeros(*s, dtype=dt)  # noqa: E731
    L, d, E, K = 8, 64, 4, 2
    ns = _norm(L, d)
    x, m, wt = t(L, d, dt=BF), t(L), t(d)

    def fwd(**kw):
        a = dict(x=x, res=None, w=wt, b=None, s=None, y=x, m=m, r=m)
        a.update(kw)
        B.layernorm_forward(ns, a["x"], a["res"], a["w"], a["b"], 1e-5, a["s"], a["y"], a["m"], a["r"])

    for kw, msg in (({"x": t(L, d)}, "x: dtype"), ({"x": t(d, L, dt=BF).t()}, "x: must be contiguous"),
                    ({"res": t(L, d + 1, dt=BF)}, "residual: shape"), ({"w": t(d, dt=BF)}, "weight: dtype"),
                    ({"b": t(d + 1)}, "bias: shape"), ({"m": t(L, 1)}, "mean: shape"), ({"w": None}, "weight: a tensor"),
                    ({}, "x: must be a CUDA tensor")):
        with pytest.raises(ValueError, match=msg):
            fwd(**kw)
    bs = B.make_shape(L, 1, 0, E, K, F, "identity")
    ids = t(L, K, dt=torch.int32)
    with pytest.raises(ValueError, match="logits: dtype"):
        B.balance_forward(bs, t(L, E, dt=BF), ids, None, t(2), t(E + 1, dt=torch.int32), t(L), t(1))
    with pytest.raises(ValueError, match="valid: dtype"):
        B.balance_forward(bs, t(L, E), ids, t(L, dt=torch.bool), t(2), t(E + 1, dt=torch.int32), t(L), t(1))
    with pytest.raises(ValueError, match="counts: shape"):
        B.balance_forward(bs, t(L, E), ids, None, t(2), t(E, dt=torch.int32), t(L), t(1))
    with pytest.raises(ValueError, match="dlogits: shape"):
        B.router_backward_logits(B.make_shape(L, d, 0, E, K, BF, "identity"), x, t(d, E), t(L, E + 1), t(d, E), None,
                                 None)
    with pytest.raises(ValueError, match="W: dtype"):
        B.int4_quantize(t(2, 128, 128, dt=torch.float64), 64)
    with pytest.raises(ValueError, match="q: expected"):
        B.int4_pack(t(128, 128, dt=torch.int8), t(1, 128, dt=BF), 128)
    with pytest.raises(B.MoEBlazeError, match="unsupported"):
        B.int4_pack(t(1, 96, 128, dt=torch.int8), t(1, 3, 128, dt=BF), 32)
    with pytest.raises(ValueError, match="scales: shape"):
        B.int4_pack(t(1, 128, 128, dt=torch.int8), t(1, 2, 128, dt=BF), 32)


def _int4_slices(L, d, h, E, K, group):
    """Slices of the down projection as the workspace has them: (slices x L K x d) fp32 behind h (L K x h) bf16,
    both rounded up to 256 bytes (d a multiple of 128 makes the first exact)."""
    n = B.moeblaze_int4_workspace_bytes(B.make_shape(L, d, h, E, K, B.BF16, "swiglu"), group)
    hidden = (L * K * h * 2 + 255) // 256 * 256
    assert n > hidden and (n - hidden) % (L * K * d * 4) == 0
    return (n - hidden) // (L * K * d * 4)


@pytest.mark.parametrize("group", [32, 64, 128])
def test_int4_slices_are_bounded(group):
    """A unit's number holds 64 slices; h / 128 need not have a divisor that fits."""
    for blocks in (1, 2, 64, 65, 67, 86, 101, 107, 109, 127, 128, 1009, 4093, 4095, 4096, 4099):
        for L in (1, 4, 16, 64):
            assert 1 <= _int4_slices(L, 128, 128 * blocks, 8, 2, group) <= min(blocks, 64), (blocks, L)
    # a slice of the widest h whose token row does not fit an SM is refused
    assert B.moeblaze_int4_workspace_bytes(B.make_shape(1, 128, 1 << 22, 8, 2, B.BF16, "swiglu"), group) == 0
    # and what one slice a piece cost, it no longer does: the partial sums of the widest layer stay below its weights
    assert _int4_slices(64, 4096, 128 * 109, 8, 8, group) <= 16


def test_balance_masked_status():
    sh = B.make_shape(8, 1, 0, 8, 2, F, "identity")

    def bwd(lg=OKP, lse=OKP, c=OKP, dl=OKP, v=OKP, ids=OKP, g=OKP, dg=OKP, out=OKP):
        return B.moeblaze_balance_backward_masked(sh, lg, lse, c, dl, v, ids, g, dg, 1, out, None)

    for k in ("lg", "lse", "c", "dl", "out", "ids", "g", "dg"):
        assert bwd(**{k: None}) == B.ERR_INVALID_ARG, k
    assert bwd(lg=BAD) == B.ERR_INVALID_ARG
    assert B.moeblaze_balance_backward_masked(B.make_shape(0, 1, 0, 8, 2, F, "identity"), None, None, OKP, OKP, None,
                                              None, None, None, 1, None, None) == B.OK


@pytest.mark.parametrize("d,h,E,K,group", [(1024, 7168, 64, 1, 128), (128, 2944, 64, 3, 64), (128, 8704, 32, 1, 64),
                                           (128, 4608, 128, 2, 32), (256, 384, 8, 2, 128), (128, 13696, 16, 4, 64)])
def test_int4_buffers_hold_every_number_of_tokens(d, h, E, K, group):
    """A batch of L <= max_tokens tokens never needs more scratch than the object made for max_tokens has."""
    from mixture_experts_atomic_gb300.int4 import Int4Experts
    need = {L: B.moeblaze_int4_workspace_bytes(B.make_shape(L, d, h, E, K, B.BF16, "swiglu"), group)
            for L in range(1, 261)}
    for most in (1, 5, 63, 64, 65, 67, 80, 100, 126, 127, 128, 200, 260):
        have = Int4Experts(most, d, h, E, K, "swiglu", group, device="cpu")._ws.numel()
        short = [L for L in range(1, most + 1) if need[L] > have]
        assert not short, (most, short, have)


def test_balance_backward_before_forward():
    from mixture_experts_atomic_gb300.block import BalanceLoss
    with pytest.raises(RuntimeError, match="run forward first"):
        BalanceLoss(8, 4, 2, device="cpu").backward(torch.zeros(8, 4), torch.ones(2))


def test_int4_load_refuses_before_it_replaces(monkeypatch):
    """A tensor that does not fit, whichever it is, leaves the weights that are loaded as they are."""
    from mixture_experts_atomic_gb300.int4 import Int4Experts
    E, d, h, G = 2, 128, 256, 64
    ex = Int4Experts(4, d, h, E, 1, "swiglu", G, device="cpu")
    packs = []
    monkeypatch.setattr(B, "int4_pack", lambda q, s, group, *old: packs.append(1) or (q, s))
    q = lambda r, n, dt=torch.int8: torch.zeros(E, r, n, dtype=dt)  # noqa: E731
    s = lambda r, n, dt=BF: torch.ones(E, r // G, n, dtype=dt)  # noqa: E731
    good = [q(d, h), s(d, h), q(d, h), s(d, h), q(h, d), s(h, d)]
    for at, bad, msg in ((1, s(2 * d, h), "s1: shape"), (3, s(d, h, F), "s2: dtype"), (5, s(d, h), "s3: shape"),
                         (5, None, "s3: a tensor"), (3, torch.ones(E, h, d // G, dtype=BF).transpose(1, 2), "s2: must be"),
                         (4, q(h, d, torch.uint8), "q3: dtype"), (2, q(h, d), "q2: expected"), (0, None, "q1: expected"),
                         (1, s(d, h), "must be a CUDA tensor")):
        args = list(good)
        args[at] = bad
        with pytest.raises(ValueError, match=msg):
            ex.load(*args)
    assert not packs and ex._weights is None
    # weights on another device than the buffers are refused too (their checks of the current device aside)
    monkeypatch.setattr(B, "_args", lambda *specs: None)
    with pytest.raises(ValueError, match="q1: on meta, but the buffers are on cpu"):
        ex.load(*[t.to("meta") for t in good])
    assert not packs
    ex.load(*good)
    assert len(packs) == 3
