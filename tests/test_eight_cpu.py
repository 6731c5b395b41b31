"""Sizes and refusals of the operators in 8 bits, on the CPU: by the library
(status codes, before anything is enqueued) and by the binding."""
import ctypes

import pytest
import torch

from mixture_experts_atomic_gb300 import binding as B
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
