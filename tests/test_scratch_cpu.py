"""Layers of a model that share one scratch, on the CPU: what they allocate, and
what is refused."""
import pytest
import torch

from mixture_experts_atomic_gb300 import binding as B
from mixture_experts_atomic_gb300.block import MoEBlock
from mixture_experts_atomic_gb300.layer import MoELayer

BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    try:
        B.lib()
    except RuntimeError:
        import __graft_entry__
        __graft_entry__.build()


def _held(layers):
    """Bytes of the layers' saved activations and scratch, each buffer once."""
    seen = {t.data_ptr(): t.nbytes for x in layers for t in (x.bufs.saved, x.bufs.fwd_ws, x.bufs.bwd_ws)}
    return sum(seen.values())


@pytest.mark.parametrize("act", ["swiglu", "silu"])
def test_checkpoints_in_8_bits_save_memory_across_layers(act):
    """The codes are half of the saved bytes; the scratch, which grows by dA and dB, is there once."""
    n = 4

    def model(**kw):
        first = MoELayer(700, 256, 384, 4, 2, BF, act, "cpu", **kw)
        return [first] + [MoELayer(700, 256, 384, 4, 2, BF, act, "cpu", scratch=first, **kw) for _ in range(n - 1)]

    eight, default = model(checkpoint8=True), model()
    one = eight[0].bufs
    assert _held(eight) == n * one.saved.nbytes + one.fwd_ws.nbytes + one.bwd_ws.nbytes
    assert len({x.bufs.saved.data_ptr() for x in eight}) == n
    assert _held(eight) < _held(default) < _held([MoELayer(700, 256, 384, 4, 2, BF, act, "cpu") for _ in range(n)])


def test_blocks_share_their_layers_scratch():
    first = MoEBlock(300, 128, 256, 4, 2, BF, device="cpu", norm="rms", checkpoint8=True)
    other = MoEBlock(200, 128, 256, 4, 2, BF, device="cpu", norm="layer", scratch=first)
    assert other.layer.bufs.bwd_ws is first.layer.bufs.bwd_ws and other.layer.bufs.fwd_ws is first.layer.bufs.fwd_ws
    assert other.layer.bufs.saved is not first.layer.bufs.saved


def test_scratch_that_does_not_fit_is_refused():
    small = MoELayer(300, 128, 256, 4, 2, BF, "swiglu", "cpu")
    with pytest.raises(ValueError, match="scratch: fwd_ws"):
        MoELayer(400, 128, 256, 4, 2, BF, "swiglu", "cpu", scratch=small)
    with pytest.raises(ValueError, match="scratch: bwd_ws"):        # the same forward, dA and dB more in the backward
        MoELayer(300, 128, 256, 4, 2, BF, "swiglu", "cpu", checkpoint8=True, scratch=small)
    with pytest.raises(ValueError, match="scratch: on cpu"):
        MoELayer(300, 128, 256, 4, 2, BF, "swiglu", "meta", scratch=small)
    MoELayer(300, 128, 256, 4, 2, BF, "swiglu", "cpu", recompute_h=True, scratch=small)
    MoELayer(300, 128, 0, 4, 2, F, "identity", "cpu", scratch=small)
