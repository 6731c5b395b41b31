"""Layers and blocks that share one scratch, run as a model runs them (forward
through all, backward in the other order), against the same with scratch of
their own, to the bit (two slots a token: sums of two have one order)."""
import pytest
import torch

from mixture_experts_atomic_gb300.block import MoEBlock
from mixture_experts_atomic_gb300.layer import MoELayer

pytestmark = pytest.mark.gpu

from gpu_util import ensure_built  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _r(g, *s):
    return torch.randn(*s, device="cuda", generator=g)


KINDS = [dict(L=700, checkpoint8=True), dict(L=512), dict(L=300, recompute_h=True), dict(L=700, checkpoint8=True)]


@pytest.mark.parametrize("act", ["swiglu", "silu"])
def test_layers_of_one_scratch(act):
    d, h, E, K = 256, 384, 4, 2

    def run(share):
        g = torch.Generator(device="cuda").manual_seed(5)
        layers, kept, out = [], [], []
        for kw in KINDS:
            kw = dict(kw)
            L = kw.pop("L")
            layer = MoELayer(L, d, h, E, K, BF16, act, scratch=layers[0] if share and layers else None, **kw)
            W = [(_r(g, E, d, h) / 16).to(BF16), (_r(g, E, d, h) / 16).to(BF16) if act == "swiglu" else None,
                 (_r(g, E, h, d) / 20).to(BF16)]
            x, dy = _r(g, L, d).to(BF16), _r(g, L, d).to(BF16)
            ids = torch.rand(L, E, device="cuda", generator=g).topk(K, 1).indices.int().contiguous()
            gates = torch.rand(L, K, device="cuda", generator=g)
            layer.dispatch(ids)
            out.append(layer.forward(x, gates, *W).clone())
            layers.append(layer)
            kept.append((dy, x, gates, *W))
        for layer, args in reversed(list(zip(layers, kept))):
            out += [None if t is None else t.clone() for t in layer.backward(*args)]
        torch.cuda.synchronize()
        assert all(layer.device_error() == 0 for layer in layers)
        return out

    for a, b in zip(run(False), run(True)):
        assert (a is None and b is None) or torch.equal(a, b)


def test_blocks_of_one_scratch_in_a_captured_step():
    """Three blocks on a residual stream, a step captured and replayed on new inputs."""
    L, d, h, E, K, n = 400, 256, 384, 4, 2, 3
    g = torch.Generator(device="cuda").manual_seed(6)
    ps = [{"norm_w": 1 + 0.1 * _r(g, d), "Wr": _r(g, d, E) / 16, "W1": (_r(g, E, d, h) / 16).to(BF16),
           "W2": (_r(g, E, d, h) / 16).to(BF16), "W3": (_r(g, E, h, d) / 20).to(BF16)} for _ in range(n)]
    x, res, dout = (_r(g, L, d).to(BF16) for _ in range(3))
    x2, res2, dout2 = (_r(g, L, d).to(BF16) for _ in range(3))
    dl = torch.tensor([0.01, 0.001], device="cuda")

    def step(blocks, x, res, dout):
        s = res
        for b, p in zip(blocks, ps):
            x, s, losses, _ = b.forward(x, s, p)
        ds, out = None, [x]
        for b, p in zip(reversed(blocks), reversed(ps)):
            grads = b.backward(dout, dl, p, ds)
            out += [grads[k] for k in sorted(grads) if grads[k] is not None]
            dout = ds = grads["x"]
        return out

    def make(share):
        blocks = []
        for _ in range(n):
            blocks.append(MoEBlock(L, d, h, E, K, BF16, norm="rms", checkpoint8=True,
                                   scratch=blocks[0] if share and blocks else None))
        return blocks

    alone, shared = make(False), make(True)
    want = [t.clone() for t in step(alone, x, res, dout)]
    got = step(shared, x, res, dout)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(shared, x, res, dout)
    want = [t.clone() for t in step(alone, x2, res2, dout2)]
    x.copy_(x2), res.copy_(res2), dout.copy_(dout2)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
