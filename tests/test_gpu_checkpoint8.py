"""The layer with its checkpoints in 8 bits, on the GPU: the codes against what
they stand for, the gradients against their definition in fp64 at the values
that the codes stand for (so that no rounding border lies between the two), and
against differences of the forward."""
import pytest
import torch

import eight_ref as R
from mixture_experts_atomic_gb300 import binding as B
from mixture_experts_atomic_gb300 import inputs as I
from mixture_experts_atomic_gb300.block import MoEBlock
from mixture_experts_atomic_gb300.layer import GraphStep, MoELayer

pytestmark = pytest.mark.gpu

from gpu_util import ensure_built  # noqa: E402

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _problem(L, d, h, E, K, act, seed, one=None):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    p = {"x": r(L, d).to(BF16), "dY": r(L, d).to(BF16), "W1": (r(E, d, h) / d ** 0.5).to(BF16),
         "W2": (r(E, d, h) / d ** 0.5).to(BF16) if act == "swiglu" else None, "W3": (r(E, h, d) / h ** 0.5).to(BF16)}
    p["ids"], p["gates"] = I.random_routing(L, E, K, seed, one_expert=one)
    return {k: None if v is None else v.cuda() for k, v in p.items()}


def _kept(layer, p):
    """Per expert the checkpoints' values in fp64, rows in the order of torch.nonzero(ids == e), and the steps."""
    qa, sa, qb, sb = layer.saved()
    _, _, pad, _ = layer.meta()
    out = [], [], [], []
    for e in range(layer.E):
        t, _ = torch.nonzero(p["ids"] == e, as_tuple=True)   # ascending tokens, as in the layer's row space
        rows = slice(int(pad[e]), int(pad[e]) + t.numel())
        for i, (q, s) in enumerate(((qa, sa), (qb, sb))):
            if q is None:
                continue
            step = s[rows].double().repeat_interleave(B.CODE_BLOCK, dim=1)
            out[2 * i].append(q[rows].double() * step)
            out[2 * i + 1].append(step)
    return out


def _args(p, *names):
    return [p[n] for n in names]


def _forward(layer, p):
    layer.dispatch(p["ids"])
    return layer.forward(*_args(p, "x", "gates", "W1", "W2", "W3"))


def _backward(layer, p):
    got = layer.backward(*_args(p, "dY", "x", "gates", "W1", "W2", "W3"))
    torch.cuda.synchronize()
    assert layer.device_error() == 0
    return dict(zip(("dX", "dW1", "dW2", "dW3", "dgates"), got))


def _check_codes(layer, p):
    """|a - s q| <= s / 2, for the kernel's own a: fp32 sums next to the exact ones; and the steps are a 127th of the
    largest."""
    A, As, Bv, Bs = _kept(layer, p)
    for vals, steps, w in ((A, As, p["W1"]), (Bv, Bs, p["W2"])):
        for e in range(layer.E):
            if not vals or vals[e].numel() == 0:
                continue
            t, _ = torch.nonzero(p["ids"] == e, as_tuple=True)
            x, we = p["x"][t].double(), w[e].double()
            a, off = x @ we, (x.abs() @ we.abs()) * R.matmul_err(layer.d)
            R.inside(vals[e], a, 0.5 * steps[e] + off + 8 * R.U32 * a.abs(), f"checkpoints of expert {e}")
            n = a.shape[0]
            top = a.abs().view(n, -1, B.CODE_BLOCK).amax(2).repeat_interleave(B.CODE_BLOCK, dim=1)
            R.inside(steps[e], top / 127, (off.view(n, -1, B.CODE_BLOCK).amax(2).repeat_interleave(B.CODE_BLOCK, dim=1)
                                           + 4 * R.U32 * top) / 127, f"steps of expert {e}")
    return A, Bv


SHAPES = [
    (1, 128, 128, 1, 1, "swiglu", None),
    (1, 128, 128, 4, 2, "silu", None),
    (130, 128, 128, 8, 2, "silu", None),          # h 128: half a SiLU tile; experts with few or no tokens
    (300, 256, 384, 5, 2, "swiglu", None),        # h % 256 == 128
    (300, 256, 384, 5, 2, "silu", None),
    (700, 384, 128, 3, 3, "swiglu", None),        # K == E
    (900, 128, 256, 16, 6, "swiglu", 3),          # skewed: expert 3 takes every token
    (2000, 512, 512, 4, 1, "swiglu", None),       # K = 1
    (2048, 128, 640, 64, 2, "silu", None),
    (10000, 2048, 512, 4, 2, "swiglu", 1),        # 256-row tiles of the up projection
    (10000, 2048, 384, 4, 2, "silu", None),
    (1300, 1024, 1408, 8, 2, "swiglu", None),     # 256-row tiles of the weight gradients at 325 rows an expert
    (1300, 1024, 2560, 8, 2, "silu", 5),
]


@pytest.mark.parametrize("L,d,h,E,K,act,one", SHAPES)
def test_checkpoint8(L, d, h, E, K, act, one):
    p = _problem(L, d, h, E, K, act, L + d + h, one)
    layer = MoELayer(L, d, h, E, K, BF16, act, checkpoint8=True)
    y = _forward(layer, p)
    torch.cuda.synchronize()
    want, bound = R.layer_forward(*_args(p, "x", "ids", "gates", "W1", "W2", "W3"))
    R.inside(y, want, bound + R.BF * (want.abs() + bound) + 1e-30, "y")
    if K <= 2:  # the forward is the default mode's
        assert torch.equal(y, _forward(MoELayer(L, d, h, E, K, BF16, act), p))
    A, Bv = _check_codes(layer, p)
    before = layer.bufs.saved.clone()
    got = {k: None if v is None else v.clone() for k, v in _backward(layer, p).items()}
    want, tol = R.layer_backward(*_args(p, "dY", "x", "ids", "gates", "W1", "W2", "W3"), A, Bv)
    for n, w in want.items():
        own = R.U32 if n == "dgates" else R.BF
        R.inside(got[n], w, tol[n] + own * (w.abs() + tol[n]) + 1e-30, n)
    # what is kept stays as it is: a second backward gives the same
    again = _backward(layer, p)
    assert torch.equal(before, layer.bufs.saved)
    assert all(torch.equal(again[n], got[n]) for n in ("dW1", "dW2", "dW3") if got[n] is not None)


def test_checkpoint8_gradient_against_differences():
    """<gradient, direction> against a central difference of the forward of the definition: the codes are off by half a
    step, so the two agree to the size of that, not of a wrong term."""
    L, d, h, E, K = 64, 128, 256, 4, 2
    p = _problem(L, d, h, E, K, "swiglu", 3)
    layer = MoELayer(L, d, h, E, K, BF16, "swiglu", checkpoint8=True)
    _forward(layer, p)
    got = _backward(layer, p)
    g = torch.Generator().manual_seed(9)
    for name, grad in (("x", "dX"), ("W1", "dW1"), ("W2", "dW2"), ("W3", "dW3"), ("gates", "dgates")):
        v = torch.randn(p[name].shape, generator=g).double().cuda()
        f = []
        for eps in (1e-4, -1e-4):
            q = {k: t if k == "ids" or t is None else t.double() for k, t in p.items()}
            q[name] = q[name] + eps * v
            y, _ = R.layer_forward(*_args(q, "x", "ids", "gates", "W1", "W2", "W3"))
            f.append(float((y * q["dY"]).sum()))
        want = (f[0] - f[1]) / 2e-4
        have = float((got[grad].double() * v).sum())
        # The gradient is off by what codes (1/254 of a block's largest, at most 4 sigma: 1.6 % of sigma, in at most
        # three factors of a term) and bf16 (two roundings, 2^-8 each) make of it, 6 % of its norm at most; on a random
        # direction of n elements that is 6 % of |gradient| |v| / sqrt(n), here within five times its spread.
        size = float(got[grad].double().norm() * v.norm()) / v.numel() ** 0.5
        assert abs(have - want) <= 5 * 0.06 * size, (name, have, want, size)


def test_checkpoint8_odd_values():
    """A token of zeros has steps of zero; one with an infinity spoils its own rows and the weights' gradients, and no
    other token's; values below 2^-100 become zeros."""
    L, d, h, E, K = 200, 128, 256, 2, 1
    p = _problem(L, d, h, E, K, "swiglu", 4)
    p["ids"] = (torch.arange(L, device="cuda", dtype=torch.int32) % 2).view(L, 1).contiguous()
    p["x"][10] = 0
    p["x"][12] = (p["x"][12].double() * 2.0 ** -110).to(BF16)
    p["x"][13, 5] = float("inf")
    layer = MoELayer(L, d, h, E, K, BF16, "swiglu", checkpoint8=True)
    _forward(layer, p)
    A, As, Bv, Bs = _kept(layer, p)
    assert float(As[0][5].abs().max()) == 0 and float(A[0][5].abs().max()) == 0   # token 10 is expert 0's sixth
    assert float(As[0][6].abs().max()) == 0 and float(Bs[0][6].abs().max()) == 0
    assert not bool(A[1][6].isfinite().any())
    got = _backward(layer, p)
    rows = torch.arange(L, device="cuda") != 13
    assert bool(got["dX"][rows].isfinite().all()) and not bool(got["dX"][13].isfinite().all())
    assert bool(got["dW1"][0].isfinite().all()) and bool(got["dW3"][0].isfinite().all())
    assert not bool(got["dW3"][1].isfinite().any())


@pytest.mark.parametrize("eight", [False, True])
def test_layer_in_buffers_that_start_on_16_bytes(eight):
    """Pointers need 16-byte alignment, not more: every buffer of the C call moved by 16 bytes gives the same bits."""
    L, d, h, E, K = 300, 256, 384, 5, 2
    p = _problem(L, d, h, E, K, "swiglu", 9)
    layer = MoELayer(L, d, h, E, K, BF16, "swiglu", checkpoint8=eight)
    y = _forward(layer, p).clone()
    want = {k: v.clone() for k, v in _backward(layer, p).items()}

    def moved(t):
        raw = torch.zeros(t.nbytes + 16, dtype=torch.uint8, device="cuda")
        out = raw[16:].view(t.dtype).view(t.shape)
        assert out.data_ptr() % 32 == 16
        return out.copy_(t)

    other = MoELayer(L, d, h, E, K, BF16, "swiglu", checkpoint8=eight)
    for n in ("y", "dX", "dW1", "dW2", "dW3", "dgates"):
        setattr(other, n, moved(getattr(other, n)))
    other.bufs = B.LayerBuffers(*[moved(t) for t in (other.bufs.saved, other.bufs.fwd_ws, other.bufs.bwd_ws)])
    q = {k: v if k in ("ids", "gates") else moved(v) for k, v in p.items()}
    assert torch.equal(_forward(other, q), y)
    got = _backward(other, q)
    for n in ("dX", "dW1", "dW2", "dW3"):
        assert torch.equal(got[n], want[n]), n


def test_checkpoint8_empty_batch():
    p = _problem(0, 128, 256, 4, 2, "swiglu", 5)
    layer = MoELayer(0, 128, 256, 4, 2, BF16, "swiglu", checkpoint8=True)
    assert _forward(layer, p).shape == (0, 128)
    got = _backward(layer, p)
    assert all(float(got[n].float().abs().max()) == 0 for n in ("dW1", "dW2", "dW3"))


def test_checkpoint8_graph_replays_on_new_inputs():
    L, d, h, E, K = 500, 128, 256, 4, 2
    p, q = (_problem(L, d, h, E, K, "swiglu", s) for s in (6, 7))
    eager = MoELayer(L, d, h, E, K, BF16, "swiglu", checkpoint8=True)
    _forward(eager, q)
    want = _backward(eager, q)
    layer = MoELayer(L, d, h, E, K, BF16, "swiglu", checkpoint8=True)
    step = GraphStep(layer, p)
    for k in p:
        p[k].copy_(q[k])
    for _ in range(3):
        step.replay()
    torch.cuda.synchronize()
    assert torch.equal(layer.y, eager.y) and torch.equal(layer.dX, want["dX"]) and torch.equal(layer.dW1, want["dW1"])
    assert torch.equal(layer.dW2, want["dW2"]) and torch.equal(layer.dW3, want["dW3"])


def test_checkpoint8_in_the_block():
    """The block keeps its checkpoints in 8 bits: the same output and losses as without, gradients near."""
    L, d, h, E, K = 512, 256, 384, 8, 2
    g = torch.Generator(device="cuda").manual_seed(8)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    p = {"norm_w": torch.ones(d, device="cuda"), "norm_b": torch.zeros(d, device="cuda"), "Wr": r(d, E) / 16,
         "W1": (r(E, d, h) / 16).to(BF16), "W2": (r(E, d, h) / 16).to(BF16), "W3": (r(E, h, d) / 20).to(BF16)}
    x, res, dout = (r(L, d).to(BF16) for _ in range(3))
    dl = torch.tensor([0.01, 0.001], device="cuda")
    grads, outs = [], []
    for eight in (False, True):
        block = MoEBlock(L, d, h, E, K, BF16, checkpoint8=eight)
        out, _, losses, _ = block.forward(x, res, p)
        outs.append((out.clone(), losses.clone()))
        grads.append({k: v.clone() for k, v in block.backward(dout, dl, p).items()})
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    for k, v in grads[0].items():
        # codes are off by at most half a 127th of the block's largest, which is at most 4 sigma of normal values:
        # 2 % of sigma in A and in B, and at most 1.1 + 0.5 and 1 of that in dA and dB
        assert float((grads[1][k].double() - v.double()).norm() / v.double().norm()) <= 0.05, k
