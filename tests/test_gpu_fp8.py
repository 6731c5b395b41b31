"""The layer's forward on 8-bit floating-point weights on the GPU against its
fp64 definition (eight_ref.experts8, which also gives the error bound), and the
weights' quantiser against its definition to the bit."""
import pytest
import torch

import eight_ref as R
from mixture_experts_atomic_gb300 import binding as B
from mixture_experts_atomic_gb300 import fp8
from mixture_experts_atomic_gb300.block import RMSNorm
from mixture_experts_atomic_gb300.fp8 import Fp8Experts
from mixture_experts_atomic_gb300.layer import MoELayer

pytestmark = pytest.mark.gpu

from gpu_util import ensure_built  # noqa: E402

BF16, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _matrix(E, N, K, g):
    q = (100 * torch.randn(E, N, K, generator=g)).clamp(-448, 448).to(F8).cuda()
    return q, ((0.5 + torch.rand(E, N // 128, K // 128, generator=g)) / (100 * K ** 0.5)).cuda()


def _problem(L, d, h, E, K, act, seed, one=None):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(L, d, generator=g) * (1 + 9 * (torch.rand(d, generator=g) < 0.02))).to(BF16).cuda()
    if one is None:
        ids = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(L)]).int() if L else torch.empty(0, K).int()
    else:  # every token's first slot on one expert
        ids = torch.stack([torch.cat([torch.tensor([one]), (one + 1 + torch.randperm(E - 1, generator=g)[:K - 1]) % E])
                           for _ in range(L)]).int()
    gates = torch.softmax(torch.randn(L, K, generator=g), 1).contiguous()
    mats = _matrix(E, h, d, g) + (_matrix(E, h, d, g) if act == "swiglu" else (None, None)) + _matrix(E, d, h, g)
    return x, ids.contiguous().cuda(), gates.cuda(), mats


def _check(y, x, ids, gates, mats):
    q, s = R.rows8(x)                       # (exact: a bf16 value over a power of two)
    want, bound = R.experts8(q * R.grown(s, x.shape[1]), ids, gates, mats)
    R.inside(y, want, bound + R.BF * (want.abs() + bound) + 1e-30, "y")


SHAPES = [
    (1, 128, 128, 1, 1, "swiglu", None),
    (1, 256, 384, 8, 2, "swiglu", None),
    (2, 128, 256, 4, 2, "silu", None),
    (3, 640, 128, 5, 3, "swiglu", None),
    (7, 384, 896, 8, 2, "silu", None),          # d and h with half a tile of 256 columns
    (16, 512, 1024, 8, 2, "swiglu", None),
    (17, 512, 640, 3, 1, "swiglu", None),
    (33, 128, 128, 2, 1, "silu", None),
    (61, 256, 384, 64, 6, "swiglu", None),
    (64, 256, 512, 8, 8, "swiglu", None),       # K == E
    (65, 128, 256, 4, 2, "swiglu", None),
    (150, 128, 128, 3, 2, "silu", None),
    (40, 128, 128, 512, 8, "swiglu", None),
    (300, 256, 384, 5, 2, "swiglu", None),
    (513, 384, 256, 2, 2, "swiglu", 1),         # 513 rows of each expert: a tile of one row
    (700, 128, 640, 16, 4, "silu", 3),          # skewed
    (2500, 256, 256, 8, 2, "swiglu", None),     # more slots than one chunk of the routing
    (5000, 384, 384, 3, 3, "swiglu", None),
    (3000, 1024, 512, 6, 2, "silu", 0),
    (5, 4096, 1408, 4, 2, "swiglu", None),
    (24, 6144, 256, 2, 1, "swiglu", None),
    (12, 1408, 7168, 2, 2, "silu", None),
    (4, 14336, 128, 2, 1, "swiglu", None),
    (900, 2048, 1408, 8, 2, "swiglu", None),
    # few tokens (at most 512 slots, 16 an expert): several tiles of an expert's tokens, tiles in parts, and the next
    # number of tokens, which goes the other way
    (64, 256, 512, 8, 2, "swiglu", 3),
    (65, 256, 512, 8, 2, "swiglu", 3),
    (64, 384, 640, 8, 2, "silu", 5),
    (32, 2048, 256, 4, 2, "silu", 1),
    (85, 128, 128, 64, 6, "swiglu", 9),
    (86, 128, 128, 64, 6, "swiglu", 9),
    (33, 640, 896, 30, 3, "silu", None),
    (3, 2048, 2816, 16, 4, "swiglu", None),
    (1, 4096, 4096, 2, 1, "silu", None),
    (16, 128, 128, 1, 1, "swiglu", None),
    (17, 128, 128, 1, 1, "swiglu", None),
]


@pytest.mark.parametrize("L,d,h,E,K,act,one", SHAPES)
def test_fp8_forward(L, d, h, E, K, act, one):
    x, ids, gates, mats = _problem(L, d, h, E, K, act, L + d + h, one)
    ex = Fp8Experts(L, d, h, E, K, act)
    ex.load(*mats)
    y = ex.forward(x, ids, gates).clone()
    torch.cuda.synchronize()
    _check(y, x, ids, gates, mats)
    q, s = fp8.quantize_rows(x)                              # the same rows, given in 8 bits
    assert torch.equal(y, ex.forward(q, ids, gates, s))
    assert torch.equal(y, ex.forward(x, ids, gates))         # repeatable to the bit


def test_fp8_rows_with_any_scales():
    """Scales that are not powers of two, and of very different sizes."""
    L, d, h, E, K = 200, 512, 256, 4, 2
    x, ids, gates, mats = _problem(L, d, h, E, K, "swiglu", 4)
    q, s = fp8.quantize_rows(x)
    g = torch.Generator().manual_seed(5)
    s = s * (0.3 + torch.rand(s.shape, generator=g)).cuda()
    s[7] *= 1e-20
    ex = Fp8Experts(L, d, h, E, K)
    ex.load(*mats)
    y = ex.forward(q, ids, gates, s)
    want, bound = R.experts8(q.double() * R.grown(s, d), ids, gates, mats)
    R.inside(y, want, bound + R.BF * (want.abs() + bound) + 1e-30, "y")


@pytest.mark.parametrize("L", [1, 40, 700])
def test_fp8_empty_slots_and_odd_values(L):
    d, h, E, K = 256, 384, 6, 3
    x, ids, gates, mats = _problem(max(L, 12), d, h, E, K, "swiglu", 6)
    x, ids, gates = x[:L].contiguous(), ids[:L].contiguous(), gates[:L].contiguous()
    ids[0] = -1                                              # a token without experts
    gates[0] = float("nan")                                  # not read where the slot is empty
    x[0] = float("inf")
    if L > 10:
        ids[3, 1] = E
        ids[4, 0] = -2 ** 31
        ids[5, 1] = 2 ** 31 - 1
        ids[6] = ids[6, 0].clone()                           # the same expert three times counts three times
        x[8, 5] = float("nan")
        x[9] = 0
    ex = Fp8Experts(L, d, h, E, K)
    ex.load(*mats)
    y = ex.forward(x, ids, gates)
    assert float(y[0].float().abs().max()) == 0
    if L > 10:
        assert y[8].isnan().all() and float(y[9].float().abs().max()) == 0
        keep = [t for t in range(L) if t not in (0, 8)]
        _check(y[keep], x[keep], ids[keep], gates[keep], mats)
    ids[:] = -1                                              # nothing at all
    assert float(ex.forward(x, ids, gates).float().abs().max()) == 0


def test_fp8_fewer_tokens_than_the_buffers_and_rows_behind():
    d, h, E, K = 256, 384, 8, 2
    x, ids, gates, mats = _problem(600, d, h, E, K, "swiglu", 5)
    ex = Fp8Experts(600, d, h, E, K)
    ex.load(*mats)
    for n in (600, 1, 40, 0, 333):
        ex._y.fill_(3.0)
        y = ex.forward(x[:n], ids[:n], gates[:n])
        assert y.shape == (n, d)
        if n:
            _check(y, x[:n], ids[:n], gates[:n], mats)
        assert bool((ex._y[n:] == 3.0).all())                # rows behind the last token stay as they were


@pytest.mark.parametrize("L", [3, 60, 900])
def test_fp8_graph_stream_and_two_objects(L):
    """A captured forward replays on new inputs; two objects on two streams at once do not meet."""
    d, h, E, K = 256, 512, 8, 2
    x, ids, gates, mats = _problem(L, d, h, E, K, "swiglu", 7)
    x2, ids2, gates2, mats2 = _problem(L, d, h, E, K, "swiglu", 8)
    one, two = Fp8Experts(L, d, h, E, K), Fp8Experts(L, d, h, E, K)
    one.load(*mats)
    two.load(*mats2)
    want, want2 = one.forward(x, ids, gates).clone(), two.forward(x2, ids2, gates2).clone()
    other = one.forward(x2, ids2, gates2).clone()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(a):
            ya = one.forward(x, ids, gates)
        with torch.cuda.stream(b):
            yb = two.forward(x2, ids2, gates2)
    torch.cuda.synchronize()
    assert torch.equal(ya, want) and torch.equal(yb, want2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = one.forward(x, ids, gates)
    x.copy_(x2), ids.copy_(ids2), gates.copy_(gates2)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, other)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("E,K,N", [(1, 128, 128), (3, 256, 640), (2, 1408, 384)])
def test_quantize_weights_to_the_bit(E, K, N, dt):
    g = torch.Generator().manual_seed(E + K)
    W = (torch.randn(E, K, N, generator=g) * torch.exp2(torch.randint(-30, 30, (E, 1, 1), generator=g).float())).to(dt).cuda()
    W[0, :128, :128] = 0
    q, s = B.fp8_quantize_weights(W)
    assert q.shape == (E, N, K) and s.shape == (E, N // 128, K // 128)
    for e in range(E):
        for i in range(N // 128):
            for j in range(K // 128):
                blk = W[e, 128 * j:128 * j + 128, 128 * i:128 * i + 128].t().double()
                # the definition of a row's block, with all 128 x 128 as the block
                f, x = torch.frexp(blk.abs().max() / 448.0)
                k = max(int(x) - (float(f) == 0.5), -126) if float(f) else -126
                assert float(s[e, i, j]) == 2.0 ** k
                got = q[e, 128 * i:128 * i + 128, 128 * j:128 * j + 128].double()
                u = blk / 2.0 ** k
                _, ue = torch.frexp(u)
                step = ((ue - 4).clamp(min=-9).long() + 1023 << 52).view(torch.float64)
                assert torch.equal(got, torch.round(u / step) * step)
    back = B.fp8_dequantize_weights(q, s)
    want = torch.stack([R.matrix8(q[e], s[e]) for e in range(E)])
    assert torch.equal(back.double(), want)                  # four bits of mantissa: exact
    packed = B.fp8_pack(q)
    assert torch.equal(packed.view(torch.uint8), q.view(torch.uint8).view(E, N // 128, 128, K // 128, 128).transpose(2, 3))
    assert torch.equal(B.fp8_dequantize_weights(packed, s), back)
    any_s = s * 0.7
    want = torch.stack([R.matrix8(q[e].float(), any_s[e]) for e in range(E)]).float().to(BF16)
    off = (B.fp8_dequantize_weights(q, any_s).double() - want.double()).abs()
    assert bool((off <= 2 * R.BF * want.double().abs()).all())
    W[0, 5, 7] = float("nan")
    q, s = B.fp8_quantize_weights(W)
    assert bool(s[0, 0, 0].isnan()) and not bool(s[1:].isnan().any())


@pytest.mark.parametrize("L,act", [(5, "swiglu"), (700, "swiglu"), (700, "silu")])
def test_fp8_in_buffers_that_start_on_16_bytes(L, act):
    d, h, E, K = 256, 384, 4, 2
    x, ids, gates, mats = _problem(L, d, h, E, K, act, 3)
    ex = Fp8Experts(L, d, h, E, K, act)
    ex.load(*mats)
    want = ex.forward(x, ids, gates).clone()

    def moved(t):
        raw = torch.zeros(t.nbytes + 16, dtype=torch.uint8, device="cuda")
        out = raw[16:].view(t.dtype).view(t.shape)
        assert out.data_ptr() % 32 == 16
        out.view(torch.uint8).copy_(t.view(torch.uint8))
        return out

    packed = {n: (moved(q), moved(s)) for n, (q, s) in ex._packed.items()}
    args = [t.data_ptr() if t is not None else None for n in "123" for t in packed.get(n, (None, None))]
    y, ws = moved(want), moved(ex._ws)
    got = B.fp8_forward(ex._shape(L), moved(x), None, ids, gates, B.Fp8Weights(*args), y, ws)
    assert torch.equal(got, want)


def test_fp8_load_replaces_weights_in_place():
    """A graph captured on one set of weights runs on the next one loaded; a refused tensor leaves all as they were."""
    L, d, h, E, K = 20, 256, 384, 4, 2
    x, ids, gates, mats = _problem(L, d, h, E, K, "swiglu", 1)
    _, _, _, mats2 = _problem(L, d, h, E, K, "swiglu", 2)
    ex, other = Fp8Experts(L, d, h, E, K), Fp8Experts(L, d, h, E, K)
    ex.load(*mats)
    other.load(*mats2)
    want, want2 = ex.forward(x, ids, gates).clone(), other.forward(x, ids, gates).clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ex.forward(x, ids, gates)
    for bad in (0, 3, 5):
        broken = list(mats2)
        broken[bad] = broken[bad][:, :1].contiguous()
        with pytest.raises(ValueError):
            ex.load(*broken)
    graph.replay()
    assert torch.equal(y, want)
    ex.load(*mats2)
    for m in mats2:
        m.view(torch.uint8).zero_()                          # the object keeps copies
    graph.replay()
    assert torch.equal(y, want2)


def test_fp8_serving_chain():
    """RMS norm with 8-bit rows, router on its bf16 rows, 8-bit experts: the same tokens as a prompt through the bf16
    layer on the weights that the 8-bit ones stand for are near, and against the definition exact to the bound."""
    L, d, h, E, K = 400, 512, 768, 8, 2
    g = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    W = [(r(E, d, h) / d ** 0.5).to(BF16), (r(E, d, h) / d ** 0.5).to(BF16), (r(E, h, d) / h ** 0.5).to(BF16)]
    ex = Fp8Experts(L, d, h, E, K)
    ex.quantize(*W)
    norm = RMSNorm(L, d, BF16)
    q, s, u, _, _ = norm.forward8(r(L, d).to(BF16), 1 + 0.1 * r(d), r(L, d).to(BF16))
    shape = B.make_shape(L, d, h, E, K, BF16, "swiglu")
    ids, gates = torch.empty(L, K, dtype=torch.int32, device="cuda"), torch.empty(L, K, device="cuda")
    B.router_forward(shape, u, r(d, E) / d ** 0.5, None, ids, gates)
    y = ex.forward(q, ids, gates, s)
    mats = [m for w in W for m in B.fp8_quantize_weights(w)]
    want, bound = R.experts8(q.double() * R.grown(s, d), ids, gates, mats)
    R.inside(y, want, bound + R.BF * (want.abs() + bound) + 1e-30, "y")
    layer = MoELayer(L, d, h, E, K, BF16, "swiglu")
    layer.dispatch(ids)
    y16 = layer.forward(u, gates, *ex.dequantize())
    # x and H in 8 bits: each value off by at most 2^-4, uniformly within a step, so 2^-4 / sqrt(3) of a norm each at most
    assert float((y.double() - y16.double()).norm() / y16.double().norm()) <= 2 ** -4


@pytest.mark.parametrize("L", [8, 600])
def test_fp8_wait_limit(L):
    """A product whose first stage is never loaded gives up after the wait limit: y is NaN, and the next call is whole."""
    d, h, E, K = 256, 1024, 4, 2
    x, ids, gates, mats = _problem(L, d, h, E, K, "swiglu", 9)
    ex = Fp8Experts(L, d, h, E, K)
    ex.load(*mats)
    want = ex.forward(x, ids, gates).clone()
    torch.cuda.synchronize()
    B.moeblaze_set_fault_injection(20_000_000, 1)
    try:
        y = ex.forward(x, ids, gates)
        torch.cuda.synchronize()
    finally:
        B.moeblaze_set_fault_injection(0, 0)
    assert bool(y.isnan().all())
    assert torch.equal(ex.forward(x, ids, gates), want)
