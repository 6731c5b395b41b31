"""Expert products on 4-bit weights on the GPU against their fp64 definition
(block_ref.int4_layer, which also gives the error bound), and the packed
layout against the values it holds, exactly."""
import pytest
import torch

import block_ref as R
from mixture_experts_atomic_gb300 import binding as B
from mixture_experts_atomic_gb300.int4 import Int4Experts
from mixture_experts_atomic_gb300.layer import MoELayer

pytestmark = pytest.mark.gpu

from gpu_util import ensure_built  # noqa: E402

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _matrix(E, rows, cols, group, g):
    q = torch.randint(-8, 8, (E, rows, cols), generator=g).to(torch.int8)
    s = ((0.5 + torch.rand(E, rows // group, cols, generator=g)) / (4.6 * rows ** 0.5)).to(BF16)
    return q, s


def _problem(L, d, h, E, K, act, group, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(L, d, generator=g).to(BF16)
    ids = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(L)]).int() if L else torch.empty(0, K).int()
    gates = torch.softmax(torch.randn(L, K, generator=g), 1).contiguous()
    mats = [_matrix(E, d, h, group, g), _matrix(E, d, h, group, g) if act == "swiglu" else (None, None),
            _matrix(E, h, d, group, g)]
    return x, ids.contiguous(), gates, mats


def _load(experts, mats):
    experts.load(*[None if t is None else t.cuda() for m in mats for t in m])


def _check(y, x, ids, gates, mats, group):
    W = [None if q is None else R.int4_weights(q, s, group) for q, s in mats]
    want, bound = R.int4_layer(x, ids, gates, *W)
    R.inside(y, want, bound + R.HALF[BF16] * (want.abs() + bound) + 1e-30, "y")


@pytest.mark.parametrize("L,d,h,E,K,act,group", [
    (1, 128, 128, 1, 1, "swiglu", 128),
    (1, 256, 384, 8, 2, "swiglu", 32),
    (2, 128, 256, 4, 2, "silu", 64),
    (3, 640, 128, 5, 3, "swiglu", 64),
    (7, 384, 896, 8, 2, "swiglu", 128),
    (8, 256, 256, 2, 2, "silu", 32),
    (9, 256, 256, 2, 2, "swiglu", 128),
    (17, 512, 640, 3, 1, "swiglu", 32),
    (33, 128, 128, 2, 1, "swiglu", 64),
    (61, 256, 384, 64, 6, "swiglu", 64),
    (64, 256, 512, 8, 8, "swiglu", 128),
    (65, 128, 256, 4, 2, "swiglu", 32),
    (150, 128, 128, 3, 2, "silu", 128),
    (20, 128, 128, 300, 4, "swiglu", 32),
    (40, 128, 128, 512, 8, "silu", 64),
    (5, 4096, 1408, 4, 2, "swiglu", 128),
    (24, 6144, 256, 2, 1, "swiglu", 64),
    (12, 1408, 7168, 2, 2, "silu", 32),
    (4, 14336, 128, 2, 1, "swiglu", 128),
])
def test_int4_forward(L, d, h, E, K, act, group):
    x, ids, gates, mats = _problem(L, d, h, E, K, act, group, L + d + h)
    ex = Int4Experts(L, d, h, E, K, act, group)
    _load(ex, mats)
    y = ex.forward(x.cuda(), ids.cuda(), gates.cuda())
    torch.cuda.synchronize()
    _check(y, x, ids, gates, mats, group)
    a = y.clone()
    assert torch.equal(a, ex.forward(x.cuda(), ids.cuda(), gates.cuda()))


@pytest.mark.parametrize("L,d,h,E,K,act,group", [
    (8, 128, 2560, 32, 4, "swiglu", 128),
    (24, 128, 2560, 32, 4, "swiglu", 64),
    (20, 256, 2688, 40, 2, "swiglu", 32),
    (9, 128, 5120, 32, 4, "silu", 32),
    (40, 5120, 128, 32, 1, "silu", 128),
])
def test_int4_units_of_a_warp(L, d, h, E, K, act, group):
    """Many units of few rows: a warp takes one by itself."""
    test_int4_forward(L, d, h, E, K, act, group)


def test_int4_fewer_tokens_than_the_buffers_and_skew():
    d, h, E, K, group = 256, 384, 8, 2, 64
    x, ids, gates, mats = _problem(64, d, h, E, K, "swiglu", group, 5)
    ids[:, 0] = 3                                            # every token on one expert
    ids[:, 1] = torch.where(ids[:, 1] == 3, torch.tensor(4, dtype=torch.int32), ids[:, 1])
    ex = Int4Experts(100, d, h, E, K, "swiglu", group)
    _load(ex, mats)
    for n in (64, 1, 40, 0, 33):
        y = ex.forward(x[:n].cuda(), ids[:n].cuda(), gates[:n].cuda())
        torch.cuda.synchronize()
        assert y.shape == (n, d)
        _check(y, x[:n], ids[:n], gates[:n], mats, group)


def test_int4_empty_slots_and_odd_values():
    d, h, E, K, group = 128, 256, 4, 2, 32
    x, ids, gates, mats = _problem(10, d, h, E, K, "swiglu", group, 6)
    ids[2] = -1                                              # a token without experts
    ids[3, 1] = E
    ids[4, 0] = -2 ** 31
    ids[5, 1] = 2 ** 31 - 1
    ids[6] = ids[6, 0]                                       # the same expert twice counts twice
    gates[2] = float("nan")                                  # not read where the slot is empty
    x[2] = float("inf")
    ex = Int4Experts(10, d, h, E, K, "swiglu", group)
    _load(ex, mats)
    y = ex.forward(x.cuda(), ids.cuda(), gates.cuda()).cpu()
    assert not y[2].any()
    keep = [i for i in range(10) if i != 2]
    _check(y[keep], x[keep], ids[keep], gates[keep], mats, group)
    y = ex.forward(x.cuda(), torch.full_like(ids, -1).cuda(), gates.cuda())
    assert not y.any()
    # a token's inf or NaN stays in its row
    x[0, 3] = float("nan")
    y2 = ex.forward(x.cuda(), ids.cuda(), gates.cuda()).cpu()
    assert y2[0].isnan().all()
    _check(y2[keep[1:]], x[keep[1:]], ids[keep[1:]], gates[keep[1:]], mats, group)


@pytest.mark.parametrize("E,rows,cols,group", [(1, 128, 128, 128), (3, 256, 384, 32), (2, 640, 128, 64)])
def test_int4_pack_round_trip(E, rows, cols, group):
    g = torch.Generator().manual_seed(rows)
    q, s = _matrix(E, rows, cols, group, g)
    packed, ps = B.int4_pack(q.cuda(), s.cuda(), group)
    W = B.int4_dequantize(packed, ps, E, rows, cols, group).cpu()
    want = (q.float() * s.float().repeat_interleave(group, dim=1)).to(BF16)
    assert torch.equal(W, want)


@pytest.mark.parametrize("dt", [torch.float32, BF16])
def test_int4_quantize(dt):
    E, rows, cols, group = 2, 256, 128, 64
    W = torch.randn(E, rows, cols, generator=torch.Generator().manual_seed(3)).to(dt)
    W[0, :64, 5] = 0
    q, s = (t.cpu() for t in B.int4_quantize(W.cuda(), group))
    m = W.float().view(E, rows // group, group, cols).abs().amax(2)
    assert torch.equal(s, (m / 7.0).to(BF16))
    sr = s.float().repeat_interleave(group, dim=1)
    want = torch.where(sr > 0, torch.round(W.float() / sr), torch.zeros(())).clamp(-8, 7)
    assert torch.equal(q.float(), want)
    # within half a step of the weight (the clamp takes at most what rounding the scale to bf16 adds)
    assert ((q.float() * sr - W.float()).abs() <= sr * (0.5 + 7 * 2.0 ** -8) + 1e-7).all()


def test_int4_serving_matches_the_layer_on_dequantised_weights():
    """Norm, router and 4-bit experts of a decode batch against the bf16 layer on the weights they stand for."""
    from mixture_experts_atomic_gb300.block import LayerNorm
    L, d, h, E, K, group = 24, 256, 512, 8, 2, 64
    g = torch.Generator().manual_seed(12)
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    W1, W2, W3 = r(E, d, h) / 16, r(E, d, h) / 16, r(E, h, d) / 22
    ex = Int4Experts(L, d, h, E, K, "swiglu", group)
    ex.quantize(W1.to(BF16), W2.to(BF16), W3.to(BF16))
    x, res = r(L, d).to(BF16), r(L, d).to(BF16)
    norm = LayerNorm(L, d, BF16)
    u, s, _, _ = norm.forward(x, torch.ones(d, device="cuda"), None, res)
    layer = MoELayer(L, d, h, E, K, BF16, "swiglu")
    ids, gates = layer.route(u, r(d, E) / 16)
    y4 = ex.forward(u, ids, gates)
    y16 = layer.forward(u, gates, *ex.dequantize())
    torch.cuda.synchronize()
    # the layer rounds its weights (2^-8), A, B, H and y to bf16: the layer's own tolerance
    assert (y4.float() - y16.float()).abs().max() <= 2e-2 * y16.float().abs().max()


def test_int4_streams_and_graph():
    d, h, E, K, group = 256, 384, 8, 2, 128
    x, ids, gates, mats = _problem(6, d, h, E, K, "swiglu", group, 21)
    ex = Int4Experts(6, d, h, E, K, "swiglu", group)
    _load(ex, mats)
    x, ids, gates = x.cuda(), ids.cuda(), gates.cuda()
    want = ex.forward(x, ids, gates).clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = ex.forward(x, ids, gates).clone()
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ex.forward(x, ids, gates)
    for _ in range(3):  # replays back to back: each has to see its own predecessor finished
        y.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("L,d,h,E,K,act,group", [
    (1, 4096, 256, 4, 2, "swiglu", 128),
    (1, 256, 384, 8, 8, "silu", 64),
    (2, 640, 128, 3, 3, "swiglu", 32),
    (3, 256, 256, 2, 2, "swiglu", 128),
    (9, 128, 256, 8, 8, "swiglu", 64),
    (64, 128, 128, 8, 8, "silu", 128),
])
def test_int4_tokens_that_name_an_expert_more_than_once(L, d, h, E, K, act, group):
    """An expert may have more pairs than there are tokens: each slot counts."""
    x, ids, gates, mats = _problem(L, d, h, E, K, act, group, 3 * L + K)
    ex = Int4Experts(L, d, h, E, K, act, group)
    _load(ex, mats)
    for same in (E - 1, 0):
        ids[:] = same
        if L > 2:
            ids[1, 0] = (same + 1) % E
        y = ex.forward(x.cuda(), ids.cuda(), gates.cuda())
        torch.cuda.synchronize()
        _check(y, x, ids, gates, mats, group)


@pytest.mark.parametrize("L,d,h,E,K,act,group", [
    (16, 128, 128 * 67, 2, 2, "swiglu", 64),
    (20, 256, 128 * 107, 2, 1, "silu", 32),
    (64, 128, 128 * 86, 3, 2, "swiglu", 128),
    (5, 128, 128 * 131, 2, 2, "silu", 128),
    (1, 256, 128 * 433, 2, 1, "swiglu", 128),
    (16, 384, 128 * 73, 4, 1, "swiglu", 32),
    (23, 1152, 128 * 59, 2, 2, "swiglu", 64),
    (33, 128, 128 * 1031, 1, 1, "silu", 64),
])
def test_int4_reductions_in_unequal_slices(L, d, h, E, K, act, group):
    """h / 128 without a divisor that fits: slices of n and n + 1 pieces."""
    test_int4_forward(L, d, h, E, K, act, group)


@pytest.mark.parametrize("dt", [torch.float32, BF16])
def test_int4_quantize_of_what_is_not_finite(dt):
    """A NaN or an infinity shows: its group's weights are NaN, and so are the rows that meet them; others are not."""
    E, d, h, group = 2, 128, 128, 64
    g = torch.Generator().manual_seed(8)
    W = torch.randn(E, d, h, generator=g)
    W[0, 5, 7], W[0, 70, 9], W[0, 127, 11] = float("nan"), float("inf"), -float("inf")
    W[0, 64:, 12] = float("nan")
    ex = Int4Experts(2, d, h, E, 1, "silu", group)
    W3 = torch.randn(E, h, d, generator=g) / 16
    ex.quantize(W.to(dt).cuda(), None, W3.to(dt).cuda())
    got = ex.dequantize()[0].cpu()
    bad = torch.zeros(E, d, h, dtype=torch.bool)
    bad[0, :64, 7] = bad[0, 64:, 9] = bad[0, 64:, 11] = bad[0, 64:, 12] = True
    assert got[bad].isnan().all() and got[~bad].isfinite().all()
    x = torch.randn(2, d, generator=g).to(BF16).cuda()
    y = ex.forward(x, torch.tensor([[0], [1]], dtype=torch.int32, device="cuda"), torch.ones(2, 1, device="cuda")).cpu()
    assert y[0].isnan().all() and y[1].isfinite().all()
