"""The two paths of the products on 8-bit weights, for few tokens and for prompts,
on either side of the number of tokens where one takes over from the other: tiles
in parts, half tiles, several tiles of an expert's tokens, both activations, even
and skewed routing, against fp64 (eight_ref.experts8).  Which path a call took
shows in its launches: four for few tokens, five or six for prompts."""
import threading

import pytest
import torch

import eight_ref as R
from mixture_experts_atomic_gb300 import binding as B
from mixture_experts_atomic_gb300 import fp8
from mixture_experts_atomic_gb300.fp8 import Fp8Experts
from test_gpu_fp8 import _check, _problem

pytestmark = pytest.mark.gpu

from gpu_util import ensure_built  # noqa: E402

BF16 = torch.bfloat16
FEW, PROMPT = 4, 5


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _call(ex, *args):
    before = B.moeblaze_kernel_launches()
    y = ex.forward(*args)
    return y, min(B.moeblaze_kernel_launches() - before, PROMPT)


# (d, h, E, K, act, most tokens of the path for few)
LAYERS = [
    (1024, 1280, 16, 2, "swiglu", 96),          # 12 slots an expert
    (640, 896, 48, 3, "swiglu", 192),           # d and h with half a tile of 256 columns
    (384, 640, 128, 4, "silu", 384),            # the same
    (256, 384, 200, 7, "swiglu", 342),          # 342.9 tokens
    (2816, 1408, 4, 1, "swiglu", 80),           # 20 slots; reductions of 22 and 11 blocks
    (4096, 2048, 8, 8, "silu", 20),             # K == E
    (128, 128, 512, 1, "swiglu", 4096),         # one block; 4,096 slots
    (2048, 2048, 1, 1, "swiglu", 20),           # one expert
]


@pytest.mark.parametrize("one", [False, True], ids=["even", "one"])
@pytest.mark.parametrize("d,h,E,K,act,most", LAYERS)
def test_either_side_of_the_border(d, h, E, K, act, most, one):
    x, ids, gates, mats = _problem(most + 1, d, h, E, K, act, d + h + E, E // 2 if one and E > 1 else None)
    if one:
        ids[most // 2:, K - 1] = ids[0, 0]       # an expert twice in a token, where K > 1
    ex = Fp8Experts(most + 1, d, h, E, K, act)
    ex.load(*mats)
    for L, path in ((most + 1, PROMPT), (most, FEW), (1, FEW), (min(3, most), FEW)):
        args = x[:L], ids[:L], gates[:L]
        y, took = _call(ex, *args)
        assert took == path, (L, took)
        y = y.clone()
        _check(y, *args, mats)
        q, s = fp8.quantize_rows(x[:L])
        assert torch.equal(y, ex.forward(q, ids[:L], gates[:L], s))
        assert torch.equal(y, ex.forward(*args))


@pytest.mark.parametrize("d,h,E,K,act", [(512, 1024, 8, 2, "swiglu"), (1024, 1024, 4, 2, "swiglu"), (128, 128, 4, 2, "silu"),
                                         (1024, 4096, 8, 2, "silu"), (128, 128, 1, 1, "swiglu")])
def test_the_smallest_layers_take_the_prompts_path(d, h, E, K, act):
    x, ids, gates, mats = _problem(33, d, h, E, K, act, d + h)
    ex = Fp8Experts(33, d, h, E, K, act)
    ex.load(*mats)
    for L in (1, 2, 33):
        y, took = _call(ex, x[:L], ids[:L], gates[:L])
        assert took == PROMPT
        _check(y, x[:L], ids[:L], gates[:L], mats)


def test_few_tokens_empty_slots_and_odd_values():
    d, h, E, K, L = 640, 896, 48, 3, 40
    x, ids, gates, mats = _problem(L, d, h, E, K, "swiglu", 6)
    ids[0] = -1                                  # a token without experts
    gates[0] = float("nan")                      # not read where the slot is empty
    x[0] = float("inf")
    ids[3, 1], ids[4, 0], ids[5, 1] = E, -2 ** 31, 2 ** 31 - 1
    ids[6] = ids[6, 0].clone()                   # the same expert three times counts three times
    x[8, 5] = float("nan")
    x[9] = 0
    ex = Fp8Experts(L, d, h, E, K)
    ex.load(*mats)
    y, took = _call(ex, x, ids, gates)
    assert took == FEW
    assert float(y[0].float().abs().max()) == 0 and y[8].isnan().all() and float(y[9].float().abs().max()) == 0
    keep = [t for t in range(L) if t not in (0, 8)]
    _check(y[keep], x[keep], ids[keep], gates[keep], mats)
    ids[:] = -1
    assert float(ex.forward(x, ids, gates).float().abs().max()) == 0


def test_few_tokens_any_scales():
    d, h, E, K, L = 640, 896, 48, 3, 61
    x, ids, gates, mats = _problem(L, d, h, E, K, "swiglu", 4)
    q, s = fp8.quantize_rows(x)
    s = s * (0.3 + torch.rand(s.shape, generator=torch.Generator().manual_seed(5))).cuda()
    s[7] *= 1e-20
    ex = Fp8Experts(L, d, h, E, K)
    ex.load(*mats)
    y, took = _call(ex, q, ids, gates, s)
    assert took == FEW
    want, bound = R.experts8(q.double() * R.grown(s, d), ids, gates, mats)
    R.inside(y, want, bound + R.BF * (want.abs() + bound) + 1e-30, "y")


def test_few_tokens_captured_on_streams_and_from_threads():
    """Two objects at once, on two streams and from host threads, and a captured call replayed on new inputs."""
    d, h, E, K, L = 640, 896, 48, 3, 61
    probs = [_problem(L, d, h, E, K, "swiglu", s) for s in (7, 8)]
    exs = [Fp8Experts(L, d, h, E, K) for _ in probs]
    want = []
    for ex, (x, ids, gates, mats) in zip(exs, probs):
        ex.load(*mats)
        y, took = _call(ex, x, ids, gates)
        assert took == FEW
        want.append(y.clone())
    other = exs[0].forward(*probs[1][:3]).clone()
    torch.cuda.synchronize()
    bad, start = [], threading.Barrier(2)

    def work(i):
        stream = torch.cuda.Stream()
        start.wait()
        with torch.cuda.stream(stream):
            for _ in range(200):
                y = exs[i].forward(*probs[i][:3])
            if not torch.equal(y, want[i]):
                bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not bad, bad
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = exs[0].forward(*probs[0][:3])
    for a, b in zip(probs[0][:3], probs[1][:3]):
        a.copy_(b)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, other)


def test_few_tokens_wait_limit():
    """A product whose first stage is never loaded gives up after the wait limit: y is NaN, and the next call is whole."""
    d, h, E, K, L = 640, 896, 48, 3, 8
    x, ids, gates, mats = _problem(L, d, h, E, K, "swiglu", 9)
    ex = Fp8Experts(L, d, h, E, K)
    ex.load(*mats)
    y, took = _call(ex, x, ids, gates)
    assert took == FEW
    want = y.clone()
    torch.cuda.synchronize()
    B.moeblaze_set_fault_injection(20_000_000, 1)
    try:
        y = ex.forward(x, ids, gates)
        torch.cuda.synchronize()
    finally:
        B.moeblaze_set_fault_injection(0, 0)
    assert bool(y.isnan().all())
    assert torch.equal(ex.forward(x, ids, gates), want)
