"""The operators in 8 bits as a program uses them, on the GPU: host threads
side by side, the training and the serving example, and the smallest calls."""
import importlib.util
import os
import threading

import pytest
import torch

import eight_ref as R
from mixture_experts_atomic_gb300 import binding as B
from mixture_experts_atomic_gb300.block import RMSNorm
from mixture_experts_atomic_gb300.fp8 import Fp8Experts
from mixture_experts_atomic_gb300.layer import MoELayer

pytestmark = pytest.mark.gpu

from gpu_util import ensure_built  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
ROUNDS = 300


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _rms(L, d, dt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, w, dy = (torch.randn(*s, device="cuda", generator=g) for s in ((L, d), (d,), (L, d)))
    x, dy, n = x.to(dt), dy.to(dt), RMSNorm(L, d, dt)

    def call():
        y, s, rstd = n.forward(x, w)
        dx, dw = n.backward(dy, s, rstd, w)
        return y, rstd, dx, dw
    return call


def _fp8(L, d, h, E, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: (torch.randn(*s, device="cuda", generator=g) / 16).to(BF16)  # noqa: E731
    ex = Fp8Experts(L, d, h, E, K)
    ex.quantize(r(E, d, h), r(E, d, h), r(E, h, d))
    x = r(L, d) * 16
    ids = torch.rand(L, E, device="cuda", generator=g).topk(K, 1).indices.int().contiguous()
    gates = torch.rand(L, K, device="cuda", generator=g)
    return lambda: (ex.forward(x, ids, gates),)


def _layer8(L, d, h, E, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: (torch.randn(*s, device="cuda", generator=g) / 16).to(BF16)  # noqa: E731
    W, x, dy = (r(E, d, h), r(E, d, h), r(E, h, d)), r(L, d) * 16, r(L, d)
    ids = torch.rand(L, E, device="cuda", generator=g).topk(K, 1).indices.int().contiguous()
    gates = torch.rand(L, K, device="cuda", generator=g)
    layer = MoELayer(L, d, h, E, K, BF16, "swiglu", checkpoint8=True)

    def call():
        layer.dispatch(ids)
        layer.forward(x, gates, *W)
        return layer.saved()
    return call


@pytest.mark.parametrize("make,shapes", [
    (_rms, [(64, 4200, BF16), (64, 5120, BF16)]),
    (_rms, [(64, 513, F32), (64, 4992, F32)]),
    (_fp8, [(5, 256, 512, 4, 2), (3, 1024, 256, 8, 3)]),
    (_fp8, [(300, 256, 512, 4, 2), (700, 512, 256, 8, 1)]),
    (_fp8, [(5, 256, 512, 4, 2), (700, 512, 256, 8, 1)]),
    (_layer8, [(300, 256, 512, 4, 2), (700, 512, 256, 2, 1)]),
], ids=["rms_bf16", "rms_f32", "few", "prompts", "both", "checkpoint8"])
def test_threads_side_by_side(make, shapes):
    """Host threads on their own streams, with buffers of their own: each one's results are those of a call alone,
    to the bit."""
    jobs = [make(*shapes[i % 2], i) for i in range(4)]
    alone = [[t.clone() for t in job()] for job in jobs]
    torch.cuda.synchronize()
    bad, start = [], threading.Barrier(len(jobs))

    def work(i):
        stream = torch.cuda.Stream()
        start.wait()
        with torch.cuda.stream(stream):
            for _ in range(ROUNDS):
                out = jobs[i]()
            if not all(torch.equal(a, b) for a, b in zip(out, alone[i])):
                bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not bad, bad


def test_example_in_8_bits():
    """The example's block with an RMS norm and checkpoints in 8 bits runs its captured steps, and its experts in 8
    bits agree with the bf16 layer on the same rows and weights."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")
    spec = importlib.util.spec_from_file_location("moe_block_example_8", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    p, history = m.train(512, 256, 256, 8, 2, 5, norm="rms", checkpoint8=True)
    assert all(torch.isfinite(torch.tensor(history[i])).all() for i in range(5))
    assert all(bool(v.isfinite().all()) for v in p.values())
    for tokens in (7, 512):
        y8, y16 = m.serve8(p, tokens, 2)
        # the hidden values round to e4m3, by 2^-4 of each at most; the rest are roundings to bf16
        assert float((y8.double() - y16.double()).norm() / y16.double().norm()) <= 2 ** -4 + 4 * 2 ** -8


@pytest.mark.parametrize("L,E,K", [(1, 1, 1), (1, 8, 8), (24, 1, 1), (25, 1, 1), (49, 2, 1), (256, 64, 6), (257, 64, 6),
                                   (4096, 400, 1), (4097, 400, 1), (1024, 300, 4)])
def test_fp8_where_the_paths_meet(L, E, K):
    """The smallest layer, and either side of the number of tokens from which the products take another path, with
    repeated slots: an expert twice in a token counts twice."""
    d = h = 128
    g = torch.Generator().manual_seed(L + E)
    mats = []
    for _ in range(3):
        mats += [(100 * torch.randn(E, 128, 128, generator=g)).clamp(-448, 448).to(torch.float8_e4m3fn).cuda(),
                 ((0.5 + torch.rand(E, 1, 1, generator=g)) / 1100).cuda()]
    x = torch.randn(L, d, generator=g).to(BF16).cuda()
    ids = torch.randint(0, E, (L, K), generator=g).int().cuda()
    gates = torch.randn(L, K, generator=g).cuda()
    ex = Fp8Experts(L, d, h, E, K)
    ex.load(*mats)
    y = ex.forward(x, ids, gates)
    q, s = R.rows8(x)
    want, bound = R.experts8(q * R.grown(s, d), ids, gates, mats)
    R.inside(y, want, bound + R.BF * (want.abs() + bound) + 1e-30, "y")
