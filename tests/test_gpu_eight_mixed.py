"""The operators in 8 bits beside each other and beside the layer's on one GPU, and
at sizes whose offsets pass 32 bits."""
import threading

import pytest
import torch

from mixture_experts_atomic_gb300.block import MoEBlock, RMSNorm
from mixture_experts_atomic_gb300.fp8 import Fp8Experts, dequantize_rows, quantize_rows
from mixture_experts_atomic_gb300.int4 import Int4Experts

pytestmark = pytest.mark.gpu

from gpu_util import ensure_built  # noqa: E402

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _r(g, *s):
    return torch.randn(*s, device="cuda", generator=g)


def _routing(g, L, E, K):
    return (torch.rand(L, E, device="cuda", generator=g).topk(K, 1).indices.int().contiguous(),
            torch.rand(L, K, device="cuda", generator=g))


def _weights(g, E, d, h):
    return ((_r(g, E, d, h) / d ** 0.5).to(BF16), (_r(g, E, d, h) / d ** 0.5).to(BF16), (_r(g, E, h, d) / h ** 0.5).to(BF16))


def _serve(cls, L, d, h, E, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ex = cls(L, d, h, E, K)
    ex.quantize(*_weights(g, E, d, h))
    x = _r(g, L, d).to(BF16)
    ids, gates = _routing(g, L, E, K)
    return lambda: [ex.forward(x, ids, gates)]


def _train(L, d, h, E, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    block = MoEBlock(L, d, h, E, K, BF16, norm="rms", checkpoint8=True)
    W1, W2, W3 = _weights(g, E, d, h)
    p = {"norm_w": 1 + 0.1 * _r(g, d), "Wr": _r(g, d, E) / d ** 0.5, "W1": W1, "W2": W2, "W3": W3}
    x, res, dout = (_r(g, L, d).to(BF16) for _ in range(3))
    dl = torch.tensor([0.01, 0.001], device="cuda")

    def call():
        out, s, losses, _ = block.forward(x, res, p)
        grads = block.backward(dout, dl, p)
        return [out, s, losses] + [grads[k] for k in ("W1", "W2", "W3", "Wr", "bias", "norm_w", "x")]
    return call


# The gradient of a gate is a sum over the hidden columns' tiles (three of them here), which are added as they come: two
# orders of three fp32 numbers differ by two half steps, 2^-23 of their sizes' sum, which may be some 2^6 times the sum
# itself; Wr and bias follow it.  Through the router it reaches x and norm_w by way of bf16, where it can tip a
# rounding: a step, 2^-7 of the value.
LOOSE = {6: 2.0 ** -17, 7: 2.0 ** -17, 8: 2.0 ** -7, 9: 2.0 ** -7}


def _same(job, got, want):
    loose = LOOSE if job == 0 else {}
    return all(float((a.double() - b.double()).norm() / b.double().norm()) <= loose[k] if k in loose else torch.equal(a, b)
               for k, (a, b) in enumerate(zip(got, want)))


def test_training_and_serving_side_by_side():
    """A training step, a decode batch and a prompt in 8 bits, and a decode batch in 4 bits, from host threads on their
    own streams: tensor memory and SMs are shared, results are those of a call alone, to the bit where sums have an
    order."""
    jobs = [_train(700, 512, 640, 8, 2, 1), _serve(Fp8Experts, 61, 640, 896, 48, 3, 2),
            _serve(Fp8Experts, 1500, 512, 640, 8, 2, 3), _serve(Int4Experts, 16, 512, 1024, 8, 2, 4)]
    alone = [[t.clone() for t in job()] for job in jobs]
    torch.cuda.synchronize()
    bad, start = [], threading.Barrier(len(jobs))

    def work(i):
        stream = torch.cuda.Stream()
        start.wait()
        with torch.cuda.stream(stream):
            for _ in range(60):
                out = jobs[i]()
            if not _same(i, out, alone[i]):
                bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not bad, bad


def test_rows_past_32_bits():
    """2.2e9 elements: rows at the start, around element 2^31 and at the end are those of a small call."""
    L, d = 540000, 4096
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.empty(L, d, dtype=BF16, device="cuda")
    for i in range(0, L, 60000):
        x[i:i + 60000] = _r(g, min(60000, L - i), d)
    w = 1 + 0.1 * _r(g, d)
    q, s = quantize_rows(x)
    v = dequantize_rows(q, s)
    big, small = RMSNorm(L, d, BF16), RMSNorm(64, d, BF16)
    q8, s8, y, _, rstd = big.forward8(x, w)
    dx, _ = big.backward(y, x, rstd, w)
    for at in (0, 2 ** 31 // d - 3, L - 64):
        part = slice(at, at + 64)
        xp = x[part].contiguous()
        qp, sp = quantize_rows(xp)
        assert torch.equal(q[part].view(torch.uint8), qp.view(torch.uint8)) and torch.equal(s[part], sp)
        assert torch.equal(v[part], dequantize_rows(qp, sp))
        qp, sp, yp, _, rp = small.forward8(xp, w)
        assert torch.equal(q8[part].view(torch.uint8), qp.view(torch.uint8)) and torch.equal(s8[part], sp)
        assert torch.equal(y[part], yp) and torch.equal(rstd[part], rp)
        assert torch.equal(dx[part], small.backward(yp, xp, rp, w)[0])


def test_experts_past_32_bits():
    """170,000 routed rows of 14,336 hidden columns: tokens anywhere in a long prompt are those of a short one."""
    L, d, h, E, K = 85000, 1024, 14336, 4, 2
    g = torch.Generator(device="cuda").manual_seed(6)
    W = _weights(g, E, d, h)
    ex, short = Fp8Experts(L, d, h, E, K), Fp8Experts(1000, d, h, E, K)
    ex.quantize(*W), short.quantize(*W)
    x = _r(g, L, d).to(BF16)
    ids, gates = _routing(g, L, E, K)
    y = ex.forward(x, ids, gates)
    for at in (0, L // 2, L - 1000):
        part = slice(at, at + 1000)
        assert torch.equal(y[part], short.forward(x[part], ids[part], gates[part]))
