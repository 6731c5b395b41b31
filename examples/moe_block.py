"""The block around the layer, as a training and as a serving program use it.

    python examples/moe_block.py [--tokens N] [--steps S]

train(): steps of a pre-norm MoE block (layer norm with the residual sum,
router with its balance and z loss, dropless experts) with a plain gradient
step on every parameter, captured once as a CUDA graph and replayed.
With norm="rms" and checkpoint8 the block has a root-mean-square norm and
keeps its checkpoints in 8 bits.
serve(): the trained experts quantised to 4 bits, and a decode batch sent
through norm, router and 4-bit experts.
serve8(): the experts in 8-bit floating point, on rows that the RMS norm
leaves in 8 bits: a prompt, or a decode batch.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from mixture_experts_atomic_gb300 import binding as B  # noqa: E402
from mixture_experts_atomic_gb300.block import LayerNorm, MoEBlock, RMSNorm  # noqa: E402
from mixture_experts_atomic_gb300.fp8 import Fp8Experts, dequantize_rows  # noqa: E402
from mixture_experts_atomic_gb300.int4 import Int4Experts  # noqa: E402


def parameters(d, h, E, dtype, seed=0, norm="layer"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    p = {"norm_w": torch.ones(d, device="cuda")}
    if norm == "layer":
        p["norm_b"] = torch.zeros(d, device="cuda")
    p.update({"Wr": r(d, E) / d ** 0.5, "bias": torch.zeros(E, device="cuda"),
              "W1": (r(E, d, h) / d ** 0.5).to(dtype), "W2": (r(E, d, h) / d ** 0.5).to(dtype),
              "W3": (r(E, h, d) / h ** 0.5).to(dtype)})
    return p


def train(L, d, h, E, K, steps, lr=0.05, dtype=torch.bfloat16, norm="layer", checkpoint8=False):
    """The block learns to map x to a fixed target; returns (parameters, history) with the mean squared error, the
    balance loss and the largest expert's share of the slots of each step."""
    p = parameters(d, h, E, dtype, norm=norm)
    block = MoEBlock(L, d, h, E, K, dtype, norm=norm, checkpoint8=checkpoint8)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, res = (torch.randn(L, d, device="cuda", generator=g).to(dtype) for _ in range(2))
    target = torch.randn(L, d, device="cuda", generator=g) * 0.5
    valid = torch.ones(L, dtype=torch.uint8, device="cuda")
    valid[-L // 16:] = 0                     # padding at the batch's end: out of the losses
    dlosses = torch.tensor([0.02, 0.002], device="cuda")
    mse = torch.zeros((), device="cuda")

    def step():
        out, _, losses, counts = block.forward(x, res, p, valid)
        err = (out.float() - target) * valid[:, None]
        mse.copy_(err.square().mean())
        grads = block.backward((err * (2.0 / L)).to(dtype), dlosses, p)
        for k, v in p.items():
            v.sub_((grads[k].float() * lr).to(v.dtype))
        return losses, counts

    step()                                   # sizes and kernel attributes are settled outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        losses, counts = step()
    history = []
    for _ in range(steps):
        graph.replay()
        history.append((float(mse), float(losses[0]), float(counts.max()) / max(1, int(counts.sum()))))
    assert block.layer.device_error() == 0
    return p, history


def serve(p, tokens, K, group=128):
    """One decode batch on the 4-bit experts; returns (y on 4 bits, y of the bf16 layer on the weights those stand for)."""
    E, d, h = p["W1"].shape
    experts = Int4Experts(tokens, d, h, E, K, "swiglu", group)
    experts.quantize(p["W1"], p["W2"], p["W3"])
    norm = LayerNorm(tokens, d, torch.bfloat16)
    x, res = (torch.randn(tokens, d, device="cuda").to(torch.bfloat16) for _ in range(2))
    u, _, _, _ = norm.forward(x, p["norm_w"], p["norm_b"], res)
    shape = B.make_shape(tokens, d, h, E, K, torch.bfloat16, "swiglu")
    ids = torch.empty(tokens, K, dtype=torch.int32, device="cuda")
    gates = torch.empty(tokens, K, device="cuda")
    B.router_forward(shape, u, p["Wr"], p["bias"], ids, gates)
    y = experts.forward(u, ids, gates)
    # the same batch as a prompt would run: the weights widened, the bf16 layer
    from mixture_experts_atomic_gb300.layer import MoELayer
    layer = MoELayer(tokens, d, h, E, K, torch.bfloat16, "swiglu")
    layer.dispatch(ids)
    return y, layer.forward(u, gates, *experts.dequantize())


def serve8(p, tokens, K):
    """tokens rows on the 8-bit experts; returns (y in 8 bits, y of the bf16 layer on the rows and weights that the
    8 bits stand for)."""
    from mixture_experts_atomic_gb300.layer import MoELayer
    E, d, h = p["W1"].shape
    experts = Fp8Experts(tokens, d, h, E, K, "swiglu")
    experts.quantize(p["W1"], p["W2"], p["W3"])
    norm = RMSNorm(tokens, d, torch.bfloat16)
    x, res = (torch.randn(tokens, d, device="cuda").to(torch.bfloat16) for _ in range(2))
    q, scales, u, _, _ = norm.forward8(x, p["norm_w"], res)
    layer = MoELayer(tokens, d, h, E, K, torch.bfloat16, "swiglu")
    ids, gates = layer.route(u, p["Wr"], p["bias"])
    y = experts.forward(q, ids, gates, scales)
    return y, layer.forward(dequantize_rows(q, scales), gates, *experts.dequantize())


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=50)
    a = ap.parse_args()
    p, history = train(a.tokens, 512, 1024, 8, 2, a.steps)
    for i in (0, len(history) // 2, len(history) - 1):
        print("step %3d  mse %.4f  balance %.4f  largest expert's share %.3f" % (i, *history[i]))
    y4, y16 = serve(p, 16, 2)
    print("4-bit experts against the bf16 layer on the same weights: rel %.2e"
          % float((y4.float() - y16.float()).norm() / y16.float().norm()))
    p, history = train(a.tokens, 512, 1024, 8, 2, a.steps, norm="rms", checkpoint8=True)
    print("RMS norm, checkpoints in 8 bits: last step's mse %.4f" % history[-1][0])
    for tokens in (a.tokens, 16):
        y8, y16 = serve8(p, tokens, 2)
        print("%d tokens: 8-bit experts against the bf16 layer on the same rows and weights: rel %.2e"
              % (tokens, float((y8.float() - y16.float()).norm() / y16.float().norm())))


if __name__ == "__main__":
    main()
