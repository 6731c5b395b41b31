"""The weight gradients on either side of the rule for 256-row tiles (on the
152 SMs of a GB300: below half of them, up to one tile each, up to one and a half,
beyond; few and many rows an expert; a last half tile), against fp64 at the
values that the 8-bit checkpoints stand for."""
import pytest
import torch

import eight_ref as R
from mixture_experts_atomic_gb300.layer import MoELayer
from test_gpu_checkpoint8 import _args, _backward, _forward, _kept, _problem

pytestmark = pytest.mark.gpu

from gpu_util import ensure_built  # noqa: E402

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


# 256-row tiles of dW1 (or dW1 || dW2) and of dW3
SHAPES = [
    (600, 512, 512, 4, 2, "silu"),          # 16 and 16
    (1100, 1024, 640, 8, 2, "silu"),        # 96 and 96, both with half tiles
    (1100, 1024, 640, 8, 2, "swiglu"),      # 160 and 96
    (1000, 1024, 640, 8, 2, "swiglu"),      # the same, below 256 rows an expert
    (1600, 512, 1024, 22, 4, "silu"),       # 176 and 176
    (1400, 1024, 1280, 8, 2, "silu"),       # 160 and 160
    (1500, 1024, 1920, 8, 2, "silu"),       # 256 and 256
    (9000, 512, 512, 2, 1, "swiglu"),       # 16 and 8, 4,500 rows an expert
    (9000, 1024, 2432, 2, 1, "silu"),       # 80 and 80, the same
]


@pytest.mark.parametrize("L,d,h,E,K,act", SHAPES)
def test_weight_gradients_on_either_tile(L, d, h, E, K, act):
    p = _problem(L, d, h, E, K, act, L + d + h)
    layer = MoELayer(L, d, h, E, K, BF16, act, checkpoint8=True)
    _forward(layer, p)
    A, _, Bv, _ = _kept(layer, p)
    got = _backward(layer, p)
    want, tol = R.layer_backward(*_args(p, "dY", "x", "ids", "gates", "W1", "W2", "W3"), A, Bv)
    for n in ("dW1", "dW2", "dW3"):
        if n in want:
            R.inside(got[n], want[n], tol[n] + R.BF * (want[n].abs() + tol[n]) + 1e-30, n)
