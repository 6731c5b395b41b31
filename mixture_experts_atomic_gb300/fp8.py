"""8-bit floating point: rows with a scale for each 128 columns, as the RMS
norm leaves them (block.RMSNorm.forward8), and the layer's forward on expert
weights with a scale for each 128 x 128 (serving, one token to long prompts):
`Fp8Experts` keeps the weights and the buffers of one layer and runs
moeblaze_fp8_forward on the current CUDA stream, straight from the router's ids
and gates."""
from __future__ import annotations

from typing import Optional

import torch

from . import binding as B


def quantize_rows(x):
    """(q, scales) of x (L,d) bf16 or fp32: q (L,d) float8_e4m3fn, scales (L, ceil(d/128)) fp32, powers of two."""
    return B.fp8_quantize_rows(x)


def dequantize_rows(q, scales, dtype=torch.bfloat16):
    """What 8-bit rows stand for, (L,d) in dtype (bf16 or fp32)."""
    return B.fp8_dequantize_rows(q, scales, dtype)


class Fp8Experts:
    def __init__(self, max_tokens: int, d: int, h: int, E: int, K: int, act: str = "swiglu", device="cuda"):
        """Buffers for up to max_tokens tokens a call; the weights come with load or quantize."""
        self.max_tokens, self.d, self.h, self.E, self.K = max_tokens, d, h, E, K
        self.act, self.device = act, device
        n = B.moeblaze_fp8_workspace_bytes(self._shape(max_tokens))
        if max_tokens > 0 and n == 0:
            raise B.MoEBlazeError(B.ERR_UNSUPPORTED, "moeblaze_fp8_workspace_bytes")
        self._ws = B._bytes(n, device)
        self._y = torch.empty((max_tokens, d), dtype=torch.bfloat16, device=device)
        self._packed: dict = {}
        self._weights: Optional[B.Fp8Weights] = None
        self._shapes: dict = {}

    def _shape(self, L: int) -> B.Shape:
        return B.make_shape(L, self.d, self.h, self.E, self.K, torch.bfloat16, self.act)

    def load(self, q1, s1, q2, s2, q3, s3):
        """Pack 8-bit weights: q1, q2 (E,h,d), q3 (E,d,h) float8_e4m3fn, each output's row along the reduction, and
        fp32 scales (E,N/128,R/128) of each 128 x 128 (q2, s2 None for SiLU).  The copies replace earlier ones in
        place, all of them or, when a tensor is refused, none."""
        mats = [("1", q1, s1, self.h, self.d), ("3", q3, s3, self.d, self.h)]
        if self.act == "swiglu":
            mats.insert(1, ("2", q2, s2, self.h, self.d))
        specs = []
        for n, q, s, N, R in mats:
            specs += [(q, "q" + n, (self.E, N, R), torch.float8_e4m3fn, False),
                      (s, "s" + n, (self.E, N // 128, R // 128), torch.float32, False)]
        B._args(*specs)
        for t, name, *_ in specs:
            if t.device != self._ws.device:  # the products read the weights beside the buffers
                raise ValueError(f"{name}: on {t.device}, but the buffers are on {self._ws.device}")
        for n, q, s, N, R in mats:
            old = self._packed.get(n)
            packed = B.fp8_pack(q, None if old is None else old[0])
            self._packed[n] = (packed, s.clone() if old is None else old[1].copy_(s))
        p = {n: tuple(t.data_ptr() for t in v) for n, v in self._packed.items()}
        w1, w2, w3 = p["1"], p.get("2", (None, None)), p["3"]
        self._weights = B.Fp8Weights(w1[0], w1[1], w2[0], w2[1], w3[0], w3[1])

    def quantize(self, W1, W2, W3):
        """Quantise bf16 or fp32 weights in the layer's layout (W2 None for SiLU)."""
        q1, s1 = B.fp8_quantize_weights(W1)
        q2, s2 = B.fp8_quantize_weights(W2) if self.act == "swiglu" else (None, None)
        q3, s3 = B.fp8_quantize_weights(W3)
        self.load(q1, s1, q2, s2, q3, s3)

    def dequantize(self):
        """(W1, W2, W3) in bf16, as MoELayer.forward takes them (W2 None for SiLU)."""
        if self._weights is None:
            raise RuntimeError("Fp8Experts: load or quantize weights first")
        return tuple(B.fp8_dequantize_weights(*self._packed[n]) if n in self._packed else None for n in "123")

    def forward(self, x, topk_ids, gates, x_scales=None) -> torch.Tensor:
        """y (L,d) for the L <= max_tokens rows of x: bf16, or 8-bit rows with their scales (RMSNorm.forward8,
        quantize_rows).  ids outside [0,E) are empty slots.  y is this object's buffer: the next call overwrites it."""
        if self._weights is None:
            raise RuntimeError("Fp8Experts: load or quantize weights first")
        L = x.shape[0]
        if L > self.max_tokens:
            raise ValueError(f"x: {L} tokens, at most {self.max_tokens}")
        shape = self._shapes.get(L)
        if shape is None:
            shape = self._shapes[L] = self._shape(L)
        return B.fp8_forward(shape, x, x_scales, topk_ids, gates, self._weights, self._y[:L], self._ws, self._ws.numel())
