"""Expert weights held in 4 bits with group scales, and the layer's forward on
them for few tokens (serving): `Int4Experts` keeps the packed weights and the
buffers of one layer and runs moeblaze_int4_forward on the current CUDA
stream, straight from the router's ids and gates."""
from __future__ import annotations

from typing import Optional

import torch

from . import binding as B


class Int4Experts:
    def __init__(self, max_tokens: int, d: int, h: int, E: int, K: int, act: str = "swiglu", group: int = 128,
                 device="cuda"):
        """Buffers for up to max_tokens tokens a call; the weights come with load or quantize."""
        self.max_tokens, self.d, self.h, self.E, self.K = max_tokens, d, h, E, K
        self.act, self.group, self.device = act, group, device
        # a call's scratch depends on its tokens: with 64 or more, on the 64 of a launch and on the rest of the last
        # one, which may take more of it than 64 do
        ws = [B.moeblaze_int4_workspace_bytes(self._shape(t), group) for t in range(1, min(max_tokens, 127) + 1)]
        if max_tokens > 0 and min(ws) == 0:
            raise B.MoEBlazeError(B.ERR_UNSUPPORTED, "moeblaze_int4_workspace_bytes")
        self._ws = B._bytes(max(ws, default=0), device)
        self._y = torch.empty((max_tokens, d), dtype=torch.bfloat16, device=device)
        self._packed: dict = {}
        self._weights: Optional[B.Int4Weights] = None
        self._shapes: dict = {}

    def _shape(self, L: int) -> B.Shape:
        return B.make_shape(L, self.d, self.h, self.E, self.K, torch.bfloat16, self.act)

    def load(self, q1, s1, q2, s2, q3, s3):
        """Pack 4-bit weights: q1, q2 (E,d,h), q3 (E,h,d) int8 in -8..7 and their scales (E,R/group,N) bf16
        (R the middle axis; q2, s2 None for SiLU).  The packed copies replace earlier ones in place, all of them or,
        when a tensor is refused, none."""
        mats = [("1", q1, s1, self.d, self.h), ("3", q3, s3, self.h, self.d)]
        if self.act == "swiglu":
            mats.append(("2", q2, s2, self.d, self.h))
        specs = []
        for n, q, s, R, N in mats:
            if not isinstance(q, torch.Tensor) or tuple(q.shape) != (self.E, R, N):
                raise ValueError(f"q{n}: expected a tensor of shape {(self.E, R, N)}")
            specs += [(q, "q" + n, (self.E, R, N), torch.int8, False),
                      (s, "s" + n, (self.E, R // self.group, N), torch.bfloat16, False)]
        B._args(*specs)
        for t, name, *_ in specs:
            if t.device != self._ws.device:  # the products read the packed copies beside the buffers
                raise ValueError(f"{name}: on {t.device}, but the buffers are on {self._ws.device}")
        for n, q, s, R, N in mats:
            old = self._packed.get(n, (None, None))
            self._packed[n] = B.int4_pack(q, s, self.group, *old)
        p = {n: tuple(t.data_ptr() for t in v) for n, v in self._packed.items()}
        w1, w2, w3 = p["1"], p.get("2", (None, None)), p["3"]
        self._weights = B.Int4Weights(w1[0], w1[1], w2[0], w2[1], w3[0], w3[1], self.group)

    def quantize(self, W1, W2, W3):
        """Quantise and pack bf16 or fp32 weights (W2 None for SiLU)."""
        q1, s1 = B.int4_quantize(W1, self.group)
        q2, s2 = B.int4_quantize(W2, self.group) if self.act == "swiglu" else (None, None)
        q3, s3 = B.int4_quantize(W3, self.group)
        self.load(q1, s1, q2, s2, q3, s3)

    def dequantize(self):
        """(W1, W2, W3) in bf16, as MoELayer.forward takes them (W2 None for SiLU): for long prompts."""
        if self._weights is None:
            raise RuntimeError("Int4Experts: load or quantize weights first")
        out = []
        for n, R, N in (("1", self.d, self.h), ("2", self.d, self.h), ("3", self.h, self.d)):
            out.append(B.int4_dequantize(*self._packed[n], self.E, R, N, self.group) if n in self._packed else None)
        return tuple(out)

    def forward(self, x, topk_ids, gates) -> torch.Tensor:
        """y (L,d) for the L <= max_tokens rows of x; ids outside [0,E) are empty slots.  y is this object's
        buffer: the next call overwrites it."""
        if self._weights is None:
            raise RuntimeError("Int4Experts: load or quantize weights first")
        L = x.shape[0]
        if L > self.max_tokens:
            raise ValueError(f"x: {L} tokens, at most {self.max_tokens}")
        shape = self._shapes.get(L)
        if shape is None:
            shape = self._shapes[L] = self._shape(L)
        return B.int4_forward(shape, x, topk_ids, gates, self._weights, self._y[:L], self._ws)
