"""8-bit floating point: rows with a scale for each 128 columns, as the RMS
norm leaves them (block.RMSNorm.forward8), and what they stand for."""
from __future__ import annotations

import torch

from . import binding as B


def quantize_rows(x):
    """(q, scales) of x (L,d) bf16 or fp32: q (L,d) float8_e4m3fn, scales (L, ceil(d/128)) fp32, powers of two."""
    return B.fp8_quantize_rows(x)


def dequantize_rows(q, scales, dtype=torch.bfloat16):
    """What 8-bit rows stand for, (L,d) in dtype (bf16 or fp32)."""
    return B.fp8_dequantize_rows(q, scales, dtype)
