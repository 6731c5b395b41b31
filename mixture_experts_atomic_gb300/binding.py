"""ctypes binding of libmoeblaze.so: the C entry points under the same names
(argument marshalling only), plus small torch helpers that allocate the
caller-owned buffers and pass their device pointers and the current stream.

Every compute step runs in the library's CUDA kernels; there is no Python or
CPU fallback.  Loading fails loudly when the library has not been built.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoeblaze.so")
_lib = None

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_BAD_ROUTING, ERR_WORKSPACE, ERR_TIMEOUT, ERR_CUDA = range(7)
F32, BF16 = 0, 1
SWIGLU, SILU, IDENTITY = 0, 1, 2
ACT = {"swiglu": SWIGLU, "silu": SILU, "identity": IDENTITY}
DTYPE = {torch.float32: F32, torch.bfloat16: BF16}

# names exported by include/moeblaze.h
EXPORTS = [
    "moeblaze_dispatch_meta_bytes", "moeblaze_dispatch_workspace_bytes", "moeblaze_saved_bytes",
    "moeblaze_forward_workspace_bytes", "moeblaze_backward_workspace_bytes", "moeblaze_dispatch_build",
    "moeblaze_forward", "moeblaze_backward", "moeblaze_device_error", "moeblaze_status_string",
    "moeblaze_version", "moeblaze_set_stage_events", "moeblaze_kernel_launches",
    "moeblaze_dispatch_build_static", "moeblaze_dispatch_meta_check", "moeblaze_set_fault_injection",
    "moeblaze_router_forward", "moeblaze_router_backward", "moeblaze_router_backward_workspace_bytes",
    "moeblaze_router_dispatch_workspace_bytes", "moeblaze_router_dispatch_build",
    "moeblaze_router_forward_logits", "moeblaze_router_dispatch_build_logits", "moeblaze_router_backward_logits",
    "moeblaze_router_backward_logits_workspace_bytes", "moeblaze_balance_workspace_bytes",
    "moeblaze_balance_forward", "moeblaze_balance_backward", "moeblaze_layernorm_forward",
    "moeblaze_layernorm_backward", "moeblaze_layernorm_backward_workspace_bytes", "moeblaze_int4_weight_bytes",
    "moeblaze_int4_scale_bytes", "moeblaze_int4_quantize", "moeblaze_int4_pack", "moeblaze_int4_dequantize",
    "moeblaze_int4_workspace_bytes", "moeblaze_int4_forward", "moeblaze_balance_backward_masked",
    "moeblaze_rmsnorm_forward", "moeblaze_rmsnorm_backward", "moeblaze_rmsnorm_backward_workspace_bytes",
    "moeblaze_fp8_quantize_rows", "moeblaze_fp8_dequantize_rows", "moeblaze_fp8_quantize_weights",
    "moeblaze_fp8_dequantize_weights", "moeblaze_fp8_workspace_bytes", "moeblaze_fp8_forward", "moeblaze_fp8_pack",
]

# fixed scratch of moeblaze_dispatch_build_static (MOEBLAZE_STATIC_SCRATCH_BYTES)
STATIC_SCRATCH_BYTES = 8 << 20


class Shape(ctypes.Structure):
    _fields_ = [("L", ctypes.c_int64), ("d", ctypes.c_int32), ("h", ctypes.c_int32), ("E", ctypes.c_int32),
                ("K", ctypes.c_int32), ("dtype", ctypes.c_int32), ("act", ctypes.c_int32), ("flags", ctypes.c_int32)]


# moeblaze_shape.flags
RECOMPUTE_H = 1
CHECKPOINT_8BIT = 4
CODE_BLOCK = 128  # columns that share a step of the 8-bit checkpoints


class Dispatch(ctypes.Structure):
    _fields_ = [("expert_token_indices", ctypes.c_void_p), ("expert_token_offsets", ctypes.c_void_p),
                ("token_expert_indices", ctypes.c_void_p), ("token_index_map", ctypes.c_void_p),
                ("meta", ctypes.c_void_p)]


class Int4Weights(ctypes.Structure):
    _fields_ = [("w1", ctypes.c_void_p), ("s1", ctypes.c_void_p), ("w2", ctypes.c_void_p), ("s2", ctypes.c_void_p),
                ("w3", ctypes.c_void_p), ("s3", ctypes.c_void_p), ("group", ctypes.c_int32)]


class Fp8Weights(ctypes.Structure):
    _fields_ = [("q1", ctypes.c_void_p), ("s1", ctypes.c_void_p), ("q2", ctypes.c_void_p), ("s2", ctypes.c_void_p),
                ("q3", ctypes.c_void_p), ("s3", ctypes.c_void_p)]


class MoEBlazeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


def lib():
    """The loaded library; raises if it is missing (build it first)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"libmoeblaze.so not built ({_LIB_PATH}); run "
                               "`python -m mixture_experts_atomic_gb300.build`")
        L = ctypes.CDLL(_LIB_PATH)
        sz = ctypes.c_size_t
        P = ctypes.c_void_p
        SP = ctypes.POINTER(Shape)
        DP = ctypes.POINTER(Dispatch)
        for n in ["moeblaze_dispatch_meta_bytes", "moeblaze_dispatch_workspace_bytes", "moeblaze_saved_bytes",
                  "moeblaze_forward_workspace_bytes", "moeblaze_backward_workspace_bytes"]:
            getattr(L, n).argtypes = [SP]
            getattr(L, n).restype = sz
        L.moeblaze_dispatch_build.argtypes = [SP, P, DP, P, sz, ctypes.c_int, P]
        L.moeblaze_dispatch_build.restype = ctypes.c_int
        L.moeblaze_dispatch_build_static.argtypes = [SP, P, DP, ctypes.c_int, P]
        L.moeblaze_dispatch_build_static.restype = ctypes.c_int
        L.moeblaze_forward.argtypes = [SP, P, P, DP, P, P, P, P, P, P, sz, P]
        L.moeblaze_forward.restype = ctypes.c_int
        L.moeblaze_backward.argtypes = [SP, P, P, P, DP, P, P, P, P, P, P, P, P, P, P, sz, P]
        L.moeblaze_backward.restype = ctypes.c_int
        L.moeblaze_router_forward.argtypes = [SP, P, P, P, P, P, P]
        L.moeblaze_router_forward.restype = ctypes.c_int
        L.moeblaze_router_backward_workspace_bytes.argtypes = [SP]
        L.moeblaze_router_backward_workspace_bytes.restype = sz
        L.moeblaze_router_backward.argtypes = [SP, P, P, P, P, P, P, P, P, P, sz, P]
        L.moeblaze_router_backward.restype = ctypes.c_int
        L.moeblaze_router_dispatch_workspace_bytes.argtypes = [SP]
        L.moeblaze_router_dispatch_workspace_bytes.restype = sz
        L.moeblaze_router_dispatch_build.argtypes = [SP, P, P, P, P, P, DP, P, sz, P]
        L.moeblaze_router_dispatch_build.restype = ctypes.c_int
        L.moeblaze_router_forward_logits.argtypes = [SP, P, P, P, P, P, P, P]
        L.moeblaze_router_dispatch_build_logits.argtypes = [SP, P, P, P, P, P, P, DP, P, sz, P]
        L.moeblaze_router_backward_logits.argtypes = [SP, P, P, P, P, P, P, ctypes.c_int32, P, sz, P]
        L.moeblaze_balance_forward.argtypes = [SP, P, P, P, P, P, P, P, sz, P]
        L.moeblaze_balance_backward.argtypes = [SP, P, P, P, P, P, P, P, P, P]
        L.moeblaze_balance_backward_masked.argtypes = [SP, P, P, P, P, P, P, P, P, ctypes.c_int32, P, P]
        L.moeblaze_layernorm_forward.argtypes = [SP, P, P, P, P, ctypes.c_float, P, P, P, P, P]
        L.moeblaze_layernorm_backward.argtypes = [SP, P, P, P, P, P, P, P, P, P, P, sz, P]
        L.moeblaze_rmsnorm_forward.argtypes = [SP, P, P, P, ctypes.c_float, P, P, P, P, P, P]
        L.moeblaze_rmsnorm_backward.argtypes = [SP, P, P, P, P, P, P, P, P, sz, P]
        i32 = ctypes.c_int32
        for n in ["moeblaze_fp8_quantize_rows", "moeblaze_fp8_dequantize_rows"]:
            getattr(L, n).argtypes = [ctypes.c_int64, i32, i32, P, P, P, P]
        L.moeblaze_fp8_quantize_weights.argtypes = [i32, i32, i32, i32, P, P, P, P]
        L.moeblaze_fp8_pack.argtypes = [i32, i32, i32, P, P, P]
        L.moeblaze_fp8_dequantize_weights.argtypes = [i32, i32, i32, P, i32, P, P, P]
        L.moeblaze_fp8_forward.argtypes = [SP, P, P, P, P, ctypes.POINTER(Fp8Weights), P, P, sz, P]
        L.moeblaze_int4_quantize.argtypes = [i32, i32, i32, i32, i32, P, P, P, P]
        L.moeblaze_int4_pack.argtypes = [i32, i32, i32, i32, P, P, P, P, P]
        L.moeblaze_int4_dequantize.argtypes = [i32, i32, i32, i32, P, P, P, P]
        L.moeblaze_int4_forward.argtypes = [SP, P, P, P, ctypes.POINTER(Int4Weights), P, P, sz, P]
        for n in ["moeblaze_router_backward_logits_workspace_bytes", "moeblaze_balance_workspace_bytes",
                  "moeblaze_layernorm_backward_workspace_bytes", "moeblaze_rmsnorm_backward_workspace_bytes",
                  "moeblaze_fp8_workspace_bytes"]:
            getattr(L, n).argtypes = [SP]
            getattr(L, n).restype = sz
        L.moeblaze_int4_workspace_bytes.argtypes = [SP, i32]
        L.moeblaze_int4_workspace_bytes.restype = sz
        L.moeblaze_int4_weight_bytes.argtypes = [i32, i32, i32]
        L.moeblaze_int4_weight_bytes.restype = sz
        L.moeblaze_int4_scale_bytes.argtypes = [i32, i32, i32, i32]
        L.moeblaze_int4_scale_bytes.restype = sz
        L.moeblaze_device_error.argtypes = [SP, DP, ctypes.POINTER(ctypes.c_int32), P]
        L.moeblaze_device_error.restype = ctypes.c_int
        L.moeblaze_dispatch_meta_check.argtypes = [SP, P]
        L.moeblaze_dispatch_meta_check.restype = ctypes.c_int
        L.moeblaze_status_string.argtypes = [ctypes.c_int]
        L.moeblaze_status_string.restype = ctypes.c_char_p
        L.moeblaze_version.argtypes = []
        L.moeblaze_version.restype = ctypes.c_int32
        L.moeblaze_set_stage_events.argtypes = [ctypes.POINTER(ctypes.c_void_p), ctypes.c_int32]
        L.moeblaze_set_stage_events.restype = None
        L.moeblaze_set_fault_injection.argtypes = [ctypes.c_int64, ctypes.c_int32]
        L.moeblaze_set_fault_injection.restype = None
        L.moeblaze_kernel_launches.argtypes = []
        L.moeblaze_kernel_launches.restype = ctypes.c_int64
        _lib = L
    return _lib


def status_string(st: int) -> str:
    return lib().moeblaze_status_string(st).decode()


# ---------------------------------------------------------------- C names

def moeblaze_dispatch_meta_bytes(shape: Shape) -> int:
    return lib().moeblaze_dispatch_meta_bytes(ctypes.byref(shape))


def moeblaze_dispatch_workspace_bytes(shape: Shape) -> int:
    return lib().moeblaze_dispatch_workspace_bytes(ctypes.byref(shape))


def moeblaze_saved_bytes(shape: Shape) -> int:
    return lib().moeblaze_saved_bytes(ctypes.byref(shape))


def moeblaze_forward_workspace_bytes(shape: Shape) -> int:
    return lib().moeblaze_forward_workspace_bytes(ctypes.byref(shape))


def moeblaze_backward_workspace_bytes(shape: Shape) -> int:
    return lib().moeblaze_backward_workspace_bytes(ctypes.byref(shape))


def moeblaze_dispatch_build(shape, topk_ids, disp, ws, ws_bytes, validate, stream) -> int:
    return lib().moeblaze_dispatch_build(ctypes.byref(shape), topk_ids, ctypes.byref(disp), ws, ws_bytes,
                                         int(validate), stream)


def moeblaze_dispatch_build_static(shape, topk_ids, disp, validate, stream) -> int:
    return lib().moeblaze_dispatch_build_static(ctypes.byref(shape), topk_ids, ctypes.byref(disp), int(validate),
                                                stream)


def moeblaze_forward(shape, x, gates, disp, W1, W2, W3, y, saved, ws, ws_bytes, stream) -> int:
    return lib().moeblaze_forward(ctypes.byref(shape), x, gates, ctypes.byref(disp), W1, W2, W3, y, saved, ws,
                                  ws_bytes, stream)


def moeblaze_backward(shape, dY, x, gates, disp, W1, W2, W3, saved, dX, dW1, dW2, dW3, dgates, ws, ws_bytes,
                      stream) -> int:
    return lib().moeblaze_backward(ctypes.byref(shape), dY, x, gates, ctypes.byref(disp), W1, W2, W3, saved, dX,
                                   dW1, dW2, dW3, dgates, ws, ws_bytes, stream)


def moeblaze_router_forward(shape, x, Wr, bias, topk_ids, gates, stream) -> int:
    return lib().moeblaze_router_forward(ctypes.byref(shape), x, Wr, bias, topk_ids, gates, stream)


def moeblaze_router_backward_workspace_bytes(shape: Shape) -> int:
    return lib().moeblaze_router_backward_workspace_bytes(ctypes.byref(shape))


def moeblaze_router_backward(shape, x, Wr, topk_ids, gates, dgates, dWr, dbias, dx, ws, ws_bytes, stream) -> int:
    return lib().moeblaze_router_backward(ctypes.byref(shape), x, Wr, topk_ids, gates, dgates, dWr, dbias, dx, ws,
                                          ws_bytes, stream)


def moeblaze_router_dispatch_workspace_bytes(shape: Shape) -> int:
    return lib().moeblaze_router_dispatch_workspace_bytes(ctypes.byref(shape))


def moeblaze_router_dispatch_build(shape, x, Wr, bias, topk_ids, gates, disp, ws, ws_bytes, stream) -> int:
    return lib().moeblaze_router_dispatch_build(ctypes.byref(shape), x, Wr, bias, topk_ids, gates, ctypes.byref(disp),
                                                ws, ws_bytes, stream)


def moeblaze_router_forward_logits(shape, x, Wr, bias, topk_ids, gates, logits, stream) -> int:
    return lib().moeblaze_router_forward_logits(ctypes.byref(shape), x, Wr, bias, topk_ids, gates, logits, stream)


def moeblaze_router_dispatch_build_logits(shape, x, Wr, bias, topk_ids, gates, logits, disp, ws, ws_bytes,
                                          stream) -> int:
    return lib().moeblaze_router_dispatch_build_logits(ctypes.byref(shape), x, Wr, bias, topk_ids, gates, logits,
                                                       ctypes.byref(disp), ws, ws_bytes, stream)


def moeblaze_router_backward_logits_workspace_bytes(shape: Shape) -> int:
    return lib().moeblaze_router_backward_logits_workspace_bytes(ctypes.byref(shape))


def moeblaze_router_backward_logits(shape, x, Wr, dlogits, dWr, dbias, dx, accumulate, ws, ws_bytes, stream) -> int:
    return lib().moeblaze_router_backward_logits(ctypes.byref(shape), x, Wr, dlogits, dWr, dbias, dx, int(accumulate),
                                                 ws, ws_bytes, stream)


def moeblaze_balance_workspace_bytes(shape: Shape) -> int:
    return lib().moeblaze_balance_workspace_bytes(ctypes.byref(shape))


def moeblaze_balance_forward(shape, logits, topk_ids, valid, losses, counts, lse, ws, ws_bytes, stream) -> int:
    return lib().moeblaze_balance_forward(ctypes.byref(shape), logits, topk_ids, valid, losses, counts, lse, ws,
                                          ws_bytes, stream)


def moeblaze_balance_backward(shape, logits, lse, counts, dlosses, topk_ids, gates, dgates, dlogits, stream) -> int:
    return lib().moeblaze_balance_backward(ctypes.byref(shape), logits, lse, counts, dlosses, topk_ids, gates, dgates,
                                           dlogits, stream)


def moeblaze_balance_backward_masked(shape, logits, lse, counts, dlosses, valid, topk_ids, gates, dgates, gates_of_all,
                                     dlogits, stream) -> int:
    return lib().moeblaze_balance_backward_masked(ctypes.byref(shape), logits, lse, counts, dlosses, valid, topk_ids,
                                                  gates, dgates, int(gates_of_all), dlogits, stream)


def moeblaze_layernorm_forward(shape, x, residual, weight, bias, eps, sum, y, mean, rstd, stream) -> int:
    return lib().moeblaze_layernorm_forward(ctypes.byref(shape), x, residual, weight, bias, eps, sum, y, mean, rstd,
                                            stream)


def moeblaze_layernorm_backward_workspace_bytes(shape: Shape) -> int:
    return lib().moeblaze_layernorm_backward_workspace_bytes(ctypes.byref(shape))


def moeblaze_layernorm_backward(shape, dy, sum, mean, rstd, weight, dsum, dx, dweight, dbias, ws, ws_bytes,
                                stream) -> int:
    return lib().moeblaze_layernorm_backward(ctypes.byref(shape), dy, sum, mean, rstd, weight, dsum, dx, dweight,
                                             dbias, ws, ws_bytes, stream)


def moeblaze_rmsnorm_forward(shape, x, residual, weight, eps, sum, y, rstd, q, q_scales, stream) -> int:
    return lib().moeblaze_rmsnorm_forward(ctypes.byref(shape), x, residual, weight, eps, sum, y, rstd, q, q_scales,
                                          stream)


def moeblaze_rmsnorm_backward_workspace_bytes(shape: Shape) -> int:
    return lib().moeblaze_rmsnorm_backward_workspace_bytes(ctypes.byref(shape))


def moeblaze_rmsnorm_backward(shape, dy, sum, rstd, weight, dsum, dx, dweight, ws, ws_bytes, stream) -> int:
    return lib().moeblaze_rmsnorm_backward(ctypes.byref(shape), dy, sum, rstd, weight, dsum, dx, dweight, ws, ws_bytes,
                                           stream)


def moeblaze_fp8_quantize_rows(L, d, dtype, x, q, scales, stream) -> int:
    return lib().moeblaze_fp8_quantize_rows(L, d, dtype, x, q, scales, stream)


def moeblaze_fp8_dequantize_rows(L, d, dtype, q, scales, x, stream) -> int:
    return lib().moeblaze_fp8_dequantize_rows(L, d, dtype, q, scales, x, stream)


def moeblaze_fp8_quantize_weights(E, R, N, dtype, W, q, scales, stream) -> int:
    return lib().moeblaze_fp8_quantize_weights(E, R, N, dtype, W, q, scales, stream)


def moeblaze_fp8_pack(E, R, N, q, packed, stream) -> int:
    return lib().moeblaze_fp8_pack(E, R, N, q, packed, stream)


def moeblaze_fp8_dequantize_weights(E, R, N, q, packed, scales, W, stream) -> int:
    return lib().moeblaze_fp8_dequantize_weights(E, R, N, q, int(packed), scales, W, stream)


def moeblaze_fp8_workspace_bytes(shape: Shape) -> int:
    return lib().moeblaze_fp8_workspace_bytes(ctypes.byref(shape))


def moeblaze_fp8_forward(shape, x, x_scales, topk_ids, gates, weights, y, ws, ws_bytes, stream) -> int:
    return lib().moeblaze_fp8_forward(ctypes.byref(shape), x, x_scales, topk_ids, gates, ctypes.byref(weights), y, ws,
                                      ws_bytes, stream)


def moeblaze_int4_weight_bytes(E: int, R: int, N: int) -> int:
    return lib().moeblaze_int4_weight_bytes(E, R, N)


def moeblaze_int4_scale_bytes(E: int, R: int, N: int, group: int) -> int:
    return lib().moeblaze_int4_scale_bytes(E, R, N, group)


def moeblaze_int4_quantize(E, R, N, group, dtype, W, q, scales, stream) -> int:
    return lib().moeblaze_int4_quantize(E, R, N, group, dtype, W, q, scales, stream)


def moeblaze_int4_pack(E, R, N, group, q, scales, packed, packed_scales, stream) -> int:
    return lib().moeblaze_int4_pack(E, R, N, group, q, scales, packed, packed_scales, stream)


def moeblaze_int4_dequantize(E, R, N, group, packed, packed_scales, W, stream) -> int:
    return lib().moeblaze_int4_dequantize(E, R, N, group, packed, packed_scales, W, stream)


def moeblaze_int4_workspace_bytes(shape: Shape, group: int) -> int:
    return lib().moeblaze_int4_workspace_bytes(ctypes.byref(shape), group)


def moeblaze_int4_forward(shape, x, topk_ids, gates, weights, y, ws, ws_bytes, stream) -> int:
    return lib().moeblaze_int4_forward(ctypes.byref(shape), x, topk_ids, gates, ctypes.byref(weights), y, ws, ws_bytes,
                                       stream)


def moeblaze_device_error(shape, disp, stream):
    code = ctypes.c_int32(0)
    st = lib().moeblaze_device_error(ctypes.byref(shape), ctypes.byref(disp), ctypes.byref(code), stream)
    return st, code.value


def moeblaze_dispatch_meta_check(shape, meta_header) -> int:
    """meta_header: a host buffer (bytes-like or ctypes pointer) holding a
    copy of the first 32 bytes of a dispatch's meta."""
    return lib().moeblaze_dispatch_meta_check(ctypes.byref(shape), meta_header)


def moeblaze_set_stage_events(events, n: int) -> None:
    lib().moeblaze_set_stage_events(events, int(n))


def moeblaze_set_fault_injection(wait_limit_ns: int, withhold: int) -> None:
    lib().moeblaze_set_fault_injection(int(wait_limit_ns), int(withhold))


def moeblaze_kernel_launches() -> int:
    return int(lib().moeblaze_kernel_launches())


# ---------------------------------------------------------------- torch helpers

def _ptr(t: Optional[torch.Tensor]):
    # the argument types of the entry points turn an int into a void*
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def make_shape(L, d, h, E, K, dtype, act, flags: int = 0) -> Shape:
    dt = DTYPE[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    a = ACT[act] if isinstance(act, str) else int(act)
    return Shape(int(L), int(d), int(h), int(E), int(K), dt, a, int(flags))


_TORCH_DTYPE = {F32: torch.float32, BF16: torch.bfloat16}


def _args(*specs):
    """Check tensor arguments before their pointers go to C.  Each spec is
    (tensor, name, shape, dtype, optional); a tensor of an empty shape may
    be None, as the library takes NULL there.  Every tensor must have exactly
    that shape and dtype and a dense row-major layout (checked for all of
    them first), and live on the current CUDA device.  The C library sees
    only pointers, so a wrong tensor would otherwise be read or written out
    of bounds on the GPU."""
    for t, name, shape, dtype, optional in specs:
        if t is None:
            # an empty buffer (no tokens) may be passed as NULL
            if optional or 0 in shape:
                continue
            raise ValueError(f"{name}: a tensor is required")
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
        if t.shape != shape:
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(int(v) for v in shape)}")
        if t.dtype is not dtype:
            raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name}: must be contiguous (row-major)")
    current = None
    for spec in specs:
        t = spec[0]
        if t is not None:
            if current is None:
                if not t.is_cuda:
                    raise ValueError(f"{spec[1]}: must be a CUDA tensor")
                current = torch._C._cuda_getDevice()
            if t.get_device() != current:  # -1 off the GPU
                if not t.is_cuda:
                    raise ValueError(f"{spec[1]}: must be a CUDA tensor")
                raise ValueError(f"{spec[1]}: on {t.device}, but the current device is cuda:{current}")


def _on_device(*named):
    for t, name in named:
        if not t.is_cuda:
            raise ValueError(f"{name}: must be a CUDA tensor")
        if t.get_device() != torch.cuda.current_device():
            raise ValueError(f"{name}: on {t.device}, but the current device is cuda:{torch.cuda.current_device()}")


def _bytes_arg(t, name: str, nbytes: int):
    """A caller-provided byte buffer: at least nbytes, contiguous, on the current CUDA device."""
    if not isinstance(t, torch.Tensor) or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    if t.nbytes < nbytes:
        raise ValueError(f"{name}: {t.nbytes} bytes, needs {nbytes}")
    if not t.is_cuda or t.get_device() != torch._C._cuda_getDevice():
        _on_device((t, name))


def _weight_specs(shape: Shape, W1, W2, W3, prefix: str = ""):
    """Specs of the expert weights the activation uses (the others go to C as NULL)."""
    if shape.act == IDENTITY:
        return []
    dt = _TORCH_DTYPE[shape.dtype]
    E, d, h = shape.E, shape.d, shape.h
    specs = [(W1, prefix + "W1", (E, d, h), dt, False), (W3, prefix + "W3", (E, h, d), dt, False)]
    if shape.act == SWIGLU:
        specs.append((W2, prefix + "W2", (E, d, h), dt, False))
    return specs


def _used_weights(shape: Shape, W1, W2, W3):
    if shape.act == IDENTITY:
        return None, None, None
    return W1, (W2 if shape.act == SWIGLU else None), W3


def _check_dispatch_bufs(shape: Shape, bufs: "DispatchBuffers"):
    LK = shape.L * shape.K
    for name in ("expert_token_indices", "token_expert_indices", "token_index_map"):
        _bytes_arg(getattr(bufs, name), name, 4 * LK)
    _bytes_arg(bufs.expert_token_offsets, "expert_token_offsets", 4 * (shape.E + 1))
    _bytes_arg(bufs.meta, "meta", moeblaze_dispatch_meta_bytes(shape))


def _check(st: int, where: str):
    if st != OK:
        raise MoEBlazeError(st, where)


@dataclass
class DispatchBuffers:
    shape: Shape
    expert_token_indices: torch.Tensor
    expert_token_offsets: torch.Tensor
    token_expert_indices: torch.Tensor
    token_index_map: torch.Tensor
    meta: torch.Tensor
    ws: torch.Tensor

    def struct(self) -> Dispatch:
        return Dispatch(self.expert_token_indices.data_ptr(), self.expert_token_offsets.data_ptr(),
                        self.token_expert_indices.data_ptr(), self.token_index_map.data_ptr(), self.meta.data_ptr())


def _bytes(n: int, device) -> torch.Tensor:
    # 256-byte aligned device buffer of at least n bytes (torch allocations are)
    return torch.empty(max(int(n), 16), dtype=torch.uint8, device=device)


def alloc_dispatch(shape: Shape, device="cuda") -> DispatchBuffers:
    LK = shape.L * shape.K
    i32 = dict(dtype=torch.int32, device=device)
    return DispatchBuffers(
        shape,
        torch.empty(max(LK, 4), **i32),
        torch.empty(shape.E + 1 + 3, **i32),
        torch.empty(max(LK, 4), **i32),
        torch.empty(max(LK, 4), **i32),
        _bytes(moeblaze_dispatch_meta_bytes(shape), device),
        _bytes(moeblaze_dispatch_workspace_bytes(shape), device),
    )


def dispatch_build(shape: Shape, topk_ids: torch.Tensor, bufs: Optional[DispatchBuffers] = None,
                   validate: bool = False, stream=None) -> DispatchBuffers:
    """Run the three-step dispatch build; returns the buffers holding the
    index structures (views: [:L*K], [:E+1])."""
    _args((topk_ids, "topk_ids", (shape.L, shape.K), torch.int32, False))
    if bufs is None:
        bufs = alloc_dispatch(shape, topk_ids.device)
    _check_dispatch_bufs(shape, bufs)
    d = bufs.struct()
    st = moeblaze_dispatch_build(shape, _ptr(topk_ids), d, _ptr(bufs.ws), bufs.ws.numel(), validate, _stream(stream))
    _check(st, "moeblaze_dispatch_build")
    return bufs


def index_views(shape: Shape, bufs: DispatchBuffers):
    LK = shape.L * shape.K
    return (bufs.expert_token_indices[:LK], bufs.expert_token_offsets[:shape.E + 1],
            bufs.token_expert_indices[:LK].view(shape.L, shape.K), bufs.token_index_map[:LK].view(shape.L, shape.K))


@dataclass
class LayerBuffers:
    saved: torch.Tensor
    fwd_ws: torch.Tensor
    bwd_ws: torch.Tensor


def alloc_layer(shape: Shape, device="cuda", scratch: Optional[LayerBuffers] = None) -> LayerBuffers:
    """The buffers of one layer.  scratch: another layer's, whose fwd_ws and bwd_ws this one then uses too (nothing
    in them outlives a call, so layers that run in turn may)."""
    need = (("fwd_ws", moeblaze_forward_workspace_bytes(shape)), ("bwd_ws", moeblaze_backward_workspace_bytes(shape)))
    saved = _bytes(moeblaze_saved_bytes(shape), device)
    if scratch is None:
        return LayerBuffers(saved, *[_bytes(n, device) for _, n in need])
    for name, n in need:
        t = getattr(scratch, name)
        if t.nbytes < n:
            raise ValueError(f"scratch: {name} has {t.nbytes} bytes, this layer needs {n}")
        if t.device != saved.device:
            raise ValueError(f"scratch: on {t.device}, but the layer is on {saved.device}")
    return LayerBuffers(saved, scratch.fwd_ws, scratch.bwd_ws)


def forward(shape: Shape, x, gates, disp: DispatchBuffers, W1, W2, W3, y, layer: LayerBuffers, stream=None):
    dt = _TORCH_DTYPE[shape.dtype]
    _args((x, "x", (shape.L, shape.d), dt, False), (gates, "gates", (shape.L, shape.K), torch.float32, False),
          (y, "y", (shape.L, shape.d), dt, False), *_weight_specs(shape, W1, W2, W3))
    W1, W2, W3 = _used_weights(shape, W1, W2, W3)
    _check_dispatch_bufs(shape, disp)
    _bytes_arg(layer.saved, "saved", moeblaze_saved_bytes(shape))
    st = moeblaze_forward(shape, _ptr(x), _ptr(gates), disp.struct(), _ptr(W1), _ptr(W2), _ptr(W3), _ptr(y),
                          _ptr(layer.saved), _ptr(layer.fwd_ws), layer.fwd_ws.numel(), _stream(stream))
    _check(st, "moeblaze_forward")
    return y


def backward(shape: Shape, dY, x, gates, disp: DispatchBuffers, W1, W2, W3, layer: LayerBuffers, dX, dW1, dW2, dW3,
             dgates=None, stream=None):
    dt = _TORCH_DTYPE[shape.dtype]
    _args((dY, "dY", (shape.L, shape.d), dt, False), (x, "x", (shape.L, shape.d), dt, False),
          (gates, "gates", (shape.L, shape.K), torch.float32, False), (dX, "dX", (shape.L, shape.d), dt, False),
          (dgates, "dgates", (shape.L, shape.K), torch.float32, True),
          *_weight_specs(shape, W1, W2, W3), *_weight_specs(shape, dW1, dW2, dW3, prefix="d"))
    W1, W2, W3 = _used_weights(shape, W1, W2, W3)
    dW1, dW2, dW3 = _used_weights(shape, dW1, dW2, dW3)
    _check_dispatch_bufs(shape, disp)
    _bytes_arg(layer.saved, "saved", moeblaze_saved_bytes(shape))
    st = moeblaze_backward(shape, _ptr(dY), _ptr(x), _ptr(gates), disp.struct(), _ptr(W1), _ptr(W2), _ptr(W3),
                           _ptr(layer.saved), _ptr(dX), _ptr(dW1), _ptr(dW2), _ptr(dW3), _ptr(dgates),
                           _ptr(layer.bwd_ws), layer.bwd_ws.numel(), _stream(stream))
    _check(st, "moeblaze_backward")


class StageEvents:
    """CUDA events the library records at its stage boundaries (see
    moeblaze_set_stage_events); use as a context manager around one call."""

    def __init__(self, n: int):
        self.events = [torch.cuda.Event(enable_timing=True) for _ in range(n)]
        for e in self.events:  # torch creates the CUDA event on its first record
            e.record()
        torch.cuda.current_stream().synchronize()
        self._arr = (ctypes.c_void_p * n)(*[ctypes.c_void_p(e.cuda_event) for e in self.events])

    def __enter__(self):
        moeblaze_set_stage_events(self._arr, len(self.events))
        return self

    def __exit__(self, *exc):
        moeblaze_set_stage_events(None, 0)
        return False

    def elapsed_ms(self):
        return [self.events[i].elapsed_time(self.events[i + 1]) for i in range(len(self.events) - 1)]


def router_forward(shape: Shape, x, Wr, bias, topk_ids, gates, stream=None, logits=None):
    """Token-choice top-K softmax router: fills topk_ids (L,K) int32 and gates (L,K) fp32, and the logits
    (L,E) fp32 when a tensor for them is given."""
    _args((x, "x", (shape.L, shape.d), _TORCH_DTYPE[shape.dtype], False),
          (Wr, "Wr", (shape.d, shape.E), torch.float32, False), (bias, "bias", (shape.E,), torch.float32, True),
          (topk_ids, "topk_ids", (shape.L, shape.K), torch.int32, False),
          (gates, "gates", (shape.L, shape.K), torch.float32, False),
          (logits, "logits", (shape.L, shape.E), torch.float32, True))
    if logits is not None:
        st = moeblaze_router_forward_logits(shape, _ptr(x), _ptr(Wr), _ptr(bias), _ptr(topk_ids), _ptr(gates),
                                            _ptr(logits), _stream(stream))
        _check(st, "moeblaze_router_forward_logits")
        return
    st = moeblaze_router_forward(shape, _ptr(x), _ptr(Wr), _ptr(bias), _ptr(topk_ids), _ptr(gates), _stream(stream))
    _check(st, "moeblaze_router_forward")


def router_dispatch_build(shape: Shape, x, Wr, bias, topk_ids, gates, bufs: Optional["DispatchBuffers"] = None,
                          ws=None, stream=None, logits=None) -> "DispatchBuffers":
    """The router fused with the dispatch build's first step: fills topk_ids
    (L,K) int32, gates (L,K) fp32, the dispatch buffers and, when a tensor is
    given for them, the logits (L,E) fp32 in one call.  `ws`
    is a device byte tensor of moeblaze_router_dispatch_workspace_bytes(shape)
    bytes (allocated here when None)."""
    _args((x, "x", (shape.L, shape.d), _TORCH_DTYPE[shape.dtype], False),
          (Wr, "Wr", (shape.d, shape.E), torch.float32, False), (bias, "bias", (shape.E,), torch.float32, True),
          (topk_ids, "topk_ids", (shape.L, shape.K), torch.int32, False),
          (gates, "gates", (shape.L, shape.K), torch.float32, False),
          (logits, "logits", (shape.L, shape.E), torch.float32, True))
    if bufs is None:
        bufs = alloc_dispatch(shape, Wr.device)
    _check_dispatch_bufs(shape, bufs)
    n = moeblaze_router_dispatch_workspace_bytes(shape)
    if n == 0:
        raise MoEBlazeError(ERR_UNSUPPORTED, "moeblaze_router_dispatch_workspace_bytes")
    if ws is None:
        ws = _bytes(n, Wr.device)
    _bytes_arg(ws, "ws", n)
    if logits is not None:
        st = moeblaze_router_dispatch_build_logits(shape, _ptr(x), _ptr(Wr), _ptr(bias), _ptr(topk_ids), _ptr(gates),
                                                   _ptr(logits), bufs.struct(), _ptr(ws), n, _stream(stream))
        _check(st, "moeblaze_router_dispatch_build_logits")
        return bufs
    st = moeblaze_router_dispatch_build(shape, _ptr(x), _ptr(Wr), _ptr(bias), _ptr(topk_ids), _ptr(gates),
                                        bufs.struct(), _ptr(ws), n, _stream(stream))
    _check(st, "moeblaze_router_dispatch_build")
    return bufs


def router_backward(shape: Shape, x, Wr, topk_ids, gates, dgates, dWr, dbias, dx, ws=None, stream=None):
    """Router gradients from the gate gradients: fills dWr (d,E) fp32, dbias (E) fp32 and dx (L,d) (dbias and dx
    may be None).  `ws` is a device byte tensor of moeblaze_router_backward_workspace_bytes(shape) bytes
    (allocated here when None)."""
    _args((x, "x", (shape.L, shape.d), _TORCH_DTYPE[shape.dtype], False),
          (Wr, "Wr", (shape.d, shape.E), torch.float32, False),
          (topk_ids, "topk_ids", (shape.L, shape.K), torch.int32, False),
          (gates, "gates", (shape.L, shape.K), torch.float32, False),
          (dgates, "dgates", (shape.L, shape.K), torch.float32, False),
          (dWr, "dWr", (shape.d, shape.E), torch.float32, False),
          (dbias, "dbias", (shape.E,), torch.float32, True),
          (dx, "dx", (shape.L, shape.d), _TORCH_DTYPE[shape.dtype], True))
    n = moeblaze_router_backward_workspace_bytes(shape)
    if ws is None:
        ws = _bytes(n, Wr.device)
    _bytes_arg(ws, "ws", n)
    st = moeblaze_router_backward(shape, _ptr(x), _ptr(Wr), _ptr(topk_ids), _ptr(gates), _ptr(dgates), _ptr(dWr),
                                  _ptr(dbias), _ptr(dx), _ptr(ws), n, _stream(stream))
    _check(st, "moeblaze_router_backward")


def router_backward_logits(shape: Shape, x, Wr, dlogits, dWr, dbias, dx, ws=None, stream=None, accumulate=False,
                           own=None):
    """Router gradients from a dense gradient of its logits: fills dWr (d,E) fp32, dbias (E) fp32 and dx (L,d)
    (dbias and dx may be None); with accumulate dx is added to what is there.  `ws` is a device byte tensor of
    moeblaze_router_backward_logits_workspace_bytes(shape) bytes (allocated here when None).
    own: the workspace's bytes, when dWr, dbias and ws are buffers made for this shape on dWr's device."""
    dt, L, d, E = _TORCH_DTYPE[shape.dtype], shape.L, shape.d, shape.E
    specs = ((x, "x", (L, d), dt, False), (Wr, "Wr", (d, E), torch.float32, False),
             (dlogits, "dlogits", (L, E), torch.float32, False), (dWr, "dWr", (d, E), torch.float32, False),
             (dx, "dx", (L, d), dt, True))
    if own is None:
        specs += ((dbias, "dbias", (E,), torch.float32, True),)
    _args(*specs)
    n = own
    if own is None:
        n = moeblaze_router_backward_logits_workspace_bytes(shape)
        if ws is None:
            ws = _bytes(n, Wr.device)
        _bytes_arg(ws, "ws", n)
    st = moeblaze_router_backward_logits(shape, _ptr(x), _ptr(Wr), _ptr(dlogits), _ptr(dWr), _ptr(dbias), _ptr(dx),
                                         accumulate, _ptr(ws), n, _stream(stream))
    _check(st, "moeblaze_router_backward_logits")


def balance_forward(shape: Shape, logits, topk_ids, valid, losses, counts, lse, ws, stream=None, own=None):
    """Load-balance and z loss of a router's logits: fills losses (2) fp32, counts (E+1) int32 (the last one the
    active tokens) and lse (L) fp32.  valid: (L) uint8 or None.
    own: the workspace's bytes, when outputs and workspace are buffers made for this shape on losses' device."""
    L, E = shape.L, shape.E
    specs = ((logits, "logits", (L, E), torch.float32, False), (topk_ids, "topk_ids", (L, shape.K), torch.int32, False),
             (valid, "valid", (L,), torch.uint8, True), (losses, "losses", (2,), torch.float32, False))
    if own is None:
        specs += ((counts, "counts", (E + 1,), torch.int32, False), (lse, "lse", (L,), torch.float32, False))
    _args(*specs)
    n = own
    if own is None:
        n = moeblaze_balance_workspace_bytes(shape)
        _bytes_arg(ws, "ws", n)
    st = moeblaze_balance_forward(shape, _ptr(logits), _ptr(topk_ids), _ptr(valid), _ptr(losses), _ptr(counts),
                                  _ptr(lse), _ptr(ws), n, _stream(stream))
    _check(st, "moeblaze_balance_forward")


def balance_backward(shape: Shape, logits, lse, counts, dlosses, topk_ids, gates, dgates, dlogits, stream=None,
                     own=False, gates_of_all=False, valid=None):
    """Gradient of the logits (L,E) fp32 from the gradients of the two losses and, when topk_ids, gates and dgates
    are given (all or none), of the gates; gates_of_all: of the gates of tokens left out of the losses too.
    valid: (L) uint8 or None, tokens left out besides those the forward left out.
    own: lse and counts are buffers made for this shape on dlogits' device."""
    L, E, K = shape.L, shape.E, shape.K
    specs = ((logits, "logits", (L, E), torch.float32, False), (dlosses, "dlosses", (2,), torch.float32, False),
             (valid, "valid", (L,), torch.uint8, True), (topk_ids, "topk_ids", (L, K), torch.int32, True),
             (gates, "gates", (L, K), torch.float32, True), (dgates, "dgates", (L, K), torch.float32, True), (dlogits, "dlogits", (L, E), torch.float32, False))
    if not own:
        specs += ((lse, "lse", (L,), torch.float32, False), (counts, "counts", (E + 1,), torch.int32, False))
    _args(*specs)
    if L > 0 and len({topk_ids is None, gates is None, dgates is None}) != 1:
        raise ValueError("topk_ids, gates and dgates: give all three or none")
    st = moeblaze_balance_backward_masked(shape, _ptr(logits), _ptr(lse), _ptr(counts), _ptr(dlosses),
                                          _ptr(valid), _ptr(topk_ids), _ptr(gates), _ptr(dgates), gates_of_all, _ptr(dlogits),
                                          _stream(stream))
    _check(st, "moeblaze_balance_backward_masked")


def layernorm_forward(shape: Shape, x, residual, weight, bias, eps, sum, y, mean, rstd, stream=None, own=False):
    """Layer norm of x (+ residual): fills y (L,d), mean and rstd (L) fp32 and, unless None, sum (L,d).
    own: the outputs are buffers made for this shape on y's device, and only y is looked at again."""
    dt, L, d = _TORCH_DTYPE[shape.dtype], shape.L, shape.d
    specs = ((x, "x", (L, d), dt, False), (residual, "residual", (L, d), dt, True),
             (weight, "weight", (d,), torch.float32, False), (bias, "bias", (d,), torch.float32, True),
             (y, "y", (L, d), dt, False))
    if not own:
        specs += ((sum, "sum", (L, d), dt, True), (mean, "mean", (L,), torch.float32, False),
                  (rstd, "rstd", (L,), torch.float32, False))
    _args(*specs)
    st = moeblaze_layernorm_forward(shape, _ptr(x), _ptr(residual), _ptr(weight), _ptr(bias), eps, _ptr(sum), _ptr(y),
                                    _ptr(mean), _ptr(rstd), _stream(stream))
    _check(st, "moeblaze_layernorm_forward")


def layernorm_backward(shape: Shape, dy, sum, mean, rstd, weight, dsum, dx, dweight, dbias, ws, stream=None, own=None):
    """Layer norm backward: fills dx (L,d), dweight (d) fp32 and, unless None, dbias (d) fp32.
    own: the workspace's bytes, when outputs and workspace are buffers made for this shape on dx's device."""
    dt, L, d = _TORCH_DTYPE[shape.dtype], shape.L, shape.d
    specs = ((dy, "dy", (L, d), dt, False), (sum, "sum", (L, d), dt, False), (mean, "mean", (L,), torch.float32, False),
             (rstd, "rstd", (L,), torch.float32, False), (weight, "weight", (d,), torch.float32, False),
             (dsum, "dsum", (L, d), dt, True), (dx, "dx", (L, d), dt, False))
    n = own
    if own is None:
        specs += ((dweight, "dweight", (d,), torch.float32, False), (dbias, "dbias", (d,), torch.float32, True))
    _args(*specs)
    if own is None:
        n = moeblaze_layernorm_backward_workspace_bytes(shape)
        _bytes_arg(ws, "ws", n)
    st = moeblaze_layernorm_backward(shape, _ptr(dy), _ptr(sum), _ptr(mean), _ptr(rstd), _ptr(weight), _ptr(dsum),
                                     _ptr(dx), _ptr(dweight), _ptr(dbias), _ptr(ws), n, _stream(stream))
    _check(st, "moeblaze_layernorm_backward")


def rmsnorm_forward(shape: Shape, x, residual, weight, eps, sum, y, rstd, q=None, q_scales=None, stream=None, own=False):
    """Root-mean-square norm of x (+ residual): fills rstd (L) fp32, y (L,d) (None: only with q), unless None sum (L,d)
    and, unless None, q (L,d) float8_e4m3fn with q_scales (L, ceil(d/128)) fp32.
    own: the outputs are buffers made for this shape on rstd's device, and only rstd is looked at again."""
    dt, L, d = _TORCH_DTYPE[shape.dtype], shape.L, shape.d
    specs = ((x, "x", (L, d), dt, False), (residual, "residual", (L, d), dt, True),
             (weight, "weight", (d,), torch.float32, False), (rstd, "rstd", (L,), torch.float32, False))
    if not own:
        specs += ((sum, "sum", (L, d), dt, True), (y, "y", (L, d), dt, q is not None),
                  (q, "q", (L, d), torch.float8_e4m3fn, True),
                  (q_scales, "q_scales", (L, blocks8(d)), torch.float32, q is None))
    _args(*specs)
    st = moeblaze_rmsnorm_forward(shape, _ptr(x), _ptr(residual), _ptr(weight), eps, _ptr(sum), _ptr(y), _ptr(rstd),
                                  _ptr(q), _ptr(q_scales), _stream(stream))
    _check(st, "moeblaze_rmsnorm_forward")


def rmsnorm_backward(shape: Shape, dy, sum, rstd, weight, dsum, dx, dweight, ws, stream=None, own=None):
    """Root-mean-square norm backward: fills dx (L,d) and dweight (d) fp32.
    own: the workspace's bytes, when outputs and workspace are buffers made for this shape on dx's device."""
    dt, L, d = _TORCH_DTYPE[shape.dtype], shape.L, shape.d
    specs = ((dy, "dy", (L, d), dt, False), (sum, "sum", (L, d), dt, False), (rstd, "rstd", (L,), torch.float32, False),
             (weight, "weight", (d,), torch.float32, False), (dsum, "dsum", (L, d), dt, True),
             (dx, "dx", (L, d), dt, False))
    n = own
    if own is None:
        specs += ((dweight, "dweight", (d,), torch.float32, False),)
    _args(*specs)
    if own is None:
        n = moeblaze_rmsnorm_backward_workspace_bytes(shape)
        _bytes_arg(ws, "ws", n)
    st = moeblaze_rmsnorm_backward(shape, _ptr(dy), _ptr(sum), _ptr(rstd), _ptr(weight), _ptr(dsum), _ptr(dx),
                                   _ptr(dweight), _ptr(ws), n, _stream(stream))
    _check(st, "moeblaze_rmsnorm_backward")


def blocks8(d: int) -> int:
    """Blocks of 128 columns, each with a scale, of 8-bit rows of d columns."""
    return (d + 127) // 128


def fp8_quantize_rows(x, q=None, scales=None, stream=None):
    """8-bit rows of x (L,d) bf16 or fp32: (q (L,d) float8_e4m3fn, scales (L, ceil(d/128)) fp32)."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x: expected a tensor of shape (L, d)")
    if x.dtype not in DTYPE:
        raise ValueError(f"x: dtype {x.dtype}, expected float32 or bfloat16")
    L, d = x.shape
    if d % 16 != 0:
        raise MoEBlazeError(ERR_UNSUPPORTED, "moeblaze_fp8_quantize_rows")
    _args((x, "x", (L, d), x.dtype, False), (q, "q", (L, d), torch.float8_e4m3fn, True),
          (scales, "scales", (L, blocks8(d)), torch.float32, True))
    q = torch.empty((L, d), dtype=torch.float8_e4m3fn, device=x.device) if q is None else q
    scales = torch.empty((L, blocks8(d)), dtype=torch.float32, device=x.device) if scales is None else scales
    st = moeblaze_fp8_quantize_rows(L, d, DTYPE[x.dtype], _ptr(x), _ptr(q), _ptr(scales), _stream(stream))
    _check(st, "moeblaze_fp8_quantize_rows")
    return q, scales


def fp8_dequantize_rows(q, scales, dtype=torch.bfloat16, out=None, stream=None):
    """What 8-bit rows q (L,d) with scales (L, ceil(d/128)) stand for, (L,d) bf16 or fp32, rounded once (with scales of
    powers of two, as the quantiser's, exactly)."""
    if not isinstance(q, torch.Tensor) or q.dim() != 2:
        raise ValueError("q: expected a tensor of shape (L, d)")
    if dtype not in DTYPE:
        raise ValueError(f"dtype {dtype}, expected float32 or bfloat16")
    L, d = q.shape
    _args((q, "q", (L, d), torch.float8_e4m3fn, False), (scales, "scales", (L, blocks8(d)), torch.float32, False),
          (out, "out", (L, d), dtype, True))
    out = torch.empty((L, d), dtype=dtype, device=q.device) if out is None else out
    st = moeblaze_fp8_dequantize_rows(L, d, DTYPE[dtype], _ptr(q), _ptr(scales), _ptr(out), _stream(stream))
    _check(st, "moeblaze_fp8_dequantize_rows")
    return out


def fp8_quantize_weights(W, stream=None):
    """8-bit weights of W (E,R,N) bf16 or fp32: (q (E,N,R) float8_e4m3fn, scales (E, N/128, R/128) fp32)."""
    if not isinstance(W, torch.Tensor) or W.dim() != 3:
        raise ValueError("W: expected a tensor of shape (E, R, N)")
    if W.dtype not in DTYPE:
        raise ValueError(f"W: dtype {W.dtype}, expected float32 or bfloat16")
    E, R, N = W.shape
    if E < 1 or R < 1 or N < 1 or R % 128 or N % 128:
        raise MoEBlazeError(ERR_UNSUPPORTED, "moeblaze_fp8_quantize_weights")
    _args((W, "W", (E, R, N), W.dtype, False))
    q = torch.empty((E, N, R), dtype=torch.float8_e4m3fn, device=W.device)
    s = torch.empty((E, N // 128, R // 128), dtype=torch.float32, device=W.device)
    st = moeblaze_fp8_quantize_weights(E, R, N, DTYPE[W.dtype], _ptr(W), _ptr(q), _ptr(s), _stream(stream))
    _check(st, "moeblaze_fp8_quantize_weights")
    return q, s


def fp8_pack(q, packed=None, stream=None):
    """The layout the 8-bit products read, of q (E,N,R): a float8_e4m3fn tensor (E, N/128, R/128, 128, 128)."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q: expected a tensor of shape (E, N, R)")
    E, N, R = q.shape
    if E < 1 or R < 1 or N < 1 or R % 128 or N % 128:
        raise MoEBlazeError(ERR_UNSUPPORTED, "moeblaze_fp8_pack")
    _args((q, "q", (E, N, R), torch.float8_e4m3fn, False))
    if packed is None:
        packed = torch.empty((E, N // 128, R // 128, 128, 128), dtype=torch.float8_e4m3fn, device=q.device)
    _args((packed, "packed", (E, N // 128, R // 128, 128, 128), torch.float8_e4m3fn, False))
    st = moeblaze_fp8_pack(E, R, N, _ptr(q), _ptr(packed), _stream(stream))
    _check(st, "moeblaze_fp8_pack")
    return packed


def fp8_dequantize_weights(q, scales, stream=None):
    """The bf16 weights (E,R,N) that q (E,N,R), or its packed layout (fp8_pack), with scales (E, N/128, R/128) stands
    for."""
    if isinstance(q, torch.Tensor) and q.dim() == 5:
        E, nb, rb = q.shape[:3]
        N, R = 128 * nb, 128 * rb
        _args((q, "q", (E, nb, rb, 128, 128), torch.float8_e4m3fn, False),
              (scales, "scales", (E, nb, rb), torch.float32, False))
        W = torch.empty((E, R, N), dtype=torch.bfloat16, device=q.device)
        st = moeblaze_fp8_dequantize_weights(E, R, N, _ptr(q), True, _ptr(scales), _ptr(W), _stream(stream))
        _check(st, "moeblaze_fp8_dequantize_weights")
        return W
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q: expected a tensor of shape (E, N, R)")
    E, N, R = q.shape
    _args((q, "q", (E, N, R), torch.float8_e4m3fn, False),
          (scales, "scales", (E, N // 128, R // 128), torch.float32, False))
    W = torch.empty((E, R, N), dtype=torch.bfloat16, device=q.device)
    st = moeblaze_fp8_dequantize_weights(E, R, N, _ptr(q), False, _ptr(scales), _ptr(W), _stream(stream))
    _check(st, "moeblaze_fp8_dequantize_weights")
    return W


def fp8_forward(shape: Shape, x, x_scales, topk_ids, gates, weights: Fp8Weights, y, ws, ws_bytes=None, stream=None):
    """The layer's forward on 8-bit weights: fills y (L,d) bf16.  x (L,d) bf16, or float8_e4m3fn with x_scales
    (L, d/128) fp32.  `weights` holds device pointers that the caller keeps alive (see fp8.Fp8Experts).
    ws_bytes: the workspace's bytes, when y and ws are buffers made for this shape (at least) on x's device."""
    L, d, K = shape.L, shape.d, shape.K
    rows = (x, "x", (L, d), torch.bfloat16, False)
    if x_scales is not None:
        rows = (x, "x", (L, d), torch.float8_e4m3fn, False)
    specs = (rows, (x_scales, "x_scales", (L, blocks8(d)), torch.float32, True),
             (topk_ids, "topk_ids", (L, K), torch.int32, False), (gates, "gates", (L, K), torch.float32, False),
             (y, "y", (L, d), torch.bfloat16, False))
    _args(*specs)
    if ws_bytes is None:
        ws_bytes = moeblaze_fp8_workspace_bytes(shape)
        _bytes_arg(ws, "ws", ws_bytes)
    st = moeblaze_fp8_forward(shape, _ptr(x), _ptr(x_scales), _ptr(topk_ids), _ptr(gates), weights, _ptr(y), _ptr(ws),
                              ws_bytes, _stream(stream))
    _check(st, "moeblaze_fp8_forward")
    return y


def _int4_matrix(E: int, R: int, N: int, group: int, where: str):
    """Sizes of a packed matrix and its scales; raises for a matrix the library does not take."""
    wb, sb = moeblaze_int4_weight_bytes(E, R, N), moeblaze_int4_scale_bytes(E, R, N, group)
    if wb == 0 or sb == 0:
        raise MoEBlazeError(ERR_UNSUPPORTED, where)
    return wb, sb


def int4_quantize(W, group: int, stream=None):
    """4-bit values and group scales of W (E,R,N): returns q (E,R,N) int8 in -8..7 and scales (E,R/group,N) bf16."""
    if not isinstance(W, torch.Tensor) or W.dim() != 3:
        raise ValueError("W: expected a tensor of shape (E, R, N)")
    E, R, N = W.shape
    if W.dtype not in DTYPE:
        raise ValueError(f"W: dtype {W.dtype}, expected float32 or bfloat16")
    _int4_matrix(E, R, N, group, "moeblaze_int4_quantize")
    _args((W, "W", (E, R, N), W.dtype, False))
    q = torch.empty((E, R, N), dtype=torch.int8, device=W.device)
    s = torch.empty((E, R // group, N), dtype=torch.bfloat16, device=W.device)
    st = moeblaze_int4_quantize(E, R, N, group, DTYPE[W.dtype], _ptr(W), _ptr(q), _ptr(s), _stream(stream))
    _check(st, "moeblaze_int4_quantize")
    return q, s


def int4_pack(q, scales, group: int, packed=None, packed_scales=None, stream=None):
    """The layout the 4-bit products read, from q (E,R,N) int8 and scales (E,R/group,N) bf16: two byte tensors."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q: expected a tensor of shape (E, R, N)")
    E, R, N = q.shape
    wb, sb = _int4_matrix(E, R, N, group, "moeblaze_int4_pack")
    _args((q, "q", (E, R, N), torch.int8, False), (scales, "scales", (E, R // group, N), torch.bfloat16, False))
    packed = _bytes(wb, q.device) if packed is None else packed
    packed_scales = _bytes(sb, q.device) if packed_scales is None else packed_scales
    _bytes_arg(packed, "packed", wb)
    _bytes_arg(packed_scales, "packed_scales", sb)
    st = moeblaze_int4_pack(E, R, N, group, _ptr(q), _ptr(scales), _ptr(packed), _ptr(packed_scales), _stream(stream))
    _check(st, "moeblaze_int4_pack")
    return packed, packed_scales


def int4_dequantize(packed, packed_scales, E: int, R: int, N: int, group: int, stream=None):
    """The bf16 weights (E,R,N) a packed matrix stands for."""
    wb, sb = _int4_matrix(E, R, N, group, "moeblaze_int4_dequantize")
    _bytes_arg(packed, "packed", wb)
    _bytes_arg(packed_scales, "packed_scales", sb)
    W = torch.empty((E, R, N), dtype=torch.bfloat16, device=packed.device)
    st = moeblaze_int4_dequantize(E, R, N, group, _ptr(packed), _ptr(packed_scales), _ptr(W), _stream(stream))
    _check(st, "moeblaze_int4_dequantize")
    return W


def int4_forward(shape: Shape, x, topk_ids, gates, weights: Int4Weights, y, ws, stream=None):
    """The layer's forward on packed 4-bit weights: fills y (L,d) bf16.  `weights` holds device pointers that the
    caller keeps alive (see int4.Int4Experts)."""
    dt = _TORCH_DTYPE[shape.dtype]
    _args((x, "x", (shape.L, shape.d), dt, False), (topk_ids, "topk_ids", (shape.L, shape.K), torch.int32, False),
          (gates, "gates", (shape.L, shape.K), torch.float32, False), (y, "y", (shape.L, shape.d), dt, False))
    if not isinstance(ws, torch.Tensor) or not ws.is_contiguous():
        raise ValueError("ws: expected a contiguous tensor")
    _on_device((ws, "ws"))
    st = moeblaze_int4_forward(shape, _ptr(x), _ptr(topk_ids), _ptr(gates), weights, _ptr(y), _ptr(ws), ws.numel(),
                               _stream(stream))
    _check(st, "moeblaze_int4_forward")
    return y


def device_error(shape: Shape, disp: DispatchBuffers, stream=None) -> int:
    """The device error word of a dispatch (0: every kernel since its build
    finished normally; bits 1 bad routing, 2 timeout, 4 shape mismatch)."""
    st, code = moeblaze_device_error(shape, disp.struct(), _stream(stream))
    if st not in (OK, ERR_BAD_ROUTING, ERR_TIMEOUT) and not (st == ERR_INVALID_ARG and code & 4):
        raise MoEBlazeError(st, "moeblaze_device_error")
    return code


def padded_rows(shape: Shape) -> int:
    """Rows of the expert-major row space: L*K plus each expert's padding to
    a multiple of 256 rows, at most."""
    r = shape.L * shape.K + shape.E * 255
    return (r + 255) // 256 * 256


def saved_views(shape: Shape, layer: LayerBuffers, dtype):
    """(A, B) views of the saved checkpoint: (padded_rows, h) each (B None for
    SiLU).  After a bf16 backward they hold dA and dB."""
    es = 4 if dtype == torch.float32 else 2
    h = shape.h
    nb = 2 if shape.act == SWIGLU else 1
    rows = padded_rows(shape)
    t = layer.saved[: rows * nb * h * es].view(dtype).view(nb, rows, h)
    return t[0], (t[1] if nb == 2 else None)


def saved_codes(shape: Shape, layer: LayerBuffers):
    """(qA, sA, qB, sB) views of the checkpoints in 8 bits (MOEBLAZE_CHECKPOINT_8BIT): codes (padded_rows, h) int8 and
    steps (padded_rows, h/128) fp32; A stands for qA sA (qB and sB None for SiLU).  Rows of no token are unspecified."""
    h, rows = shape.h, padded_rows(shape)
    nb = 2 if shape.act == SWIGLU else 1
    n = nb * rows * h
    q = layer.saved[:n].view(torch.int8).view(nb, rows, h)
    s = layer.saved[n:n + n // CODE_BLOCK * 4].view(torch.float32).view(nb, rows, h // CODE_BLOCK)
    return (q[0], s[0]) + ((q[1], s[1]) if nb == 2 else (None, None))


def meta_arrays(shape: Shape, disp: DispatchBuffers):
    """Host copies of (num_m_tiles, n_e, pad_off, order) from the meta buffer."""
    m = disp.meta.view(torch.int32).cpu()
    E = shape.E
    n_e = m[8:8 + E]
    pad = m[8 + E:8 + 2 * E + 1]
    order = m[8 + 2 * E + 1:8 + 3 * E + 1]
    return int(m[1]), n_e, pad, order
