"""The pre-norm block around the layer: layer or RMS norm with the residual sum, the
router with its losses, the layer, and the backward of it all.  Each class
owns the buffers of one shape and runs on the current CUDA stream, as
layer.MoELayer does; outputs are the object's own buffers, which the next call
overwrites."""
from __future__ import annotations

from typing import Optional

import torch

from . import binding as B
from .layer import MoELayer


class LayerNorm:
    def __init__(self, L: int, d: int, dtype: torch.dtype, eps: float = 1e-5, device="cuda"):
        self.shape = B.make_shape(L, d, 0, 1, 1, dtype, "identity")
        self.L, self.d, self.dtype, self.eps = L, d, dtype, eps
        f32 = dict(dtype=torch.float32, device=device)
        self.y = torch.empty((L, d), dtype=dtype, device=device)
        self.mean = torch.empty((L,), **f32)
        self.rstd = torch.empty((L,), **f32)
        self.dw = torch.empty((d,), **f32)
        self.db = torch.empty((d,), **f32)
        # (what a call writes is kept here too, so that its checks, made once, hold whatever becomes of the names)
        self._fwd = (self.y, self.mean, self.rstd)
        self._bwd = (self.dw, self.db)
        self._s: Optional[torch.Tensor] = None
        self._dx: Optional[torch.Tensor] = None
        self._ws: Optional[torch.Tensor] = None
        self._ws_bytes = B.moeblaze_layernorm_backward_workspace_bytes(self.shape)

    def forward(self, x, weight, bias=None, residual=None):
        """(y, s, mean, rstd) of s = x (+ residual); without a residual s is x itself."""
        s = None
        y, mean, rstd = self._fwd
        if residual is not None:
            if self._s is None:
                self._s = torch.empty_like(y)
            s = self._s
        B.layernorm_forward(self.shape, x, residual, weight, bias, self.eps, s, y, mean, rstd, own=True)
        return y, (x if s is None else s), mean, rstd

    def backward(self, dy, s, mean, rstd, weight, dsum=None):
        """(dx, dweight, dbias); dsum is a gradient that reaches s besides the norm and is added to dx."""
        if self._dx is None:
            self._dx = torch.empty_like(self._fwd[0])
            self._ws = B._bytes(self._ws_bytes, self._dx.device)
        dw, db = self._bwd
        B.layernorm_backward(self.shape, dy, s, mean, rstd, weight, dsum, self._dx, dw, db, self._ws, own=self._ws_bytes)
        return self._dx, dw, db


class RMSNorm:
    """Root-mean-square norm with the residual sum, its rows in 8 bits where wanted (forward8), and its backward."""

    def __init__(self, L: int, d: int, dtype: torch.dtype, eps: float = 1e-5, device="cuda"):
        self.shape = B.make_shape(L, d, 0, 1, 1, dtype, "identity")
        self.L, self.d, self.dtype, self.eps = L, d, dtype, eps
        self.y = torch.empty((L, d), dtype=dtype, device=device)
        self.rstd = torch.empty((L,), dtype=torch.float32, device=device)
        self.dw = torch.empty((d,), dtype=torch.float32, device=device)
        # (what a call writes is kept here too, so that its checks, made once, hold whatever becomes of the names)
        self._fwd = (self.y, self.rstd)
        self._dw = self.dw
        self._s: Optional[torch.Tensor] = None
        self._q: Optional[tuple] = None
        self._dx: Optional[torch.Tensor] = None
        self._ws: Optional[torch.Tensor] = None
        self._ws_bytes = B.moeblaze_rmsnorm_backward_workspace_bytes(self.shape)

    def _sum(self, residual):
        if residual is None:
            return None
        if self._s is None:
            self._s = torch.empty_like(self._fwd[0])
        return self._s

    def forward(self, x, weight, residual=None):
        """(y, s, rstd) of s = x (+ residual); without a residual s is x itself."""
        s = self._sum(residual)
        y, rstd = self._fwd
        B.rmsnorm_forward(self.shape, x, residual, weight, self.eps, s, y, rstd, own=True)
        return y, (x if s is None else s), rstd

    def forward8(self, x, weight, residual=None, with_y: bool = True):
        """(q, scales, y, s, rstd): the normed rows in 8-bit floating point too, q (L,d) float8_e4m3fn with scales
        (L, ceil(d/128)) fp32, as fp8.Fp8Experts takes them; with_y=False leaves y out (None).  d is a multiple of 16."""
        if self._q is None:
            if self.d % 16 != 0:
                raise ValueError(f"forward8: d {self.d} is not a multiple of 16")
            dev = self._fwd[0].device
            self._q = (torch.empty((self.L, self.d), dtype=torch.float8_e4m3fn, device=dev),
                       torch.empty((self.L, B.blocks8(self.d)), dtype=torch.float32, device=dev))
        q, scales = self._q
        s = self._sum(residual)
        y, rstd = self._fwd
        if not with_y:
            y = None
        B.rmsnorm_forward(self.shape, x, residual, weight, self.eps, s, y, rstd, q, scales, own=True)
        return q, scales, y, (x if s is None else s), rstd

    def backward(self, dy, s, rstd, weight, dsum=None):
        """(dx, dweight); dsum is a gradient that reaches s besides the norm and is added to dx."""
        if self._dx is None:
            self._dx = torch.empty_like(self._fwd[0])
            self._ws = B._bytes(self._ws_bytes, self._dx.device)
        B.rmsnorm_backward(self.shape, dy, s, rstd, weight, dsum, self._dx, self._dw, self._ws, own=self._ws_bytes)
        return self._dx, self._dw


class BalanceLoss:
    """Load-balance and z loss of a router on its logits, and the tokens per expert."""

    def __init__(self, L: int, E: int, K: int, device="cuda"):
        self.shape = B.make_shape(L, 1, 0, E, K, torch.float32, "identity")
        self.E = E
        f32 = dict(dtype=torch.float32, device=device)
        self.losses = torch.empty((2,), **f32)
        self._counts = torch.empty((E + 1,), dtype=torch.int32, device=device)
        self.counts = self._counts[:E]
        self.active = self._counts[E:]
        self._lse = torch.empty((L,), **f32)
        self.dlogits = torch.empty((L, E), **f32)
        self._ws_bytes = B.moeblaze_balance_workspace_bytes(self.shape)
        self._ws = B._bytes(self._ws_bytes, device)
        self._ran = False  # until then there are no statistics for backward
        self._out = (self.losses, self.dlogits)  # what the calls write, whatever becomes of the names

    def forward(self, logits, topk_ids, valid=None):
        """(losses, counts): losses = [balance, z]; valid (L) uint8 leaves tokens out."""
        losses = self._out[0]
        B.balance_forward(self.shape, logits, topk_ids, valid, losses, self._counts, self._lse, self._ws,
                          own=self._ws_bytes)
        self._ran = True
        return losses, self.counts

    def backward(self, logits, dlosses, valid=None, topk_ids=None, gates=None, dgates=None, gates_of_all=False):
        """dlogits after a forward on the same logits: of the losses, with gradients dlosses (2), and of the
        gates when topk_ids, gates and dgates are given.  The tokens left out are those the forward left out
        (its mask need not be given again) and those that valid leaves out here: their rows are 0, or, with
        gates_of_all, the gates' share."""
        if not self._ran:
            raise RuntimeError("BalanceLoss: run forward first")
        dlogits = self._out[1]
        B.balance_backward(self.shape, logits, self._lse, self._counts, dlosses, topk_ids, gates, dgates, dlogits,
                           own=True, gates_of_all=gates_of_all, valid=valid)
        return dlogits


class RouterGrad:
    """The router's gradients from a dense gradient of its logits."""

    def __init__(self, L: int, d: int, E: int, dtype: torch.dtype, device="cuda"):
        self.shape = B.make_shape(L, d, 0, E, 1, dtype, "identity")
        self._dx: Optional[torch.Tensor] = None
        self.dWr = torch.empty((d, E), dtype=torch.float32, device=device)
        self.dbias = torch.empty((E,), dtype=torch.float32, device=device)
        self._grads = (self.dWr, self.dbias)  # what a call writes, whatever becomes of the names
        self._ws_bytes = B.moeblaze_router_backward_logits_workspace_bytes(self.shape)
        self._ws = B._bytes(self._ws_bytes, device)

    def backward(self, x, Wr, dlogits, add_to=None):
        """(dx, dWr, dbias); with add_to (L,d) dx is added to it in place, and it is returned."""
        dx = add_to
        if dx is None:
            if self._dx is None:
                self._dx = torch.empty_like(x)
            dx = self._dx
        dWr, dbias = self._grads
        B.router_backward_logits(self.shape, x, Wr, dlogits, dWr, dbias, dx, self._ws,
                                 accumulate=add_to is not None, own=self._ws_bytes)
        return dx, dWr, dbias


class MoEBlock:
    """s = x + residual;  out = MoE(Norm(s)) (the caller adds s in its next norm), with the router's losses.

    forward keeps what backward needs in the parts' buffers; one step is forward, then backward."""

    def __init__(self, L: int, d: int, h: int, E: int, K: int, dtype: torch.dtype, act: str = "swiglu",
                 eps: float = 1e-5, device="cuda", recompute_h: bool = False, checkpoint8: bool = False,
                 norm: str = "layer", scratch: Optional["MoEBlock"] = None):
        """recompute_h, checkpoint8: what the layer keeps for its backward; scratch: a block whose layer's scratch this
        one's uses too (see MoELayer); norm: "layer" or "rms"."""
        if norm not in ("layer", "rms"):
            raise ValueError(f"norm: {norm!r}, expected 'layer' or 'rms'")
        self.rms = norm == "rms"
        self.norm = (RMSNorm if self.rms else LayerNorm)(L, d, dtype, eps, device)
        self.layer = MoELayer(L, d, h, E, K, dtype, act, device, recompute_h=recompute_h, checkpoint8=checkpoint8,
                              scratch=None if scratch is None else scratch.layer)
        self.loss = BalanceLoss(L, E, K, device)
        self.grad = RouterGrad(L, d, E, dtype, device)
        self.logits = torch.empty((L, E), dtype=torch.float32, device=device)
        self._kept = None

    def forward(self, x, residual, p, valid=None):
        """(out, s, losses, counts).  p: dict of parameters: norm_w, norm_b (or None; layer norm), Wr, bias (or None), W1, W2, W3.
        valid (L) uint8: tokens that count for the losses (all of them are routed and have a row of out)."""
        if self.rms:
            if p.get("norm_b") is not None:
                raise ValueError("norm_b: the RMS norm has no bias")
            (u, s, rstd), mean = self.norm.forward(x, p["norm_w"], residual), None
        else:
            u, s, mean, rstd = self.norm.forward(x, p["norm_w"], p.get("norm_b"), residual)
        ids, gates = self.layer.route(u, p["Wr"], p.get("bias"), self.logits)
        losses, counts = self.loss.forward(self.logits, ids, valid)
        out = self.layer.forward(u, gates, p["W1"], p.get("W2"), p["W3"])
        self._kept = (u, s, mean, rstd, ids, gates)
        return out, s, losses, counts

    def backward(self, dout, dlosses, p, dsum=None):
        """Gradients as a dict: x (of x and of the residual alike), norm_w, norm_b (layer norm), Wr, bias, W1, W2, W3.
        dout: of out; dlosses (2): of the two losses; dsum: what reaches s besides the norm."""
        if self._kept is None:
            raise RuntimeError("MoEBlock: run forward first")
        u, s, mean, rstd, ids, gates = self._kept
        self._kept = None
        du, dW1, dW2, dW3, dgates = self.layer.backward(dout, u, gates, p["W1"], p.get("W2"), p["W3"])
        # the mask is the losses' alone: the gates of every token made its row of out
        dlogits = self.loss.backward(self.logits, dlosses, None, ids, gates, dgates, gates_of_all=True)
        du, dWr, dbias = self.grad.backward(u, p["Wr"], dlogits, add_to=du)
        if self.rms:
            dx, dnw = self.norm.backward(du, s, rstd, p["norm_w"], dsum)
            return {"x": dx, "norm_w": dnw, "Wr": dWr, "bias": dbias, "W1": dW1, "W2": dW2, "W3": dW3}
        dx, dnw, dnb = self.norm.backward(du, s, mean, rstd, p["norm_w"], dsum)
        return {"x": dx, "norm_w": dnw, "norm_b": dnb, "Wr": dWr, "bias": dbias, "W1": dW1, "W2": dW2, "W3": dW3}
