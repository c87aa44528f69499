"""Feed-forward block on the library's kernels, for training and for decoding.

    h = x + residual;  n = rmsnorm(h);  (g, u) = n W_gate_up^T;
    a = g / (1 + exp(-g)) * u;  y = a W_down^T

The block returns (y, h): y joins the residual stream h in the next block's
norm (y as its x, h as its residual), so that no addition runs by itself.

Training (`forward`): both products through the MXFP4 linear layer, the norm
and the activation through their fused kernels, gradients for everything.

Decoding (`decode`): a few rows of x against weights quantized once
(`quantize_weights`). The norm and the activation write MXFP8 (E4M3) codes
with their scales, which the few-row product reads as they are; the weights
stay in the codes and tensor-core scale layout of the training products.
"""
from __future__ import annotations

import torch

from .binding import (BLOCK_1X32, FORMAT_E4M3, LAYOUT_ROWMAJOR, ROUND_RTN, SCALE_ROUNDUP, QuantParams,
                      mxfp4_gemv, mxfp4_quantize, mxfp4_rmsnorm_backward, mxfp4_rmsnorm_quantize,
                      mxfp4_swiglu_backward, mxfp4_swiglu_quantize)
from .linear import LinearRecipe, Mxfp4Linear


def _readable(t: torch.Tensor) -> torch.Tensor:
    """The matrix t, or a copy of it that the kernels can read (unit column
    stride, rows on 16-byte boundaries): autograd may hand over expanded
    gradients, and a view may begin anywhere."""
    rows = t.shape[0] <= 1 or (t.stride(0) >= t.shape[1] and t.stride(0) % 8 == 0)
    return t if rows and t.stride(1) == 1 and t.data_ptr() % 16 == 0 else t.clone(memory_format=torch.contiguous_format)


def _readable_vector(t: torch.Tensor | None) -> torch.Tensor | None:
    """The same for a norm's weight (a slice of a flat parameter buffer, say)."""
    if t is None or (t.is_contiguous() and t.data_ptr() % 16 == 0):
        return t
    return t.clone(memory_format=torch.contiguous_format)


class _FirstOrder(torch.autograd.Function):
    @staticmethod
    def forward(ctx, what, anchors, *tensors):
        ctx.what = what
        return tensors[anchors:]

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError(f"second derivatives of {ctx.what} are not provided")


def _first_order(what: str, anchors, *grads):
    """Gradients that a library kernel computed, on their way out of a backward
    pass. Where a graph of that pass is wanted (create_graph) and they depend on
    the tensors `anchors` (those that require grad count), they get a node that
    raises, so that a second derivative is refused; without one they would pass
    for constants and their part of it would be missing without a word."""
    if not torch.is_grad_enabled():
        return grads
    anchors = [t for t in anchors if t is not None and t.requires_grad]
    if not anchors:
        return grads
    out = iter(_FirstOrder.apply(what, len(anchors), *anchors, *[g for g in grads if g is not None]))
    return tuple(None if g is None else next(out) for g in grads)


class _RmsNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, eps, out_dtype):
        ctx.set_materialize_grads(False)
        _, _, y, h, rstd = mxfp4_rmsnorm_quantize(x, weight, residual=residual, eps=eps, y_dtype=out_dtype,
                                                  with_rstd=True)
        ctx.save_for_backward(x if h is None else h, weight, rstd)
        return y if h is None else (y, h)

    @staticmethod
    def backward(ctx, dy, dh=None):
        h, weight, rstd = ctx.saved_tensors
        need_x, need_r, need_w = ctx.needs_input_grad[:3]
        if dy is None:                                   # y unused: only the stream's gradient passes
            return dh if need_x else None, dh if need_r else None, None, None, None
        dx, dw = mxfp4_rmsnorm_backward(_readable(dy), h, weight, rstd, dh=None if dh is None else _readable(dh),
                                        with_dw=need_w)
        # (dw alone is linear in what the weight multiplies: it depends on dy only)
        dx, dw = _first_order("rmsnorm", (dy, dh, h, weight) if need_x or need_r else (dy,), dx, dw)
        return dx if need_x else None, dx if need_r else None, dw, None, None


def rmsnorm(x: torch.Tensor, weight: torch.Tensor | None = None, residual: torch.Tensor | None = None,
            eps: float = 1e-6, out_dtype: torch.dtype = torch.bfloat16):
    """Differentiable root-mean-square norm over the last dimension (a multiple
    of 32): y in out_dtype, or (y, h) with h = x + residual when a residual is
    given. x and residual share one type (bf16 or fp32). First derivatives
    only: a graph of the backward pass raises where it is differentiated."""
    lead, D = x.shape[:-1], x.shape[-1]
    r = None if residual is None else _readable(residual.reshape(-1, D))
    out = _RmsNormFn.apply(_readable(x.reshape(-1, D)), r, _readable_vector(weight), eps, out_dtype)
    if residual is None:
        return out.reshape(*lead, D)
    return out[0].reshape(*lead, D), out[1].reshape(*lead, D)


class _SwigluFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, gate, up, out_dtype):
        ctx.save_for_backward(gate, up)
        return mxfp4_swiglu_quantize(gate, up, y_dtype=out_dtype)[2]

    @staticmethod
    def backward(ctx, dy):
        gate, up = ctx.saved_tensors
        dgate, dup = mxfp4_swiglu_backward(_readable(dy), gate, up)
        # (dup alone depends on gate and dy)
        return *_first_order("swiglu", (dy, gate, up) if ctx.needs_input_grad[0] else (dy,), dgate, dup), None


def swiglu(gate: torch.Tensor, up: torch.Tensor, out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """Differentiable gate / (1 + exp(-gate)) * up in out_dtype; the last
    dimension is a multiple of 32, gate and up share one type (bf16 or fp32).
    First derivatives only, as rmsnorm."""
    lead, F = gate.shape[:-1], gate.shape[-1]
    return _SwigluFn.apply(_readable(gate.reshape(-1, F)), _readable(up.reshape(-1, F)), out_dtype).reshape(*lead, F)


class Mxfp4FeedForward(torch.nn.Module):
    """Pre-norm feed-forward block (see the module's text). dim and hidden are
    multiples of 128; training rows too, decoding rows are free."""

    def __init__(self, dim: int, hidden: int, recipe: LinearRecipe | None = None, eps: float = 1e-6,
                 device=None, dtype: torch.dtype = torch.bfloat16):
        super().__init__()
        if dim % 128 or hidden % 128:
            raise ValueError(f"dim and hidden must be multiples of 128 (got {dim}, {hidden})")
        self.dim, self.hidden, self.eps = dim, hidden, eps
        self.norm = torch.nn.Parameter(torch.ones(dim, device=device, dtype=dtype))
        self.gate_up = Mxfp4Linear(dim, 2 * hidden, recipe, device=device, dtype=dtype, out_dtype=torch.bfloat16)
        self.down = Mxfp4Linear(hidden, dim, recipe, device=device, dtype=dtype, out_dtype=torch.bfloat16)
        self._decode_params = None
        for name in self._DECODE:                        # (they follow the module to a device; not its state)
            self.register_buffer(name, None, persistent=False)

    _DECODE = ("gate_up_codes", "gate_up_scales", "down_codes", "down_scales")

    @property
    def _decode(self):
        """(codes, scales, parameters) of both weights, None before quantize_weights."""
        if self._decode_params is None:
            return None
        t = [getattr(self, name) for name in self._DECODE]
        return [(t[0], t[1], self._decode_params[0]), (t[2], t[3], self._decode_params[1])]

    def forward(self, x: torch.Tensor, residual: torch.Tensor | None = None):
        """(y, h) for bf16 x (and residual) [..., dim] with a multiple of 128 rows."""
        if residual is None:
            n, h = rmsnorm(x, self.norm, None, self.eps), x
        else:
            n, h = rmsnorm(x, self.norm, residual, self.eps)
        # (the backward pass of the two slices fills and adds two tensors of gu's size beside the activation's kernel)
        gu = self.gate_up(n)
        return self.down(swiglu(gu[..., :self.hidden], gu[..., self.hidden:])), h

    @torch.no_grad()
    def quantize_weights(self) -> None:
        """Quantizes the weights for `decode`, once; call it again after they change."""
        done = []
        for layer in (self.gate_up, self.down):
            p = layer.recipe.w_row
            if p.wht:
                raise ValueError("decoding needs weights quantized without rotation along their rows")
            q, s, _, _ = mxfp4_quantize(layer.weight.detach(), p)
            done += [q, s]
        for name, t in zip(self._DECODE, done):
            setattr(self, name, t)
        self._decode_params = [layer.recipe.w_row for layer in (self.gate_up, self.down)]

    @torch.no_grad()
    def decode(self, x: torch.Tensor, residual: torch.Tensor | None = None):
        """(y, h) for a few rows of bf16 x (and residual) [..., dim], without gradients."""
        if self._decode is None:
            raise RuntimeError("quantize_weights() has not been called")
        lead = x.shape[:-1]
        x2 = _readable(x.reshape(-1, self.dim))
        r2 = None if residual is None else _readable(residual.reshape(-1, self.dim))
        p8 = QuantParams(BLOCK_1X32, SCALE_ROUNDUP, ROUND_RTN, LAYOUT_ROWMAJOR, elem_format=FORMAT_E4M3)
        q, s, _, h, _ = mxfp4_rmsnorm_quantize(x2, _readable_vector(self.norm), p8, residual=r2, eps=self.eps)
        (qg, sg, pg), (qd, sd, pd) = self._decode
        gu = mxfp4_gemv(q, qg, sg, 2 * self.hidden, self.dim, pg, sx=s)
        qa, sa, _ = mxfp4_swiglu_quantize(gu[:, :self.hidden], gu[:, self.hidden:], p8)
        y = mxfp4_gemv(qa, qd, sd, self.dim, self.hidden, pd, sx=sa)
        return y.reshape(*lead, self.dim), (x if h is None else h.reshape(*lead, self.dim))
