"""Attention for decoding: a cache of keys and values in 8 bits, and the
attention half of a layer on weights quantized once.

    h = x + residual;  n = rmsnorm(h);  (q, k, v) = n W_qkv^T;
    k, v into the cache;  o = attention(q, cache);  y = o W_out^T

The block returns (y, h) like the feed-forward block (ffn.py), so that the two
alternate: y joins the residual stream h in the next block's norm.

The cache lies in pages of tokens that the caller hands out: a table names each
sequence's pages in order, lens its tokens (the new ones included), starts the
rows of its new tokens (None: one row each). The same three go to every call of
a step.
"""
from __future__ import annotations

import torch

from .binding import (BLOCK_1X32, FORMAT_E4M3, LAYOUT_ROWMAJOR, ROUND_RTN, SCALE_ROUNDUP, QuantParams,
                      mxfp4_gemv, mxfp4_quantize, mxfp4_rmsnorm_quantize, mxfp8_cache_append, mxfp8_cache_attention,
                      mxfp8_cache_read)
from .ffn import _readable, _readable_vector
from .linear import LinearRecipe, Mxfp4Linear


def _check_head_dim(head_dim: int) -> None:
    if head_dim not in (64, 96, 128, 192, 256):
        raise ValueError(f"head_dim must be 64, 96, 128, 192 or 256 (got {head_dim})")


class KvCache:
    """Keys and values of one layer in 8 bits: E4M3 codes [pages, 2, heads,
    page_tokens, head_dim] and one E8M0 scale for each page, kind and head,
    scales [pages, 2, heads]. page_tokens is 16, 32, 64 or 128, head_dim 64, 96,
    128, 192 or 256."""

    def __init__(self, pages: int, heads: int, head_dim: int, page_tokens: int = 64, device=None):
        if page_tokens not in (16, 32, 64, 128):
            raise ValueError(f"page_tokens must be 16, 32, 64 or 128 (got {page_tokens})")
        _check_head_dim(head_dim)
        self.codes = torch.zeros((pages, 2, heads, page_tokens, head_dim), dtype=torch.uint8, device=device)
        self.scales = torch.zeros((pages, 2, heads), dtype=torch.uint8, device=device)

    @property
    def page_tokens(self) -> int:
        return self.codes.shape[3]

    def append(self, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor, lens: torch.Tensor,
               starts: torch.Tensor | None = None) -> None:
        """Quantizes new keys and values into their pages (mxfp8_cache_append)."""
        mxfp8_cache_append(k, v, self.codes, self.scales, page_table, lens, starts=starts)

    def attend(self, q: torch.Tensor, page_table: torch.Tensor, lens: torch.Tensor,
               starts: torch.Tensor | None = None, **options):
        """(out, lse) of the new tokens' queries over the cache (mxfp8_cache_attention)."""
        return mxfp8_cache_attention(q, self.codes, self.scales, page_table, lens, starts=starts, **options)

    def read(self, page_table: torch.Tensor, starts: torch.Tensor, rows: int, **options):
        """(k, v) of each sequence's first tokens (mxfp8_cache_read)."""
        return mxfp8_cache_read(self.codes, self.scales, page_table, starts, rows, **options)


class Mxfp4Attention(torch.nn.Module):
    """The attention half of a pre-norm layer, for decoding (see the module's
    text). `heads` query heads share `kv_heads` heads of the cache (default: as
    many), of head_dim channels (default: dim // heads; 64, 96, 128, 192 or 256).
    slopes: [heads], kept as fp32. dim, heads * head_dim and (heads + 2 kv_heads) *
    head_dim are multiples of 128. The projections' parameters are those of Mxfp4Linear; no backward pass
    through the attention is provided."""

    _DECODE = ("qkv_codes", "qkv_scales", "out_codes", "out_scales")

    def __init__(self, dim: int, heads: int, kv_heads: int | None = None, head_dim: int | None = None,
                 recipe: LinearRecipe | None = None, eps: float = 1e-6, window: int = 0, softcap: float = 0.0,
                 slopes: torch.Tensor | None = None, device=None, dtype: torch.dtype = torch.bfloat16):
        super().__init__()
        kv_heads = heads if kv_heads is None else kv_heads
        if heads < 1 or kv_heads < 1 or heads % kv_heads:
            raise ValueError(f"heads must be a multiple of kv_heads (got {heads}, {kv_heads})")
        head_dim = dim // heads if head_dim is None else head_dim
        _check_head_dim(head_dim)
        wide = (heads + 2 * kv_heads) * head_dim
        if dim % 128 or heads * head_dim % 128 or wide % 128:
            raise ValueError(f"dim, heads * head_dim and (heads + 2 kv_heads) * head_dim must be multiples of 128 "
                             f"(got {dim}, {heads * head_dim}, {wide})")
        self.dim, self.heads, self.kv_heads, self.head_dim, self.eps = dim, heads, kv_heads, head_dim, eps
        self.window, self.softcap = window, softcap
        self.norm = torch.nn.Parameter(torch.ones(dim, device=device, dtype=dtype))
        self.qkv = Mxfp4Linear(dim, wide, recipe, device=device, dtype=dtype, out_dtype=torch.bfloat16)
        self.out = Mxfp4Linear(heads * head_dim, dim, recipe, device=device, dtype=dtype, out_dtype=torch.bfloat16)
        if slopes is not None:
            if slopes.shape != (heads,):
                raise ValueError(f"slopes must be [{heads}] (got {list(slopes.shape)})")
            slopes = slopes.detach().to(device=device, dtype=torch.float32, copy=True).contiguous()
        self.register_buffer("slopes", slopes)
        self._decode_params = None
        for name in self._DECODE:                        # (they follow the module to a device; not its state)
            self.register_buffer(name, None, persistent=False)

    def _apply(self, fn, recurse=True):
        """The slopes follow the block to a device, not to a type: the kernel reads fp32, and
        rounded ones would not come back."""
        slopes = self.slopes
        super()._apply(fn, recurse)
        if slopes is not None and self.slopes.dtype != slopes.dtype:
            self.slopes = slopes.to(self.slopes.device)
        return self

    def cache(self, pages: int, page_tokens: int = 64) -> KvCache:
        """A cache for this layer, on its device."""
        return KvCache(pages, self.kv_heads, self.head_dim, page_tokens, self.norm.device)

    @torch.no_grad()
    def quantize_weights(self) -> None:
        """Quantizes the weights for `decode`, once; call it again after they change."""
        done = []
        for layer in (self.qkv, self.out):
            p = layer.recipe.w_row
            if p.wht:
                raise ValueError("decoding needs weights quantized without rotation along their rows")
            q, s, _, _ = mxfp4_quantize(layer.weight.detach(), p)
            done += [q, s]
        for name, t in zip(self._DECODE, done):
            setattr(self, name, t)
        self._decode_params = (self.qkv.recipe.w_row, self.out.recipe.w_row)

    @torch.no_grad()
    def decode(self, x: torch.Tensor, cache: KvCache, page_table: torch.Tensor, lens: torch.Tensor,
               residual: torch.Tensor | None = None, starts: torch.Tensor | None = None, rotate=None):
        """(y, h) for the new tokens' rows of bf16 x (and residual) [tokens, dim],
        whose keys and values join the cache. `rotate` (None: nothing) takes the
        step's (q, k) [tokens, heads, head_dim] and returns them with their
        positions' rotation applied."""
        if self._decode_params is None:
            raise RuntimeError("quantize_weights() has not been called")
        H, G, D = self.kv_heads, self.heads, self.head_dim
        x2 = _readable(x)
        r2 = None if residual is None else _readable(residual)
        p8 = QuantParams(BLOCK_1X32, SCALE_ROUNDUP, ROUND_RTN, LAYOUT_ROWMAJOR, elem_format=FORMAT_E4M3)
        n, s, _, h, _ = mxfp4_rmsnorm_quantize(x2, _readable_vector(self.norm), p8, residual=r2, eps=self.eps)
        qkv = mxfp4_gemv(n, self.qkv_codes, self.qkv_scales, (G + 2 * H) * D, self.dim, self._decode_params[0], sx=s)
        qkv = qkv.view(-1, G + 2 * H, D)
        q, k, v = qkv[:, :G], qkv[:, G:G + H], qkv[:, G + H:]
        if rotate is not None:
            q, k = rotate(q, k)
        cache.append(k, v, page_table, lens, starts)
        o, _ = cache.attend(q, page_table, lens, starts, window=self.window, softcap=self.softcap, slopes=self.slopes)
        y = mxfp4_gemv(o.view(-1, G * D), self.out_codes, self.out_scales, self.dim, G * D, self._decode_params[1])
        return y, (x if h is None else h)
