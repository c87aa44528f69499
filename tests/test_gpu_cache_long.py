"""Attention over long runs of tokens: tiles that more CTAs share than the join's
warps have lanes (one head of keys and values, 11 thousand tokens and more at
128 channels), by themselves and among short sequences."""
from __future__ import annotations

import pytest
import torch

from _cache import DEV, gen, make_cache
from test_gpu_cache import check

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32

RUNS = [
    # L, n, Hq, H, D, P
    ([20000], [1], 8, 1, 128, 64), ([100003], [1], 8, 1, 128, 128), ([33333], [1], 1, 1, 64, 32), ([99999], [1], 5, 1, 64, 128),
    ([20011], [1], 4, 1, 256, 64), ([70001], [1], 16, 1, 96, 128), ([25000], [3], 6, 1, 192, 64), ([40000], [1], 6, 3, 128, 128),
    ([3, 50001, 700], [1, 2, 1], 4, 1, 128, 64), ([30] * 20 + [60007] + [45] * 20, [1] * 41, 4, 1, 128, 128),
]


@pytest.mark.parametrize("L,n,Hq,H,D,P", RUNS, ids=lambda v: str(v) if isinstance(v, int) else f"{max(v)}x{len(v)}")
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_long_runs(L, n, Hq, H, D, P, dtype):
    import gemm_pt_block_gb300 as mx

    c = make_cache(L, n, H, D, P, seed=70)
    q = torch.randn((c.T, Hq, D), device=DEV, generator=gen(71)).to(BF16)
    out, lse = mx.mxfp8_cache_attention(q, c.codes, c.scales, c.table, c.lens, starts=c.starts, out_dtype=dtype, with_lse=True)
    assert mx.device_status() == 0
    check(c, q, out, lse, dtype)


@pytest.mark.parametrize("kw", [dict(window=30000), dict(softcap=5.0), dict(slopes=1e-4)], ids=str)
def test_long_runs_with_options(kw):
    import gemm_pt_block_gb300 as mx

    c = make_cache([65000], [1], 1, 128, 128, seed=72)
    q = torch.randn((1, 8, 128), device=DEV, generator=gen(73)).to(BF16)
    kw = dict(kw)
    if "slopes" in kw:
        kw["slopes"] = kw["slopes"] * torch.exp2(-torch.arange(8, device=DEV, dtype=torch.float32))
    out, lse = mx.mxfp8_cache_attention(q, c.codes, c.scales, c.table, c.lens, out_dtype=F32, with_lse=True, **kw)
    assert mx.device_status() == 0
    check(c, q, out, lse, F32, **kw)


def test_the_first_and_the_last_part_alone_count():
    """All the weight in one token, at either end of a run that 152 CTAs share."""
    import gemm_pt_block_gb300 as mx

    c = make_cache([80000], [1], 1, 128, 128, seed=74)
    k = c.tokens(0, 80000)[0][0]
    q = torch.stack([k[0], k[-1], k[40000], -k[0]]).float().mul(20).to(BF16)[None]
    for dtype in (BF16, F32):
        out, lse = mx.mxfp8_cache_attention(q, c.codes, c.scales, c.table, c.lens, out_dtype=dtype, with_lse=True)
        check(c, q, out, lse, dtype)
    assert mx.device_status() == 0
