"""The calls on the 8-bit cache of keys and values against their definition in
64 bits: appends and reads bit for bit, attention within bounds that follow
from its roundings (tests/_cache.py)."""
from __future__ import annotations

import math

import pytest
import torch

from _cache import DEV, append, attend, attention_bounds, gen, make_cache, values

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def same(a, b):
    assert a.shape == b.shape and a.dtype == b.dtype
    if a.dtype.is_floating_point:
        assert torch.equal(torch.isnan(a), torch.isnan(b))
        a, b = torch.nan_to_num(a.double()), torch.nan_to_num(b.double())
    bad = torch.nonzero(a != b)
    assert not len(bad), f"{len(bad)} differ, first at {bad[0].tolist()}: {a[tuple(bad[0])]} for {b[tuple(bad[0])]}"


# ------------------------------------------------------------------ append ---

APPENDS = [
    # L, n, H, D, P
    ([1], [1], 1, 64, 16), ([700], [1], 8, 128, 64), ([64, 65, 128, 1], [1, 1, 1, 1], 2, 128, 64),
    ([17, 16, 33, 40, 15], [17, 16, 1, 25, 15], 3, 64, 16), ([200, 0, 90, 31], [130, 0, 90, 0], 2, 96, 32),
    ([1000, 555], [1000, 300], 4, 192, 128), ([129, 7, 300], [129, 3, 172], 5, 256, 128),
    ([2000], [1999], 1, 256, 16), ([63, 64, 65], [62, 63, 64], 16, 96, 64),
    ([50, 3, 100, 17], [50, 2, 41, 17], 3, 96, 16), ([300, 9, 64], [3, 2, 4], 9, 256, 64),
    ([i % 70 + 1 for i in range(700)], [i % 3 if i % 70 > 3 else 1 for i in range(700)], 2, 64, 16),
    ([300 + i for i in range(40)], [100 + 3 * i for i in range(40)], 2, 128, 32),
]


@pytest.mark.parametrize("L,n,H,D,P", APPENDS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_append(L, n, H, D, P, dtype):
    import gemm_pt_block_gb300 as mx

    c = make_cache(L, n, H, D, P, seed=len(L), filled=[a - b for a, b in zip(L, n)])
    kv = torch.randn((c.T, 2, H, D), device=DEV, generator=gen(3))
    kv[:, :, 0] *= 40.0                                     # pages whose scale grows, and pages whose does not
    kv[..., 3] *= 2.0 ** -9
    kv = kv.to(dtype)
    want = append(c, kv[:, 0], kv[:, 1])
    one = all(m == 1 for m in n)
    for starts in ([None, c.starts] if one else [c.starts]):
        codes, scales = c.codes.clone(), c.scales.clone()
        mx.mxfp8_cache_append(kv[:, 0], kv[:, 1], codes, scales, c.table, c.lens, starts=starts)
        assert mx.device_status() == 0
        same(scales, want[1])
        same(codes, want[0])


def test_append_again_changes_nothing():
    import gemm_pt_block_gb300 as mx

    c = make_cache([50, 100], [10, 70], 2, 128, 32, filled=[40, 30])
    kv = (torch.randn((80, 2, 2, 128), device=DEV, generator=gen(4)) * 30).to(BF16)
    mx.mxfp8_cache_append(kv[:, 0], kv[:, 1], c.codes, c.scales, c.table, c.lens, starts=c.starts)
    once = c.codes.clone(), c.scales.clone()
    mx.mxfp8_cache_append(kv[:, 0], kv[:, 1], c.codes, c.scales, c.table, c.lens, starts=c.starts)
    same(c.codes, once[0])
    same(c.scales, once[1])


@pytest.mark.parametrize("dtype,at,step", [(F32, 2.0 ** -149, 1), (F32, 2.0 ** -130, 1), (F32, 3.0e38, 2), (BF16, 2.0 ** -133, 1),
                                           (BF16, 3.3e38, 3), (F32, 448.0, 1), (F32, 448.00003, 1)])
def test_append_of_the_smallest_and_largest_values(dtype, at, step):
    import gemm_pt_block_gb300 as mx

    c = make_cache([20], [20], 1, 64, 16, filled=[0])
    kv = torch.randn((20, 2, 1, 64), device=DEV, generator=gen(5)).clamp(-1, 1).double()
    kv[0, :, :, 0] = 1.0
    kv = (kv * at).to(dtype)
    want = append(c, kv[:, 0], kv[:, 1])
    mx.mxfp8_cache_append(kv[:, 0], kv[:, 1], c.codes, c.scales, c.table, c.lens, starts=c.starts)
    same(c.scales, want[1])
    same(c.codes, want[0])


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_append_of_what_is_no_number(bad):
    """The page's scale becomes NaN, its new codes 0; its neighbours and the other heads are untouched; and it stays."""
    import gemm_pt_block_gb300 as mx

    c = make_cache([70, 5], [40, 5], 2, 64, 32, filled=[30, 0])
    kv = torch.randn((45, 2, 2, 64), device=DEV, generator=gen(6)).to(BF16)
    kv[1, 0, 1, 7] = bad                                    # a token of the page that holds older ones
    kv[42, 1, 0, 63] = bad
    want = append(c, kv[:, 0], kv[:, 1])
    mx.mxfp8_cache_append(kv[:, 0], kv[:, 1], c.codes, c.scales, c.table, c.lens, starts=c.starts)
    same(c.scales, want[1])
    same(c.codes, want[0])
    assert int((c.scales == 255).sum()) - 3 * 2 * 2 == 2
    # later tokens of the page
    c.L, c.n = [70, 9], [0, 4]
    c.lens, c.starts = torch.tensor([70, 9], dtype=torch.int32, device=DEV), torch.tensor([0, 0, 4], dtype=torch.int32, device=DEV)
    kv = torch.randn((4, 2, 2, 64), device=DEV, generator=gen(7))
    want = append(c, kv[:, 0], kv[:, 1])
    mx.mxfp8_cache_append(kv[:, 0], kv[:, 1], c.codes, c.scales, c.table, c.lens, starts=c.starts)
    same(c.scales, want[1])
    same(c.codes, want[0])


def test_append_of_zeros_and_scales_far_apart():
    import gemm_pt_block_gb300 as mx

    c = make_cache([10, 40], [4, 8], 1, 64, 16, filled=[6, 32])
    kv = torch.zeros((12, 2, 1, 64), device=DEV)
    kv[4:] = torch.randn((8, 2, 1, 64), device=DEV, generator=gen(8)) * 2.0 ** 100
    c.scales[c.table[1, 1].long()] = 3                      # 2^-124
    want = append(c, kv[:, 0], kv[:, 1])
    mx.mxfp8_cache_append(kv[:, 0], kv[:, 1], c.codes, c.scales, c.table, c.lens, starts=c.starts)
    same(c.scales, want[1])
    same(c.codes, want[0])


# -------------------------------------------------------------------- read ---

@pytest.mark.parametrize("L,H,D,P", [([1], 1, 64, 16), ([777], 8, 128, 64), ([17, 0, 300, 16, 15], 3, 96, 16),
                                     ([128, 129, 127, 1], 2, 256, 128), ([1000, 33], 5, 192, 32)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_read(L, H, D, P, dtype):
    import gemm_pt_block_gb300 as mx

    c = make_cache(L, L, H, D, P, seed=9)
    c.scales[c.table[0, 0].long(), 1, 0] = 255
    want = torch.cat([c.tokens(b, x) for b, x in enumerate(L)], 2).transpose(1, 2)    # [2, T, H, D]
    k, v = mx.mxfp8_cache_read(c.codes, c.scales, c.table, c.starts, c.T, out_dtype=dtype)
    assert mx.device_status() == 0
    same(k, want[0].float().to(dtype))
    same(v, want[1].float().to(dtype))
    # a part of each sequence, into rows of its own; the rows behind the last are left
    part = [x // 2 for x in L]
    starts = torch.tensor([0] + [sum(part[:i + 1]) for i in range(len(L))], dtype=torch.int32, device=DEV)
    rows = sum(part) + 5
    k, v = (torch.full((rows, H, D), 7.0, dtype=dtype, device=DEV) for _ in range(2))
    mx.mxfp8_cache_read(c.codes, c.scales, c.table, starts, rows, k=k, v=v)
    want = torch.cat([c.tokens(b, x) for b, x in enumerate(part)] + [torch.full((2, H, 5, D), 7.0, device=DEV)], 2)
    same(k, want[0].transpose(0, 1).float().to(dtype))
    same(v, want[1].transpose(0, 1).float().to(dtype))


@pytest.mark.parametrize("scale", [0, 1, 20, 127, 247])
def test_read_of_every_code_and_far_scales(scale):
    import gemm_pt_block_gb300 as mx

    codes = torch.arange(512, device=DEV).to(torch.uint8)
    codes[codes & 0x7F == 0x7F] = 0
    codes = codes.view(1, 1, 1, 8, 64).repeat(1, 2, 1, 2, 1).contiguous()
    scales = torch.full((1, 2, 1), scale, dtype=torch.uint8, device=DEV)
    table = torch.zeros((1, 1), dtype=torch.int32, device=DEV)
    starts = torch.tensor([0, 16], dtype=torch.int32, device=DEV)
    want = values(codes, scales)[0, 0].transpose(0, 1)
    for dtype in (BF16, F32):
        k, v = mx.mxfp8_cache_read(codes, scales, table, starts, 16, out_dtype=dtype)
        same(k, want.float().to(dtype))
        same(v, want.float().to(dtype))


# --------------------------------------------------------------- attention ---

def check(c, q, got, lse, dtype, **kw):
    ref, want_lse, weight, reach = attend(c, q, **kw)
    lim, lse_lim = attention_bounds(dtype, max(c.L + [1]), ref, weight, reach)
    assert got.dtype == dtype and got.shape == ref.shape
    off = (got.double() - ref).abs()
    worst = (off / lim.clamp_min(1e-300)).max()
    assert bool((off <= lim).all()), f"out up to {float(worst):.3g} of its bound"
    if lse is not None:
        empty = torch.isinf(want_lse)
        assert torch.equal(empty, torch.isinf(lse)) and bool((lse[empty] < 0).all())
        off = torch.where(empty, 0.0, (lse.double() - want_lse).abs())
        lim = torch.where(empty, 0.0, lse_lim + 2.0 ** -23 * want_lse.abs())
        assert bool((off <= lim).all()), f"lse off by {float((off - lim).max()):.3g} more than its bound"


ATTENTIONS = [
    # L, n, Hq, H, D, P
    ([1], [1], 1, 1, 64, 16), ([1, 2, 15, 16, 17], [1] * 5, 4, 2, 64, 16), ([777], [1], 32, 8, 128, 64),
    ([31, 32, 33, 63, 64, 65, 255, 256, 257], [1] * 9, 8, 1, 128, 32), ([0, 5, 0, 300], [0, 1, 0, 1], 6, 2, 96, 32),
    ([2000, 3], [1, 1], 16, 1, 256, 128), ([513, 40], [1, 1], 7, 7, 192, 64), ([4000], [1], 5, 1, 128, 16),
    ([100, 7, 333], [4, 7, 1], 8, 2, 128, 64), ([2, 1], [5, 3], 4, 4, 64, 32), ([0], [3], 4, 2, 64, 16),
    ([600], [40], 12, 4, 128, 32), ([90, 1000, 1], [33, 2, 1], 20, 1, 64, 16), ([700, 70], [9, 17], 3, 1, 256, 64),
    ([40, 300], [2, 3], 64, 1, 96, 128), ([500] * 40, [1] * 40, 8, 8, 64, 64),
]


@pytest.mark.parametrize("L,n,Hq,H,D,P", ATTENTIONS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention(L, n, Hq, H, D, P, dtype):
    import gemm_pt_block_gb300 as mx

    c = make_cache(L, n, H, D, P, seed=11)
    q = torch.randn((c.T, Hq, D), device=DEV, generator=gen(12)).to(BF16)
    out, lse = mx.mxfp8_cache_attention(q, c.codes, c.scales, c.table, c.lens, starts=c.starts, out_dtype=dtype,
                                        with_lse=True)
    assert mx.device_status() == 0
    check(c, q, out, lse, dtype)
    if n == [1] * len(n):
        again, none = mx.mxfp8_cache_attention(q, c.codes, c.scales, c.table, c.lens, out_dtype=dtype)
        assert none is None
        same(again, out)


@pytest.mark.parametrize("L,n,Hq,H,D,P", [([300, 5, 70], [1, 1, 1], 8, 2, 128, 64), ([200, 3], [6, 4], 4, 1, 64, 16),
                                          ([1100], [3], 6, 3, 256, 128)])
@pytest.mark.parametrize("kw", [dict(window=1), dict(window=33), dict(window=64), dict(window=300), dict(softcap=2.0),
                                dict(softcap=50.0), dict(slopes=0.3), dict(slopes=-0.01), dict(scale=0.5), dict(scale=0.0),
                                dict(scale=-0.1), dict(window=100, softcap=5.0, slopes=0.05, scale=0.2)], ids=str)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_options(L, n, Hq, H, D, P, kw, dtype):
    import gemm_pt_block_gb300 as mx

    c = make_cache(L, n, H, D, P, seed=13)
    q = torch.randn((c.T, Hq, D), device=DEV, generator=gen(14)).to(BF16)
    kw = dict(kw)
    if "slopes" in kw:
        kw["slopes"] = kw["slopes"] * torch.exp2(-torch.arange(Hq, device=DEV, dtype=torch.float32))
    out, lse = mx.mxfp8_cache_attention(q, c.codes, c.scales, c.table, c.lens, starts=c.starts, out_dtype=dtype,
                                        with_lse=True, **kw)
    check(c, q, out, lse, dtype, **kw)


def test_attention_of_peaked_and_far_apart_scores():
    """One token takes all the weight, the first or the last; scores that fall by thousands."""
    import gemm_pt_block_gb300 as mx

    c = make_cache([900, 900, 400], [1, 1, 1], 2, 128, 64, seed=15)
    q = torch.randn((3, 8, 128), device=DEV, generator=gen(16))
    k = [c.tokens(b, x)[0] for b, x in enumerate(c.L)]
    q[0, :4] = k[0][0, 0].float() * 20
    q[1, 4:] = k[1][1, -1].float() * 20
    q[2] *= 300
    q = q.to(BF16)
    for dtype in (BF16, F32):
        out, lse = mx.mxfp8_cache_attention(q, c.codes, c.scales, c.table, c.lens, out_dtype=dtype, with_lse=True)
        check(c, q, out, lse, dtype)


def test_attention_of_queries_of_far_sizes():
    """Queries are scaled row by row: tiny and huge rows beside one another, zeros, and wide ranges inside a row."""
    import gemm_pt_block_gb300 as mx

    c = make_cache([333], [6], 1, 64, 32, seed=17)
    q = torch.randn((6, 2, 64), device=DEV, generator=gen(18))
    q[0] *= 2.0 ** -120
    q[1] *= 2.0 ** 20
    q[2] = 0
    q[3] *= torch.exp2(-torch.arange(64, device=DEV).float() / 3)
    q = q.to(BF16)
    for scale in (0.125, 2.0 ** -18):
        out, lse = mx.mxfp8_cache_attention(q, c.codes, c.scales, c.table, c.lens, starts=c.starts, out_dtype=F32,
                                            with_lse=True, scale=scale)
        check(c, q, out, lse, F32, scale=scale)


def test_attention_of_pages_with_far_scales():
    import gemm_pt_block_gb300 as mx

    c = make_cache([200], [1], 2, 64, 16, seed=19)
    pages = c.table[0, :13].long()
    c.scales[pages[3], 1] = 60                              # values of 2^-67
    c.scales[pages[5], 0] = 40                              # keys that count for nothing
    c.scales[pages[7], 1] = 0
    c.scales[pages[8], 0] = 133
    q = torch.randn((1, 4, 64), device=DEV, generator=gen(20)).to(BF16)
    out, lse = mx.mxfp8_cache_attention(q, c.codes, c.scales, c.table, c.lens, out_dtype=F32, with_lse=True)
    check(c, q, out, lse, F32)


def test_attention_of_what_is_no_number():
    """NaN where it is attended, and nowhere else: a page of scale 0xFF behind a
    query's own position or before its window, other heads, other sequences."""
    import gemm_pt_block_gb300 as mx

    c = make_cache([64, 64], [20, 20], 2, 64, 16, seed=21)
    page = c.table[0].long()
    c.scales[page[3], 1, 0] = 255                           # values of tokens 48 .. 63, head 0
    c.scales[page[2], 0, 1] = 255                           # keys of tokens 32 .. 47, head 1
    q = torch.randn((40, 4, 64), device=DEV, generator=gen(22)).to(BF16)
    out, lse = mx.mxfp8_cache_attention(q, c.codes, c.scales, c.table, c.lens, starts=c.starts, with_lse=True, window=10)
    p = torch.arange(20, device=DEV) + 44
    want = torch.zeros((40, 4), dtype=torch.bool, device=DEV)
    want[:20, :2] = (p >= 48)[:, None]
    want[:20, 2:] = (p - 9 <= 47)[:, None]
    nan = torch.isnan(out)
    assert torch.equal(nan.any(-1), want) and torch.equal(nan.all(-1), want)
    keys = want.clone()
    keys[:, :2] = False
    assert torch.equal(torch.isnan(lse), keys)
    # a query that is no number
    c = make_cache([64, 40], [2, 1], 1, 64, 16, seed=23)
    for bad in (math.nan, math.inf, -math.inf):
        q = torch.randn((3, 3, 64), device=DEV, generator=gen(24)).to(BF16)
        q[1, 2, 9] = bad
        out, lse = mx.mxfp8_cache_attention(q, c.codes, c.scales, c.table, c.lens, starts=c.starts, with_lse=True)
        want = torch.zeros((3, 3), dtype=torch.bool, device=DEV)
        want[1, 2] = True
        assert torch.equal(torch.isnan(out).all(-1), want) and torch.equal(torch.isnan(out).any(-1), want)
        assert torch.equal(torch.isnan(lse), want)


def test_attention_leaves_other_rows():
    import gemm_pt_block_gb300 as mx

    c = make_cache([30, 50], [2, 3], 2, 64, 16, seed=25)
    q = torch.randn((11, 4, 64), device=DEV, generator=gen(26)).to(BF16)
    starts = c.starts + 2
    out, lse = torch.full((11, 4, 64), 9.0, device=DEV), torch.full((11, 4), 9.0, device=DEV)
    mx.mxfp8_cache_attention(q, c.codes, c.scales, c.table, c.lens, starts=starts, out=out, lse=lse)
    check(c, q[2:7], out[2:7], lse[2:7], F32)
    assert bool((out[:2] == 9).all()) and bool((out[7:] == 9).all()) and bool((lse[:2] == 9).all()) and bool((lse[7:] == 9).all())


def test_strides():
    """Slices of one product's output, heads before tokens, a wide table."""
    import gemm_pt_block_gb300 as mx

    c = make_cache([40, 100, 70], [10, 1, 20], 2, 64, 32, seed=27, filled=[30, 99, 50])
    qkv = torch.randn((c.T, 8, 64), device=DEV, generator=gen(28)).to(BF16)
    k, v = qkv[:, 4:6], qkv[:, 6:]
    want = append(c, k, v)
    wide = torch.full((3, 40), 1 << 29, dtype=torch.int32, device=DEV)
    wide[:, :c.table.shape[1]] = c.table
    for kk, vv in ((k, v), (k.transpose(0, 1).contiguous().transpose(0, 1), v.contiguous())):
        codes, scales = c.codes.clone(), c.scales.clone()
        mx.mxfp8_cache_append(kk, vv, codes, scales, wide[:, :c.table.shape[1]], c.lens, starts=c.starts)
        same(codes, want[0])
        same(scales, want[1])
    c.codes, c.scales = want
    ref, lse = mx.mxfp8_cache_attention(qkv[:, :4].contiguous(), c.codes, c.scales, c.table, c.lens, starts=c.starts,
                                        with_lse=True)
    check(c, qkv[:, :4], ref, lse, BF16)
    for q in (qkv[:, :4], qkv[:, :4].transpose(0, 1).contiguous().transpose(0, 1)):
        out = torch.empty((4, c.T + 3, 72), dtype=BF16, device=DEV)[:, :c.T, 8:].transpose(0, 1)
        got, _ = mx.mxfp8_cache_attention(q, c.codes, c.scales, wide[:, :c.table.shape[1]], c.lens, starts=c.starts, out=out)
        assert got.data_ptr() == out.data_ptr()
        same(got.contiguous(), ref)
    n = [40, 3, 70]
    starts = torch.tensor([0, 40, 43, 113], dtype=torch.int32, device=DEV)
    k, v = mx.mxfp8_cache_read(c.codes, c.scales, c.table, starts, 113)
    kk, vv = torch.zeros((2, 113, 64), dtype=BF16, device=DEV).transpose(0, 1), torch.zeros((113, 6, 64), dtype=BF16, device=DEV)[:, 2:4]
    mx.mxfp8_cache_read(c.codes, c.scales, c.table, starts, 113, k=kk, v=vv)
    same(kk.contiguous(), k)
    same(vv.contiguous(), v)
    assert sum(n) == 113


def test_codes_past_four_gigabytes():
    """Pages whose bytes lie beyond 2^32 of the cache's beginning."""
    import gemm_pt_block_gb300 as mx

    small = make_cache([100], [30], 1, 256, 128, seed=29, filled=[70])
    kv = torch.randn((30, 2, 1, 256), device=DEV, generator=gen(30)).to(BF16)
    q = torch.randn((30, 2, 256), device=DEV, generator=gen(31)).to(BF16)
    pages = (1 << 32) // (2 * 128 * 256) + 7
    codes = torch.empty((pages, 2, 1, 128, 256), dtype=torch.uint8, device=DEV)
    scales = torch.empty((pages, 2, 1), dtype=torch.uint8, device=DEV)
    codes[-3], scales[-3] = small.codes[small.table[0, 0].long()], small.scales[small.table[0, 0].long()]
    table = torch.full((1, 1), pages - 3, dtype=torch.int32, device=DEV)
    want = append(small, kv[:, 0], kv[:, 1])
    mx.mxfp8_cache_append(kv[:, 0], kv[:, 1], codes, scales, table, small.lens, starts=small.starts)
    small.codes, small.scales = want
    same(codes[-3], small.codes[small.table[0, 0].long()])
    out, lse = mx.mxfp8_cache_attention(q, codes, scales, table, small.lens, starts=small.starts, with_lse=True)
    check(small, q, out, lse, BF16)
    starts = torch.tensor([0, 100], dtype=torch.int32, device=DEV)
    k, _ = mx.mxfp8_cache_read(codes, scales, table, starts, 100, out_dtype=F32)
    same(k, small.tokens(0, 100)[0].transpose(0, 1).float())
