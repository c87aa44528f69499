"""The 8-bit cache's calls at their limits: what the device's arrays say wrong
(pages, lengths, rows: skipped, reported, and nothing else touched), buffers that
the binding refuses, the bounds-checking build, many sequences."""
from __future__ import annotations

import pytest
import torch

from _cache import DEV, append, attend, attention_bounds, gen, make_cache
from test_gpu_bounds_check import _both, _equal, _using, bc_lib  # noqa: F401  (bc_lib is a fixture)
from test_gpu_cache import check, same

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
BAD = 1                                                     # MXFP4_ERR_INVALID_ARG


def setup(P=32, D=64, H=2):
    c = make_cache([100, 70, 40], [3, 1, 2], H, D, P, seed=1, filled=[97, 69, 38])
    g = gen(2)
    kv = torch.randn((c.T, 2, H, D), device=DEV, generator=g).to(BF16)
    q = torch.randn((c.T, 2 * H, D), device=DEV, generator=g).to(BF16)
    return c, kv, q


def spoil(c, what):
    """The sequences that a fault concerns; the others must not notice."""
    if what == "page below":
        c.table[1, 2] = -7
    elif what == "page above":
        c.table[1, 2] = c.codes.shape[0]
    elif what == "largest page":
        c.table[1, 2] = 2 ** 31 - 1
    elif what == "length below":
        c.lens[1] = -5
    elif what == "length above":
        c.lens[1] = c.table.shape[1] * c.P + 1
    elif what == "largest length":
        c.lens[1] = 2 ** 31 - 1
    return 1


@pytest.mark.parametrize("what", ["page below", "page above", "largest page", "length below", "length above", "largest length"])
def test_a_wrong_page_or_length(what):
    import gemm_pt_block_gb300 as mx

    c, kv, q = setup()
    want = append(c, kv[:, 0], kv[:, 1])
    spared = c.codes.clone(), c.scales.clone()
    b = spoil(c, what)
    mx.mxfp8_cache_append(kv[:, 0], kv[:, 1], c.codes, c.scales, c.table, c.lens, starts=c.starts)
    assert mx.device_status() == BAD
    assert mx.device_status() == 0
    wrong = make_cache([100, 70, 40], [3, 1, 2], 2, 64, 32, seed=1, filled=[97, 69, 38]).table[b].long()
    wrong = wrong[(wrong >= 0) & (wrong < c.codes.shape[0])]
    want[0][wrong], want[1][wrong] = spared[0][wrong], spared[1][wrong]     # (its pages stay as they were)
    same(c.codes, want[0])
    same(c.scales, want[1])
    out, lse = mx.mxfp8_cache_attention(q, c.codes, c.scales, c.table, c.lens, starts=c.starts, with_lse=True)
    assert mx.device_status() == BAD
    ref, ref_lse, weight, reach = attend(make_view(c, b), q)
    lim, _ = attention_bounds(BF16, 100, ref, weight, reach)
    rows = torch.ones(c.T, dtype=torch.bool, device=DEV)
    rows[3:4] = False                                       # sequence 1's
    assert bool(((out.double() - ref).abs() <= lim)[rows].all())
    if what == "length below":
        assert bool((out[3] == 0).all()) and bool(torch.isinf(lse[3]).all())
    else:
        assert bool(torch.isnan(out[3]).all())
    starts = torch.tensor([0, 10, 80, 90], dtype=torch.int32, device=DEV)
    k = torch.full((90, 2, 64), 5.0, device=DEV)
    v = k.clone()
    mx.mxfp8_cache_read(c.codes, c.scales, c.table, starts, 90, k=k, v=v)
    assert mx.device_status() == (BAD if "page" in what else 0)
    both = c.tokens(0, 10)[0].transpose(0, 1).float()
    same(k[:10], both)
    if "page" in what:
        assert bool((k[10 + 64:80] == 5).all())


def make_view(c, without):
    """The cache with one sequence's tokens out of the way of the reference."""
    from _cache import Cache

    L, n = [100, 70, 40], [3, 1, 2]
    table = c.table.clone()
    table[without] = table[0, 0]
    return Cache(c.codes, c.scales, table, c.lens, c.starts, L, n)


@pytest.mark.parametrize("starts", [[0, 3, 2, 6], [-1, 3, 4, 6], [0, 3, 4, 7], [5, 3, 4, 6], [0, 2 ** 31 - 1, 4, 6],
                                    [-2 ** 31, 2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1], [0, 6, 6, 5]])
def test_wrong_row_starts_stay_inside(starts):
    """Nothing past the tensors, no endless walk; the error is reported."""
    import gemm_pt_block_gb300 as mx

    c, kv, q = setup()
    bad = torch.tensor(starts, dtype=torch.int32, device=DEV)
    room = torch.full((c.T + 2, 4, 64), 7.0, device=DEV)
    mx.mxfp8_cache_attention(q, c.codes, c.scales, c.table, c.lens, starts=bad, out=room[1:-1])
    assert mx.device_status() == BAD
    assert bool((room[0] == 7).all()) and bool((room[-1] == 7).all())
    mx.mxfp8_cache_append(kv[:, 0], kv[:, 1], c.codes, c.scales, c.table, c.lens, starts=bad)
    k = torch.full((c.T + 2, 2, 64), 7.0, device=DEV)
    v = k.clone()
    mx.mxfp8_cache_read(c.codes, c.scales, c.table, bad, c.T, k=k[1:-1], v=v[1:-1])
    torch.cuda.synchronize()
    mx.device_status()
    for t in (k, v):
        assert bool((t[0] == 7).all()) and bool((t[-1] == 7).all())


def test_a_length_shorter_than_its_rows():
    """An append skips the sequence; attention gives the rows before its first token nothing to attend."""
    import gemm_pt_block_gb300 as mx

    c, kv, q = setup()
    spared = c.codes.clone(), c.scales.clone()
    want = append(c, kv[:, 0], kv[:, 1])
    c.lens[0] = 2
    pages = c.table[0].long()
    pages = pages[(pages >= 0) & (pages < c.codes.shape[0])]
    want[0][pages], want[1][pages] = spared[0][pages], spared[1][pages]
    mx.mxfp8_cache_append(kv[:, 0], kv[:, 1], c.codes, c.scales, c.table, c.lens, starts=c.starts)
    assert mx.device_status() == BAD
    same(c.codes, want[0])
    same(c.scales, want[1])
    c.L = [2, 70, 40]
    out, lse = mx.mxfp8_cache_attention(q, c.codes, c.scales, c.table, c.lens, starts=c.starts, with_lse=True)
    assert mx.device_status() == 0
    check(c, q, out, lse, BF16)
    assert bool((out[0] == 0).all())


def test_a_cache_without_pages():
    import gemm_pt_block_gb300 as mx

    codes, scales = torch.empty((0, 2, 2, 16, 64), dtype=torch.uint8, device=DEV), torch.empty((0, 2, 2), dtype=torch.uint8, device=DEV)
    table, lens = torch.empty((3, 0), dtype=torch.int32, device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV)
    q = torch.randn((3, 4, 64), device=DEV).to(BF16)
    out, lse = mx.mxfp8_cache_attention(q, codes, scales, table, lens, with_lse=True)
    assert mx.device_status() == 0
    assert bool((out == 0).all()) and bool(torch.isinf(lse).all())
    lens[1] = 4
    out, _ = mx.mxfp8_cache_attention(q, codes, scales, table, lens)
    assert mx.device_status() == BAD
    assert bool(torch.isnan(out[1]).all()) and bool((out[0] == 0).all())


@pytest.mark.parametrize("B,H,G,D,P", [(33, 2, 4, 64, 16), (385, 1, 8, 128, 32), (700, 2, 2, 64, 16), (2500, 1, 1, 96, 16)])
def test_many_sequences(B, H, G, D, P):
    import gemm_pt_block_gb300 as mx

    L = [(i * 37) % 90 if i % 11 else 0 for i in range(B)]
    n = [1 if x else 0 for x in L]
    L[B // 2], n[B // 2] = 900, 3
    c = make_cache(L, n, H, D, P, seed=3)
    q = torch.randn((c.T, H * G, D), device=DEV, generator=gen(4)).to(BF16)
    out, lse = mx.mxfp8_cache_attention(q, c.codes, c.scales, c.table, c.lens, starts=c.starts, with_lse=True)
    assert mx.device_status() == 0
    check(c, q, out, lse, BF16)


def test_the_largest_sequence_count():
    import gemm_pt_block_gb300 as mx

    B = 65535
    codes = torch.full((2, 2, 1, 16, 64), 0x30, dtype=torch.uint8, device=DEV)
    scales = torch.full((2, 2, 1), 127, dtype=torch.uint8, device=DEV)
    table = torch.arange(B, device=DEV).remainder(2).int()[:, None].contiguous()
    lens = torch.arange(B, device=DEV).remainder(17).int()
    q = torch.randn((B, 1, 64), device=DEV).to(BF16)
    out, lse = mx.mxfp8_cache_attention(q, codes, scales, table, lens, with_lse=True, out_dtype=F32)
    assert mx.device_status() == 0
    some = lens > 0
    assert bool((out[some] - 0.5).abs().max() < 1e-5) and bool((out[~some] == 0).all())
    s = (q.float().sum(-1)[:, 0] * 0.5 * 0.125 + torch.log(lens.float()))[some]
    assert bool(((lse[some, 0] - s).abs() <= 1e-4 * (1 + s.abs())).all())


def test_buffers_are_checked():
    import gemm_pt_block_gb300 as mx

    c, kv, q = setup()
    args = (c.codes, c.scales, c.table, c.lens)
    k, v = kv[:, 0], kv[:, 1]

    def refused(error, match, f, *a, **kw):
        with pytest.raises(error, match=match):
            f(*a, **kw)

    A, R, F = mx.mxfp8_cache_append, mx.mxfp8_cache_read, mx.mxfp8_cache_attention
    refused(ValueError, "codes must be \\[pages", A, k, v, c.codes[:, :1], c.scales, c.table, c.lens, starts=c.starts)
    refused(ValueError, "contiguous", A, k, v, c.codes[:, :, :, ::2], c.scales, c.table, c.lens, starts=c.starts)
    refused(TypeError, "codes must be", A, k, v, c.codes.float(), c.scales, c.table, c.lens, starts=c.starts)
    refused(ValueError, "scales must be \\[", A, k, v, c.codes, c.scales[:-1], c.table, c.lens, starts=c.starts)
    refused(TypeError, "page_table must be int32", A, k, v, c.codes, c.scales, c.table.long(), c.lens, starts=c.starts)
    refused(ValueError, "lens must be a contiguous vector", A, k, v, c.codes, c.scales, c.table, c.lens[:2], starts=c.starts)
    refused(ValueError, "starts must be a contiguous vector", A, k, v, *args, starts=c.starts[:3])
    refused(TypeError, "v must have k's type", A, k, v.float(), *args, starts=c.starts)
    refused(ValueError, "v must be \\[", A, k, v[:-1], *args, starts=c.starts)
    refused(ValueError, "k must be \\[", A, k[:, :1], v, *args, starts=c.starts)
    refused(TypeError, "k must be bfloat16 or float32", A, k.half(), v.half(), *args, starts=c.starts)
    refused(mx.Mxfp4Error, "without starts", A, k, v, *args)
    refused(ValueError, "unit stride", A, k.transpose(1, 2).contiguous().transpose(1, 2), v, *args, starts=c.starts)
    refused(ValueError, "rows -1", R, *args[:3], c.starts, -1)
    refused(ValueError, "k must be \\[", R, *args[:3], c.starts, 6, k=torch.empty((5, 2, 64), device=DEV))
    refused(TypeError, "must be a torch dtype", R, *args[:3], c.starts, 6, out_dtype="bf16")
    refused(TypeError, "q must be bfloat16", F, q.float(), *args, starts=c.starts)
    refused(mx.Mxfp4Error, "multiple of heads", F, q[:, :3], *args, starts=c.starts)
    refused(ValueError, "lse holds", F, q, *args, starts=c.starts, lse=torch.empty(5, device=DEV))
    refused(ValueError, "out must be \\[", F, q, *args, starts=c.starts, out=q[:-1])
    refused(TypeError, "slopes must be float32", F, q, *args, starts=c.starts, slopes=torch.ones(4, device=DEV, dtype=BF16))
    refused(ValueError, "slopes must be a contiguous vector", F, q, *args, starts=c.starts, slopes=torch.ones(3, device=DEV))
    refused(ValueError, "workspace holds", F, q, *args, starts=c.starts, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    refused(ValueError, "window -1", F, q, *args, starts=c.starts, window=-1)
    refused(mx.Mxfp4Error, "softcap", F, q, *args, starts=c.starts, softcap=-2.0)
    refused(ValueError, "on device", F, q, *args, starts=c.starts.cpu())
    with pytest.raises(ValueError):
        mx.KvCache(4, 1, 80)
    with pytest.raises(ValueError):
        mx.KvCache(4, 1, 64, 24)
    out, _ = F(q, *args, starts=c.starts)
    assert out.shape == q.shape


def calls():
    import gemm_pt_block_gb300 as mx

    out = {}
    for L, n, H, G, D, P in (([300, 7], [1, 1], 2, 4, 128, 64), ([4000, 31], [1, 3], 1, 5, 64, 16), ([700], [20], 3, 2, 96, 32),
                             ([1500], [2], 1, 9, 256, 128), ([333], [1], 2, 1, 192, 16)):
        c = make_cache(L, n, H, D, P, seed=5, table_cols=1)
        c.table[:, -1] = -1
        q = torch.randn((c.T, H * G, D), device=DEV, generator=gen(6)).to(BF16)
        for dt in (BF16, F32):
            out[f"attention {L} {D} {dt}"] = lambda c=c, q=q, dt=dt: mx.mxfp8_cache_attention(
                q, c.codes, c.scales, c.table, c.lens, starts=c.starts, out_dtype=dt, with_lse=True)
            rows = torch.tensor([0] + list(torch.tensor(L).cumsum(0)), dtype=torch.int32, device=DEV)
            out[f"read {L} {D} {dt}"] = lambda c=c, rows=rows, L=L, dt=dt: mx.mxfp8_cache_read(
                c.codes, c.scales, c.table, rows, sum(L), out_dtype=dt)
            for few in (False, True):
                m = [1 if few else min(x, 90) for x in L]
                L2 = [-(-x // P) * P for x in L]                        # (pages full to their last token)
                kv = torch.randn((sum(m), 2, H, D), device=DEV, generator=gen(7)).to(dt)
                at = torch.tensor([0] + list(torch.tensor(m).cumsum(0)), dtype=torch.int32, device=DEV)
                lens = torch.tensor(L2, dtype=torch.int32, device=DEV)

                def write(c=c, kv=kv, at=at, lens=lens, table=c.table):
                    codes, scales = c.codes[:int(table.max()) + 1].clone(), c.scales[:int(table.max()) + 1].clone()
                    mx.mxfp8_cache_append(kv[:, 0], kv[:, 1], codes, scales, table, lens, starts=at)
                    return codes, scales
                out[f"append {L} {D} {dt} {few}"] = write
    return out


def test_no_store_outside_and_the_same_bits(bc_lib):  # noqa: F811
    for name, fn in calls().items():
        want, got, status = _both(bc_lib, fn)
        assert status == 0, name
        assert _equal([torch.nan_to_num(x.float()) for x in want], [torch.nan_to_num(x.float()) for x in got]), name


def test_the_check_fires(bc_lib):  # noqa: F811
    import gemm_pt_block_gb300 as mx

    fired = set()
    for name, fn in calls().items():
        with _using(bc_lib):
            try:
                assert bc_lib.mxfp4_bounds_check_shrink(1) == 0
                fn()
                status = mx.device_status()
            finally:
                assert bc_lib.mxfp4_bounds_check_shrink(0) == 0
            assert status in (0, 7), name
            if status == 7:
                fired.add(name.split()[0])
            else:
                assert name.startswith("append"), name     # (the last page of the cache is not always the one written)
            fn()
            assert mx.device_status() == 0, name
    assert fired == {"attention", "read", "append"}


@pytest.mark.parametrize("L,n,H,G,D,P,window", [([200, 77, 33], [1, 1, 1], 2, 2, 64, 16, 5), ([300, 95], [4, 9], 1, 4, 128, 16, 20),
                                                ([300, 130], [3, 40], 2, 1, 64, 32, 40), ([500, 200], [1, 7], 1, 8, 96, 64, 64),
                                                ([700], [1], 1, 16, 256, 128, 200)])
def test_pages_before_the_window_may_be_gone(L, n, H, G, D, P, window):
    import gemm_pt_block_gb300 as mx

    c = make_cache(L, n, H, D, P, seed=40)
    q = torch.randn((c.T, H * G, D), device=DEV, generator=gen(41)).to(BF16)
    gone = make_cache(L, n, H, D, P, seed=40)
    for b in range(len(L)):
        first = max(0, L[b] - n[b] - window + 1)            # that a query attends
        gone.table[b, :first // P] = torch.tensor([-1, 1 << 30], device=DEV).int().repeat(first // P)[:first // P]
    for dtype in (BF16, F32):
        out, lse = mx.mxfp8_cache_attention(q, c.codes, c.scales, gone.table, c.lens, starts=c.starts, with_lse=True,
                                            out_dtype=dtype, window=window)
        assert mx.device_status() == 0
        check(c, q, out, lse, dtype, window=window)


def test_a_missing_page_beside_rows_that_do_not_attend_it():
    import gemm_pt_block_gb300 as mx

    # (what lies in shared memory in its place: NaN codes behind other sequences' ends)
    c = make_cache([49], [1], 1, 64, 16, seed=42)
    B = 152 * 14 * 3
    q = torch.randn((B, 1, 64), device=DEV, generator=gen(43)).to(BF16)
    mx.mxfp8_cache_attention(q, c.codes, c.scales, c.table.expand(B, -1).contiguous(), c.lens.expand(B).contiguous())
    c = make_cache([51], [5], 1, 64, 16, seed=44)
    c.table[0, 3] = -1
    out, lse = mx.mxfp8_cache_attention(q[:5], c.codes, c.scales, c.table, c.lens, starts=c.starts, with_lse=True)
    assert mx.device_status() == BAD
    assert bool(torch.isnan(out[2:]).all()) and bool(torch.isnan(lse[2:]).all())
    c.table[0, 3] = c.table[0, 0]
    c.L, c.n = [48], [2]
    check(c, q[:2], out[:2], lse[:2], BF16)


@pytest.mark.parametrize("B,rows", [(4, 1600), (34, 600)])
def test_falling_starts_of_more_work_than_is_counted(B, rows):
    """Rows named again and again, each time with as many tokens as a call may have: nothing is done."""
    import gemm_pt_block_gb300 as mx

    codes = torch.zeros((1, 2, 1, 128, 64), dtype=torch.uint8, device=DEV)
    scales = torch.zeros((1, 2, 1), dtype=torch.uint8, device=DEV)
    table = torch.zeros((B, (1 << 22) - 1 if B == 4 else 1 << 21), dtype=torch.int32, device=DEV)
    lens = torch.full((B,), table.shape[1] * 128, dtype=torch.int32, device=DEV)
    starts = (torch.arange(B + 1, device=DEV) % 2 * rows).int()
    q = torch.zeros((rows, 1, 64), dtype=BF16, device=DEV)
    out = torch.full((rows, 1, 64), 7.0, device=DEV)
    mx.mxfp8_cache_attention(q, codes, scales, table, lens, starts=starts, out=out)
    assert mx.device_status() == BAD
    assert bool((out == 7).all())


@pytest.mark.parametrize("B,H,G,n,D,L,window", [(19, 8, 4, 1, 128, 700, 0), (20, 8, 4, 1, 128, 700, 0), (19, 8, 1, 1, 64, 1500, 0),
                                                (32, 1, 20, 2, 96, 900, 0), (16, 3, 9, 2, 64, 650, 300), (3, 2, 8, 1, 256, 30, 0)])
def test_as_many_tiles_as_processors(B, H, G, n, D, L, window):
    """A tile to a processor, one more, sequences without rows or tokens among them."""
    import gemm_pt_block_gb300 as mx

    Ls, ns = [L - 3 * (i % 5) for i in range(B)], [n] * B
    Ls[2], ns[1] = 0, 0
    c = make_cache(Ls, ns, H, D, 32, seed=50)
    q = torch.randn((c.T, H * G, D), device=DEV, generator=gen(51)).to(BF16)
    out, lse = mx.mxfp8_cache_attention(q, c.codes, c.scales, c.table, c.lens, starts=c.starts, with_lse=True, window=window)
    assert mx.device_status() == 0
    check(c, q, out, lse, BF16, window=window)


@pytest.mark.parametrize("B,H,D,P,few,many", [(130, 2, 128, 64, 13, 300), (130, 2, 64, 128, 24, 500), (9, 4, 256, 64, 3, 6),
                                              (260, 1, 96, 32, 20, 90), (128, 2, 256, 64, 7, 60), (5, 8, 128, 64, 8, 9)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_appends_of_a_few_tokens(B, H, D, P, few, many, dtype):
    """A few tokens a sequence, more than a warp holds in one of them, none in others."""
    import gemm_pt_block_gb300 as mx

    n = [few - i % 3 for i in range(B)]
    n[B // 2], n[1] = many, 0
    L = [n[i] + 11 * i % 150 for i in range(B)]
    c = make_cache(L, n, H, D, P, seed=60, filled=[a - b for a, b in zip(L, n)])
    kv = torch.randn((c.T, 2, H, D), device=DEV, generator=gen(61))
    kv[:, :, 0] *= torch.exp2(torch.randint(-4, 9, (c.T, 2, 1), device=DEV, generator=gen(62)).float())
    kv = kv.to(dtype)
    want = append(c, kv[:, 0], kv[:, 1])
    mx.mxfp8_cache_append(kv[:, 0], kv[:, 1], c.codes, c.scales, c.table, c.lens, starts=c.starts)
    same(c.codes, want[0])
    same(c.scales, want[1])
    assert mx.device_status() == 0
