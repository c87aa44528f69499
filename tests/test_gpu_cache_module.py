"""The attention block for decoding, and the cache's calls together as a server
makes them: prompts, then steps, sequences that end and pages that are used
again, captured steps, several streams and threads."""
from __future__ import annotations

import threading

import pytest
import torch

from _cache import DEV, Cache, append, attend, attention_bounds, gen

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


class Pages:
    """Hands out pages and takes them back; the table and lengths of the sequences that run."""

    def __init__(self, pages, page_tokens, sequences, columns):
        self.free, self.P = list(range(pages))[::-1], page_tokens
        self.table = torch.full((sequences, columns), -1, dtype=torch.int32)
        self.lens = [0] * sequences

    def grow(self, b, n):
        for i in range(-(-self.lens[b] // self.P), -(-(self.lens[b] + n) // self.P)):
            self.table[b, i] = self.free.pop()
        self.lens[b] += n

    def end(self, b):
        for i in range(-(-self.lens[b] // self.P)):
            self.free.append(int(self.table[b, i]))
            self.table[b, i] = -1
        self.lens[b] = 0

    def step(self, new):
        for b, n in enumerate(new):
            self.grow(b, n)
        starts = torch.tensor([0] + list(torch.tensor(new).cumsum(0)), dtype=torch.int32)
        return self.table.to(DEV), torch.tensor(self.lens, dtype=torch.int32, device=DEV), starts.to(DEV)


def view(cache, table, lens, starts, L, n):
    return Cache(cache.codes, cache.scales, table, lens, starts, list(L), list(n))


@pytest.mark.parametrize("H,G,D,P", [(2, 4, 128, 32), (1, 3, 64, 16)])
def test_a_run_of_steps(H, G, D, P):
    """Each step's cache bit for bit and its attention within its bounds, from the state that the definition has."""
    import gemm_pt_block_gb300 as mx

    cache = mx.KvCache(60, H, D, P, DEV)
    cache.codes.fill_(0x7F)
    cache.scales.fill_(255)
    pages = Pages(60, P, 3, 12)
    g = gen(40)
    want = cache.codes.clone(), cache.scales.clone()
    for step, new in enumerate([[37, 1, 0], [1, 1, 5], [1, 1, 1], [4, 2, 1], [1, 60, 1], "end", [1, 3, 70], [1, 1, 1]]):
        if new == "end":
            pages.end(0)
            pages.end(1)
            continue
        table, lens, starts = pages.step(new)
        kv = torch.randn((sum(new), 2, H, D), device=DEV, generator=g) * 2.0 ** (step % 4)
        q = torch.randn((sum(new), G * H, D), device=DEV, generator=g).to(BF16)
        c = Cache(*want, table, lens, starts, list(pages.lens), new)
        want = append(c, kv[:, 0], kv[:, 1])
        cache.append(kv[:, 0], kv[:, 1], table, lens, starts)
        out, lse = cache.attend(q, table, lens, starts, with_lse=True)
        assert torch.equal(cache.codes, want[0]) and torch.equal(cache.scales, want[1]), step
        c = view(cache, table, lens, starts, pages.lens, new)
        ref, ref_lse, weight, reach = attend(c, q)
        lim, lse_lim = attention_bounds(BF16, max(pages.lens), ref, weight, reach)
        assert bool(((out.double() - ref).abs() <= lim).all()), step
        assert bool(((lse.double() - ref_lse).abs() <= lse_lim + 2.0 ** -23 * ref_lse.abs()).all()), step
        rows = torch.tensor([0] + list(torch.tensor(pages.lens).cumsum(0)), dtype=torch.int32, device=DEV)
        k, v = cache.read(table, rows, sum(pages.lens), out_dtype=torch.float32)
        both = torch.cat([c.tokens(b, n) for b, n in enumerate(pages.lens)], 2).transpose(1, 2)
        assert torch.equal(k.double(), both[0]) and torch.equal(v.double(), both[1]), step
    assert mx.device_status() == 0


def rotate_by(angle):
    def rotate(q, k):
        c, s = torch.cos(angle), torch.sin(angle)
        return tuple(torch.cat((x[..., ::2].float() * c - x[..., 1::2].float() * s,
                                x[..., ::2].float() * s + x[..., 1::2].float() * c), -1).to(x.dtype) for x in (q, k))
    return rotate


@pytest.mark.parametrize("rotate", [False, True])
@pytest.mark.parametrize("options", [{}, dict(window=20, softcap=30.0), dict(slopes=True)], ids=str)
def test_the_block_is_its_parts(rotate, options):
    import gemm_pt_block_gb300 as mx

    torch.manual_seed(0)
    options = dict(options)
    if "slopes" in options:
        options["slopes"] = torch.exp2(-torch.arange(1, 5).float())
    block = mx.Mxfp4Attention(256, 4, 2, 64, device=DEV, **options)
    with pytest.raises(RuntimeError, match="quantize_weights"):
        block.decode(torch.zeros(1, 256, device=DEV, dtype=BF16), block.cache(1), None, None)
    block.quantize_weights()
    cache, other = block.cache(20, 16), block.cache(20, 16)
    pages = Pages(20, 16, 2, 8)
    p8 = mx.QuantParams(scale_mode=mx.SCALE_ROUNDUP, elem_format=mx.FORMAT_E4M3)
    (wq, ws), (oq, os_) = (block.qkv_codes, block.qkv_scales), (block.out_codes, block.out_scales)
    p = block.qkv.recipe.w_row
    for new in ([30, 3], [1, 1], [2, 5]):
        table, lens, starts = pages.step(new)
        T = sum(new)
        x, r = (torch.randn((T, 256), device=DEV, generator=gen(T + i)).to(BF16) for i in range(2))
        turn = rotate_by(torch.rand((T, 1, 32), device=DEV, generator=gen(T + 2))) if rotate else None
        y, h = block.decode(x, cache, table, lens, r, starts, rotate=turn)
        n, s, _, hh, _ = mx.mxfp4_rmsnorm_quantize(x, block.norm, p8, residual=r, eps=block.eps)
        qkv = mx.mxfp4_gemv(n, wq, ws, 512, 256, p, sx=s).view(T, 8, 64)
        q, k, v = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
        if rotate:
            q, k = turn(q, k)
        mx.mxfp8_cache_append(k, v, other.codes, other.scales, table, lens, starts=starts)
        o, _ = mx.mxfp8_cache_attention(q, other.codes, other.scales, table, lens, starts=starts, **{
            **options, **({"slopes": block.slopes} if "slopes" in options else {})})
        want = mx.mxfp4_gemv(o.view(T, 256), oq, os_, 256, 256, block.out.recipe.w_row)
        assert torch.equal(h, hh) and torch.equal(y, want)
        assert torch.equal(cache.codes, other.codes) and torch.equal(cache.scales, other.scales)
        # and the parts are what they should be, from the weights' values
        c = view(cache, table, lens, starts, pages.lens, new)
        ref, _, weight, reach = attend(c, q, **({**options, "slopes": block.slopes} if "slopes" in options else options))
        lim, _ = attention_bounds(BF16, max(pages.lens), ref, weight, reach)
        assert bool(((o.double() - ref).abs() <= lim).all())
        w = mx.mxfp4_dequantize(oq, os_, 256, 256, params=block.out.recipe.w_row).double()
        ref = o.reshape(T, 256).double() @ w.t()
        room = 1e-4 * (o.reshape(T, 256).double().abs() @ w.abs().t())
        assert bool(((y.double() - ref).abs() <= room + 2.0 ** -8 * (ref.abs() + room)).all())
    assert mx.device_status() == 0


def test_a_layer_of_two_blocks():
    """Attention and feed-forward blocks in turn, a token at a time, as a model's layer decodes."""
    import gemm_pt_block_gb300 as mx

    torch.manual_seed(1)
    attention, ff = mx.Mxfp4Attention(256, 2, 1, 128, device=DEV), mx.Mxfp4FeedForward(256, 512, device=DEV)
    attention.quantize_weights()
    ff.quantize_weights()
    cache, pages = attention.cache(8, 16), Pages(8, 16, 2, 4)
    stream = torch.zeros((2, 256), device=DEV, dtype=BF16)
    y = torch.randn((2, 256), device=DEV, generator=gen(50)).to(BF16)
    for _ in range(20):
        table, lens, _ = pages.step([1, 1])
        y, stream = attention.decode(y, cache, table, lens, stream)
        y, stream = ff.decode(y, stream)
    assert bool(torch.isfinite(stream.float()).all()) and stream.shape == (2, 256)
    assert mx.device_status() == 0


def test_a_captured_step_replays():
    """A step captured once, replayed with new lengths, pages, keys and queries in place; two
    captured steps share nothing; an eager one between them."""
    import gemm_pt_block_gb300 as mx

    H, D, P, B = 2, 128, 64, 5
    cache, eager = mx.KvCache(400, H, D, P, DEV), mx.KvCache(400, H, D, P, DEV)
    for c in (cache, eager):
        x = torch.randint(0, 120, c.codes.shape, device=DEV, generator=gen(60), dtype=torch.uint8)
        c.codes.copy_(x)
        c.scales.fill_(120)
    table = torch.randperm(400, device=DEV, generator=gen(61)).int()[:B * 60].view(B, 60).contiguous()
    lens = torch.tensor([1, 3000, 64, 65, 700], dtype=torch.int32, device=DEV)
    kv = torch.randn((B, 2, H, D), device=DEV, generator=gen(62)).to(BF16)
    q = torch.randn((B, 8, D), device=DEV, generator=gen(63)).to(BF16)

    def step(c):
        c.append(kv[:, 0], kv[:, 1], table, lens)
        return c.attend(q, table, lens, with_lse=True)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(cache)
    torch.cuda.current_stream().wait_stream(side)
    cache.codes.copy_(eager.codes)
    cache.scales.copy_(eager.scales)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(cache)
        graphs.append((g, out))
    for i in range(6):
        graphs[i % 2][0].replay()
        got = graphs[i % 2][1]
        want = step(eager)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(cache.codes, eager.codes) and torch.equal(cache.scales, eager.scales)
        lens += torch.tensor([1, 1, 50, 7, 300], dtype=torch.int32, device=DEV)
        kv.normal_(generator=gen(64 + i))
        q.normal_(generator=gen(70 + i))
    assert mx.device_status() == 0


def test_the_same_bits_on_every_call_and_stream():
    import gemm_pt_block_gb300 as mx
    from _cache import make_cache

    c = make_cache([5000, 17, 900, 1, 333], [1] * 5, 2, 128, 64, seed=80)
    q = torch.randn((5, 16, 128), device=DEV, generator=gen(81)).to(BF16)
    want, want_lse = mx.mxfp8_cache_attention(q, c.codes, c.scales, c.table, c.lens, with_lse=True)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [mx.mxfp8_cache_attention(q, c.codes, c.scales, c.table, c.lens, with_lse=True, stream=s)
           for _ in range(5) for s in streams]
    torch.cuda.synchronize()
    for out, lse in got:
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    need = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    need.random_(generator=gen(82))                         # (a workspace's contents are nobody's)
    out, lse = mx.mxfp8_cache_attention(q, c.codes, c.scales, c.table, c.lens, with_lse=True, workspace=need)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_several_threads():
    import gemm_pt_block_gb300 as mx
    from _cache import make_cache

    caches = [make_cache([400 + 100 * i, 30], [1, 1], 1 + i % 2, (64, 128)[i % 2], 32, seed=90 + i) for i in range(4)]
    qs = [torch.randn((2, 4, c.codes.shape[4]), device=DEV, generator=gen(95)).to(BF16) for c in caches]
    want = [mx.mxfp8_cache_attention(q, c.codes, c.scales, c.table, c.lens)[0] for c, q in zip(caches, qs)]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                out, _ = mx.mxfp8_cache_attention(qs[i], caches[i].codes, caches[i].scales, caches[i].table, caches[i].lens)
                k, _ = mx.mxfp8_cache_read(caches[i].codes, caches[i].scales, caches[i].table, caches[i].starts, 2)
                torch.cuda.current_stream().synchronize()
                if not torch.equal(out, want[i]) or not bool(torch.isfinite(k.float()).all()):
                    bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
    assert mx.device_status() == 0


def test_a_step_captured_from_two_streams():
    """Keys and queries made on streams of their own: the attention follows two kernels, or a copy."""
    import gemm_pt_block_gb300 as mx

    H, D, P, B = 2, 64, 32, 40
    cache, eager = mx.KvCache(B * 20, H, D, P, DEV), mx.KvCache(B * 20, H, D, P, DEV)
    table = torch.randperm(B * 20, device=DEV, generator=gen(110)).int().view(B, 20).contiguous()
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    kv, q = torch.zeros((B, 2, H, D), device=DEV, dtype=BF16), torch.zeros((B, 4, D), device=DEV, dtype=BF16)
    given = torch.zeros_like(q)

    def step(c, side, copies):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            c.append(kv[:, 0], kv[:, 1], table, lens)
        if copies:
            q.copy_(given)
        else:
            torch.mul(given, 1.0, out=q)
        main.wait_stream(side)
        return c.attend(q, table, lens, with_lse=True)

    graphs = []
    warm, side = torch.cuda.Stream(), torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        step(cache, side, False)
    assert mx.device_status() == 1                          # (lengths of no token yet: nothing was appended)
    for copies in (False, True):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(cache, side, copies)
        graphs.append((g, out))
    for i in range(300):
        lens += 1 + torch.arange(B, device=DEV).int() % 2
        kv.normal_(generator=gen(111 + i))
        given.normal_(generator=gen(500 + i))
        graphs[i % 2][0].replay()
        got, lse = graphs[i % 2][1]
        eager.append(kv[:, 0], kv[:, 1], table, lens)
        want, want_lse = eager.attend(given, table, lens, with_lse=True)
        if i % 7 == 0:
            torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(lse, want_lse), i
    assert torch.equal(cache.codes, eager.codes) and torch.equal(cache.scales, eager.scales)
    assert mx.device_status() == 0


def test_pages_behind_the_window_are_used_again():
    """Steps of a model with a window: pages that no query reaches any more go to other sequences."""
    import gemm_pt_block_gb300 as mx

    H, G, D, P, window, B = 2, 2, 64, 16, 40, 3
    pages, whole = Pages(B * 5, P, B, 30), Pages(200, P, B, 30)
    cache, full = mx.KvCache(B * 5, H, D, P, DEV), mx.KvCache(200, H, D, P, DEV)
    g = gen(120)
    new = [30, 17, 1]
    for i in range(90):
        table, lens, starts = pages.step(new)
        table2, lens2, _ = whole.step(new)
        x = torch.randn((sum(new), 2, H, D), device=DEV, generator=g).to(BF16)
        q = torch.randn((sum(new), H * G, D), device=DEV, generator=g).to(BF16)
        cache.append(x[:, 0], x[:, 1], table, lens, starts)
        full.append(x[:, 0], x[:, 1], table2, lens2, starts)
        out, lse = cache.attend(q, table, lens, starts, with_lse=True, window=window)
        want, want_lse = full.attend(q, table2, lens2, starts, with_lse=True, window=window)
        assert torch.equal(out, want) and torch.equal(lse, want_lse), i
        for b in range(B):
            for j in range(max(0, pages.lens[b] - window + 1) // P):
                if int(pages.table[b, j]) >= 0:
                    pages.free.append(int(pages.table[b, j]))
                    pages.table[b, j] = -1
        new = [1 + (i + b) % 3 for b in range(B)]
        if max(pages.lens) + 3 > 30 * P:
            break
    assert mx.device_status() == 0
