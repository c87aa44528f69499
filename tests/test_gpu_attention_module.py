"""The attention block as a user's program handles it: cast to another type, moved, captured."""
from __future__ import annotations

import copy

import pytest
import torch

from _cache import DEV, gen

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def a_token(block, cache, x, lens):
    table = torch.tensor([[3, 1], [0, 2]], dtype=torch.int32, device=DEV)
    return block.decode(x, cache, table, lens)


@pytest.mark.parametrize("cast", [lambda m: m.to(BF16), lambda m: m.half().to(BF16), lambda m: m.cpu().to(BF16).to(DEV)])
def test_decoding_with_slopes_after_a_cast(cast):
    import gemm_pt_block_gb300 as mx

    torch.manual_seed(0)
    slopes = torch.tensor([1 / 3, 0.7, 1e-2, 0.1])
    block = mx.Mxfp4Attention(256, 4, 2, 64, slopes=slopes, device=DEV)
    with torch.no_grad():
        for p in block.parameters():
            p.copy_(p.half().to(BF16))                      # (so that a cast to fp16 and back changes nothing)
    block.quantize_weights()
    other = cast(copy.deepcopy(block))
    caches = [b.cache(4, 16) for b in (block, other)]
    lens = torch.tensor([1, 1], dtype=torch.int32, device=DEV)
    for i in range(20):
        x = torch.randn((2, 256), device=DEV, generator=gen(i)).to(BF16)
        want, got = a_token(block, caches[0], x, lens), a_token(other, caches[1], x, lens)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        lens += 1
    assert mx.device_status() == 0


@pytest.mark.parametrize("options", [{}, dict(window=24, softcap=20.0, slopes=True)], ids=str)
@pytest.mark.parametrize("sequences", [1, 5, 40])
def test_a_captured_step_of_the_block(options, sequences):
    """decode captured once and replayed, with tokens, lengths and pages that change in place, beside eager steps."""
    import gemm_pt_block_gb300 as mx

    torch.manual_seed(1)
    options = dict(options)
    if "slopes" in options:
        options["slopes"] = torch.exp2(-torch.arange(1, 5).float())
    block = mx.Mxfp4Attention(256, 4, 2, 64, device=DEV, **options)
    block.quantize_weights()
    captured, eager = block.cache(sequences * 6, 16), block.cache(sequences * 6, 16)
    pages = torch.randperm(sequences * 6, device=DEV, generator=gen(2)).int().view(sequences, 6)
    table = torch.full((sequences, 6), -1, dtype=torch.int32, device=DEV)
    lens = torch.ones(sequences, dtype=torch.int32, device=DEV)
    table[:, 0] = pages[:, 0]
    x, stream = (torch.randn((sequences, 256), device=DEV, generator=gen(i)).to(BF16) for i in (3, 4))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block.decode(x, captured, table, lens, stream)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = block.decode(x, captured, table, lens, stream)
    for i in range(60):
        graph.replay()
        want = block.decode(x, eager, table, lens, stream)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), i
        lens += 1
        at = ((lens - 1) // 16).long()[:, None]
        table.scatter_(1, at, pages.gather(1, at))
        x.normal_(generator=gen(100 + i))
        stream.copy_(want[1])
    assert torch.equal(captured.codes, eager.codes) and torch.equal(captured.scales, eager.scales)
    assert mx.device_status() == 0
