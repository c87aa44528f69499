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
