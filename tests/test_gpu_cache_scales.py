"""Appends onto pages whose older tokens lie under scales that an append itself
never needs: every scale but 0xFF is a value's scale."""
from __future__ import annotations

import pytest
import torch

from _cache import DEV, append, gen, make_cache
from test_gpu_cache import same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [0, 1, 126, 246, 247, 248, 253, 254])
@pytest.mark.parametrize("P,D,older,new", [(16, 64, 3, 1), (64, 128, 10, 5), (64, 64, 10, 54), (128, 256, 1, 120)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_onto_every_scale(scale, P, D, older, new, dtype):
    import gemm_pt_block_gb300 as mx

    c = make_cache([older + new], [new], 2, D, P, seed=1, filled=[older])
    c.scales[c.table[0, 0].long(), :, 0] = scale
    kv = torch.randn((new, 2, 2, D), device=DEV, generator=gen(2)).clamp(-1, 1)
    # (of the largest finite values' size, where scale 254 gives codes up to 2; and down from there)
    kv = kv * torch.exp2(torch.randint(0, 6, (new, 1, 1, D), device=DEV, generator=gen(3)).float() - 5) * 3.3e38
    kv[0, ..., 0] = 3.3e38
    kv = kv.to(dtype)
    want = append(c, kv[:, 0], kv[:, 1])
    one = [dict(starts=c.starts)] + ([{}] if new == 1 else [])
    for kw in one:
        codes, scales = c.codes.clone(), c.scales.clone()
        mx.mxfp8_cache_append(kv[:, 0], kv[:, 1], codes, scales, c.table, c.lens, **kw)
        same(scales, want[1])
        same(codes, want[0])
    if scale == 254:
        assert int((codes[c.table[0, 0].long(), :, 0, older:older + new] & 0x7F).max()) == 0x40   # (2: the values were not lost)
    assert mx.device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("new,P", [(1, 64), (3, 16), (90, 64)])
def test_scales_at_the_border(dtype, new, P):
    """The largest magnitude is 448 * 2^e, or the next value on either side: the smallest scale that does not
    clip. (By whole-number arithmetic; a quotient's logarithm in 64 bits may fall on the wrong side.)"""
    import gemm_pt_block_gb300 as mx

    H, D = 7, 64
    c = make_cache([new], [new], H, D, P, filled=[0])
    step = torch.finfo(dtype).eps                           # of values in [1, 2)
    for e in (-90, -15, -6, -1, 0, 1, 8, 100):
        kv = torch.randn((new, 2, H, D), device=DEV, generator=gen(4)).clamp(-1, 1)
        want = torch.zeros((2, H), dtype=torch.int64, device=DEV)
        for h, (top, up) in enumerate([(1.75, 0), (1.75 - step, 0), (1.75 + step, 1), (1.0, 0), (2 - step, 1), (1.75 + 2 * step, 1), (1.5, 0)]):
            kv[:, :, h] *= top
            kv[new // 2, 0, h, 5], kv[new // 2, 1, h, 50] = -top, top
            want[:, h] = e + up + 127                       # top * 2^(8 + e) <= 448 * 2^(e + up)
        kv = (kv * 2.0 ** (8 + e)).to(dtype)
        codes, scales = c.codes.clone(), c.scales.clone()
        mx.mxfp8_cache_append(kv[:, 0], kv[:, 1], codes, scales, c.table, c.lens, starts=c.starts)
        page = c.table[0, (new // 2) // P].long()
        assert torch.equal(scales[page].long(), want), e
        assert not bool(((codes[page] & 0x7F) == 0x7F)[:, :, :min(P, new)].any())
        at = codes[page, :, :, new // 2 % P]
        assert torch.equal(at[0, 0, 5], torch.tensor(0xFE, dtype=torch.uint8, device=DEV)) and int(at[1, 0, 50]) == 0x7E   # 448
    assert mx.device_status() == 0
