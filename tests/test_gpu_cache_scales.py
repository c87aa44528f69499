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
