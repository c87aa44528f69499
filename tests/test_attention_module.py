"""The attention block's arguments and buffers (no GPU needed)."""
from __future__ import annotations

import copy

import pytest
import torch


def block(slopes, **kw):
    import gemm_pt_block_gb300 as mx

    return mx.Mxfp4Attention(256, 4, 2, 64, slopes=slopes, **kw)


SLOPES = torch.tensor([1 / 3, -0.7, 1e-3, 2.0 ** 20 + 1])     # (three of them do not fit bf16)


@pytest.mark.parametrize("cast", [lambda m: m.to(torch.bfloat16), lambda m: m.bfloat16(), lambda m: m.half(), lambda m: m.double(),
                                  lambda m: m.to(torch.bfloat16).float(), lambda m: torch.nn.Sequential(m).bfloat16()[0],
                                  lambda m: copy.deepcopy(m).half()])
def test_slopes_keep_their_type_and_values(cast):
    m = cast(block(SLOPES))
    assert m.slopes.dtype == torch.float32 and torch.equal(m.slopes, SLOPES)
    assert "slopes" in dict(m.named_buffers())


def test_the_rest_of_the_block_is_cast():
    m = block(SLOPES).half()
    assert m.norm.dtype == m.qkv.weight.dtype == m.out.weight.dtype == torch.float16
    assert block(None).half().slopes is None


def test_slopes_follow_the_block_to_a_device():
    m = block(SLOPES).to("meta", torch.bfloat16)
    assert m.slopes.device.type == "meta" and m.slopes.dtype == torch.float32
    m = m.to_empty(device="cpu")
    assert m.slopes.device.type == "cpu" and m.slopes.dtype == torch.float32
    m.load_state_dict(block(SLOPES).state_dict())
    assert torch.equal(m.slopes, SLOPES)


@pytest.mark.parametrize("kw", [dict(dim=256, heads=4, kv_heads=2, head_dim=32), dict(dim=1280, heads=16, head_dim=80),
                                dict(dim=512, heads=4, kv_heads=2, head_dim=512), dict(dim=1024, heads=64), dict(dim=512, heads=1)],
                         ids=str)
def test_head_sizes_that_no_cache_has_are_refused(kw):
    import gemm_pt_block_gb300 as mx

    with pytest.raises(ValueError, match="head_dim must be 64, 96, 128, 192 or 256"):
        mx.Mxfp4Attention(**kw)


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
def test_head_sizes_of_a_cache_are_taken(dim):
    import gemm_pt_block_gb300 as mx

    m = mx.Mxfp4Attention(256, 4, 2, dim)
    assert m.cache(3, 16).codes.shape == (3, 2, 2, 16, dim)


@pytest.mark.parametrize("heads,kv_heads", [(0, None), (-2, 1), (4, 0), (4, -4), (4, 3)])
def test_head_counts_are_checked(heads, kv_heads):
    import gemm_pt_block_gb300 as mx

    with pytest.raises(ValueError, match="multiple of kv_heads"):
        mx.Mxfp4Attention(256, heads, kv_heads)


@pytest.mark.parametrize("slopes", [torch.ones(3), torch.ones(5), torch.ones(1, 4), torch.tensor(1.0)], ids=lambda t: str(tuple(t.shape)))
def test_slopes_of_another_number_are_refused(slopes):
    with pytest.raises(ValueError, match=r"slopes must be \[4\]"):
        block(slopes)


@pytest.mark.parametrize("slopes", [torch.ones(1).expand(4), torch.arange(8.0)[::2], torch.nn.Parameter(torch.arange(4.0)),
                                    torch.arange(4).double()], ids=["expanded", "every other", "parameter", "double"])
def test_slopes_are_the_blocks_own(slopes):
    want = slopes.detach().float().clone()
    m = block(slopes)
    assert m.slopes.dtype == torch.float32 and m.slopes.is_contiguous() and not m.slopes.requires_grad
    with torch.no_grad():
        slopes[:1] = 9.0
    assert torch.equal(m.slopes, want)
    assert "slopes" not in dict(m.named_parameters())
