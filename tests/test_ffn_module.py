"""The feed-forward block's decode weights as part of the module (no GPU: the
quantizer is stood in for by one that returns bytes)."""
from __future__ import annotations

import copy

import pytest
import torch


@pytest.fixture
def block(monkeypatch):
    import gemm_pt_block_gb300 as mx
    from gemm_pt_block_gb300 import ffn

    def quantize(w, p):
        rows, cols = w.shape
        return (torch.full((rows, cols // 2), 3, dtype=torch.uint8, device=w.device),
                torch.full((rows * cols // 32,), 127, dtype=torch.uint8, device=w.device), None, None)

    monkeypatch.setattr(ffn, "mxfp4_quantize", quantize)
    return mx.Mxfp4FeedForward(128, 256, dtype=torch.float32)


def tensors(block):
    return [t for q, s, _ in block._decode for t in (q, s)]


def test_decode_weights_follow_the_module(block):
    assert block._decode is None
    with pytest.raises(RuntimeError, match="quantize_weights"):
        block.decode(torch.zeros(1, 128))
    block.quantize_weights()
    assert [t.device.type for t in tensors(block)] == ["cpu"] * 4
    other = copy.deepcopy(block).to("meta")
    assert [t.device.type for t in tensors(other)] == ["meta"] * 4
    assert [t.device.type for t in tensors(block)] == ["cpu"] * 4
    # a change of the parameters' type leaves the codes alone
    block.to(torch.bfloat16)
    assert all(t.dtype == torch.uint8 for t in tensors(block))


def test_decode_weights_are_no_part_of_the_state(block):
    before = set(block.state_dict())
    block.quantize_weights()
    assert set(block.state_dict()) == before
    block.load_state_dict(block.state_dict())
    assert len(tensors(block)) == 4


def test_a_refused_weight_leaves_the_last_ones(block):
    from dataclasses import replace

    block.quantize_weights()
    old = tensors(block)
    p = block.down.recipe.w_row
    block.down.recipe = replace(block.down.recipe, w_row=replace(p, wht=True))
    with pytest.raises(ValueError):
        block.quantize_weights()
    assert all(a is b for a, b in zip(tensors(block), old))
