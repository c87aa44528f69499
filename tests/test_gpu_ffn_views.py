"""The feed-forward functions and the block take views that begin or step
anywhere: the same bits as from a copy on the kernels' boundaries."""
from __future__ import annotations

import pytest
import torch

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


def rnd(*shape, dtype, seed, dev=DEV):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(dev)


def off(t, elements=1):
    """t's values one element past a boundary (contiguous, as a view)."""
    buf = torch.empty(t.numel() + elements, dtype=t.dtype, device=t.device)
    v = buf[elements:].view(t.shape)
    with torch.no_grad():
        v.copy_(t)
    return v


def every_second(t):
    wide = torch.zeros((*t.shape[:-1], 2 * t.shape[-1]), dtype=t.dtype, device=t.device)
    wide[..., ::2] = t
    return wide[..., ::2]


@pytest.mark.parametrize("rows", [1, 3])
@pytest.mark.parametrize("form", [off, every_second, lambda t: t])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_a_readable_matrix_is_one_the_kernels_take(rows, form, dt):
    from gemm_pt_block_gb300.ffn import _readable, _readable_vector

    t = rnd(rows, 64, dtype=dt, seed=1, dev="cpu")
    r, v = _readable(form(t)), _readable_vector(form(t[0]))
    assert r.data_ptr() % 16 == 0 and r.stride(1) == 1 and (rows == 1 or r.stride(0) % 8 == 0) and torch.equal(r, t)
    assert v.data_ptr() % 16 == 0 and v.is_contiguous() and torch.equal(v, t[0])
    assert _readable(r) is r and _readable_vector(v) is v and _readable_vector(None) is None


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 5])
@pytest.mark.parametrize("form", [off, every_second])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_functions_of_views(rows, form, dt):
    import gemm_pt_block_gb300 as mx

    x, r, w = rnd(rows, 96, dtype=dt, seed=2), rnd(rows, 96, dtype=dt, seed=3), rnd(96, dtype=dt, seed=4)
    gy, gh = rnd(rows, 96, dtype=dt, seed=5), rnd(rows, 96, dtype=dt, seed=6)

    def run(f):
        leaves = [t.clone().requires_grad_() for t in (x, r, w)]
        y, h = mx.rmsnorm(f(leaves[0]), f(leaves[2]), f(leaves[1]), out_dtype=dt)
        a = mx.swiglu(f(y), f(h), out_dtype=dt)
        return [y, h, a, *torch.autograd.grad([y, h, a], leaves, [f(gy), f(gh), f(gy)])]

    def view(t):
        if not t.requires_grad:
            return form(t)
        if form is off:                                   # differentiable, one element past a boundary
            return torch.cat((t.detach().reshape(-1)[:1], t.reshape(-1)))[1:].view(t.shape)
        return torch.stack((t, t.detach()), -1)[..., 0]

    for got, want in zip(run(view), run(lambda t: t)):
        assert torch.equal(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("form", [off, every_second])
def test_decode_of_views_and_a_norm_weight_in_a_flat_buffer(form):
    import gemm_pt_block_gb300 as mx

    block = mx.Mxfp4FeedForward(128, 256, device=DEV)
    block.quantize_weights()
    x, r = rnd(2, 128, dtype=BF16, seed=7), rnd(2, 128, dtype=BF16, seed=8)
    want = block.decode(x, r)
    block.norm.data = off(block.norm.data)
    got = block.decode(form(x), form(r))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    one = block.decode(form(x[:1]), form(r[:1]))
    assert torch.equal(one[1], want[1][:1])
