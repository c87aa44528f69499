"""The feed-forward block: its training pass against autograd in plain PyTorch,
and decoding against the training weights."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16


def leaf(*shape, dtype=torch.float32, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, device=DEV, generator=g).to(dtype).requires_grad_()


def plain_norm(h, w, eps):
    return h * w / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)


def test_rmsnorm_autograd_with_residual_and_unused_outputs():
    import gemm_pt_block_gb300 as mx

    x, r, w = leaf(3, 5, 96, seed=1), leaf(3, 5, 96, seed=2), leaf(96, seed=3)
    x2, r2, w2 = (t.detach().double().requires_grad_() for t in (x, r, w))
    gy, gh = leaf(3, 5, 96, seed=4).detach(), leaf(3, 5, 96, seed=5).detach()
    for use_y, use_h in ((True, True), (True, False), (False, True)):
        for t in (x, r, w, x2, r2, w2):
            t.grad = None
        y, h = mx.rmsnorm(x, w, r, eps=1e-5, out_dtype=torch.float32)
        h2 = x2 + r2
        y2 = plain_norm(h2, w2, 1e-5)
        ((y * gy).sum() * use_y + (h * gh).sum() * use_h).backward()
        ((y2 * gy.double()).sum() * use_y + (h2 * gh.double()).sum() * use_h).backward()
        for a, b in ((x, x2), (r, r2), (w, w2)):
            # fp32 throughout: 96-term sums, gradients of order one
            assert torch.allclose(a.grad.double(), b.grad, rtol=1e-4, atol=1e-5)
    # only h used at all: no gradient reaches y
    x.grad = None
    mx.rmsnorm(x, w, r)[1].sum().backward()
    assert (x.grad == 1).all()


def test_autograd_of_expanded_gradients_and_frozen_inputs():
    import gemm_pt_block_gb300 as mx

    x, w = leaf(4, 64, seed=6), leaf(64, seed=7)
    y = mx.rmsnorm(x, w, out_dtype=torch.float32)
    y.sum().backward()                                     # dy is an expanded scalar
    x2, w2 = x.detach().double().requires_grad_(), w.detach().double().requires_grad_()
    plain_norm(x2, w2, 1e-6).sum().backward()
    assert torch.allclose(x.grad.double(), x2.grad, rtol=1e-4, atol=1e-5)
    assert torch.allclose(w.grad.double(), w2.grad, rtol=1e-4, atol=1e-5)
    frozen = w.detach()
    x.grad = None
    mx.rmsnorm(x, frozen, out_dtype=torch.float32).sum().backward()
    assert torch.allclose(x.grad.double(), x2.grad, rtol=1e-4, atol=1e-5)
    # the two halves of one projection
    gu = leaf(2, 3, 128, seed=8)
    a = mx.swiglu(gu[..., :64], gu[..., 64:], out_dtype=torch.float32)
    a.sum().backward()
    gu2 = gu.detach().double().requires_grad_()
    (torch.nn.functional.silu(gu2[..., :64]) * gu2[..., 64:]).sum().backward()
    assert torch.allclose(gu.grad.double(), gu2.grad, rtol=1e-4, atol=1e-5)


def test_block_trains_and_decodes():
    import gemm_pt_block_gb300 as mx

    torch.manual_seed(0)
    dim, hidden, T = 256, 384, 256
    block = mx.Mxfp4FeedForward(dim, hidden, device=DEV)
    x = leaf(2, T // 2, dim, dtype=BF16, seed=9)
    r = leaf(2, T // 2, dim, dtype=BF16, seed=10)
    y, h = block(x, r)
    assert y.shape == x.shape and torch.equal(h, (x.float() + r.float()).to(BF16))
    (y.float().square().mean() + h.float().mean()).backward()
    for t in (x, r, block.norm, block.gate_up.weight, block.down.weight):
        assert t.grad is not None and torch.isfinite(t.grad.float()).all() and t.grad.float().abs().max() > 0
    assert torch.equal(x.grad, r.grad)

    # decoding reads the same weight codes: against their dequantized values in 64 bits
    with pytest.raises(RuntimeError):
        block.decode(x[0, :1])
    block.quantize_weights()
    (qg, sg, pg), (qd, sd, pd) = block._decode
    wg = mx.mxfp4_dequantize(qg, sg, 2 * hidden, dim, params=pg).double()
    wd = mx.mxfp4_dequantize(qd, sd, dim, hidden, params=pd).double()
    for M in (1, 3, 17):
        xm, rm = x.detach().reshape(-1, dim)[:M], r.detach().reshape(-1, dim)[:M]
        ym, hm = block.decode(xm, rm)
        assert torch.equal(hm, (xm.float() + rm.float()).to(BF16))
        n = plain_norm(hm.double(), block.norm.detach().double(), block.eps)
        gu = n @ wg.t()
        want = (torch.nn.functional.silu(gu[:, :hidden]) * gu[:, hidden:]) @ wd.t()
        # two roundings to E4M3 (relative 2^-4 each at most, random in sign) and two to bf16:
        # well within a tenth of the output's norm
        assert ((ym.double() - want).norm() <= 0.1 * want.norm()).item()
    assert mx.device_status() == 0


def test_decode_in_a_graph_follows_its_input():
    import gemm_pt_block_gb300 as mx

    block = mx.Mxfp4FeedForward(128, 256, device=DEV)
    block.quantize_weights()
    xs = [leaf(2, 128, dtype=BF16, seed=20 + i).detach() for i in range(3)]
    want = [block.decode(t) for t in xs]
    buf = xs[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, h = block.decode(buf)
    for t, (wy, wh) in zip(xs, want):
        buf.copy_(t)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, wy) and torch.equal(h, wh)
