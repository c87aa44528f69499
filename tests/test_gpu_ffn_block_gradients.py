"""The feed-forward block's training pass, stage by stage, against 64 bits.

The block's own tensors between its stages and their gradients are caught by
hooks; each stage's gradients are then computed from what that stage was given:
the linear layers on the same codes (the quantizer is called with the layer's
parameters and its result dequantized), the activation and the norm from their
formulas. So a gradient that went to the wrong half, row or weight shows, and
the bounds are those of one stage: the GEMM's 1e-5 of the products' magnitudes,
24 u and (D / 64 + 76) u of the terms' for activation and norm (u = 2^-24,
derived in test_gpu_ffn.py), each with half a unit of bf16 (2^-8).
"""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16
U = 2.0 ** -24


def rnd(*shape, seed, dtype=BF16):
    return torch.randn(shape, device=DEV, generator=torch.Generator(device=DEV).manual_seed(seed)).to(dtype)


def near(got, want, mag, rel):
    t = rel * mag
    bad = (got.double() - want).abs() > t + 2.0 ** -8 * (want.abs() + t)
    assert not bad.any(), (int(bad.sum()), got[bad][:4], want[bad][:4])


def quantized(t, row=None, col=None):
    """The values of t's codes, [rows, cols] or [cols, rows] (column-wise)."""
    import gemm_pt_block_gb300 as mx

    q, s, qc, sc = mx.mxfp4_quantize(t, row, col)
    rows, cols = t.shape
    if row is not None:
        return mx.mxfp4_dequantize(q, s, rows, cols, params=row).double()
    return mx.mxfp4_dequantize(qc, sc, cols, rows, params=col).double()


def check_linear(layer, x, dy, dx):
    r, w = layer.recipe, layer.weight.detach()
    g, wt = quantized(dy, r.dy_row), quantized(w, None, r.w_col)
    near(dx, g @ wt.t(), g.abs() @ wt.abs().t(), 1e-5)
    gt, xt = quantized(dy, None, r.dy_col), quantized(x, None, r.x_col)
    near(layer.weight.grad, gt @ xt.t(), gt.abs() @ xt.abs().t(), 1e-5)


@pytest.mark.parametrize("recipe", ["default", "1d"])
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("T,dim,hidden", [(128, 128, 256), (256, 256, 384)])
def test_every_stage_of_the_backward_pass(recipe, residual, T, dim, hidden):
    import gemm_pt_block_gb300 as mx

    torch.manual_seed(1)
    block = mx.Mxfp4FeedForward(dim, hidden, mx.recipe_1d(0x5A5A1234, 3) if recipe == "1d" else None, device=DEV)
    with torch.no_grad():
        block.norm.copy_(1 + 0.2 * rnd(dim, seed=2))
    x, r = rnd(T, dim, seed=3).requires_grad_(), rnd(T, dim, seed=4).requires_grad_() if residual else None
    seen, grads = {}, {}

    def catch(name):
        def hook(module, args, out):
            for key, t in ((name + " in", args[0]), (name + " out", out)):
                seen[key] = t.detach().reshape(T, -1)
                t.register_hook(lambda g, key=key: grads.__setitem__(key, g.detach().reshape(T, -1).clone()))
        return hook

    block.gate_up.register_forward_hook(catch("gate_up"))
    block.down.register_forward_hook(catch("down"))
    y, h = block(x, r)
    gy, gh = rnd(T, dim, seed=5), rnd(T, dim, seed=6)
    torch.autograd.backward([y, h], [gy, gh])

    assert torch.equal(grads["down out"], gy)
    check_linear(block.down, seen["down in"], gy, grads["down in"])

    # the activation: its two halves beside one another in the product's gradient
    gu, da, dgu = seen["gate_up out"].double(), grads["down in"].double(), grads["gate_up out"]
    g, u = gu[:, :hidden], gu[:, hidden:]
    s = 1 / (1 + torch.exp(-g))
    near(seen["down in"], g * s * u, (g * s * u).abs(), 16 * U)
    near(dgu[:, :hidden], da * u * s * (1 + g * (1 - s)), (da * u * s).abs() * (1 + g.abs()), 24 * U)
    near(dgu[:, hidden:], da * g * s, (da * g * s).abs(), 24 * U)

    check_linear(block.gate_up, seen["gate_up in"], dgu, grads["gate_up in"])

    # the norm, with the stream's gradient
    hh, dn = h.detach().double(), grads["gate_up in"].double()
    rstd = 1 / torch.sqrt((hh * hh).mean(1, keepdim=True) + block.eps)
    n, w = hh * rstd, block.norm.detach().double()
    d = dn * w
    mean = (d * n).mean(1, keepdim=True)
    dx = (d - n * mean) * rstd + gh.double()
    mag = (d.abs() + n.abs() * (d * n).abs().mean(1, keepdim=True)) * rstd + gh.double().abs()
    if residual:
        near(x.grad, dx, mag, (dim / 64 + 76) * U)
        assert torch.equal(x.grad, r.grad)
    else:                                                 # the two gradients of x are added by autograd, in bf16
        own = dx - gh.double()
        assert ((x.grad.double() - dx).abs() <= 2.0 ** -7 * (own.abs() + gh.double().abs()) + (dim / 64 + 76) * U * mag).all()
    near(block.norm.grad, (dn * n).sum(0), (dn * n).abs().sum(0), (T + dim / 64 + 76) * U)
    assert mx.device_status() == 0
