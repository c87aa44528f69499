"""Second derivatives through the norm and the activation:
refused, never dropped. (The kernels are stood in for by plain PyTorch on the
CPU: what is tested is what autograd is told.)"""
from __future__ import annotations

import pytest
import torch


@pytest.fixture
def mx(monkeypatch):
    import gemm_pt_block_gb300 as mx
    from gemm_pt_block_gb300 import ffn

    def norm(x, weight, residual=None, eps=1e-6, y_dtype=None, with_rstd=False, **kw):
        h = x if residual is None else x + residual
        rstd = 1 / torch.sqrt((h * h).mean(1) + eps)
        y = h * rstd[:, None] * (1 if weight is None else weight)
        return None, None, y.detach(), None if residual is None else h.detach(), rstd.detach()

    def norm_backward(dy, h, weight, rstd, dh=None, with_dw=True, **kw):
        dy, h, rstd = dy.detach(), h.detach(), rstd[:, None]
        n, dn = h * rstd, dy * (1 if weight is None else weight.detach())
        dx = (dn - n * (dn * n).mean(1, keepdim=True)) * rstd + (0 if dh is None else dh.detach())
        return dx, (dy * n).sum(0) if with_dw and weight is not None else None

    def act(gate, up, y_dtype=None, **kw):
        return None, None, (torch.nn.functional.silu(gate) * up).detach()

    def act_backward(dy, gate, up, dgate=None, dup=None, **kw):
        dy, g, u = dy.detach(), gate.detach(), up.detach()
        s = torch.sigmoid(g)
        dgate = torch.empty_like(g) if dgate is None else dgate
        dup = torch.empty_like(g) if dup is None else dup
        dgate.copy_(dy * u * s * (1 + g * (1 - s)))
        dup.copy_(dy * g * s)
        return dgate, dup

    for name, fake in (("mxfp4_rmsnorm_quantize", norm), ("mxfp4_rmsnorm_backward", norm_backward),
                       ("mxfp4_swiglu_quantize", act), ("mxfp4_swiglu_backward", act_backward)):
        monkeypatch.setattr(ffn, name, fake)
    return mx


def leaf(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float32).requires_grad_()


def forms(mx):
    x, r, w, u = leaf(8, 64, seed=1), leaf(8, 64, seed=2), leaf(64, seed=3), leaf(8, 64, seed=4)
    wide = leaf(8, 128, seed=5)
    f32 = torch.float32
    return {
        "norm": (lambda: mx.rmsnorm(x, w, out_dtype=f32), (x, w)),
        "norm, residual": (lambda: sum(t.sum(1).square() for t in mx.rmsnorm(x, w, r, out_dtype=f32)), (x, r, w)),
        "norm, weight alone": (lambda: mx.rmsnorm(x.detach(), w, out_dtype=f32).square(), (w,)),
        "activation": (lambda: mx.swiglu(x, u, out_dtype=f32), (x, u)),
        "activation, up alone": (lambda: mx.swiglu(x.detach(), u, out_dtype=f32).square(), (u,)),
        "of every second column": (lambda: mx.rmsnorm(wide[:, ::2], w, out_dtype=f32), (wide, w)),
    }


NAMES = ["norm", "norm, residual", "norm, weight alone", "activation", "activation, up alone", "of every second column"]


@pytest.mark.parametrize("name", NAMES)
def test_a_loss_of_gradients_is_refused(mx, name):
    call, leaves = forms(mx)[name]
    grads = torch.autograd.grad(call().sum(), leaves, create_graph=True)
    # first derivatives are there as ever, the same with and without a graph
    for g, plain in zip(grads, torch.autograd.grad(call().sum(), leaves)):
        assert torch.equal(g, plain)
    for i, g in enumerate(grads):
        loss = g.square().sum() + leaves[0].sum()
        with pytest.raises(RuntimeError, match="second derivatives"):
            torch.autograd.grad(loss, leaves, retain_graph=True, allow_unused=True)


@pytest.mark.parametrize("name", ["norm, weight alone", "activation, up alone"])
def test_gradients_that_are_constants_stay_constants(mx, name):
    """With a loss linear in the output, the gradient of what enters linearly
    depends on nothing that requires grad: nothing is refused."""
    x, u, w = leaf(8, 64, seed=1).detach(), leaf(8, 64, seed=4), leaf(64, seed=3)
    y, t = {"norm, weight alone": lambda: (mx.rmsnorm(x, w, out_dtype=torch.float32), w),
            "activation, up alone": lambda: (mx.swiglu(x, u, out_dtype=torch.float32), u)}[name]()
    g, = torch.autograd.grad(y.sum(), (t,), create_graph=True)
    assert not g.requires_grad
    torch.autograd.grad((g * t).sum(), (t,))


def test_training_passes_carry_no_extra_node(mx):
    x, w = leaf(8, 64, seed=1), leaf(64, seed=3)
    mx.rmsnorm(x, w, out_dtype=torch.float32).sum().backward()
    assert x.grad.grad_fn is None and not x.grad.requires_grad and not w.grad.requires_grad
