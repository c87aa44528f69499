"""SwiGLU over the whole range of its inputs: tiny gates under large `up`, and
gates so negative that the sigmoid is below fp32's normal numbers.

y = (g sigma(g)) u with sigma(g), silu(g) and y rounded to fp32, so the bound is
the arithmetic's 16 u relative to |y| (u = 2^-24, derived in test_gpu_ffn.py)
and, where one of the three is subnormal, half of fp32's last place there
(2^-150) times what it is multiplied by afterwards. No absolute slack beyond.
"""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


def silu64(g):
    return g.double() / (1 + torch.exp(-g.double()))


def check(gate, up, cols=None):
    import gemm_pt_block_gb300 as mx

    y = mx.mxfp4_swiglu_quantize(gate, up, y_dtype=F32)[2].double()
    s, u = silu64(gate), up.double()
    sig = 1 / (1 + torch.exp(-gate.double()))
    bound = 16 * U * (s * u).abs() + 2.0 ** -150 * (
        (gate.double() * u).abs() * (sig < 2.0 ** -125) + u.abs() * (s.abs() < 2.0 ** -125)
        + 1.0 * ((s * u).abs() < 2.0 ** -125))
    bad = (y - s * u).abs() > bound
    assert not bad.any(), (gate[bad][:4], up[bad][:4], y[bad][:4], (s * u)[bad][:4])


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_tiny_gates_under_large_up(dt, sign):
    g = torch.Generator(device=DEV).manual_seed(1)
    e = torch.linspace(-126, -100, 27, device=DEV).repeat_interleave(32).view(27, 32)
    m = 1 + torch.rand((27, 32), device=DEV, generator=g)
    gate = (sign * m.double() * torch.exp2(e.double())).to(dt)
    gate[-1, :4] = 0.0
    up = ((1 + torch.rand((27, 32), device=DEV, generator=g)) * 2.0 ** 100).to(dt)
    assert (gate[:-1].abs() >= 2.0 ** -126).all()
    check(gate, up)


@pytest.mark.parametrize("dt", [BF16, F32])
def test_subnormal_gates(dt):
    step = 2.0 ** -133 if dt == BF16 else 2.0 ** -149
    k = torch.arange(1, 129, device=DEV, dtype=torch.float64).view(4, 32)
    gate = (k * step).to(dt)
    check(gate, torch.full((4, 32), 2.0 ** 100, device=DEV, dtype=dt))


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("up", [1.0, 2.0 ** 60, 2.0 ** -20])
def test_gates_of_the_smallest_sigmoids(dt, up):
    """Alone, and in one row with ordinary and with tiny gates."""
    gate = torch.linspace(-103.5, -60.0, 512, device=DEV).view(4, 128).to(dt)
    check(gate, torch.full((4, 128), up, device=DEV, dtype=dt))
    mixed = gate.clone()
    mixed[:, ::3] = 2.0 ** -120
    mixed[:, 1::3] = 1.25
    check(mixed, torch.full((4, 128), up, device=DEV, dtype=dt))


def test_codes_of_tiny_gates():
    """Quantized outputs come from the same values: 2^-120 under 2^100 counts."""
    import gemm_pt_block_gb300 as mx

    gate = torch.full((2, 128), 1.5 * 2.0 ** -120, device=DEV)
    up = torch.full((2, 128), 2.0 ** 100, device=DEV)
    q, s, _ = mx.mxfp4_swiglu_quantize(gate, up, mx.QuantParams(scale_mode=mx.SCALE_ROUNDUP, elem_format=mx.FORMAT_E4M3))
    d = mx.mxfp4_dequantize(q, s, 2, 128, params=mx.QuantParams(elem_format=mx.FORMAT_E4M3))
    assert (d == 0.75 * 2.0 ** -20).all()
