"""Few-row products at the ends of their range: scales whose product passes
fp32, tensor exponents against the size of x, tiny x, and elements far above
their block."""
from __future__ import annotations

import pytest
import torch

from test_gpu_gemv import E2M1, activations, check, gen, weights, wparams

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


def space(on, x_kind, nv, M, N, K):
    import gemm_pt_block_gb300 as mx

    if not on:
        return False
    need = mx.lib().mxfp4_gemv_workspace_size(x_kind, 3 if nv else 0, M, N, K)
    return torch.empty(need, dtype=torch.uint8, device=DEV) if need else False


@pytest.mark.parametrize("M", [1, 5, 8, 12, 32])
@pytest.mark.parametrize("ws", [False, True])
def test_block_scales_whose_product_passes_fp32(M, ws):
    """x in MXFP8 under 2^100, weights under 2^30: the products are finite (two
    nonzero weights of each row meet x values of 2^-6), and a block of zero
    weights gives zero. All values are powers of two times small integers, so
    the sums are exact."""
    import gemm_pt_block_gb300 as mx

    N, K = 96, 256
    x = torch.full((M, K), 0x08, dtype=torch.uint8, device=DEV)          # E4M3 2^-6
    sx = torch.full((M, K // 32), 127 + 100, dtype=torch.uint8, device=DEV)
    q = torch.zeros((N, K // 2), dtype=torch.uint8, device=DEV)
    q[1:, 20] = 0x12                                                      # 1.0 and 0.5 in block 1
    s = torch.full((N, K // 32), 127 + 30, dtype=torch.uint8, device=DEV)
    y = mx.mxfp4_gemv(x, q, s, N, K, sx=sx, out_dtype=F32, workspace=space(ws, 1, False, M, N, K))
    want = torch.full((M, N), 1.5 * 2.0 ** (94 + 30), dtype=torch.float64, device=DEV)
    want[:, 0] = 0.0
    assert torch.equal(y.double(), want)
    assert mx.device_status() == 0


@pytest.mark.parametrize("M", [1, 8, 12, 32])
@pytest.mark.parametrize("ws", [False, True])
def test_bf16_blocks_whose_scale_product_passes_fp32(M, ws):
    """bf16 x near 2^110 under weights of 2^17: zero weights give zero, and one
    small element that meets the only nonzero weight gives its finite product."""
    import gemm_pt_block_gb300 as mx

    N, K = 64, 128
    x = torch.full((M, K), 2.0 ** 118, device=DEV, dtype=BF16)
    x[:, 32:64] = 2.0 ** 100
    q = torch.zeros((N, K // 2), dtype=torch.uint8, device=DEV)
    q[1:, 20] = 0x02                                                      # element 40: 1.0
    s = torch.full((N, K // 32), 127 + 26, dtype=torch.uint8, device=DEV)
    y = mx.mxfp4_gemv(x, q, s, N, K, out_dtype=F32, workspace=space(ws, 0, False, M, N, K))
    assert (y[:, 0] == 0).all() and (y[:, 1:] == 2.0 ** 126).all()


@pytest.mark.parametrize("exp,shift", [(100, -90), (60, -60), (-100, 90), (0, 0)])
@pytest.mark.parametrize("M", [3, 12])
@pytest.mark.parametrize("ws", [False, True])
def test_tensor_exponents_against_the_size_of_x(exp, shift, M, ws):
    """NVFP4's 2^tensor_exp with x of the opposite size: the product is of order
    one, and nothing on the way passes fp32 either way."""
    import gemm_pt_block_gb300 as mx

    N, K = 130, 512
    q, s, w64 = weights(N, K, True, 71)
    x, _, _, _ = activations(M, K, "bf16", 72)
    x = (x.double() * 2.0 ** shift).to(BF16)
    y = mx.mxfp4_gemv(x, q, s, N, K, wparams(True, 0, exp), out_dtype=F32, workspace=space(ws, 0, True, M, N, K))
    check(y, x.double(), w64 * 2.0 ** exp)


@pytest.mark.parametrize("M", [3, 12])
@pytest.mark.parametrize("ws", [False, True])
def test_large_tensor_exponent_with_sums_of_one_sign(M, ws):
    """Weights and x of one sign and size: the sums are as large as they get."""
    import gemm_pt_block_gb300 as mx

    N, K = 130, 4096
    q, s, _ = weights(N, K, True, 75)
    q &= 0x77
    v = E2M1.to(DEV)[torch.stack((q & 15, q >> 4), -1).view(N, K).long()]
    w64 = v * s.view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)
    x = torch.full((M, K), 1.5 * 2.0 ** -90, device=DEV, dtype=BF16)
    y = mx.mxfp4_gemv(x, q, s, N, K, wparams(True, 0, 100), out_dtype=F32, workspace=space(ws, 0, True, M, N, K))
    check(y, x.double(), w64 * 2.0 ** 100)


@pytest.mark.parametrize("nv", [False, True], ids=["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M", [3, 12, 20])
def test_x_near_the_smallest_normal_numbers(nv, M):
    """Rows of x around 2^-116 under weights of order one: the sums are normal
    fp32 numbers and keep their bits."""
    import gemm_pt_block_gb300 as mx

    N, K = 130, 1024
    q, _, _ = weights(N, K, nv, 73)
    s = torch.full((N, K // (16 if nv else 32)), 0x38 if nv else 127, dtype=torch.uint8, device=DEV)
    w64 = E2M1.to(DEV)[torch.stack((q & 15, q >> 4), -1).view(N, K).long()]
    x = (torch.randn((M, K), device=DEV, generator=gen(74)).double() * 2.0 ** -116).to(BF16)
    y = mx.mxfp4_gemv(x, q, s, N, K, wparams(nv), out_dtype=F32, workspace=False)
    check(y, x.double(), w64)
