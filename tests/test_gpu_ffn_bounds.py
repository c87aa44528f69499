"""The norm, activation and few-row kernels in the bounds-checking build: no
store outside its output on shapes ragged against their tiles and the regular
library's bits; with the checked extents shrunk the check fires (and skips the
stores past them)."""
from __future__ import annotations

import pytest
import torch

from test_gpu_bounds_check import _both, _equal, _using, bc_lib  # noqa: F401  (bc_lib is a fixture)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


def rnd(rows, cols, dtype=BF16, seed=1):
    return torch.randn((rows, cols), device=DEV, generator=torch.Generator(device=DEV).manual_seed(seed)).to(dtype)


def codes(rows, cols, seed, hi=256):
    return torch.randint(0, hi, (rows, cols), dtype=torch.uint8, device=DEV,
                         generator=torch.Generator(device=DEV).manual_seed(seed))


def calls():
    import gemm_pt_block_gb300 as mx

    p8 = mx.QuantParams(elem_format=mx.FORMAT_E4M3)
    p4 = mx.QuantParams(block=mx.BLOCK_1X16)
    pm = mx.QuantParams(scale_layout=mx.LAYOUT_MMA)
    out = {}
    for rows, cols, dt, p in ((7, 96, BF16, p8), (33, 2080, F32, p4), (128, 1152, BF16, pm), (200, 8192, BF16, p8),
                              (3, 40032, F32, p8)):
        x, r, w = rnd(rows, cols, dt), rnd(rows, cols, dt, 2), torch.ones(cols, device=DEV)
        out[f"norm {rows}x{cols}"] = lambda x=x, r=r, w=w, p=p: mx.mxfp4_rmsnorm_quantize(
            x, w, p, residual=r, y_dtype=F32, with_rstd=True)
        rstd = torch.ones(rows, device=DEV)
        out[f"norm backward {rows}x{cols}"] = lambda x=x, r=r, w=w, s=rstd: mx.mxfp4_rmsnorm_backward(r, x, w, s, dh=r)
        out[f"swiglu {rows}x{cols}"] = lambda x=x, r=r, p=p: mx.mxfp4_swiglu_quantize(x, r, p, y_dtype=BF16)
        out[f"swiglu backward {rows}x{cols}"] = lambda x=x, r=r: mx.mxfp4_swiglu_backward(r, x, r)
    for M, N, K, nv in ((3, 77, 160, False), (8, 129, 512, True), (20, 200, 544, False), (12, 130, 256, True),
                        (5, 300, 1024, False), (40, 70, 384, False)):
        q, s = codes(N, K // 2, 3), codes(N, K // (16 if nv else 32), 4, 120)
        x = rnd(M, K)
        w = p4 if nv else mx.QuantParams()
        ws = torch.empty(int(mx.lib().mxfp4_gemv_workspace_size(0, 3 if nv else 0, M, N, K)), dtype=torch.uint8,
                         device=DEV)
        out[f"gemv {M}x{N}x{K}"] = lambda x=x, q=q, s=s, N=N, K=K, w=w: mx.mxfp4_gemv(x, q, s, N, K, w, out_dtype=F32,
                                                                                     workspace=False)
        out[f"gemv {M}x{N}x{K} ws"] = lambda x=x, q=q, s=s, N=N, K=K, w=w, ws=ws: mx.mxfp4_gemv(
            x, q, s, N, K, w, out_dtype=F32, workspace=ws)
    return out


def test_no_store_outside_and_the_same_bits(bc_lib):  # noqa: F811
    for name, fn in calls().items():
        want, got, status = _both(bc_lib, fn)
        assert status == 0, name
        assert _equal(want, got), name


def test_the_check_fires(bc_lib):  # noqa: F811
    import gemm_pt_block_gb300 as mx

    for name, fn in calls().items():
        with _using(bc_lib):
            try:
                assert bc_lib.mxfp4_bounds_check_shrink(8) == 0
                fn()
                assert mx.device_status() == 7, name
            finally:
                assert bc_lib.mxfp4_bounds_check_shrink(0) == 0
            fn()
            assert mx.device_status() == 0, name
