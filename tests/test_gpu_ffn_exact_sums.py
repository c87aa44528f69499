"""The norm's weight gradient with integers, so that every sum over rows is
exact whatever its order: one missing, doubled or misplaced row shows.

dy and h are small integers and rstd is 1, so each row adds an integer of at
most 6 to each column, and the sums stay below 2^24."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


def integers(rows, cols, dtype, seed, most):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(-most, most + 1, (rows, cols), device=DEV, generator=g).to(dtype)


@pytest.mark.parametrize("rows,cols", [
    (1, 32), (40001, 96), (40000, 512), (7, 544), (1825, 544), (40000, 1024), (151, 4096), (153, 4096), (305, 8192),
    (1300, 8192), (2001, 16384), (300, 32768)])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("stream", [False, True])
def test_every_row_counts_once(rows, cols, dt, stream):
    import gemm_pt_block_gb300 as mx

    dy, h = integers(rows, cols, dt, 1, 2), integers(rows, cols, dt, 2, 3)
    dh = integers(rows, cols, dt, 3, 2) if stream else None
    w, rstd = torch.ones(cols, device=DEV), torch.ones(rows, device=DEV)
    _, dw = mx.mxfp4_rmsnorm_backward(dy, h, w, rstd, dh=dh)
    want = torch.zeros(cols, device=DEV, dtype=torch.float64)
    for lo in range(0, rows, 4096):                        # (in parts: 64-bit copies of all rows are large)
        want += (dy[lo:lo + 4096].double() * h[lo:lo + 4096].double()).sum(0)
    assert torch.equal(dw.double(), want)
    assert mx.device_status() == 0


def test_a_row_alone_reaches_its_columns():
    """One row of ones among zeros, at the rows' ends and the groups' seams."""
    import gemm_pt_block_gb300 as mx

    rows, cols = 3000, 1024
    h, w, rstd = torch.ones((rows, cols), device=DEV, dtype=BF16), torch.ones(cols, device=DEV), torch.ones(rows, device=DEV)
    for row in (0, 1, 151, 152, 1823, 1824, 2999):
        dy = torch.zeros_like(h)
        dy[row] = torch.arange(cols, device=DEV) % 200
        _, dw = mx.mxfp4_rmsnorm_backward(dy, h, w, rstd)
        assert torch.equal(dw, dy[row].float())
