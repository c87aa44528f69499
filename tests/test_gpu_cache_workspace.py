"""A workspace that the attention over the 8-bit cache did not ask for stays as it is, and so does what lies behind it."""
from __future__ import annotations

import pytest
import torch

from _cache import DEV, gen, make_cache
from test_gpu_bounds_check import _using, bc_lib  # noqa: F401  (bc_lib is a fixture)
from test_gpu_cache import check

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.mark.parametrize("L,n,H,G,D,P", [([40, 3, 17], [1, 1, 1], 2, 4, 64, 16), ([16, 9], [2, 3], 1, 3, 128, 16),
                                         ([13] * 40, [1] * 40, 2, 1, 256, 16)])
@pytest.mark.parametrize("room", [0, 16, 5000])
def test_a_workspace_that_is_not_needed(bc_lib, L, n, H, G, D, P, room):  # noqa: F811
    import gemm_pt_block_gb300 as mx

    c = make_cache(L, n, H, D, P, seed=1, table_cols=0)
    q = torch.randn((c.T, G * H, D), device=DEV, generator=gen(2)).to(BF16)

    def run():
        bytes_ = torch.full((1 << 16,), 0xA5, dtype=torch.uint8, device=DEV)
        out, lse = mx.mxfp8_cache_attention(q, c.codes, c.scales, c.table, c.lens, starts=c.starts, with_lse=True,
                                            workspace=bytes_[:room])
        assert mx.device_status() == 0
        assert bool((bytes_ == 0xA5).all())
        check(c, q, out, lse, BF16)

    run()
    with _using(bc_lib):
        run()
