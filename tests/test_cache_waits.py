"""The self-test of the bounded waits of the attention over the 8-bit cache:
its launch, on a runtime that launches nothing, and its outcome on the GPU,
where waits of whole warps run out by their own limit (nothing signals them)
and the context goes on working."""
from __future__ import annotations

import time

import pytest
import torch

from test_launch_errors import ERR_CUDA, L as fake  # noqa: F401  (a fixture)

TIMEOUT = 6   # MXFP4_ERR_TIMEOUT


def test_a_failed_launch_is_reported(fake):  # noqa: F811
    fake.fake_fail_at(-1)
    assert fake.mxfp8_selftest_cache_wait_timeout(None) == 0 and fake.fake_launches() == 1
    fake.fake_fail_at(0)
    assert fake.mxfp8_selftest_cache_wait_timeout(None) == ERR_CUDA
    assert b"mxfp8_selftest_cache_wait_timeout" in fake.mxfp4_last_error()


@pytest.mark.gpu
def test_waits_of_whole_warps_run_out_and_say_so():
    import gemm_pt_block_gb300 as mx
    from _cache import DEV, gen, make_cache
    from test_gpu_cache import check

    assert mx.device_status() == 0
    t0 = time.perf_counter()
    mx.selftest_cache_wait_timeout()
    status = mx.device_status()
    waited = time.perf_counter() - t0
    assert status == TIMEOUT                                # (1 where a lane went on alone)
    assert b"bounded device-side wait ran out" in mx.lib().mxfp4_last_error()
    assert 1.0 < waited < 30.0                              # the limit is 2 s; both warps wait side by side
    assert mx.device_status() == 0
    c = make_cache([700, 3], [1, 1], 2, 64, 16, seed=1)
    q = torch.randn((2, 8, 64), device=DEV, generator=gen(2)).to(torch.bfloat16)
    out, lse = mx.mxfp8_cache_attention(q, c.codes, c.scales, c.table, c.lens, with_lse=True)
    check(c, q, out, lse, torch.bfloat16)
    assert mx.device_status() == 0
