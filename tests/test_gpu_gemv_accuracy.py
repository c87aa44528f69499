"""What each form of the few-row product keeps of x, against the bounds that
the header states for it. W has one scale, so that Sum |W| shows what an error
of x costs. A large element of every block (or row) meets a zero weight: the
sums do not hold it, and what its size costs its neighbours is seen.

  every form          1e-5 sum_k |x w|                      (fp32 sums)
  up to eight rows    + 2^-39 of each 32-block's largest |x|, times its |W|
  MXFP8 form          + 2^-25 of each 32-block's largest |x|, at least 2^-137
  f16 rows (NVFP4)    + 2^-39 of each row's largest |x|

2^-25: the last of three E4M3 digits ends at 2^-17 steps (half of one: 2^-18)
in units in which the block's largest magnitude is above 224.
"""
from __future__ import annotations

import pytest
import torch

from test_gpu_gemv import E2M1, gen, wparams

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


def weights(N, K, nv, seed, zero):
    """Random codes under one scale (1), zero in the columns `zero` of every block."""
    q = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=DEV, generator=gen(seed))
    if zero:
        q.view(N, K // 32, 16)[:, :, 0] &= 0xF0
    s = torch.full((N, K // (16 if nv else 32)), 0x38 if nv else 127, dtype=torch.uint8, device=DEV)
    return q, s


def values(q, rows):
    return E2M1.to(DEV)[torch.stack((q[rows] & 15, q[rows] >> 4), -1).view(len(rows), -1).long()]


def bound(x, w, form):
    """x [M, K], w [n, K] in 64 bits -> [M, n]."""
    M, K = x.shape
    b = 1e-5 * (x.abs() @ w.abs().t())
    top = x.abs().view(M, K // 32, 32).amax(2, keepdim=True)
    if form == "f16 rows":
        top = top.amax(1, keepdim=True).expand(M, K // 32, 1)
    each = {"few": 2.0 ** -39 * top, "digits": (2.0 ** -25 * top).clamp_min(2.0 ** -137), "f16 rows": 2.0 ** -39 * top,
            "bf16": 0.0 * top}[form]
    return b + each.expand(M, K // 32, 32).reshape(M, K) @ w.abs().t()


FORMS = [(1, False, True, "digits"), (5, False, True, "digits"), (12, False, True, "digits"), (32, False, True, "digits"),
         (12, True, True, "f16 rows"), (31, True, True, "f16 rows"), (1, False, False, "few"), (7, True, False, "few"),
         (12, False, False, "bf16"), (12, True, False, "bf16")]


@pytest.mark.parametrize("M,nv,ws,form", FORMS)
@pytest.mark.parametrize("above", [4, 12, 20, 30])
@pytest.mark.parametrize("at", [0, -114])
def test_elements_far_above_their_block(M, nv, ws, form, above, at):
    """Elements of order 2^at, one of each block 2^above larger at a zero weight."""
    import gemm_pt_block_gb300 as mx

    N, K = 200, 1024
    q, s = weights(N, K, nv, 1, True)
    x = torch.randn((M, K), device=DEV, generator=gen(2)).double()
    x.view(M, K // 32, 32)[:, :, 0] = 2.0 ** above
    x = (x * 2.0 ** at).to(BF16)
    need = mx.lib().mxfp4_gemv_workspace_size(0, 3 if nv else 0, M, N, K)
    space = torch.empty(need, dtype=torch.uint8, device=DEV) if ws else False
    y = mx.mxfp4_gemv(x, q, s, N, K, wparams(nv), out_dtype=F32, workspace=space).double()
    w = values(q, list(range(N)))
    assert ((y - x.double() @ w.t()).abs() <= bound(x.double(), w, form)).all()


@pytest.mark.parametrize("M,N,K,nv,form", [(1, 28672, 4096, False, "digits"), (12, 8192, 4096, False, "digits"),
                                           (12, 4096, 4096, True, "f16 rows"), (1, 4096, 4096, False, "few")])
def test_the_default_call(M, N, K, nv, form):
    """Sizes at which the call takes a workspace by itself, and one at which it
    does not."""
    import gemm_pt_block_gb300 as mx

    q, s = weights(N, K, nv, 3, True)
    x = torch.randn((M, K), device=DEV, generator=gen(4))
    x.view(M, K // 32, 32)[:, :, 0] = 2.0 ** 20
    x = x.to(BF16)
    y = mx.mxfp4_gemv(x, q, s, N, K, wparams(nv), out_dtype=F32).double()
    rows = list(range(0, N, 61))
    w = values(q, rows)
    assert ((y[:, rows] - x.double() @ w.t()).abs() <= bound(x.double(), w, form)).all()


@pytest.mark.parametrize("M,N,K,nv,ws", [
    (1, 8192, 8192, False, False), (8, 28672, 4096, False, True), (9, 8192, 4096, False, True), (12, 4096, 4096, False, False),
    (16, 8192, 4096, False, True), (17, 8192, 4096, False, False), (24, 4096, 8192, False, False), (32, 8192, 4096, False, False),
    (24, 11264, 4096, False, True), (33, 8192, 4096, False, True), (24, 2048, 4096, True, False), (24, 4096, 4096, True, True)])
def test_the_form_that_the_default_call_takes(M, N, K, nv, ws):
    """The faster one of the two that were measured at these sizes (a workspace
    or none), seen by the bits of its result."""
    import gemm_pt_block_gb300 as mx

    q, s = weights(N, K, nv, 7, True)
    x = torch.randn((M, K), device=DEV, generator=gen(8))
    x.view(M, K // 32, 32)[:, :, 0] = 2.0 ** 36             # meets zero weights: its neighbours lose bits in either form
    x = x.to(BF16)
    need = mx.lib().mxfp4_gemv_workspace_size(0, 3 if nv else 0, M, N, K)
    space = torch.empty(need, dtype=torch.uint8, device=DEV)
    w = wparams(nv)
    got, one, none = (mx.mxfp4_gemv(x, q, s, N, K, w, out_dtype=F32, workspace=t) for t in (None, space, False))
    assert not torch.equal(one, none)
    assert torch.equal(got, one if ws else none)


@pytest.mark.parametrize("M,nv,ws", [(1, False, True), (12, False, True), (12, True, True), (12, False, False), (1, True, False)])
def test_long_sums_of_one_sign(M, nv, ws):
    """fp32 sums of K = 65536 products of one sign: where the tensor cores add
    (from nine rows on, and in the MXFP8 form) each step rounds toward zero,
    which one sign does not average out."""
    import gemm_pt_block_gb300 as mx

    N, K = 40, 65536
    q, s = weights(N, K, nv, 5, False)
    q &= 0x77
    x = torch.rand((M, K), device=DEV, generator=gen(6)).to(BF16)
    need = mx.lib().mxfp4_gemv_workspace_size(0, 3 if nv else 0, M, N, K)
    space = torch.empty(need, dtype=torch.uint8, device=DEV) if ws else False
    y = mx.mxfp4_gemv(x, q, s, N, K, wparams(nv), out_dtype=F32, workspace=space).double()
    w = values(q, list(range(N)))
    ref = x.double() @ w.t()
    rel = ((y - ref).abs() / ref).max().item()
    print(f"long sums M={M} nv={nv} ws={ws}: {rel:.2e}")
    assert rel <= 1e-5
