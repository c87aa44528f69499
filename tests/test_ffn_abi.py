"""Host-side refusals of the norm, activation and few-row entry points (no GPU
needed: every call fails validation before any pointer is used)."""
from __future__ import annotations

import ctypes

import pytest


@pytest.fixture(scope="module")
def L():
    from gemm_pt_block_gb300 import build as b

    b.build()
    import gemm_pt_block_gb300 as mx

    return mx.lib()


G = ctypes.c_void_p(1 << 20)
OFF = ctypes.c_void_p((1 << 20) + 2)


def params(**kw):
    import gemm_pt_block_gb300 as mx

    return ctypes.byref(mx.QuantParams(**kw)._c())


def norm(L, x=G, dt=0, rows=4, cols=64, ld=64, r=None, ldr=64, w=None, wdt=0, eps=1e-6, h=None, ldh=64, y=G, ydt=0,
         ldy=64, rstd=None, row=None, q=None, s=None):
    return L.mxfp4_rmsnorm_quantize(x, dt, rows, cols, ld, r, ldr, w, wdt, eps, h, ldh, y, ydt, ldy, rstd, row, q, s,
                                    None)


@pytest.mark.parametrize("status,kw", [
    (2, dict(cols=48)), (2, dict(rows=-1)), (2, dict(ld=32)), (2, dict(cols=1 << 31, ld=1 << 31)),
    (2, dict(rows=1 << 30, cols=1 << 20, ld=1 << 20, ldy=1 << 20)), (2, dict(ld=(1 << 40) + 8)), (2, dict(ldy=40)),
    (1, dict(dt=2)), (1, dict(ydt=5)), (1, dict(x=None)), (1, dict(w=G, wdt=9)), (1, dict(y=None)),
    (1, dict(eps=float("inf"))), (1, dict(eps=float("nan"))), (1, dict(eps=-1e-6)),
    (3, dict(x=OFF)), (3, dict(y=OFF)), (3, dict(w=OFF)), (3, dict(r=OFF)), (3, dict(h=OFF)), (3, dict(rstd=OFF)),
    (3, dict(ld=68)), (3, dict(r=G, ldr=68)), (2, dict(r=G, ldr=32)), (2, dict(h=G, ldh=32)),
])
def test_norm_refusals(L, status, kw):
    assert norm(L, **kw) == status
    assert len(L.mxfp4_last_error()) > 0


def test_quantized_output_refusals(L):
    import gemm_pt_block_gb300 as mx

    assert norm(L, row=params(), q=None, s=G) == 1
    assert norm(L, row=params(), q=OFF, s=G) == 3
    assert norm(L, row=params(rounding=mx.ROUND_SR), q=G, s=G) == 4
    assert norm(L, row=params(wht=True), q=G, s=G) == 4
    assert norm(L, row=params(block=mx.BLOCK_32X32), q=G, s=G) == 4
    assert norm(L, row=params(scale_layout=mx.LAYOUT_MMA), q=G, s=G) == 2
    assert norm(L, row=params(scale_mode=3), q=G, s=G) == 1
    assert norm(L, row=params(block=mx.BLOCK_1X16, elem_format=mx.FORMAT_E4M3), q=G, s=G) == 4
    assert norm(L, row=params(tensor_exp=3), q=G, s=G) == 1


def grad(L, dy=G, ydt=0, ldy=64, h=G, hdt=0, ldh=64, w=None, wdt=0, rstd=G, dh=None, ldd=64, rows=4, cols=64, dx=G,
         ldx=64, dw=None, ws=None, n=0):
    return L.mxfp4_rmsnorm_backward(dy, ydt, ldy, h, hdt, ldh, w, wdt, rstd, dh, ldd, rows, cols, dx, ldx, dw, ws, n,
                                    None)


@pytest.mark.parametrize("status,kw", [
    (2, dict(cols=40)), (2, dict(ldy=32)), (2, dict(ldh=32)), (2, dict(ldx=32)), (2, dict(dh=G, ldd=32)),
    (1, dict(rstd=None)), (1, dict(dx=None)), (1, dict(h=None)), (1, dict(dy=None)), (1, dict(hdt=4)),
    (1, dict(w=G, dw=G)), (1, dict(w=G, dw=G, ws=G, n=16)), (3, dict(w=G, dw=OFF)), (3, dict(rstd=OFF)),
    (3, dict(w=G, dw=G, ws=OFF, n=1 << 30)), (3, dict(ldx=68)), (3, dict(w=OFF)),
])
def test_norm_gradient_refusals(L, status, kw):
    assert grad(L, **kw) == status


def test_workspace_size(L):
    size = L.mxfp4_rmsnorm_backward_workspace_size
    assert size(0, 64) == 0 and size(-1, 64) == 0 and size(4, 0) == 0 and size(4, 1 << 31) == 0
    assert size(1, 64) >= 4 * 64 and size(100000, 64) >= size(4, 64)


def test_activation_refusals(L):
    def act(g=G, ldg=64, u=G, ldu=64, dt=0, rows=4, cols=64, y=G, ydt=0, ldy=64, row=None, q=None, s=None):
        return L.mxfp4_swiglu_quantize(g, ldg, u, ldu, dt, rows, cols, y, ydt, ldy, row, q, s, None)

    for status, kw in [(2, dict(cols=33)), (2, dict(ldg=32)), (2, dict(ldu=32)), (2, dict(ldy=32)), (1, dict(dt=2)),
                       (1, dict(g=None)), (1, dict(u=None)), (1, dict(y=None)), (3, dict(g=OFF)), (3, dict(u=OFF)),
                       (3, dict(ldu=70)), (4, dict(row=params(wht=True), q=G, s=G))]:
        assert act(**kw) == status, kw

    def back(dy=G, ydt=0, ldy=64, g=G, ldg=64, u=G, ldu=64, dt=0, rows=4, cols=64, dg=G, lddg=64, du=G, lddu=64):
        return L.mxfp4_swiglu_backward(dy, ydt, ldy, g, ldg, u, ldu, dt, rows, cols, dg, lddg, du, lddu, None)

    for status, kw in [(2, dict(rows=-4)), (2, dict(lddg=32)), (1, dict(du=None)), (1, dict(dy=None)), (1, dict(ydt=7)),
                       (3, dict(dg=OFF)), (3, dict(ldy=66))]:
        assert back(**kw) == status, kw


def test_gemv_refusals(L):
    def gemv(x=G, kind=0, ldx=256, sx=None, qw=G, sw=G, block=0, layout=0, exp=0, M=2, N=128, K=256, y=G, ydt=0,
             ldy=128):
        return L.mxfp4_gemv(x, kind, ldx, sx, qw, sw, block, layout, exp, M, N, K, y, ydt, ldy, None)

    for status, kw in [(1, dict(kind=3)), (1, dict(kind=-1)), (1, dict(ydt=2)), (1, dict(block=4)), (1, dict(layout=2)),
                       (1, dict(exp=1)), (1, dict(block=3, exp=101)), (2, dict(K=48)), (2, dict(M=-1)),
                       (2, dict(M=65537)), (2, dict(N=1 << 31)), (2, dict(ldx=128)), (2, dict(ldy=64)),
                       (2, dict(layout=1, N=100, ldy=100)), (2, dict(layout=1, K=96)),
                       (2, dict(ldx=(1 << 40) + 16)), (1, dict(y=None)), (1, dict(x=None)), (1, dict(qw=None)),
                       (1, dict(sw=None)), (1, dict(kind=1)), (3, dict(x=OFF)), (3, dict(qw=OFF)), (3, dict(ldx=260)),
                       (3, dict(kind=1, sx=G, ldx=264)), (3, dict(y=ctypes.c_void_p((1 << 20) + 1))),
                       (3, dict(y=OFF, ydt=1))]:
        assert gemv(**kw) == status, kw


def test_module_refuses_sizes_off_the_tiles():
    import gemm_pt_block_gb300 as mx

    with pytest.raises(ValueError):
        mx.Mxfp4FeedForward(100, 256)
    with pytest.raises(ValueError):
        mx.mxfp4_rmsnorm_quantize(__import__("torch").zeros(4, 64), None)
