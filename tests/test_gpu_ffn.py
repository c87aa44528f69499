"""The norm and activation kernels against plain implementations in 64 bits.

Quantized outputs are checked exactly: the call also returns its fp32 values,
and codes and scales must equal the oracle's quantization of those, bit for
bit. The fp32 values are checked against 64 bits with bounds that follow from
the arithmetic (u = 2^-24, the unit roundoff of fp32):

  rstd  A sum of n squares whose longest chain of additions has L terms is off
        by at most (L + 1) u relative to itself (all terms are positive); with
        the division, the addition of eps and the square root's reciprocal,
        rstd is off by at most (L + 1) u / 2 + 3 u. L <= n / 64 + 64 for every
        kernel here.
  y     two more roundings: rstd's bound + 2 u; and half a unit of the type it
        is stored in (bf16 has 8 significant bits: 2^-8 of the value at most).
  SwiGLU  expf and the division are within 2 ulp each and four products and
        sums follow: 16 u relative to |y|.
  dx    each factor within rstd's bound + 4 u, the mean's sum off by
        (L + 4) u sum|dn n|, added to terms that may cancel: the bound is over
        the sum of the terms' magnitudes.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from _util import assert_same, cuda_params
from test_gpu_canary import Arena

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


def chain(n):
    return n / 64 + 64


def half_ulp(dtype):
    return 2.0 ** -8 if dtype == BF16 else 0.0


def rand(rows, cols, dtype, seed, std=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((rows, cols), device=DEV, generator=g) * std
    if cols >= 64:
        x[:, 7] *= 50.0                                  # an outlier channel
    return x.to(dtype)


def strided(t, extra):
    """t in a wider buffer: the same values with row stride cols + extra."""
    wide = torch.zeros((t.shape[0], t.shape[1] + extra), dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


FORMATS = {
    "e2m1": oracle.Params(scale_mode=oracle.SCALE_FLOOR),
    "e4m3": oracle.Params(scale_mode=oracle.SCALE_ROUNDUP, elem_format=oracle.FORMAT_E4M3),
    "e4m3floor": oracle.Params(scale_mode=oracle.SCALE_FLOOR, elem_format=oracle.FORMAT_E4M3),
    "e5m2": oracle.Params(scale_mode=oracle.SCALE_ROUNDUP, elem_format=oracle.FORMAT_E5M2),
    "nvfp4": oracle.Params(block=oracle.BLOCK_1X16, scale_mode=oracle.SCALE_ROUNDUP, tensor_exp=-8),
}


def check_codes(y32, q, s, fmt, layout, what):
    rq, rs = oracle.quantize_rows(y32.cpu().numpy(), FORMATS[fmt])
    rs = oracle.scales_to_mma(rs) if layout else rs
    assert_same([q.cpu().numpy(), s.cpu().numpy()], [rq, rs], what)


# ------------------------------------------------------------------- norm ---

NORM_CASES = [
    # rows, cols, type, weight type, residual, format, layout, extra columns
    (1, 32, BF16, BF16, False, "e4m3", 0, 0),
    (1, 8192, BF16, BF16, True, "e4m3", 0, 0),
    (3, 96, BF16, F32, True, "e2m1", 0, 8),
    (5, 160, F32, BF16, True, "e5m2", 0, 16),
    (7, 1024, BF16, BF16, True, "nvfp4", 0, 0),
    (9, 1056, F32, F32, False, "e4m3floor", 0, 8),
    (128, 128, BF16, None, True, "e4m3", 1, 0),
    (256, 384, F32, F32, True, "nvfp4", 1, 0),
    (129, 2080, BF16, BF16, True, "e4m3", 0, 24),
    (33, 4096, BF16, F32, False, "e5m2", 0, 0),
    (300, 4128, BF16, BF16, True, "e2m1", 0, 0),
    (17, 8224, F32, BF16, True, "e4m3", 0, 0),
    (640, 8192, BF16, BF16, True, "e4m3", 1, 0),
    (4, 16384, BF16, BF16, True, "e4m3", 0, 0),
    (3, 20000, BF16, BF16, True, "e4m3", 0, 0),
    (2, 32768, F32, F32, True, "e4m3", 0, 0),
    (2, 40032, BF16, BF16, True, "e4m3", 0, 0),
    (3, 65536, F32, BF16, False, "nvfp4", 0, 0),
    (2000, 64, BF16, BF16, True, "e4m3", 0, 0),
]


def norm_reference(h, w, eps):
    h64 = h.double()
    rstd = 1.0 / torch.sqrt((h64 * h64).sum(1) / h.shape[1] + eps)
    y = h64 * rstd[:, None]
    return (y if w is None else y * w.double()), rstd


@pytest.mark.parametrize("rows,cols,dt,wdt,res,fmt,layout,extra", NORM_CASES)
def test_norm_forward(rows, cols, dt, wdt, res, fmt, layout, extra):
    import gemm_pt_block_gb300 as mx

    x = strided(rand(rows, cols, dt, 1), extra)
    r = strided(rand(rows, cols, dt, 2, 3.0), 2 * extra) if res else None
    w = None if wdt is None else (1 + 0.2 * torch.randn(cols, device=DEV)).to(wdt)
    p = cuda_params(FORMATS[fmt], layout)
    q, s, y, h, rstd = mx.mxfp4_rmsnorm_quantize(x, w, p, residual=r, eps=1e-5, y_dtype=F32, with_rstd=True)
    want_h = x if r is None else (x.float() + r.float()).to(dt)
    if res:
        assert torch.equal(h, want_h)
    else:
        assert h is None
    ref, ref_rstd = norm_reference(want_h, w, 1e-5)
    tol = (chain(cols) + 1) * U / 2 + 3 * U
    assert ((rstd.double() - ref_rstd).abs() <= tol * ref_rstd).all()
    assert ((y.double() - ref).abs() <= (tol + 2 * U) * ref.abs() + 1e-40).all()
    check_codes(y, q, s, fmt, layout, f"norm {rows}x{cols} {fmt}")
    # y in bf16, and every output asked for by itself: the same values
    _, _, yb, _, _ = mx.mxfp4_rmsnorm_quantize(x, w, residual=r, eps=1e-5, y_dtype=BF16)
    assert torch.equal(yb, y.to(BF16))
    q2, s2, _, _, none = mx.mxfp4_rmsnorm_quantize(x, w, p, residual=r, eps=1e-5)
    assert torch.equal(q2, q) and torch.equal(s2, s) and none is None
    assert mx.device_status() == 0


@pytest.mark.parametrize("rows,cols,dt,layout", [
    (37, 288, BF16, 0), (256, 512, F32, 1), (11, 544, BF16, 0), (19, 640, F32, 0), (128, 768, BF16, 1),
    (200, 1056, BF16, 0), (155, 1280, F32, 0), (153, 2592, BF16, 0), (3, 8224, BF16, 0), (2, 16416, F32, 0),
    (2, 24608, BF16, 0)])
def test_norm_of_rows_that_fill_their_threads_in_part(rows, cols, dt, layout):
    test_norm_forward(rows, cols, dt, BF16, True, "e4m3", layout, 0)


def test_norm_of_many_rows_takes_every_row():
    """More rows than a grid of resident CTAs, every row different."""
    import gemm_pt_block_gb300 as mx

    for rows, cols in ((20011, 128), (5003, 2048), (3001, 8192)):
        x = rand(rows, cols, BF16, 3)
        y = mx.mxfp4_rmsnorm_quantize(x, None, y_dtype=F32)[2]
        ref, _ = norm_reference(x, None, 1e-6)
        assert ((y.double() - ref).abs() <= ((chain(cols) + 1) * U / 2 + 5 * U) * ref.abs() + 1e-40).all()


def test_norm_in_place_and_single_outputs():
    import gemm_pt_block_gb300 as mx

    x, r = rand(37, 2048, BF16, 4), rand(37, 2048, BF16, 5)
    w = torch.randn(2048, device=DEV).to(BF16)
    p = mx.QuantParams(elem_format=mx.FORMAT_E4M3)
    q, s, _, h, rstd = mx.mxfp4_rmsnorm_quantize(x, w, p, residual=r, with_rstd=True)
    for target in (0, 1):
        xc, rc = x.clone(), r.clone()
        dst = (xc, rc)[target]
        q2, s2, _, h2, _ = mx.mxfp4_rmsnorm_quantize(xc, w, p, residual=rc, h=dst)
        assert h2 is dst and torch.equal(dst, h) and torch.equal(q2, q) and torch.equal(s2, s)
    only = mx.mxfp4_rmsnorm_quantize(x, None, residual=r)
    assert torch.equal(only[3], h) and only[0] is None and only[2] is None
    assert torch.equal(mx.mxfp4_rmsnorm_quantize(x, None, residual=r, with_rstd=True)[4], rstd)
    empty = mx.mxfp4_rmsnorm_quantize(x[:0], w, p, residual=r[:0], with_rstd=True)
    assert empty[0].shape == (0, 2048) and empty[3].shape == (0, 2048) and empty[4].shape == (0,)


def test_norm_of_zero_rows_tiny_values_and_non_finite_values():
    import gemm_pt_block_gb300 as mx

    x = rand(8, 256, BF16, 6)
    x[1] = 0.0                                           # a row of zeros: y = 0, smallest scale
    x[2] = 1e-30                                         # below eps: y = h w / sqrt(eps)
    x[3, 5] = float("inf")
    x[4, 6] = float("nan")
    x[5, 7] = -float("inf")
    p = mx.QuantParams(scale_mode=mx.SCALE_ROUNDUP, elem_format=mx.FORMAT_E4M3)
    q, s, y, _, rstd = mx.mxfp4_rmsnorm_quantize(x, None, p, y_dtype=F32, with_rstd=True, eps=1e-6)
    assert (q[1] == 0).all() and (s[1] == 0).all() and (y[1] == 0).all()
    fine = [0, 1, 2, 6, 7]
    rq, rs = oracle.quantize_rows(y[fine].cpu().numpy(), FORMATS["e4m3"])
    assert np.array_equal(q[fine].cpu().numpy(), rq) and np.array_equal(s[fine].cpu().numpy(), rs)
    assert torch.isnan(rstd[4]) and (s[4] == 255).all() and (q[4] == 0).all()
    # an infinity makes rstd 0: inf * 0 is NaN in its own block, the others are 0
    for r, c in ((3, 5), (5, 7)):
        assert rstd[r] == 0 and s[r, c // 32] == 255 and (s[r, 1:] == 0).all()
    d = mx.mxfp4_dequantize(q, s, 8, 256, params=p)
    assert torch.isnan(d[4]).all() and torch.isnan(d[3, :32]).all() and (d[3, 32:] == 0).all()
    pn = mx.QuantParams(block=mx.BLOCK_1X16, scale_mode=mx.SCALE_ROUNDUP)
    qn, sn, _, _, _ = mx.mxfp4_rmsnorm_quantize(x, None, pn)
    assert (sn[4] == 0x7F).all() and (qn[4] == 0).all() and sn[3, 0] == 0x7F and (sn[3, 1:] == 0).all()


GRAD_CASES = [
    # rows, cols, type of h, of dy, of w, stream gradient, extra columns
    (1, 32, BF16, BF16, BF16, True, 0),
    (1, 8192, BF16, BF16, BF16, False, 0),
    (5, 96, F32, BF16, F32, True, 8),
    (70, 256, BF16, F32, F32, False, 16),
    (2000, 64, BF16, BF16, F32, True, 0),
    (1001, 1024, F32, F32, F32, True, 0),
    (777, 4096, BF16, BF16, F32, True, 24),
    (400, 4128, BF16, BF16, BF16, False, 0),
    (650, 8192, BF16, BF16, F32, True, 0),
    (31, 16384, F32, F32, BF16, True, 0),
    (5, 20000, BF16, BF16, F32, True, 0),
    (9, 32768, BF16, F32, F32, True, 0),
    (3, 40032, F32, F32, F32, True, 0),
]


def norm_grad_reference(dy, h, w, rstd, dh):
    d, h, r = dy.double(), h.double(), rstd.double()[:, None]
    n, dn = h * r, d * (1.0 if w is None else w.double())
    mean = (dn * n).sum(1, keepdim=True) / h.shape[1]
    dx = (dn - n * mean) * r
    mag = (dn.abs() + n.abs() * (dn * n).abs().sum(1, keepdim=True) / h.shape[1]) * r
    if dh is not None:
        dx, mag = dx + dh.double(), mag + dh.double().abs()
    return dx, mag, (d * n).sum(0), (d * n).abs().sum(0)


@pytest.mark.parametrize("rows,cols,dt,gdt,wdt,stream,extra", GRAD_CASES)
def test_norm_backward(rows, cols, dt, gdt, wdt, stream, extra):
    import gemm_pt_block_gb300 as mx

    h = strided(rand(rows, cols, dt, 11), extra)
    dy = strided(rand(rows, cols, gdt, 12, 1e-2), 2 * extra)
    dh = strided(rand(rows, cols, dt, 13, 1e-2), extra) if stream else None
    w = (1 + 0.2 * torch.randn(cols, device=DEV)).to(wdt)
    rstd = mx.mxfp4_rmsnorm_quantize(h, None, with_rstd=True)[4]
    dx, dw = mx.mxfp4_rmsnorm_backward(dy, h, w, rstd, dh=dh)
    ref, mag, refw, magw = norm_grad_reference(dy, h, w, rstd, dh)
    tol = (chain(cols) + 12) * U
    assert ((dx.double() - ref).abs() <= tol * mag + half_ulp(dt) * (ref.abs() + tol * mag)).all()
    # dw: at most rows additions in a chain, three roundings in each term
    tolw = (rows + 4) * U
    assert ((dw.double() - refw).abs() <= tolw * magw + half_ulp(wdt) * (refw.abs() + tolw * magw)).all()
    dx2, dw2 = mx.mxfp4_rmsnorm_backward(dy, h, w, rstd, dh=dh)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)          # a fixed order of sums
    if dh is not None:                                            # in place of the stream's gradient
        buf = dh.clone()
        dx3, _ = mx.mxfp4_rmsnorm_backward(dy, h, w, rstd, dh=buf, dx=buf)
        assert dx3 is buf and torch.equal(buf, dx)
    dx4, none = mx.mxfp4_rmsnorm_backward(dy, h, w, rstd, dh=dh, with_dw=False)
    assert none is None and torch.equal(dx4, dx)
    dx5, none = mx.mxfp4_rmsnorm_backward(dy, h, None, rstd, dh=dh)
    ref, mag, _, _ = norm_grad_reference(dy, h, None, rstd, dh)
    assert none is None
    assert ((dx5.double() - ref).abs() <= tol * mag + half_ulp(dt) * (ref.abs() + tol * mag)).all()
    assert mx.device_status() == 0


@pytest.mark.parametrize("rows,cols,dt", [
    (1825, 544, BF16), (40000, 1024, BF16), (151, 1024, F32), (153, 4096, BF16), (304, 2080, F32), (305, 8192, BF16),
    (1300, 8192, BF16), (700, 8192, F32), (700, 16384, BF16)])
def test_norm_backward_of_row_counts_around_the_sms_and_their_groups(rows, cols, dt):
    """Each row's dx has the same bits alone and among others, whichever group
    of threads and slot of its ring takes it; dw is the sum over all rows."""
    import gemm_pt_block_gb300 as mx

    h, dy, dh = rand(rows, cols, dt, 31), rand(rows, cols, dt, 32, 1e-2), rand(rows, cols, dt, 33, 1e-2)
    w = (1 + 0.2 * torch.randn(cols, device=DEV)).to(dt)
    rstd = mx.mxfp4_rmsnorm_quantize(h, None, with_rstd=True)[4]
    dx, dw = mx.mxfp4_rmsnorm_backward(dy, h, w, rstd, dh=dh)
    for lo in range(0, rows, 100):
        hi = min(lo + 100, rows)
        part, _ = mx.mxfp4_rmsnorm_backward(dy[lo:hi], h[lo:hi], w, rstd[lo:hi], dh=dh[lo:hi])
        assert torch.equal(part, dx[lo:hi])
    _, _, refw, magw = norm_grad_reference(dy, h, w, rstd, None)
    tolw = (rows + 4) * U
    assert ((dw.double() - refw).abs() <= tolw * magw + half_ulp(dt) * (refw.abs() + tolw * magw)).all()
    assert mx.device_status() == 0


def test_norm_backward_of_no_rows():
    import gemm_pt_block_gb300 as mx

    w = torch.ones(96, device=DEV)
    z = torch.empty((0, 96), device=DEV)
    dx, dw = mx.mxfp4_rmsnorm_backward(z, z, w, torch.empty(0, device=DEV))
    assert dx.shape == (0, 96) and (dw == 0).all()


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("cols", [96, 512, 1056, 4096, 20000])
def test_matrices_on_any_16_bytes(cols, dt):
    """Inputs and outputs 16 bytes past a 32-byte boundary: the same bits."""
    import gemm_pt_block_gb300 as mx

    rows, at = 9, 16 // (2 if dt == BF16 else 4)

    def moved(t):
        buf = torch.empty(t.numel() + at, dtype=t.dtype, device=DEV)
        assert buf.data_ptr() % 32 == 0
        v = buf[at:].view(t.shape)
        return v.copy_(t)

    x, r, g = rand(rows, cols, dt, 71), rand(rows, cols, dt, 72), rand(rows, cols, dt, 73, 1e-2)
    w = (1 + 0.2 * torch.randn(cols, device=DEV)).to(dt)
    p = mx.QuantParams(elem_format=mx.FORMAT_E4M3)
    q, s, y, h, rstd = mx.mxfp4_rmsnorm_quantize(x, w, p, residual=r, y_dtype=dt, with_rstd=True)
    hm, ym = moved(torch.zeros_like(x)), moved(torch.zeros_like(x))
    q2, s2, _, _, rstd2 = mx.mxfp4_rmsnorm_quantize(moved(x), w, p, residual=moved(r), h=hm, y=ym, with_rstd=True)
    assert torch.equal(q, q2) and torch.equal(s, s2) and torch.equal(rstd, rstd2)
    assert torch.equal(hm, h) and torch.equal(ym, y)
    dx, dw = mx.mxfp4_rmsnorm_backward(g, h, w, rstd, dh=r)
    dxm = moved(torch.zeros_like(x))
    _, dw2 = mx.mxfp4_rmsnorm_backward(moved(g), moved(h), w, rstd, dh=moved(r), dx=dxm)
    assert torch.equal(dx, dxm) and torch.equal(dw, dw2)
    q, s, y = mx.mxfp4_swiglu_quantize(x, r, p, y_dtype=dt)
    q2, s2, _ = mx.mxfp4_swiglu_quantize(moved(x), moved(r), p, y=ym)
    assert torch.equal(q, q2) and torch.equal(s, s2) and torch.equal(y, ym)
    dg, du = mx.mxfp4_swiglu_backward(g, x, r)
    dgm, dum = moved(torch.zeros_like(x)), moved(torch.zeros_like(x))
    mx.mxfp4_swiglu_backward(moved(g), moved(x), moved(r), dgate=dgm, dup=dum)
    assert torch.equal(dg, dgm) and torch.equal(du, dum)
    assert mx.device_status() == 0


def test_gradients_match_differences_of_the_forward_kernels():
    """Central differences of the fp32 forward kernels along random directions.

    L(t) = sum dy y(p + t v) with |t| = 2^-7: the third derivative's term is
    t^2 / 6 = 1e-5 of comparable size; the fp32 roundings of y enter as
    sqrt(n) u |y dy| / t, below 2e-5 of |grad||v| here. 1e-3 holds both."""
    import gemm_pt_block_gb300 as mx

    rows, cols, t = 24, 512, 2.0 ** -7
    g = torch.Generator(device=DEV).manual_seed(5)

    def rnd(*shape):
        return torch.randn(shape, device=DEV, generator=g)

    x, w, dy = rnd(rows, cols), 1 + 0.3 * rnd(cols), rnd(rows, cols)

    def norm_loss(a, b):
        return (mx.mxfp4_rmsnorm_quantize(a, b, y_dtype=F32)[2].double() * dy.double()).sum()

    rstd = mx.mxfp4_rmsnorm_quantize(x, w, with_rstd=True)[4]
    dx, dw = mx.mxfp4_rmsnorm_backward(dy, x, w, rstd)
    vx, vw = rnd(rows, cols), rnd(cols)
    for grad, v, lo, hi in ((dx, vx, norm_loss(x - t * vx, w), norm_loss(x + t * vx, w)),
                            (dw, vw, norm_loss(x, w - t * vw), norm_loss(x, w + t * vw))):
        want = (hi - lo) / (2 * t)
        got = (grad.double() * v.double()).sum()
        assert abs(got - want) <= 1e-3 * grad.double().norm() * v.double().norm()

    gate, up = 2 * rnd(rows, cols), rnd(rows, cols)

    def act_loss(a, b):
        return (mx.mxfp4_swiglu_quantize(a, b, y_dtype=F32)[2].double() * dy.double()).sum()

    dg, du = mx.mxfp4_swiglu_backward(dy, gate, up)
    for grad, v, lo, hi in ((dg, vx, act_loss(gate - t * vx, up), act_loss(gate + t * vx, up)),
                            (du, vx, act_loss(gate, up - t * vx), act_loss(gate, up + t * vx))):
        want = (hi - lo) / (2 * t)
        got = (grad.double() * v.double()).sum()
        assert abs(got - want) <= 1e-3 * grad.double().norm() * v.double().norm()


# ----------------------------------------------------------------- SwiGLU ---

ACT_CASES = [
    (1, 32, BF16, "e4m3", 0, 0),
    (1, 28672, BF16, "e4m3", 0, 0),
    (3, 96, F32, "e2m1", 0, 8),
    (8, 14336, BF16, "e4m3", 0, 0),
    (65, 160, BF16, "nvfp4", 0, 16),
    (128, 256, BF16, "e4m3", 1, 0),
    (384, 1152, F32, "nvfp4", 1, 8),
    (1000, 2080, BF16, "e5m2", 0, 24),
    (33, 8192, BF16, "e4m3floor", 0, 0),
    (20011, 64, BF16, "e4m3", 0, 0),
]


@pytest.mark.parametrize("rows,cols,dt,fmt,layout,extra", ACT_CASES)
def test_swiglu(rows, cols, dt, fmt, layout, extra):
    import gemm_pt_block_gb300 as mx

    both = strided(rand(rows, 2 * cols, dt, 21, 2.0), extra)
    gate, up = both[:, :cols], both[:, cols:]
    p = cuda_params(FORMATS[fmt], layout)
    q, s, y = mx.mxfp4_swiglu_quantize(gate, up, p, y_dtype=F32)
    g64, u64 = gate.double(), up.double()
    ref = g64 / (1 + torch.exp(-g64)) * u64
    assert ((y.double() - ref).abs() <= 16 * U * ref.abs() + 1e-37).all()
    check_codes(y, q, s, fmt, layout, f"swiglu {rows}x{cols} {fmt}")
    assert torch.equal(mx.mxfp4_swiglu_quantize(gate, up, y_dtype=BF16)[2], y.to(BF16))
    q2, s2, none = mx.mxfp4_swiglu_quantize(gate, up, p)
    assert none is None and torch.equal(q2, q) and torch.equal(s2, s)

    # gradients: t within 4 ulp, 1 - t rounded once more, up to seven products and sums; 1 - t
    # and 1 + g (1 - t) may cancel, so the bound is over the terms' magnitudes
    for gdt in (BF16, F32):
        dy = strided(rand(rows, cols, gdt, 22, 1e-2), extra)
        dg, du = mx.mxfp4_swiglu_backward(dy, gate, up)
        d64, t64 = dy.double(), 1 / (1 + torch.exp(-g64))
        rg, ru = d64 * u64 * t64 * (1 + g64 * (1 - t64)), d64 * g64 * t64
        mg = (d64 * u64 * t64).abs() * (1 + g64.abs())
        assert ((dg.double() - rg).abs() <= 24 * U * mg + half_ulp(dt) * (rg.abs() + 24 * U * mg) + 1e-37).all()
        assert ((du.double() - ru).abs() <= (16 * U + half_ulp(dt) * (1 + 16 * U)) * ru.abs() + 1e-37).all()
    # in place of the inputs
    buf = both.clone()
    mx.mxfp4_swiglu_backward(dy, buf[:, :cols], buf[:, cols:], dgate=buf[:, :cols], dup=buf[:, cols:])
    assert torch.equal(buf, torch.cat((dg, du), 1))
    assert mx.device_status() == 0


@pytest.mark.parametrize("rows,cols,dt,fmt,layout", [
    (70, 1056, BF16, "e4m3", 0), (256, 4480, BF16, "e4m3", 1), (128, 1152, BF16, "nvfp4", 1), (37, 544, F32, "nvfp4", 0),
    (300, 2336, BF16, "e2m1", 0), (9, 5440, F32, "e5m2", 0), (128, 640, F32, "e4m3floor", 1), (41, 8352, BF16, "nvfp4", 0)])
def test_swiglu_of_rows_in_parts(rows, cols, dt, fmt, layout):
    """Rows whose threads come in parts of 8, 16 and whole warps."""
    test_swiglu(rows, cols, dt, fmt, layout, 0)


def test_swiglu_of_large_and_non_finite_values():
    import gemm_pt_block_gb300 as mx

    gate = torch.zeros((4, 64), device=DEV)
    up = torch.ones((4, 64), device=DEV)
    gate[0] = torch.linspace(-104.0, 104.0, 64, device=DEV)       # the exponential's whole range
    gate[1] = -1e30                                               # no overflow on the way to -0
    gate[2] = 3e38
    gate[3, 3], up[3, 40] = float("nan"), float("inf")
    gate[3, 40] = 1.0
    p = mx.QuantParams(scale_mode=mx.SCALE_ROUNDUP, elem_format=mx.FORMAT_E4M3)
    q, s, y = mx.mxfp4_swiglu_quantize(gate, up, p, y_dtype=F32)
    ref = gate[0].double() / (1 + torch.exp(-gate[0].double()))
    # below 2^-126 fp32 is subnormal: absolute bound there
    assert ((y[0].double() - ref).abs() <= 16 * U * ref.abs() + 2.0 ** -126).all()
    assert (y[1] == 0).all() and (y[2] == 3e38).all()
    assert torch.isnan(y[3, 3]) and torch.isinf(y[3, 40])
    assert (s[3] == 255).all() and (q[3] == 0).all()
    dg, du = mx.mxfp4_swiglu_backward(up, gate, up)
    assert torch.isfinite(dg[:3]).all() and torch.isfinite(du[:3]).all()
    assert (dg[1] == 0).all() and (dg[2] == 1).all()
    e = mx.mxfp4_swiglu_quantize(gate[:0], up[:0], p, y_dtype=F32)
    assert e[0].shape == (0, 64) and e[2].shape == (0, 64)


# ------------------------------------------- strides, streams, guard bytes ---

@pytest.mark.parametrize("rows,cols", [(5, 96), (130, 2080)])
def test_outputs_stay_inside_their_buffers(rows, cols):
    import gemm_pt_block_gb300 as mx

    ld = cols + 24
    es = 2
    spans = [(r * ld * es, (r * ld + cols) * es) for r in range(rows)]
    a = Arena([rows * ld * es] * 2 + [rows * cols, rows * cols // 32, rows * 4] + [rows * ld * es] * 3 + [cols * 4])
    mats = [a.region(i, BF16, (rows, ld), spans)[:, :cols] for i in (0, 1, 5, 6, 7)]
    q = a.region(2, torch.uint8, (rows, cols))
    s = a.region(3, torch.uint8, (rows, cols // 32))
    rstd = a.region(4, F32, (rows,))
    dw = a.region(8, F32, (cols,))
    x, r = rand(rows, cols, BF16, 31), rand(rows, cols, BF16, 32)
    w = torch.ones(cols, device=DEV)
    p = mx.QuantParams(elem_format=mx.FORMAT_E4M3)
    mx.mxfp4_rmsnorm_quantize(x, w, p, residual=r, h=mats[0], y=mats[1], rstd=rstd, q=q, s=s)
    mx.mxfp4_rmsnorm_backward(r, mats[0], w, rstd, dx=mats[2], dw=dw)
    mx.mxfp4_swiglu_quantize(x, r, p, q=q, s=s, y=mats[1])
    mx.mxfp4_swiglu_backward(x, x, r, dgate=mats[3], dup=mats[4])
    a.check(f"norm and activation {rows}x{cols}")


def test_calls_run_on_the_given_stream():
    import gemm_pt_block_gb300 as mx

    side = torch.cuda.Stream()
    p = mx.QuantParams(elem_format=mx.FORMAT_E4M3)
    x, r = rand(512, 4096, BF16, 41), rand(512, 4096, BF16, 42)
    w = torch.ones(4096, device=DEV)
    want = mx.mxfp4_rmsnorm_quantize(x, w, p, residual=r, with_rstd=True)
    gwant = mx.mxfp4_rmsnorm_backward(x, want[3], w, want[4])
    torch.cuda.synchronize()
    for _ in range(3):
        src = torch.empty_like(x)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)
            src.copy_(x)
        got = mx.mxfp4_rmsnorm_quantize(src, w, p, residual=r, with_rstd=True, stream=side)
        ggot = mx.mxfp4_rmsnorm_backward(src, got[3], w, got[4], stream=side)
        side.synchronize()
        for g, v in zip(got[:2] + got[3:] + ggot, want[:2] + want[3:] + gwant):
            assert torch.equal(g, v)


def test_refusals():
    import gemm_pt_block_gb300 as mx

    x = rand(8, 128, BF16, 51)
    w = torch.ones(128, device=DEV)
    p = mx.QuantParams(elem_format=mx.FORMAT_E4M3)
    rs = torch.ones(8, device=DEV)
    bad = [
        (TypeError, lambda: mx.mxfp4_rmsnorm_quantize(x.half(), w, p)),
        (TypeError, lambda: mx.mxfp4_rmsnorm_quantize(x, w, p, residual=x.float())),
        (TypeError, lambda: mx.mxfp4_rmsnorm_quantize(x, w.half(), p)),
        (TypeError, lambda: mx.mxfp4_rmsnorm_quantize(x, w, p, h=x.float())),
        (ValueError, lambda: mx.mxfp4_rmsnorm_quantize(x, w[:64], p)),
        (ValueError, lambda: mx.mxfp4_rmsnorm_quantize(x, w, p, residual=x[:4])),
        (ValueError, lambda: mx.mxfp4_rmsnorm_quantize(x.cpu(), w, p)),
        (ValueError, lambda: mx.mxfp4_rmsnorm_quantize(x, w.cpu(), p)),
        (ValueError, lambda: mx.mxfp4_rmsnorm_quantize(x.t(), None, p)),
        (ValueError, lambda: mx.mxfp4_rmsnorm_quantize(x, w, p, q=torch.empty(8, dtype=torch.uint8, device=DEV))),
        (ValueError, lambda: mx.mxfp4_rmsnorm_quantize(x, w, p, rstd=rs[:4])),
        (mx.Mxfp4Error, lambda: mx.mxfp4_rmsnorm_quantize(x, w)),                          # no output
        (mx.Mxfp4Error, lambda: mx.mxfp4_rmsnorm_quantize(x[:, :48].contiguous(), None, y_dtype=F32)),
        (mx.Mxfp4Error, lambda: mx.mxfp4_rmsnorm_quantize(x[:, 4:100], None, y_dtype=F32)),  # 8 bytes off
        (mx.Mxfp4Error, lambda: mx.mxfp4_rmsnorm_quantize(x, w, p, eps=float("nan"))),
        (mx.Mxfp4Error, lambda: mx.mxfp4_rmsnorm_quantize(x, w, p, eps=-1.0)),
        (mx.Mxfp4Error, lambda: mx.mxfp4_rmsnorm_quantize(x, w, mx.QuantParams(rounding=mx.ROUND_SR))),
        (mx.Mxfp4Error, lambda: mx.mxfp4_rmsnorm_quantize(x, w, mx.QuantParams(wht=True))),
        (mx.Mxfp4Error, lambda: mx.mxfp4_rmsnorm_quantize(x, w, mx.QuantParams(block=mx.BLOCK_32X32))),
        (mx.Mxfp4Error, lambda: mx.mxfp4_rmsnorm_quantize(x, w, mx.QuantParams(scale_layout=mx.LAYOUT_MMA))),
        (ValueError, lambda: mx.mxfp4_rmsnorm_backward(x[:4], x, w, rs)),
        (ValueError, lambda: mx.mxfp4_rmsnorm_backward(x, x, w, rs[:4])),
        (ValueError, lambda: mx.mxfp4_rmsnorm_backward(x, x, None, rs, dw=torch.empty(128, device=DEV))),
        (ValueError, lambda: mx.mxfp4_rmsnorm_backward(x, x, w, rs, workspace=torch.empty(8, dtype=torch.uint8, device=DEV))),
        (TypeError, lambda: mx.mxfp4_rmsnorm_backward(x, x, w, rs, dh=x.float())),
        (TypeError, lambda: mx.mxfp4_rmsnorm_backward(x, x, w, rs, dx=x.float())),
        (TypeError, lambda: mx.mxfp4_rmsnorm_backward(x, x, w, rs.double())),
        (TypeError, lambda: mx.mxfp4_swiglu_quantize(x, x.float(), p)),
        (ValueError, lambda: mx.mxfp4_swiglu_quantize(x, x[:, :64], p)),
        (mx.Mxfp4Error, lambda: mx.mxfp4_swiglu_quantize(x, x)),
        (mx.Mxfp4Error, lambda: mx.mxfp4_swiglu_quantize(x, x, mx.QuantParams(block=mx.BLOCK_64X64))),
        (TypeError, lambda: mx.mxfp4_swiglu_backward(x, x, x, dgate=x.float())),
        (ValueError, lambda: mx.mxfp4_swiglu_backward(x[:2], x, x)),
    ]
    for i, (err, call) in enumerate(bad):
        with pytest.raises(err):
            call()
            raise AssertionError(f"refusal {i} did not raise")
    assert mx.device_status() == 0
