"""Few-row products with 4-bit weights against 64-bit sums.

The products are exact in fp32 and summed in fp32, so the error bound is the
block-scaled GEMM's: |err| <= 1e-5 sum_k |x_k w_k|, plus bf16's half unit
where y is bf16. Weights, activations and scales are drawn as codes, so the
reference dequantizes them exactly.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from _util import gemm_tolerance_check, gemm_tolerance_check_bf16
from test_gpu_canary import Arena

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def weights(N, K, nv, seed, lo=110, hi=135):
    """Random codes and scales, and their values in 64 bits."""
    g = gen(seed)
    q = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=DEV, generator=g)
    per = 16 if nv else 32
    if nv:
        s = torch.randint(0, 127, (N, K // per), dtype=torch.uint8, device=DEV, generator=g)
        f = s.view(torch.float8_e4m3fn).double()
    else:
        s = torch.randint(lo, hi, (N, K // per), dtype=torch.uint8, device=DEV, generator=g)
        f = torch.exp2(s.double() - 127)
    v = E2M1.to(DEV)[torch.stack((q & 15, q >> 4), -1).view(N, K).long()]
    return q, s, v * f.repeat_interleave(per, 1)


def activations(M, K, kind, seed):
    """(x, sx, values in 64 bits, keyword arguments of the call)"""
    import gemm_pt_block_gb300 as mx

    g = gen(seed)
    if kind == "bf16":
        x = torch.randn((M, K), device=DEV, generator=g)
        if K >= 64:
            x[:, 40] *= 1000.0
        x = x.to(BF16)
        return x, None, x.double(), {}
    fmt = torch.float8_e4m3fn if kind == "e4m3" else torch.float8_e5m2
    x = (torch.randn((M, K), device=DEV, generator=g) * 30).to(fmt)
    sx = torch.randint(115, 130, (M, K // 32), dtype=torch.uint8, device=DEV, generator=g)
    val = x.double() * torch.exp2(sx.double() - 127).repeat_interleave(32, 1)
    return (x.view(torch.uint8), sx, val,
            {"sx": sx, "x_format": mx.FORMAT_E4M3 if kind == "e4m3" else mx.FORMAT_E5M2})


def check(y, x64, w64, what=""):
    ref, mag = (x64 @ w64.t()).cpu().numpy(), (x64.abs() @ w64.abs().t()).cpu().numpy()
    got = y.float().cpu().numpy()
    if y.dtype == F32:
        gemm_tolerance_check(got, ref, mag)
    else:
        gemm_tolerance_check_bf16(got.astype(np.float64), ref, mag)


def wparams(nv, layout=0, tensor_exp=0):
    import gemm_pt_block_gb300 as mx

    return mx.QuantParams(mx.BLOCK_1X16 if nv else mx.BLOCK_1X32, scale_layout=layout, tensor_exp=tensor_exp)


SHAPES = [(1, 1, 32), (1, 7, 64), (2, 16, 96), (3, 130, 160), (1, 1000, 1024), (4, 129, 4096), (5, 257, 288),
          (8, 300, 8192), (9, 64, 544), (13, 1000, 2080), (16, 513, 1024), (17, 96, 4128), (24, 200, 512),
          (31, 333, 800), (32, 1024, 1024), (33, 128, 256), (70, 65, 320), (1, 40, 28672), (130, 17, 64)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("nv", [False, True], ids=["mxfp4", "nvfp4"])
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e5m2"])
def test_row_major_scales(M, N, K, nv, kind):
    import gemm_pt_block_gb300 as mx

    q, s, w64 = weights(N, K, nv, 1)
    x, _, x64, kw = activations(M, K, kind, 2)
    y = mx.mxfp4_gemv(x, q, s, N, K, wparams(nv), out_dtype=F32, **kw)
    check(y, x64, w64)
    yb = mx.mxfp4_gemv(x, q, s, N, K, wparams(nv), **kw)
    assert yb.dtype == BF16 and torch.equal(yb, y.to(BF16))
    assert torch.equal(mx.mxfp4_gemv(x, q, s, N, K, wparams(nv), out_dtype=F32, **kw), y)
    assert mx.device_status() == 0


@pytest.mark.parametrize("M,N,K", [(1, 128, 128), (3, 256, 384), (8, 384, 4096), (20, 1024, 640), (32, 128, 8192),
                                   (2, 4096, 256)])
@pytest.mark.parametrize("nv", [False, True], ids=["mxfp4", "nvfp4"])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_tensor_core_scales(M, N, K, nv, kind):
    import gemm_pt_block_gb300 as mx

    q, s, w64 = weights(N, K, nv, 3)
    x, _, x64, kw = activations(M, K, kind, 4)
    tiles = torch.from_numpy(oracle.scales_to_mma(s.cpu().numpy())).to(DEV)
    y = mx.mxfp4_gemv(x, q, tiles, N, K, wparams(nv, 1), out_dtype=F32, **kw)
    check(y, x64, w64)
    assert torch.equal(y, mx.mxfp4_gemv(x, q, s, N, K, wparams(nv), out_dtype=F32, **kw))


WORKSPACE_SHAPES = [(1, 1, 128), (1, 130, 256), (2, 128, 1024), (5, 1000, 128), (7, 257, 2176), (10, 64, 640),
                    (16, 300, 384), (17, 129, 4096), (21, 513, 1152), (22, 128, 256), (32, 1024, 1024), (33, 96, 512),
                    (64, 200, 256), (65, 128, 896), (130, 65, 384), (9, 40, 96), (31, 200, 800), (40, 128, 224)]


@pytest.mark.parametrize("M,N,K", WORKSPACE_SHAPES)
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e5m2"])
@pytest.mark.parametrize("nv", [False, True], ids=["mxfp4", "nvfp4"])
@pytest.mark.parametrize("layout", [0, 1], ids=["rows", "tiles"])
def test_with_a_workspace(M, N, K, kind, nv, layout):
    import gemm_pt_block_gb300 as mx

    if layout and (N % 128 or K % 128):
        pytest.skip("the tensor-core layout has whole tiles")
    need = mx.lib().mxfp4_gemv_workspace_size({"bf16": 0, "e4m3": 1, "e5m2": 2}[kind], 3 if nv else 0, M, N, K)
    if not need:
        pytest.skip("no workspace would be used")
    q, s, w64 = weights(N, K, nv, 27)
    x, _, x64, kw = activations(M, K, kind, 28)
    sw = torch.from_numpy(oracle.scales_to_mma(s.cpu().numpy())).to(DEV) if layout else s
    a = Arena([need, M * N * 4])
    ws, y = a.region(0, torch.uint8, (need,)), a.region(1, F32, (M, N))
    mx.mxfp4_gemv(x, q, sw, N, K, wparams(nv, layout), y=y, workspace=ws, **kw)
    check(y, x64, w64)
    a.check(f"gemv {M}x{N}x{K} with a workspace")
    first = y.clone()
    y.fill_(7.0)
    ws.fill_(0xFF)                                          # nothing of it is kept from call to call
    mx.mxfp4_gemv(x, q, sw, N, K, wparams(nv, layout), y=y, workspace=ws, **kw)
    assert torch.equal(y, first)
    # one byte short: not used
    mx.mxfp4_gemv(x, q, sw, N, K, wparams(nv, layout), y=y, workspace=ws[:need - 1], **kw)
    assert torch.equal(y, mx.mxfp4_gemv(x, q, sw, N, K, wparams(nv, layout), out_dtype=F32, workspace=False, **kw))
    assert mx.device_status() == 0


def test_workspace_non_finite_rows_scales_and_zero_rows():
    import gemm_pt_block_gb300 as mx

    M, N, K = 12, 200, 512
    for nv in (False, True):
        q, s, w64 = weights(N, K, nv, 29)
        x, _, x64, _ = activations(M, K, "bf16", 30)
        x = x.clone()
        x[1, 40], x[2, 41], x[3] = float("inf"), float("nan"), 0.0
        x[4] = x[4] * 2.0 ** -100
        x[5] = (x[5].float() * 2.0 ** 100).to(BF16)
        s[7, 2] = 0x7F if nv else 255
        need = mx.lib().mxfp4_gemv_workspace_size(0, 3 if nv else 0, M, N, K)
        assert need > 0
        ws = torch.empty(need, dtype=torch.uint8, device=DEV)
        y = mx.mxfp4_gemv(x, q, s, N, K, wparams(nv), out_dtype=F32, workspace=ws)
        fine = [m for m in range(M) if m not in (1, 2)]
        cols = [n for n in range(N) if n != 7]
        assert torch.isnan(y[:, 7]).all() and torch.isnan(y[2]).all() and not torch.isfinite(y[1]).any()
        check(y[fine][:, cols], x[fine].double(), w64[cols])
        assert (y[3][cols] == 0).all()


@pytest.mark.parametrize("block", ["1x32", "32x32", "64x64", "1x16"])
def test_weights_of_the_quantizer(block):
    """The codes and scales that the training products use, as they are."""
    import gemm_pt_block_gb300 as mx

    N, K, M = 256, 512, 5
    w = (torch.randn((N, K), device=DEV, generator=gen(5)) * 0.02).to(BF16)
    b = {"1x32": mx.BLOCK_1X32, "32x32": mx.BLOCK_32X32, "64x64": mx.BLOCK_64X64, "1x16": mx.BLOCK_1X16}[block]
    p = mx.QuantParams(b, mx.SCALE_ROUNDUP, scale_layout=mx.LAYOUT_MMA, tensor_exp=-12 if block == "1x16" else 0)
    q, s, _, _ = mx.mxfp4_quantize(w, p)
    w64 = mx.mxfp4_dequantize(q, s, N, K, params=p).double()
    x, _, x64, _ = activations(M, K, "bf16", 6)
    check(mx.mxfp4_gemv(x, q, s, N, K, p, out_dtype=F32), x64, w64)


def test_scales_over_their_whole_range():
    """Scales from 2^-127 up, x of every size that bf16 has: nothing is lost on
    the way that the 64-bit sum keeps and fp32 can hold."""
    import gemm_pt_block_gb300 as mx

    N, K = 96, 512
    q, s, w64 = weights(N, K, False, 7, 0, 100)
    s[:, :4] = 0
    _, _, _ = q, s, w64
    v = E2M1.to(DEV)[torch.stack((q & 15, q >> 4), -1).view(N, K).long()]
    w64 = v * torch.exp2(s.double() - 127).repeat_interleave(32, 1)
    e = torch.randint(-60, 100, (4, K // 32), device=DEV, generator=gen(8)).double()
    x = (torch.randn((4, K), device=DEV, generator=gen(9)).double() * torch.exp2(e).repeat_interleave(32, 1)).to(BF16)
    y = mx.mxfp4_gemv(x, q, s, N, K, wparams(False), out_dtype=F32)
    check(y, x.double(), w64)
    # within one block: elements 2^20 below their block's largest still count exactly
    x = torch.zeros((1, K), device=DEV, dtype=BF16)
    x[0, 0] = 2.0 ** 20
    x[0, 1:32] = 1.375
    q[:, 0] &= 0xF0                                        # the large element meets a zero weight
    s[:] = 127
    v = E2M1.to(DEV)[torch.stack((q & 15, q >> 4), -1).view(N, K).long()]
    y = mx.mxfp4_gemv(x, q, s, N, K, wparams(False), out_dtype=F32)
    assert torch.equal(y.double(), x.double() @ v.t())     # few bits: every sum is exact


def test_non_finite_values_stay_in_their_rows():
    import gemm_pt_block_gb300 as mx

    M, N, K = 4, 48, 256
    q, s, w64 = weights(N, K, False, 10)
    q[:, 20] = 0x22                                        # weight 1.0 (codes 40, 41) everywhere
    x, _, x64, _ = activations(M, K, "bf16", 11)
    x = x.clone()
    x[1, 40], x[2, 41] = float("inf"), float("nan")
    y = mx.mxfp4_gemv(x, q, s, N, K, wparams(False), out_dtype=F32)
    w64 = E2M1.to(DEV)[torch.stack((q & 15, q >> 4), -1).view(N, K).long()] * torch.exp2(
        s.double() - 127).repeat_interleave(32, 1)
    keep = [0, 3]
    check(y[keep], x[keep].double(), w64)
    assert (y[1] == float("inf")).all() and torch.isnan(y[2]).all()
    # NaN scales: of one weight block, and of one activation block
    s2 = s.clone()
    s2[5, 3] = 255
    y2 = mx.mxfp4_gemv(x[keep], q, s2, N, K, wparams(False), out_dtype=F32)
    assert torch.isnan(y2[:, 5]).all() and torch.equal(y2[:, :5], y[keep][:, :5]) and torch.equal(y2[:, 6:], y[keep][:, 6:])
    c, sx, _, kw = activations(M, K, "e4m3", 12)
    sx[2, 1] = 255
    y3 = mx.mxfp4_gemv(c, q, s, N, K, wparams(False), **kw)
    assert torch.isnan(y3[2]).all() and torch.isfinite(y3[[0, 1, 3]]).all()
    qn, sn, _ = weights(N, K, True, 13)
    sn[7, 2] = 0x7F
    y4 = mx.mxfp4_gemv(x[keep], qn, sn, N, K, wparams(True))
    assert torch.isnan(y4[:, 7]).all() and torch.isfinite(y4[:, :7]).all() and torch.isfinite(y4[:, 8:]).all()


@pytest.mark.parametrize("M,N,K", [(1, 130, 4096), (3, 256, 3872), (12, 100, 16384), (20, 1200, 4000), (33, 600, 2816),
                                   (5, 1217, 8192)])
@pytest.mark.parametrize("nv", [False, True], ids=["mxfp4", "nvfp4"])
def test_few_row_tiles_and_long_sums(M, N, K, nv):
    """K over more slices than stages divide evenly, up to the largest cluster."""
    import gemm_pt_block_gb300 as mx

    q, s, w64 = weights(N, K, nv, 61)
    for kind in ("bf16", "e4m3"):
        x, _, x64, kw = activations(M, K, kind, 62)
        y = mx.mxfp4_gemv(x, q, s, N, K, wparams(nv), out_dtype=F32, workspace=False, **kw)
        check(y, x64, w64)
        z = mx.mxfp4_gemv(x, q, s, N, K, wparams(nv), out_dtype=F32, workspace=False, **kw)
        assert torch.equal(y, z)
    assert mx.device_status() == 0


@pytest.mark.parametrize("K", [32, 96, 160, 544, 1056, 4128, 4160])
@pytest.mark.parametrize("nv", [False, True], ids=["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M", [3, 12])
def test_scales_of_the_next_row_stay_out(M, nv, K):
    """Rows of scales of any length, a NaN row after each finite one: what lies
    past a row's end in memory enters nothing."""
    import gemm_pt_block_gb300 as mx

    N = 139
    q, s, w64 = weights(N, K, nv, 41)
    x, _, x64, _ = activations(M, K, "bf16", 42)
    s = s.clone()
    s[1::2] = 0x7F if nv else 255
    y = mx.mxfp4_gemv(x, q, s, N, K, wparams(nv), out_dtype=F32, workspace=False)
    check(y[:, ::2].contiguous(), x64, w64[::2])
    assert torch.isnan(y[:, 1::2]).all()
    space = torch.zeros(1 << 22, dtype=torch.uint8, device=DEV)
    z = mx.mxfp4_gemv(x, q, s, N, K, wparams(nv), out_dtype=F32, workspace=space)
    check(z[:, ::2].contiguous(), x64, w64[::2])
    assert torch.isnan(z[:, 1::2]).all()


@pytest.mark.parametrize("exp", [-100, -10, 0, 30])
def test_tensor_exponent(exp):
    import gemm_pt_block_gb300 as mx

    q, s, w64 = weights(64, 256, True, 14)
    x, _, x64, _ = activations(3, 256, "bf16", 15)
    y = mx.mxfp4_gemv(x, q, s, 64, 256, wparams(True, 0, exp), out_dtype=F32)
    check(y, x64, w64 * 2.0 ** exp)


@pytest.mark.parametrize("M,N,K,dt", [(3, 77, 96, BF16), (9, 130, 512, F32), (1, 33, 64, BF16)])
def test_strides_and_guard_bytes(M, N, K, dt):
    import gemm_pt_block_gb300 as mx

    es, ld = (2, N + 5) if dt == BF16 else (4, N + 3)
    spans = [(m * ld * es, (m * ld + N) * es) for m in range(M)]
    a = Arena([M * ld * es])
    y = a.region(0, dt, (M, ld), spans)[:, :N]
    q, s, w64 = weights(N, K, False, 16)
    for kind, extra in (("bf16", 8), ("e4m3", 16)):
        x, _, x64, kw = activations(M, K, kind, 17)
        wide = torch.zeros((M, K + extra), dtype=x.dtype, device=DEV)
        wide[:, :K] = x
        mx.mxfp4_gemv(wide[:, :K], q, s, N, K, wparams(False), y=y, **kw)
        check(y, x64, w64)
    a.check(f"gemv {M}x{N}x{K}")


@pytest.mark.parametrize("M,nv,layout", [(1, False, 0), (2, False, 0), (8, True, 0), (3, False, 1), (12, False, 0),
                                         (32, True, 0), (20, False, 1)])
def test_every_stage_of_a_long_sum_on_every_run(M, nv, layout):
    """Long K, many CTAs, many runs: a slot of a kernel's ring that is refilled
    under its readers shows as an element of another stage."""
    import gemm_pt_block_gb300 as mx

    N, K = 28672, 16384
    q, s, _ = weights(N, K, nv, 25, 120, 124)
    sw = torch.from_numpy(oracle.scales_to_mma(s.cpu().numpy())).to(DEV) if layout else s
    x, _, x64, _ = activations(M, K, "bf16", 26)
    y = mx.mxfp4_gemv(x, q, sw, N, K, wparams(nv, layout), out_dtype=F32)
    rows = list(range(0, N, 997))
    v = E2M1.to(DEV)[torch.stack((q[rows] & 15, q[rows] >> 4), -1).view(len(rows), K).long()]
    f = s[rows].view(torch.float8_e4m3fn).double() if nv else torch.exp2(s[rows].double() - 127)
    check(y[:, rows], x64, v * f.repeat_interleave(16 if nv else 32, 1))
    for _ in range(30):
        assert torch.equal(mx.mxfp4_gemv(x, q, sw, N, K, wparams(nv, layout), out_dtype=F32), y)
    assert mx.device_status() == 0


def test_empty_sizes():
    import gemm_pt_block_gb300 as mx

    q, s, _ = weights(16, 64, False, 18)
    x = torch.ones((2, 64), device=DEV, dtype=BF16)
    assert mx.mxfp4_gemv(x[:0], q, s, 16, 64).shape == (0, 16)
    assert mx.mxfp4_gemv(x, q[:0], s[:0], 0, 64).shape == (2, 0)
    y = torch.full((2, 16), 7.0, device=DEV)
    mx.mxfp4_gemv(x[:, :0], q[:, :0].contiguous(), s[:, :0].contiguous(), 16, 0, y=y)
    assert (y == 0).all()


def test_refusals():
    import gemm_pt_block_gb300 as mx

    N, K = 128, 128
    q, s, _ = weights(N, K, False, 19)
    x, _, _, _ = activations(2, K, "bf16", 20)
    c, sx, _, kw = activations(2, K, "e4m3", 21)
    bad = [
        (TypeError, lambda: mx.mxfp4_gemv(x.float(), q, s, N, K)),
        (TypeError, lambda: mx.mxfp4_gemv(x, q, s, N, K, out_dtype=torch.float16)),
        (TypeError, lambda: mx.mxfp4_gemv(x, q.int(), s, N, K)),
        (ValueError, lambda: mx.mxfp4_gemv(x[:, :64], q, s, N, K)),
        (ValueError, lambda: mx.mxfp4_gemv(x, q[:64], s, N, K)),
        (ValueError, lambda: mx.mxfp4_gemv(x, q, s[:64], N, K)),
        (ValueError, lambda: mx.mxfp4_gemv(x, q, s, N, K, sx=sx)),
        (ValueError, lambda: mx.mxfp4_gemv(c, q, s, N, K)),
        (ValueError, lambda: mx.mxfp4_gemv(c, q, s, N, K, sx=sx[:1])),
        (ValueError, lambda: mx.mxfp4_gemv(c, q, s, N, K, sx=sx, x_format=mx.FORMAT_E2M1)),
        (ValueError, lambda: mx.mxfp4_gemv(x, q, s, N, K, mx.QuantParams(elem_format=mx.FORMAT_E4M3))),
        (ValueError, lambda: mx.mxfp4_gemv(x, q, s, N, K, y=torch.empty((2, 64), device=DEV))),
        (ValueError, lambda: mx.mxfp4_gemv(x.cpu(), q, s, N, K)),
        (mx.Mxfp4Error, lambda: mx.mxfp4_gemv(x[:, 4:100], q, s, N, 96)),        # x 8 bytes off
        (mx.Mxfp4Error, lambda: mx.mxfp4_gemv(x, q, s, N, K, mx.QuantParams(tensor_exp=1))),
        (mx.Mxfp4Error, lambda: mx.mxfp4_gemv(x[:, :48].contiguous(), q, s, N, 48)),
        (mx.Mxfp4Error, lambda: mx.mxfp4_gemv(x, q, s, 64, K, mx.QuantParams(scale_layout=mx.LAYOUT_MMA))),
    ]
    for i, (err, call) in enumerate(bad):
        with pytest.raises(err):
            call()
            raise AssertionError(f"refusal {i} did not raise")
    assert mx.device_status() == 0


def test_side_stream_and_graph_capture():
    import gemm_pt_block_gb300 as mx

    N, K = 640, 1024
    q, s, _ = weights(N, K, False, 22)
    x = [activations(4, K, "bf16", 30 + i)[0] for i in range(3)]
    want = [mx.mxfp4_gemv(t, q, s, N, K) for t in x]
    torch.cuda.synchronize()
    side, buf, out = torch.cuda.Stream(), torch.empty_like(x[0]), torch.empty((4, N), dtype=BF16, device=DEV)
    side.wait_stream(torch.cuda.current_stream())
    for t, v in zip(x, want):
        with torch.cuda.stream(side):
            torch.cuda._sleep(1_000_000)
            buf.copy_(t)
        got = mx.mxfp4_gemv(buf, q, s, N, K, stream=side)
        side.synchronize()
        assert torch.equal(got, v)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mx.mxfp4_gemv(buf, q, s, N, K, y=out)
    for t, v in zip(x, want):
        buf.copy_(t)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, v)


@pytest.mark.parametrize("M,nv", [(2, False), (12, False), (12, True)])
def test_workspace_forms_on_a_side_stream_and_in_a_graph(M, nv):
    """The two kernels of the forms with a workspace, one launched under the
    other, follow what the stream wrote before them."""
    import gemm_pt_block_gb300 as mx

    N, K = 640, 1024
    q, s, _ = weights(N, K, nv, 24)
    x = [activations(M, K, "bf16", 50 + i)[0] for i in range(3)]
    w = wparams(nv)
    space = torch.empty(1 << 22, dtype=torch.uint8, device=DEV)
    want = [mx.mxfp4_gemv(t, q, s, N, K, w, workspace=space) for t in x]
    plain = [mx.mxfp4_gemv(t, q, s, N, K, w, workspace=False) for t in x]
    for a, b in zip(want, plain):
        assert (a.float() - b.float()).abs().max() <= b.float().abs().max() / 64
    torch.cuda.synchronize()
    side, buf, out = torch.cuda.Stream(), torch.empty_like(x[0]), torch.empty((M, N), dtype=BF16, device=DEV)
    side.wait_stream(torch.cuda.current_stream())
    for t, v in zip(x, want):
        with torch.cuda.stream(side):
            torch.cuda._sleep(1_000_000)
            buf.copy_(t)
        got = mx.mxfp4_gemv(buf, q, s, N, K, w, workspace=space, stream=side)
        side.synchronize()
        assert torch.equal(got, v)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(2):                                # the second call's workspace is the first one's
            mx.mxfp4_gemv(buf, q, s, N, K, w, y=out, workspace=space)
    for t, v in zip(x, want):
        buf.copy_(t)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, v)


def test_offsets_beyond_32_bits():
    """A weight matrix whose codes pass 4 GiB: rows past the 2^32nd byte are
    read, and land in their own columns."""
    import gemm_pt_block_gb300 as mx

    K, N = 16384, 540_000                                  # 4.4e9 code bytes
    q = torch.zeros((N, K // 2), dtype=torch.uint8, device=DEV)
    s = torch.full((N, K // 32), 127, dtype=torch.uint8, device=DEV)
    x, _, x64, _ = activations(2, K, "bf16", 23)
    rows = [0, 1, 262_143, 262_144, 524_287, 524_288, 524_289, N - 1]
    qr, sr, w64 = weights(len(rows), K, False, 24)
    q[rows], s[rows] = qr, sr
    y = mx.mxfp4_gemv(x, q, s, N, K, out_dtype=F32)
    check(y[:, rows], x64, w64)
    other = torch.ones(N, dtype=torch.bool, device=DEV)
    other[rows] = False
    assert (y[:, other] == 0).all()
