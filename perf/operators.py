"""Timed cases of the operators around the MXFP4 products of a feed-forward block.

Five operators, in the order in which a block runs them (T tokens, D model
width, F feed-forward width, M tokens of one decode step):

  norm_fwd    h = x + r;  y = (h * w) / sqrt(mean(h^2) + eps), quantized along D
  norm_bwd    gradients of y with respect to x (and r) and w
  swiglu_fwd  a = g / (1 + exp(-g)) * u, quantized along F
  swiglu_bwd  gradients of a with respect to g and u
  gemv        y[m, n] = sum_k x[m, k] W[n, k], W held as 4-bit codes and block scales

With `own` false, `run` computes them with elementary torch operations in 32
bits, rounded once at the end; with `own` true it makes the library's calls.
One-byte codes are returned as float8 tensors and E8M0 scales as
float8_e8m0fnu tensors: the values that the bytes stand for.
"""
from __future__ import annotations

import math

import torch

own = False

EPS = 1e-5
# One-byte element formats: (torch type, largest value = 0.875 * 2^TOP).
FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0, 9), "e5m2": (torch.float8_e5m2, 57344.0, 16)}
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases ---

def _norm(name, T, D, fmt="e4m3", residual=True, layout="row", mode="roundup", w="bf16", x="bf16"):
    return {"name": name, "op": "norm_fwd", "T": T, "D": D, "fmt": fmt, "residual": residual,
            "layout": layout, "mode": mode, "w": w, "x": x}


def _norm_bwd(name, T, D, stream=True, w="bf16", x="bf16"):
    return {"name": name, "op": "norm_bwd", "T": T, "D": D, "stream": stream, "w": w, "x": x}


def _swiglu(name, T, F, fmt="e4m3", layout="row", mode="roundup", x="bf16"):
    return {"name": name, "op": "swiglu_fwd", "T": T, "F": F, "fmt": fmt, "layout": layout,
            "mode": mode, "x": x}


def _swiglu_bwd(name, T, F, x="bf16"):
    return {"name": name, "op": "swiglu_bwd", "T": T, "F": F, "x": x}


def _gemv(name, M, N, K, w="mxfp4", x="bf16", layout="row", y="bf16"):
    return {"name": name, "op": "gemv", "M": M, "N": N, "K": K, "w": w, "x": x, "layout": layout,
            "y": y}


def listed():
    return [
        # One token of a decode step, model width of the 70B-shaped layer: all latency.
        _norm("norm 1x8192", 1, 8192),
        # A short ragged prompt on an 8B-shaped layer, fp32 norm weights, E5M2 codes, no residual.
        _norm("norm 777x4096", 777, 4096, fmt="e5m2", residual=False, mode="floor", w="f32"),
        # The training batch of the 70B-shaped layer; scales as the matrix product reads them.
        _norm("norm 16384x8192", 16384, 8192, layout="mma"),
        # Backward of the 8B-shaped layer's norm on a ragged batch, no gradient from the residual stream.
        _norm_bwd("norm bwd 1001x4096", 1001, 4096, stream=False, w="f32"),
        # Backward of the training batch, with the residual stream's gradient added.
        _norm_bwd("norm bwd 16384x8192", 16384, 8192),
        # Eight sequences decoding together: the activation between the two 4-bit products.
        _swiglu("swiglu 8x14336", 8, 14336),
        # A prefill of the 70B-shaped layer; scales as the matrix product reads them.
        _swiglu("swiglu 8192x28672", 8192, 28672, layout="mma"),
        # Its training backward pass on a quarter of the batch.
        _swiglu_bwd("swiglu bwd 4096x28672", 4096, 28672),
        # A small projection for one token, an odd number of output rows: launch latency.
        _gemv("gemv 1x1000x1024", 1, 1000, 1024, y="f32"),
        # One token through the 70B-shaped up-projection: the stream of 4-bit weights.
        _gemv("gemv 1x28672x8192", 1, 28672, 8192, layout="mma"),
        # Eight tokens through the 70B-shaped down-projection, MXFP8 activations.
        _gemv("gemv 8x8192x28672 e4m3", 8, 8192, 28672, x="e4m3", layout="mma"),
        # Twenty-three tokens of a larger decode batch, NVFP4 weights of the 8B-shaped layer.
        _gemv("gemv 23x14336x4096 nvfp4", 23, 14336, 4096, w="nvfp4", layout="row"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "swiglu_fwd", "swiglu_bwd", "gemv", "gemv"])
    if op == "gemv":
        M = rng.randint(1, 32)
        layout = rng.choice(["row", "mma"])
        step = 128 if layout == "mma" else 32
        N = _log_int(rng, 128, 28672)
        N = max(128, N // 128 * 128) if layout == "mma" else N
        K = max(step, _log_int(rng, 256, 28672) // step * step)
        while N * K > 28672 * 8192:
            K = max(step, K // 2 // step * step)
        return {k: v for k, v in _gemv("", M, N, K, rng.choice(["mxfp4", "mxfp4", "nvfp4"]),
                                       rng.choice(["bf16", "e4m3"]), layout,
                                       rng.choice(["bf16", "bf16", "f32"])).items() if k != "name"}
    T = _log_int(rng, 1, 16384)
    W = max(32, _log_int(rng, 128, 16384 if op.startswith("norm") else 28672) // 32 * 32)
    x = rng.choice(["bf16", "bf16", "bf16", "f32"])
    most = 16384 * 8192 // (2 if x == "f32" else 1)
    T = max(1, min(T, most // W))
    layout = rng.choice(["row", "mma"])
    if layout == "mma" and op in ("norm_fwd", "swiglu_fwd"):
        W = max(128, W // 128 * 128)
        T = max(128, T // 128 * 128)
    fmt, mode, w = rng.choice(["e4m3", "e4m3", "e5m2"]), rng.choice(["roundup", "floor"]), rng.choice(["bf16", "f32"])
    c = {"norm_fwd": lambda: _norm("", T, W, fmt, rng.random() < 0.7, layout, mode, w, x),
         "norm_bwd": lambda: _norm_bwd("", T, W, rng.random() < 0.7, w, x),
         "swiglu_fwd": lambda: _swiglu("", T, W, fmt, layout, mode, x),
         "swiglu_bwd": lambda: _swiglu_bwd("", T, W, x)}[op]()
    return {k: v for k, v in c.items() if k != "name"}


# ----------------------------------------------------------------- inputs ---

def _activations(shape, dtype, g, std=1.0):
    """Activations of a layer: normal, with a few channels of thirty times the spread."""
    x = torch.randn(shape, device="cuda", generator=g) * std
    cols = torch.randint(0, shape[1], (max(1, shape[1] // 1024),), device="cuda", generator=g)
    x[:, cols] *= 30.0
    return x.to(dtype)


def _blocks_of_weights(N, K, kind, layout, g):
    """A weight matrix N(0, 0.02) in 4-bit codes (two per byte, the even index
    low) with its block scales: E8M0 per 32 elements, or E4M3 per 16 under a
    factor 2^-10 of the whole tensor."""
    W = torch.randn((N, K), device="cuda", generator=g).mul_(0.02)
    per = 16 if kind == "nvfp4" else 32
    B = W.view(N, K // per, per)
    M = B.abs().amax(-1)
    if kind == "nvfp4":
        scale = (M * (1024.0 / 6.0)).to(torch.float8_e4m3fn)
        s, factor = scale.view(torch.uint8), scale.float() / 1024.0
    else:
        m, e = torch.frexp(M / 6.0)
        e = e - (m == 0.5).int()
        s, factor = (e + 127).to(torch.uint8), torch.ldexp(torch.ones_like(M), e)
    B = B / factor.clamp_min(1e-30)[..., None]
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    code = torch.bucketize(B.abs(), edges).to(torch.uint8)
    code |= (B < 0).to(torch.uint8) << 3
    code = code.view(N, K // 2, 2)
    q = code[..., 0] | (code[..., 1] << 4)
    return q.contiguous(), (_tiles(s) if layout == "mma" else s.contiguous())


def _tiles(s):
    """Scales [R, C] as 128 x 4 tiles of 512 bytes, as the matrix product reads them."""
    R, C = s.shape
    return s.reshape(R // 128, 4, 32, C // 4, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _rows(s, R, C):
    """The inverse of _tiles."""
    return s.view(R // 128, C // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(R, C)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "gemv":
        M, N, K = case["M"], case["N"], case["K"]
        s["qw"], s["sw"] = _blocks_of_weights(N, K, case["w"], case["layout"], g)
        x = _activations((M, K), torch.bfloat16, g)
        if case["x"] == "bf16":
            s["x"], s["sx"] = x, None
        else:
            x = x.float().view(M, K // 32, 32)
            m, e = torch.frexp(x.abs().amax(-1))
            e = e - 9 + (m > 0.875).int()
            s["sx"] = (e + 127).to(torch.uint8)
            s["x"] = (x * torch.ldexp(torch.ones_like(m), -e)[..., None]).view(M, K).to(
                torch.float8_e4m3fn).view(torch.uint8)
        return s
    dt = TYPES[case["x"]]
    if case["op"].startswith("norm"):
        T, D = case["T"], case["D"]
        s["w"] = (1.0 + 0.1 * torch.randn(D, device="cuda", generator=g)).to(TYPES[case["w"]])
        s["h" if case["op"] == "norm_bwd" else "x"] = _activations((T, D), dt, g)
        if case["op"] == "norm_fwd":
            s["r"] = _activations((T, D), dt, g, 2.0) if case["residual"] else None
        else:
            # what the forward pass left: the stream and its reciprocal root mean squares
            s["rstd"] = torch.rsqrt(s["h"].float().square().mean(-1) + EPS)
            s["dy"] = (torch.randn((T, D), device="cuda", generator=g) * 1e-3).to(dt)
            s["dh"] = (torch.randn((T, D), device="cuda", generator=g) * 1e-3).to(dt) if case["stream"] else None
        return s
    T, F = case["T"], case["F"]
    # gate and up projections side by side, as one product writes them
    gu = _activations((T, 2 * F), dt, g)
    s["g"], s["u"] = gu[:, :F], gu[:, F:]
    if case["op"] == "swiglu_bwd":
        s["dy"] = (torch.randn((T, F), device="cuda", generator=g) * 1e-3).to(dt)
    return s


# ------------------------------------------------------------------- runs ---

def _plain_quantize(y, fmt, mode, layout):
    """Codes and E8M0 scales of fp32 y along its rows, 32 elements a block."""
    dtype, largest, top = FP8[fmt]
    T, D = y.shape
    b = y.view(T, D // 32, 32)
    m, e = torch.frexp(b.abs().amax(-1))
    e = e - top
    if mode == "roundup":
        e = e + (m > 0.875).int()
    e = torch.where(m == 0, -127, e).clamp(-127, 126)
    v = (b * torch.ldexp(torch.ones_like(m), -e)[..., None]).clamp(-largest, largest)
    s = (e + 127).to(torch.uint8)
    s = _tiles(s) if layout == "mma" else s
    return v.view(T, D).to(dtype), s.view(torch.float8_e8m0fnu)


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _values(q, sw, N, K, kind, layout, dtype):
    """The weight matrix that codes and scales stand for."""
    grid = torch.tensor(_E2M1, device=q.device, dtype=dtype)
    v = grid[torch.stack((q & 15, q >> 4), -1).view(N, K).int()]
    per = 16 if kind == "nvfp4" else 32
    s = _rows(sw, N, K // per) if layout == "mma" else sw
    if kind == "nvfp4":
        f = s.contiguous().view(torch.float8_e4m3fn).to(dtype) / 1024.0
    else:
        f = torch.ldexp(torch.ones((), device=q.device, dtype=dtype), s.int() - 127)
    return (v.view(N, K // per, per) * f[..., None]).view(N, K)


def _plain(s):
    c = s["case"]
    if c["op"] == "norm_fwd":
        h = s["x"]
        if s["r"] is not None:
            h = (h.float() + s["r"].float()).to(h.dtype)
        f = h.float()
        rstd = torch.rsqrt(f.square().mean(-1) + EPS)
        q, sc = _plain_quantize(f * rstd[:, None] * s["w"].float(), c["fmt"], c["mode"], c["layout"])
        return {"q": q, "s": sc, "rstd": rstd, **({"h": h} if s["r"] is not None else {})}
    if c["op"] == "norm_bwd":
        h, dy, rstd = s["h"].float(), s["dy"].float(), s["rstd"][:, None]
        n = h * rstd
        dn = dy * s["w"].float()
        dx = (dn - n * (dn * n).mean(-1, keepdim=True)) * rstd
        if s["dh"] is not None:
            dx = dx + s["dh"].float()
        return {"dx": dx.to(s["h"].dtype), "dw": (dy * n).sum(0).to(s["w"].dtype)}
    if c["op"] == "swiglu_fwd":
        g = s["g"].float()
        q, sc = _plain_quantize(g / (1.0 + torch.exp(-g)) * s["u"].float(), c["fmt"], c["mode"], c["layout"])
        return {"q": q, "s": sc}
    if c["op"] == "swiglu_bwd":
        g, u, dy = s["g"].float(), s["u"].float(), s["dy"].float()
        sig = 1.0 / (1.0 + torch.exp(-g))
        return {"dg": (dy * u * sig * (1.0 + g * (1.0 - sig))).to(s["g"].dtype),
                "du": (dy * g * sig).to(s["u"].dtype)}
    x = s["x"].float()
    if s["sx"] is not None:
        M, K = c["M"], c["K"]
        x = s["x"].view(torch.float8_e4m3fn).float().view(M, K // 32, 32)
        x = (x * torch.ldexp(torch.ones((), device=x.device), s["sx"].int() - 127)[..., None]).view(M, K)
    W = _values(s["qw"], s["sw"], c["N"], c["K"], c["w"], c["layout"], torch.float32)
    return {"y": (x @ W.t()).to(TYPES[c["y"]])}


def _own(s):
    import gemm_pt_block_gb300 as mx

    c = s["case"]
    if c["op"] in ("norm_fwd", "swiglu_fwd"):
        p = mx.QuantParams(mx.BLOCK_1X32, mx.SCALE_ROUNDUP if c["mode"] == "roundup" else mx.SCALE_FLOOR,
                           mx.ROUND_RTN, mx.LAYOUT_MMA if c["layout"] == "mma" else mx.LAYOUT_ROWMAJOR,
                           elem_format=mx.FORMAT_E4M3 if c["fmt"] == "e4m3" else mx.FORMAT_E5M2)
        out = {}
        if c["op"] == "norm_fwd":
            q, sc, _, h, out["rstd"] = mx.mxfp4_rmsnorm_quantize(s["x"], s["w"], p, residual=s["r"], eps=EPS,
                                                                 with_rstd=True)
            if h is not None:
                out["h"] = h
        else:
            q, sc, _ = mx.mxfp4_swiglu_quantize(s["g"], s["u"], p)
        return {"q": q.view(FP8[c["fmt"]][0]), "s": sc.view(torch.float8_e8m0fnu), **out}
    if c["op"] == "norm_bwd":
        dx, dw = mx.mxfp4_rmsnorm_backward(s["dy"], s["h"], s["w"], s["rstd"], dh=s["dh"])
        return {"dx": dx, "dw": dw}
    if c["op"] == "swiglu_bwd":
        dg, du = mx.mxfp4_swiglu_backward(s["dy"], s["g"], s["u"])
        return {"dg": dg, "du": du}
    nv = c["w"] == "nvfp4"
    w = mx.QuantParams(mx.BLOCK_1X16 if nv else mx.BLOCK_1X32, tensor_exp=-10 if nv else 0,
                       scale_layout=mx.LAYOUT_MMA if c["layout"] == "mma" else mx.LAYOUT_ROWMAJOR)
    return {"y": mx.mxfp4_gemv(s["x"], s["qw"], s["sw"], c["N"], c["K"], w, sx=s["sx"],
                               out_dtype=TYPES[c["y"]])}


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------- what it has to do ---

def work(case):
    if case["op"] == "gemv":
        M, N, K = case["M"], case["N"], case["K"]
        x = M * K * (2 if case["x"] == "bf16" else 1 + 1 / 32)
        w = N * K * (0.5 + 1 / (16 if case["w"] == "nvfp4" else 32))
        return {"bytes": x + w + M * N * (2 if case["y"] == "bf16" else 4), "flops": 2 * M * N * K}
    e = 2 if case["x"] == "bf16" else 4
    if case["op"].startswith("norm"):
        n, T, D = case["T"] * case["D"], case["T"], case["D"]
        wb = D * (2 if case["w"] == "bf16" else 4)
        if case["op"] == "norm_fwd":
            moved = n * e * (3 if case["residual"] else 1) + n * (1 + 1 / 32) + 4 * T + wb
            return {"bytes": moved, "flops": 8 * n}
        return {"bytes": n * e * (4 if case["stream"] else 3) + 4 * T + 2 * wb, "flops": 12 * n}
    n = case["T"] * case["F"]
    if case["op"] == "swiglu_fwd":
        return {"bytes": n * (2 * e + 1 + 1 / 32), "flops": 8 * n}
    return {"bytes": n * 5 * e, "flops": 14 * n}


# ------------------------------------------------- the definition in 64 bits ---

def _exact_quantize(y, fmt, mode, layout):
    mant, low, largest = {"e4m3": (3, -6, 448.0), "e5m2": (2, -14, 57344.0)}[fmt]
    T, D = y.shape
    b = y.view(T, -1, 32)
    M = b.abs().amax(-1).clamp_min(2.0 ** -126)
    if mode == "roundup":
        e = torch.ceil(torch.log2(M / largest))
    else:
        e = torch.floor(torch.log2(M)) - math.floor(math.log2(largest))
    scale = torch.pow(2.0, e)
    v = b / scale[..., None]
    step = torch.pow(2.0, torch.floor(torch.log2(v.abs().clamp_min(2.0 ** low))) - mant)
    v = (torch.round(v / step) * step).clamp(-largest, largest)
    return v.reshape(T, D), (_tiles(scale) if layout == "mma" else scale)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_fwd":
        h = s["x"].double()
        out = {}
        if s["r"] is not None:
            h = (h + s["r"].double()).to(s["x"].dtype)   # the stream is held in its own type
            out["h"] = h.double()
            h = out["h"]
        rms = torch.sqrt((h * h).sum(1) / case["D"] + EPS)
        out["q"], out["s"] = _exact_quantize(s["w"].double() * (h / rms[:, None]), case["fmt"], case["mode"],
                                             case["layout"])
        out["rstd"] = 1.0 / rms
        return out
    if case["op"] == "norm_bwd":
        # dx_i = w_i dy_i / rms - h_i sum_j(w_j dy_j h_j) / (D rms^3)
        h, dy, r = s["h"].double(), s["dy"].double(), s["rstd"].double()
        gw = dy * s["w"].double()
        dx = gw * r[:, None] - h * ((gw * h).sum(1) * r ** 3 / case["D"])[:, None]
        if s["dh"] is not None:
            dx += s["dh"].double()
        return {"dx": dx, "dw": torch.einsum("td,t->d", dy * h, r)}
    if case["op"] == "swiglu_fwd":
        q, sc = _exact_quantize(torch.nn.functional.silu(s["g"].double()) * s["u"].double(), case["fmt"],
                                case["mode"], case["layout"])
        return {"q": q, "s": sc}
    if case["op"] == "swiglu_bwd":
        g, u, dy = s["g"].double(), s["u"].double(), s["dy"].double()
        sig = torch.sigmoid(g)
        return {"dg": dy * u * (sig + g * sig * torch.sigmoid(-g)), "du": dy * torch.nn.functional.silu(g)}
    M, N, K, per = case["M"], case["N"], case["K"], 16 if case["w"] == "nvfp4" else 32
    x = s["x"]
    if s["sx"] is not None:
        x = x.view(torch.float8_e4m3fn).double() * torch.exp2(s["sx"].double() - 127.0).repeat_interleave(32, 1)
    x = x.double()
    lo, hi = (s["qw"] & 15).long(), (s["qw"] >> 4).long()
    code = torch.empty((N, K), dtype=torch.long, device=x.device)
    code[:, 0::2], code[:, 1::2] = lo, hi
    mag = code & 7
    val = torch.where(mag < 2, mag * 0.5, (2.0 + (mag & 1)) * torch.exp2((mag >> 1).double() - 2.0))
    val = torch.where(code >= 8, -val, val)
    sw = _rows(s["sw"], N, K // per) if case["layout"] == "mma" else s["sw"]
    f = sw.contiguous().view(torch.float8_e4m3fn).double() * 2.0 ** -10 if per == 16 else torch.exp2(sw.double() - 127.0)
    return {"y": x @ (val * f.repeat_interleave(per, 1)).t()}
