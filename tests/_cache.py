"""The 8-bit cache's definition in 64 bits, and caches to test on: pages in a
mixed order, everything that no sequence holds filled with bytes that would
show (E4M3's NaN codes, scale 0xFF, pages outside the cache)."""
from __future__ import annotations

import math
from dataclasses import dataclass

import torch

DEV = "cuda:0"


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def e4m3(x: torch.Tensor) -> torch.Tensor:
    """Nearest E4M3 value of 64-bit x (|x| <= 448), ties to even."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def code_bytes(v: torch.Tensor) -> torch.Tensor:
    """The bytes of E4M3 values."""
    return v.float().to(torch.float8_e4m3fn).view(torch.uint8)


def scale_exp(M: torch.Tensor) -> torch.Tensor:
    """The smallest e >= -127 with 448 * 2^e >= M, 64-bit."""
    return torch.ceil(torch.log2(M.clamp_min(448 * 2.0 ** -127) / 448.0))


def values(codes: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    """64-bit values of pages [..., P, D] with scales [...]; NaN under 0xFF."""
    s = torch.where(scales == 255, torch.nan, torch.exp2(scales.double() - 127.0))
    return codes.view(torch.float8_e4m3fn).double() * s[..., None, None]


@dataclass
class Cache:
    codes: torch.Tensor
    scales: torch.Tensor
    table: torch.Tensor          # int32 [B, max_pages]
    lens: torch.Tensor           # int32 [B]
    starts: torch.Tensor         # int32 [B + 1]
    L: list
    n: list

    @property
    def P(self):
        return self.codes.shape[3]

    @property
    def T(self):
        return sum(self.n)

    def tokens(self, b, count):
        """Keys and values [2, H, count, D] of sequence b's first tokens."""
        pages = self.table[b, :-(-count // self.P)].long()
        x = values(self.codes[pages], self.scales[pages])
        return x.permute(1, 2, 0, 3, 4).reshape(2, x.shape[2], -1, x.shape[4])[:, :, :count]


def make_cache(L, n, H, D, P, seed=0, filled=None, extra_pages=3, table_cols=2):
    """A cache of sequences of L tokens, n of them new; `filled` tokens of each
    (default: all) hold values, the rest poison."""
    g = gen(seed)
    B = len(L)
    filled = L if filled is None else filled
    used = [max(0, -(-x // P)) for x in L]
    pages, cols = sum(used) + extra_pages, max(used + [0]) + table_cols
    order = torch.randperm(pages, device=DEV, generator=g).int()
    table = torch.full((B, cols), -1, dtype=torch.int32, device=DEV)
    table[:, -1] = 1 << 30
    at = 0
    for b in range(B):
        table[b, :used[b]] = order[at:at + used[b]]
        at += used[b]
    codes = torch.full((pages, 2, H, P, D), 0x7F, dtype=torch.uint8, device=DEV)
    scales = torch.full((pages, 2, H), 255, dtype=torch.uint8, device=DEV)
    for b in range(B):
        for i in range(-(-filled[b] // P)):
            m = min(P, filled[b] - i * P)
            x = torch.randn((2, H, m, D), device=DEV, generator=g, dtype=torch.float64)
            x[..., 5] *= 12.0
            x *= torch.exp2(torch.randint(-3, 3, (2, H, 1, 1), device=DEV, generator=g).double())
            e = scale_exp(x.abs().amax((2, 3)))
            page = int(table[b, i])
            codes[page, :, :, :m] = code_bytes(e4m3(x * torch.exp2(-e)[..., None, None]))
            scales[page] = (e + 127).to(torch.uint8)
    starts = torch.tensor([0] + [sum(n[:i + 1]) for i in range(B)], dtype=torch.int32, device=DEV)
    return Cache(codes, scales, table, torch.tensor(L, dtype=torch.int32, device=DEV), starts, list(L), list(n))


def attend(c: Cache, q, scale=None, window=0, softcap=0.0, slopes=None):
    """(out, lse, weight, reach): the definition in 64 bits; weight = sum_j p_j |v_j|
    and reach, the largest of what a score is summed from, bound the errors."""
    T, Hq, D = q.shape
    H = c.codes.shape[2]
    scale = D ** -0.5 if scale is None else scale
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device=DEV)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=DEV)
    weight, reach = torch.zeros_like(out), torch.zeros_like(lse)
    t = 0
    for b, (L, n) in enumerate(zip(c.L, c.n)):
        kv = c.tokens(b, L).repeat_interleave(Hq // H, 1)
        for i in range(n):
            p = L - n + i
            lo = max(0, p - window + 1) if window else 0
            if p >= 0:
                k, v = kv[0][:, lo:p + 1], kv[1][:, lo:p + 1]
                x = q[t].double()
                z = torch.einsum("hd,hld->hl", x, k) * scale
                r = torch.einsum("hd,hld->hl", x.abs(), k.abs()) * abs(scale)
                if softcap:
                    z = softcap * torch.tanh(z / softcap)
                    r = r + softcap
                if slopes is not None:
                    bias = slopes.double()[:, None] * (torch.arange(lo, p + 1, device=DEV) - p)
                    z, r = z + bias, r + bias.abs()
                lse[t] = torch.logsumexp(z, 1)
                w = torch.exp(z - lse[t][:, None])
                out[t] = torch.einsum("hl,hld->hd", w, v)
                weight[t] = torch.einsum("hl,hld->hd", w, v.abs())
                reach[t] = r.amax(1)
            t += 1
    return out, lse, weight, reach


def attention_bounds(dtype, tokens, ref, weight, reach):
    """How far out and lse may be from the definition. A score is a sum of exact
    products in fp32, at most 16 steps and a few roundings, each of 2^-23 of what
    it is summed from: ds = 2^-18 reach. A weight then is off by 2 ds (its own
    score and the maximum's) and by the exponential's and the scale's roundings
    (2^-20); for bf16 outputs it goes into the second product in 11 bits (half a
    step: 2^-11), for fp32 in 22. Sums over tokens round at each step of 16 (2^-23),
    in the numerator and in the sum of weights alike. Then the output's own half step."""
    ds = 2.0 ** -18 * reach
    each = 2 * torch.expm1(ds) + 2.0 ** -19 + (2.0 ** -11 if dtype == torch.bfloat16 else 2.0 ** -20) + \
        2 * (tokens / 16 + 64) * 2.0 ** -23
    half = torch.finfo(dtype).eps / 2
    out = half * ref.abs() + (1 + half) * each[..., None] * weight
    return out, torch.expm1(ds) + 2.0 ** -20 + (tokens / 16 + 64) * 2.0 ** -23


def append(c: Cache, k, v):
    """(codes, scales) after the new tokens k, v, by the definition."""
    P = c.P
    codes, scales = c.codes.clone(), c.scales.clone()
    x = torch.stack((k, v), 1).double()                          # [T, 2, H, D]
    t = 0
    for b, (L, n) in enumerate(zip(c.L, c.n)):
        for i in range(max(0, L - n) // P, -(-L // P) if n else 0):
            lo, hi = max(L - n, i * P), min(L, i * P + P)
            page = int(c.table[b, i])
            new = x[t + lo - (L - n):t + hi - (L - n)].permute(1, 2, 0, 3)
            bad = ~torch.isfinite(new).all(-1).all(-1)
            e = scale_exp(torch.where(torch.isfinite(new), new, 0.0).abs().amax((2, 3))) + 127
            e = torch.where(bad, 255.0, e)
            old = scales[page].double()
            now = torch.maximum(e, old) if lo > i * P else e
            if lo > i * P:
                was = codes[page, :, :, :lo - i * P]
                f = torch.where((old < now) & (now < 255), torch.exp2(old - now), 1.0)
                codes[page, :, :, :lo - i * P] = code_bytes(
                    e4m3(was.view(torch.float8_e4m3fn).double() * f[..., None, None]))
            y = torch.where((now < 255)[..., None, None], torch.nan_to_num(new, 0.0, 0.0, 0.0), 0.0)
            codes[page, :, :, lo - i * P:hi - i * P] = code_bytes(e4m3(y * torch.exp2(127 - now.clamp_max(254))[..., None, None]))
            scales[page] = now.to(torch.uint8)
        t += n
    return codes, scales
