"""Timed cases of the operators on a cache of keys and values in 8 bits.

The cache lies in pages of P tokens: E4M3 codes [pages, 2 (keys, values), H, P, D]
and one E8M0 scale for each page, kind and head [pages, 2, H]. A table gives each
sequence's pages in order; lens[b] is its number of tokens, the new ones included;
its new tokens are rows starts[b] .. starts[b + 1] - 1 of the step's tensors.

  append  quantizes the new keys and values into their pages; a page that holds
          older tokens keeps the larger of its scale and the new tokens', and the
          older codes are brought to it
  attend  query i of n stands at position p = lens - n + i and attends tokens
          j in [max(0, p - window + 1), p]:  s = scale q.k_j, capped by
          cap tanh(s / cap), plus slope_h (j - p);  o = sum_j softmax(s)_j v_j,
          lse = ln sum_j exp(s_j)
  read    keys and values of whole sequences as bf16 or fp32

With `own` false, `run` computes them with elementary torch operations in 32
bits, rounded once at the end; with `own` true it makes the library's calls.
Codes are returned as float8_e4m3fn tensors and scales as float8_e8m0fnu
tensors: the values that the bytes stand for.
"""
from __future__ import annotations

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases ---

def _attend(name, B, lo, hi, n=1, Hq=32, H=8, D=128, P=64, window=0, cap=0.0, slopes=False, out="bf16", lse=False):
    return {"name": name, "op": "attend", "B": B, "lo": lo, "hi": hi, "n": n, "Hq": Hq, "H": H, "D": D, "P": P,
            "window": window, "cap": cap, "slopes": slopes, "out": out, "lse": lse}


def _append(name, B, lo, hi, new_lo, new_hi, H=8, D=128, P=64, x="bf16"):
    return {"name": name, "op": "append", "B": B, "lo": lo, "hi": hi, "new_lo": new_lo, "new_hi": new_hi, "H": H,
            "D": D, "P": P, "x": x}


def _read(name, B, lo, hi, H=8, D=128, P=64, out="bf16"):
    return {"name": name, "op": "read", "B": B, "lo": lo, "hi": hi, "H": H, "D": D, "P": P, "out": out}


def listed():
    return [
        # One token of one short conversation on an 8B-shaped layer (32 query heads on 8): latency.
        _attend("attend 1x777", 1, 777, 777),
        # One token on a very long document, 70B-shaped layer (64 query heads on 8): the cache's stream.
        _attend("attend 1x131072", 1, 131072, 131072, Hq=64),
        # A serving batch of ragged lengths, 70B-shaped layer, with the sums that joining parts needs.
        _attend("attend 64 x 130..8192", 64, 130, 8192, Hq=64, lse=True),
        # One to four proposed tokens of each sequence checked at once, small pages, fp32 result.
        _attend("attend 16 x 1000..16384, 4 tokens", 16, 1000, 16384, n=4, P=32, out="f32"),
        # Many short requests, a head of keys for each query head, a bias that falls with the distance.
        _attend("attend 200 x 9..601 d64 slopes", 200, 9, 601, Hq=24, H=24, D=64, P=16, slopes=True),
        # Wide heads, the last 1024 tokens alone, capped scores.
        _attend("attend 40 x 100..10000 d256 window", 40, 100, 10000, Hq=16, D=256, window=1024, cap=50.0),
        # One token of one sequence into its page: latency.
        _append("append 1x1", 1, 700, 700, 1, 1),
        # One token each of a large decode batch.
        _append("append 256x1", 256, 1, 600, 1, 1),
        # Prompts of five requests, 16 thousand tokens together, into fresh pages.
        _append("append prompts 5 x 500..8000", 5, 0, 0, 500, 8000),
        # Chunks of prompts that go on where a page is partly filled, fp32 keys and values, small pages.
        _append("append 13 x 21..900 f32 d64", 13, 11, 1777, 21, 900, H=5, D=64, P=16, x="f32"),
        # One short sequence back to fp32.
        _read("read 1x777 f32", 1, 777, 777, out="f32"),
        # A batch of sequences back to bf16, for a pass that works on whole prompts.
        _read("read 24 x 300..9000", 24, 300, 9000),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "read"])
    D, P = rng.choice([64, 96, 128, 128, 192, 256]), rng.choice([16, 32, 64, 128])
    H = rng.choice([1, 2, 3, 4, 8, 8, 16])
    B = _log_int(rng, 1, 256)
    hi = _log_int(rng, 16, 131072)
    most = 131072 * 8 * 128 // (H * D)
    if op == "attend":
        G, n = rng.choice([1, 2, 3, 4, 5, 7, 8, 16]), rng.choice([1, 1, 1, 2, 4, 7])
        hi = max(16, min(hi, most // (B * max(1, G * n // 8))))
        lo = _log_int(rng, 8, hi)
        c = _attend("", B, lo, hi, n, G * H, H, D, P,
                    rng.choice([0, 0, 0, _log_int(rng, 16, 8192)]), rng.choice([0.0, 0.0, 30.0]),
                    rng.random() < 0.25, rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.3)
    elif op == "append":
        new_hi = max(1, min(_log_int(rng, 1, 8192), 16384 * 1024 // (H * D) // B))
        c = _append("", B, 0, min(hi, 2000, most // 4 // B), _log_int(rng, 1, new_hi), new_hi, H, D, P,
                    rng.choice(["bf16", "bf16", "f32"]))
    else:
        hi = max(16, min(hi, most // 2 // B))
        c = _read("", B, _log_int(rng, 1, hi), hi, H, D, P, rng.choice(["bf16", "bf16", "f32"]))
    return {k: v for k, v in c.items() if k != "name"}


def _spread(B, lo, hi, shift):
    """B whole numbers from lo to hi, even on their logarithm, in a mixed order."""
    v = [int(round((lo + 1) * ((hi + 1) / (lo + 1)) ** (i / max(1, B - 1)))) - 1 for i in range(B)]
    return [v[(i * 37 + shift) % B] for i in range(B)] if B % 37 else v


def _sizes(case):
    """Tokens of each sequence (the new ones included), and how many of them are new."""
    B = case["B"]
    if case["op"] == "attend":
        new = [1 + (b * 5 + 3) % case["n"] if b else case["n"] for b in range(B)]
        return _spread(B, case["lo"], case["hi"], 0), new
    if case["op"] == "append":
        before, new = _spread(B, case["lo"], case["hi"], 1), _spread(B, case["new_lo"], case["new_hi"], 5)
        return [a + b for a, b in zip(before, new)], new
    lens = _spread(B, case["lo"], case["hi"], 0)
    return lens, lens


# ----------------------------------------------------------------- inputs ---

def _normal(shape, g, dtype):
    """Keys and values [..., D]: normal, one channel in 64 with eight times the spread."""
    x = torch.randn(shape, device="cuda", generator=g)
    cols = torch.randint(0, shape[-1], (max(1, shape[-1] // 64),), device="cuda", generator=g)
    x[..., cols] *= 8.0
    return x.to(dtype)


def _scale_exp(M):
    """The smallest e with 448 2^e >= M (448 = 0.875 2^9)."""
    m, e = torch.frexp(M)
    e = e - 9 + (m > 0.875).int()
    return torch.where(m == 0, -127, e).clamp(-127, 126)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, H, D, P = (case[k] for k in ("B", "H", "D", "P"))
    lens, new = _sizes(case)
    used = [-(-n // P) for n in lens]
    pages, most = sum(used) + 7, max(used)
    # pages in the order in which an allocator that has run for a while hands them out
    order = torch.randperm(pages, device="cuda", generator=g).int()
    row = torch.tensor([b for b in range(B) for _ in range(used[b])], device="cuda")
    col = torch.tensor([i for b in range(B) for i in range(used[b])], device="cuda")
    table = torch.full((B, most), -1, dtype=torch.int32, device="cuda")
    table[row, col] = order[:len(row)]
    codes = torch.empty((pages, 2, H, P, D), dtype=torch.uint8, device="cuda")
    scales = torch.empty((pages, 2, H), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // (2 * H * P * D))
    for i in range(0, pages, step):
        x = _normal((min(step, pages - i), 2, H, P, D), g, torch.float32)
        e = _scale_exp(x.abs().amax((3, 4)))
        codes[i:i + step] = torch.ldexp(x, -e[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        scales[i:i + step] = (e + 127).to(torch.uint8)
    at = [0]
    for n in new:
        at.append(at[-1] + n)
    s = {"case": case, "codes": codes, "scales": scales, "table": table, "T": at[-1],
         "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
         "starts": torch.tensor(at, dtype=torch.int32, device="cuda")}
    if case["op"] == "attend":
        # queries, keys and values side by side, as one product writes them
        Hq = case["Hq"]
        qkv = torch.randn((s["T"], Hq + 2 * H, D), device="cuda", generator=g).to(torch.bfloat16)
        s["q"] = qkv[:, :Hq]
        s["scale"] = D ** -0.5
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, Hq + 1, device="cuda") / Hq) if case["slopes"] else None
    elif case["op"] == "append":
        kv = _normal((s["T"], 2, H, D), g, TYPES[case["x"]])
        s["k"], s["v"] = kv[:, 0], kv[:, 1]
    return s


# ------------------------------------------------------------------- runs ---

def _values(codes, scales):
    """fp32 values of pages [..., P, D] with scales [...]."""
    return torch.ldexp(codes.view(torch.float8_e4m3fn).float(), scales.int()[..., None, None] - 127)


def _plain_append(s):
    c = s["case"]
    codes, scales, P = s["codes"], s["scales"], c["P"]
    x = torch.stack((s["k"], s["v"]), 1).float()                             # [T, 2, H, D]
    new = s["starts"][1:] - s["starts"][:-1]
    before = (s["lens"] - new).long()
    t = torch.arange(s["T"], device="cuda")
    b = torch.bucketize(t, s["starts"][1:].long(), right=True)
    pos = before[b] + t - s["starts"][b].long()
    page = s["table"][b, pos // P].long()
    # largest magnitude of the new tokens in each page
    M = torch.zeros(scales.shape, device="cuda").index_reduce_(0, page, x.abs().amax(3), "amax")
    need = _scale_exp(M) + 127
    # the page in which a sequence goes on: older tokens in its first before % P places
    first = s["table"].gather(1, (before // P)[:, None])[:, 0].long()
    older = before % P
    was = scales[first].int()
    now = torch.where((older > 0)[:, None, None], torch.maximum(was, need[first]), need[first])
    old = codes[first]
    v = torch.ldexp(old.view(torch.float8_e4m3fn).float(), (was - now)[..., None, None]).to(torch.float8_e4m3fn)
    keep = (torch.arange(P, device="cuda") < older[:, None])[:, None, None, :, None]
    codes[first] = torch.where(keep, v.view(torch.uint8), old)
    need[first] = now
    scales[page] = need[page].to(torch.uint8)
    codes[page, :, :, pos % P] = torch.ldexp(x, 127 - need[page][..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return {"codes": codes.view(torch.float8_e4m3fn), "scales": scales.view(torch.float8_e8m0fnu)}


def _plain_attend(s):
    c = s["case"]
    B, n, Hq, H, D, P = (c[k] for k in ("B", "n", "Hq", "H", "D", "P"))
    G = Hq // H
    pages = s["table"].clamp_min(0).long()                                    # [B, most]
    kv = _values(s["codes"][pages], s["scales"][pages])                       # [B, most, 2, H, P, D]
    L = pages.shape[1] * P
    k = kv[:, :, 0].permute(0, 2, 1, 3, 4).reshape(B, H, L, D)
    v = kv[:, :, 1].permute(0, 2, 1, 3, 4).reshape(B, H, L, D)
    new = (s["starts"][1:] - s["starts"][:-1]).long()
    i = torch.arange(n, device="cuda")
    rows = (s["starts"][:-1].long()[:, None] + torch.minimum(i, new[:, None] - 1))   # [B, n], the last one repeated
    q = s["q"][rows].float().view(B, n, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, n * G, D)
    z = (q @ k.transpose(2, 3)).view(B, H, n, G, L) * s["scale"]
    if c["cap"]:
        z = c["cap"] * torch.tanh(z / c["cap"])
    p = (s["lens"].long()[:, None] - new[:, None] + i)[:, None, :, None, None]        # positions
    j = torch.arange(L, device="cuda")
    if s["slopes"] is not None:
        z = z + s["slopes"].view(1, H, 1, G, 1) * (j - p).float()
    seen = (j <= p) & (j > p - c["window"]) if c["window"] else j <= p
    z = z.masked_fill(~seen, -math.inf)
    m = z.amax(-1, keepdim=True)
    e = torch.exp(z - m)
    sums = e.sum(-1, keepdim=True)
    o = (e.view(B, H, n * G, L) @ v).view(B, H, n, G, D) / sums
    o = o.permute(0, 2, 1, 3, 4).reshape(B * n, Hq, D)
    t = torch.arange(s["T"], device="cuda")
    b = torch.bucketize(t, s["starts"][1:].long(), right=True)
    at = b * n + t - s["starts"][b].long()
    out = {"out": o[at].to(TYPES[c["out"]])}
    if c["lse"]:
        out["lse"] = (m + torch.log(sums)).permute(0, 2, 1, 3, 4).reshape(B * n, Hq)[at]
    return out


def _plain_read(s):
    c = s["case"]
    P = c["P"]
    t = torch.arange(s["T"], device="cuda")
    b = torch.bucketize(t, s["starts"][1:].long(), right=True)
    pos = t - s["starts"][b].long()
    page = s["table"][b, pos // P].long()
    x = s["codes"][page, :, :, pos % P].view(torch.float8_e4m3fn).float()     # [T, 2, H, D]
    x = torch.ldexp(x, s["scales"][page].int()[..., None] - 127).to(TYPES[c["out"]])
    return {"k": x[:, 0].contiguous(), "v": x[:, 1].contiguous()}


def _own(s):
    import gemm_pt_block_gb300 as mx

    c = s["case"]
    if c["op"] == "attend":
        starts = None if c["n"] == 1 else s["starts"]
        out, lse = mx.mxfp8_cache_attention(s["q"], s["codes"], s["scales"], s["table"], s["lens"], starts=starts,
                                            scale=s["scale"], window=c["window"], softcap=c["cap"],
                                            slopes=s["slopes"], out_dtype=TYPES[c["out"]], with_lse=c["lse"])
        return {"out": out, "lse": lse} if c["lse"] else {"out": out}
    if c["op"] == "append":
        starts = None if c["new_hi"] == 1 else s["starts"]
        mx.mxfp8_cache_append(s["k"], s["v"], s["codes"], s["scales"], s["table"], s["lens"], starts=starts)
        return {"codes": s["codes"].view(torch.float8_e4m3fn), "scales": s["scales"].view(torch.float8_e8m0fnu)}
    k, v = mx.mxfp8_cache_read(s["codes"], s["scales"], s["table"], s["starts"], s["T"], out_dtype=TYPES[c["out"]])
    return {"k": k, "v": v}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return _plain_attend(state) if op == "attend" else _plain_append(state) if op == "append" else _plain_read(state)


# --------------------------------------------------------- what it has to do ---

def work(case):
    B, H, D, P = (case[k] for k in ("B", "H", "D", "P"))
    lens, new = _sizes(case)
    T = sum(new)
    if case["op"] == "attend":
        w, Hq = case["window"], case["Hq"]
        tokens = sum(L - (max(0, L - n - w + 1) if w else 0) for L, n in zip(lens, new))
        pairs = sum(min(max(0, L - n + i + 1), w or L) for L, n in zip(lens, new) for i in range(n))
        moved = 2 * tokens * H * D + 2 * tokens * H / P + 2 * T * Hq * D + T * Hq * D * (2 if case["out"] == "bf16" else 4)
        return {"bytes": moved + (4 * T * Hq if case["lse"] else 0), "flops": 4 * pairs * Hq * D}
    n = 2 * T * H * D
    each = 2 if case["x" if case["op"] == "append" else "out"] == "bf16" else 4
    return {"bytes": n * (each + 1) + 2 * T * H / P, "flops": 2 * n}


# ------------------------------------------------- the definition in 64 bits ---

def _tokens(s, b, count):
    """Keys and values [2, H, count, D] of a sequence's first tokens, in 64 bits."""
    P = s["case"]["P"]
    pages = s["table"][b, :-(-count // P)].long()
    x = s["codes"][pages].view(torch.float8_e4m3fn).double() * torch.exp2(s["scales"][pages].double() - 127.0)[..., None, None]
    return x.permute(1, 2, 0, 3, 4).reshape(2, x.shape[2], -1, x.shape[4])[:, :, :count]


def _exact_attend(s):
    c = s["case"]
    G = c["Hq"] // c["H"]
    lens, new = _sizes(c)
    out, lse, t = [], [], 0
    for b, (L, n) in enumerate(zip(lens, new)):
        kv = _tokens(s, b, L)
        k, v = kv[0].repeat_interleave(G, 0), kv[1].repeat_interleave(G, 0)    # [Hq, L, D]
        j = torch.arange(L, device="cuda", dtype=torch.float64)
        for i in range(n):
            p = L - n + i
            if p < 0:                                       # nothing to attend
                out.append(torch.zeros(c["Hq"], c["D"], device="cuda", dtype=torch.float64))
                lse.append(torch.full((c["Hq"],), -math.inf, device="cuda", dtype=torch.float64))
                continue
            lo = max(0, p - c["window"] + 1) if c["window"] else 0
            z = torch.einsum("hd,hld->hl", s["q"][t + i].double(), k[:, lo:p + 1]) * s["scale"]
            if c["cap"]:
                z = c["cap"] * torch.tanh(z / c["cap"])
            if s["slopes"] is not None:
                z = z + s["slopes"].double()[:, None] * (j[lo:p + 1] - p)
            lse.append(torch.logsumexp(z, 1))
            out.append(torch.einsum("hl,hld->hd", torch.exp(z - lse[-1][:, None]), v[:, lo:p + 1]))
        t += n
    return {"out": torch.stack(out), **({"lse": torch.stack(lse)} if c["lse"] else {})}


def _grid(v):
    """The nearest E4M3 value, ties to the even one."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def _exact_append(s):
    c = s["case"]
    P = c["P"]
    lens, new = _sizes(c)
    codes = s["codes"].view(torch.float8_e4m3fn).double()
    scales = torch.exp2(s["scales"].double() - 127.0)
    x = torch.stack((s["k"], s["v"]), 1).double()                              # [T, 2, H, D]
    table, t = s["table"].tolist(), 0
    for b, (L, n) in enumerate(zip(lens, new)):
        for at in range((L - n) // P, -(-L // P)):
            lo, hi = max(L - n, at * P), min(L, at * P + P)
            page, part = table[b][at], x[t + lo - (L - n):t + hi - (L - n)].permute(1, 2, 0, 3)
            scale = torch.exp2(torch.ceil(torch.log2(part.abs().amax((2, 3)).clamp_min(448 * 2.0 ** -127) / 448.0)))
            if lo > at * P:
                scale = torch.maximum(scale, scales[page])
                old = codes[page, :, :, :lo - at * P]
                codes[page, :, :, :lo - at * P] = _grid(old * (scales[page] / scale)[..., None, None])
            codes[page, :, :, lo - at * P:hi - at * P] = _grid(part / scale[..., None, None])
            scales[page] = scale
        t += n
    return {"codes": codes, "scales": scales}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attend":
        return _exact_attend(s)
    if case["op"] == "append":
        return _exact_append(s)
    parts = [_tokens(s, b, L) for b, L in enumerate(_sizes(case)[0])]
    return {"k": torch.cat([p[0].transpose(0, 1) for p in parts]), "v": torch.cat([p[1].transpose(0, 1) for p in parts])}
