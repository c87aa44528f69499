// cache.cu -- keys and values in 8 bits (sm_103a): quantization as they are
// written, reading them back, and attention over them.
#include <cstdint>
#include <cuda_runtime.h>
#include <mutex>

#include "internal.h"
#include "mx_device.cuh"
#include "ptx.cuh"
#include "tma_host.h"

namespace mx {
namespace {
// Error word of this translation unit (read and cleared by mxfp4_device_status).
__device__ uint32_t g_cache_error;
}  // namespace
}  // namespace mx
#define MX_BOUNDS_FAIL() atomicExch(&::mx::g_cache_error, ::mx::kErrBounds)
#include "row_device.cuh"

namespace mx {
namespace {

constexpr int kSms = 152;

__device__ __forceinline__ void index_fail() { atomicExch(&g_cache_error, kErrIndex); }

// One sequence of a call: its rows, its first row's position and its length.
struct Seq {
  int32_t row, n, pos, len;
};

// Sequence b's rows; false (and the error word) where starts leaves the tensor or falls.
__device__ __forceinline__ bool rows_of(const CacheArgs& c, int32_t b, Seq* s) {
  s->row = b;
  s->n = 1;
  if (c.starts) {
    s->row = __ldg(c.starts + b);
    const int32_t end = __ldg(c.starts + b + 1);
    if (s->row < 0 || end < s->row || end > c.tokens) {
      index_fail();
      return false;
    }
    s->n = end - s->row;
  }
  return true;
}

// Page i of sequence b, or -1 (and the error word) where there is none.
__device__ __forceinline__ int32_t page_of(const CacheArgs& c, int32_t b, int32_t i) {
  const int32_t p = i < c.max_pages ? __ldg(c.table + (int64_t)b * c.ld_table + i) : -1;
  if (p >= 0 && p < c.pages) return p;
  index_fail();
  return -1;
}

__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t v) {
  uint32_t r;
  asm("{.reg .b16 t, u;\n\tmov.b32 {t, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;}" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ float2 f16x2_f32(uint32_t v) {
  float2 r;
  asm("{.reg .b16 t, u;\n\tmov.b32 {t, u}, %2;\n\tcvt.f32.f16 %0, t;\n\tcvt.f32.f16 %1, u;}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(v));
  return r;
}
__device__ __forceinline__ void values4(uint32_t codes, float (&f)[4]) {
  const float2 a = f16x2_f32(e4m3x2_f16x2(codes)), b = f16x2_f32(e4m3x2_f16x2(codes >> 16));
  f[0] = a.x;
  f[1] = a.y;
  f[2] = b.x;
  f[3] = b.y;
}

// 2^(s - 127) of an E8M0 scale (0xFF: NaN).
__device__ __forceinline__ float scale_value(uint32_t s) {
  return s == 0 ? __uint_as_float(0x400000u) : s == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float(s << 23);
}

// ---------------------------------------------------------- append and read ---
//
// What one call writes (or reads) of a page is a slot; a slot's keys and values of
// all heads lie block by block, 2 heads of them. Streams of bytes, bound by HBM:
// 2 + 1 bytes an element for bf16. For long appends and reads some threads take a
// block, 32 elements each, and a CTA goes from block to block of its slot with the
// next one's loads under way; for a token or so a sequence a warp takes a block.

// A slot's sequence and page, tokens [lo, hi) of the page.
struct Slot {
  Seq s;
  int32_t page, at, lo, hi;
};

// Where each sequence's slots of the grid begin: one for each page that its n
// rows may touch. Rows that go on inside a page (kExtra 2) touch at most
// floor(n / P) + 2 pages, rows from a page's start (kExtra 1) floor(n / P) + 1,
// and floor(end / P) - floor(begin / P) >= floor(n / P).
template <int kExtra>
__device__ __forceinline__ int64_t first_slot(const CacheArgs& c, int32_t b, int shift) {
  return (int64_t)(__ldg(c.starts + b) >> shift) + (int64_t)kExtra * b;
}

// The last sequence whose slots begin at or before `slot` (where starts falls, some
// sequence), by whole warps: 32 places at a time.
template <int kExtra>
__device__ __forceinline__ int32_t find_sequence(const CacheArgs& c, int64_t slot, int shift, int lane) {
  int32_t lo = 0, count = c.sequences;
  while (count > 1) {
    const int32_t step = (count + 31) >> 5, at = lo + lane * step;
    const bool before = at < lo + count && first_slot<kExtra>(c, at, shift) <= slot;
    const int32_t k = max(__popc(__ballot_sync(0xffffffffu, before)) - 1, 0) * step;
    count = min(step, count - k);
    lo += k;
  }
  return lo;
}

// All lanes of a warp; false: nothing to do there.
template <int kExtra>
__device__ __forceinline__ bool slot_of(const CacheArgs& c, int lane, Slot* t) {
  const int shift = 31 - __clz(c.page_tokens);
  const int64_t slot = blockIdx.x;
  const int32_t b = c.starts ? find_sequence<kExtra>(c, slot, shift, lane) : (int32_t)slot;
  if (!rows_of(c, b, &t->s)) return false;
  if (kExtra == 2) {
    t->s.len = __ldg(c.lens + b);
    t->s.pos = t->s.len - t->s.n;
  } else {
    t->s.len = t->s.n;
    t->s.pos = 0;
  }
  if (t->s.pos < 0 || t->s.len > c.max_pages << shift) {
    index_fail();
    return false;
  }
  const int64_t k = c.starts ? slot - first_slot<kExtra>(c, b, shift) : 0;
  const int32_t first = t->s.pos >> shift;
  if (t->s.n == 0 || k < 0 || first + k > (t->s.len - 1) >> shift) return false;
  t->at = (first + (int32_t)k) << shift;
  t->page = page_of(c, b, first + (int32_t)k);
  if (t->page < 0) return false;
  t->lo = max(t->s.pos - t->at, 0);
  t->hi = min(t->s.len - t->at, c.page_tokens);
  return true;
}

// The E8M0 scale of a block whose largest magnitude has the bits m (as whole
// numbers: magnitudes, then infinity, then NaN): 448 = 1.75 * 2^8, one more where
// the fraction passes it.
__device__ __forceinline__ uint32_t scale_for(uint32_t m) {
  return m >= 0x7F800000u ? 255u : (uint32_t)max((int)(m >> 23) - 8 + ((m & 0x7FFFFFu) > 0x600000u), 0);
}
// What values are multiplied by under a scale (254, which only a page's older tokens can
// bring: 2^-127, below the normal numbers), and older codes where it grows (below 2^-30
// every code rounds to zero).
__device__ __forceinline__ float scale_factor(uint32_t scale) {
  return scale == 255u ? 0.0f : __uint_as_float(max((254u - scale) << 23, 0x400000u));
}
__device__ __forceinline__ float older_factor(uint32_t old, uint32_t scale) {
  return __uint_as_float((127u - min(scale - old, 64u)) << 23);
}
__device__ __forceinline__ uint32_t scaled4(uint32_t codes, float f) {
  float v[4];
  values4(codes, v);
  return e4m3x4(v[0] * f, v[1] * f, v[2] * f, v[3] * f);
}
__device__ __forceinline__ float most8(float m, const float (&f)[8]) {
  return absmax3_nan(absmax3_nan(m, f[0], f[1]), absmax3_nan(f[2], f[3], f[4]), absmax3_nan(f[5], f[6], f[7]));
}
__device__ __forceinline__ uint2 quantized8(const float (&f)[8], float mul, uint32_t scale) {
  if (scale == 255u) return make_uint2(0u, 0u);
  return make_uint2(e4m3x4(f[0] * mul, f[1] * mul, f[2] * mul, f[3] * mul),
                    e4m3x4(f[4] * mul, f[5] * mul, f[6] * mul, f[7] * mul));
}

// Largest magnitude's bits of sixteen elements (as fp32; bf16 two at a time, as the
// whole numbers that its bits are).
__device__ __forceinline__ uint32_t most16(const Vec16<uint16_t>& v) {
  const uint32_t w[8] = {v.v.a.x, v.v.a.y, v.v.a.z, v.v.a.w, v.v.b.x, v.v.b.y, v.v.b.z, v.v.b.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
  return max(m << 16, m & 0xFFFF0000u);
}
__device__ __forceinline__ uint32_t most16(const Vec16<float>& v) {
  float2 f[8];
  unpack16(v, f);
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = absmax3_nan(m, f[i].x, f[i].y);
  return __float_as_uint(m) & 0x7FFFFFFFu;
}

// A few new tokens a page: a warp takes a block, eight elements a lane at a time.
// Values past the first 256 * kHeld are read twice.
template <typename T, int kHeld>
__global__ void __launch_bounds__(256) cache_append_few_kernel(CacheArgs c, Heads k, Heads v) {
  const int lane = threadIdx.x & 31, task = blockIdx.y * 8 + (threadIdx.x >> 5);
  ptx::launch_dependents();
  if (task >= 2 * c.heads) return;
  Slot t;
  if (!slot_of<2>(c, lane, &t)) return;
  const int kind = task >= c.heads, h = task - kind * c.heads, per = c.head_dim >> 3;
  const Heads& x = kind ? v : k;
  const int64_t block = (int64_t)t.page * 2 * c.heads + task;
  uint8_t* codes = c.codes + block * c.page_tokens * c.head_dim;
  const uint32_t old = t.lo > 0 ? c.scales[block] : 0u;
  const T* from = static_cast<const T*>(x.p) + (int64_t)(t.s.row + (t.at + t.lo - t.s.pos)) * x.ld_t + (int64_t)h * x.ld_h;
  const int count = (t.hi - t.lo) * per;
  auto take = [&](int i, Vec8<T>& w) {
    const int token = i / per;
    load8(from + token * x.ld_t + (i - token * per) * 8, w);
  };
  Vec8<T> held[kHeld], w;
  float f[8], m = 0.0f;
#pragma unroll
  for (int z = 0; z < kHeld; ++z)
    if (lane + 32 * z < count) take(lane + 32 * z, held[z]);
#pragma unroll
  for (int z = 0; z < kHeld; ++z)
    if (lane + 32 * z < count) {
      unpack8(held[z], f);
      m = most8(m, f);
    }
  for (int i = lane + 32 * kHeld; i < count; i += 32) {
    take(i, w);
    unpack8(w, f);
    m = most8(m, f);
  }
  const uint32_t scale = max(scale_for(__reduce_max_sync(0xffffffffu, __float_as_uint(m) & 0x7FFFFFFFu)), old);
  const float mul = scale_factor(scale);
  uint2* to = reinterpret_cast<uint2*>(codes) + t.lo * per;
#pragma unroll
  for (int z = 0; z < kHeld; ++z)
    if (lane + 32 * z < count) {
      unpack8(held[z], f);
      put_at(to + lane + 32 * z, quantized8(f, mul, scale), c.codes, c.codes_bytes);
    }
  for (int i = lane + 32 * kHeld; i < count; i += 32) {
    take(i, w);
    unpack8(w, f);
    put_at(to + i, quantized8(f, mul, scale), c.codes, c.codes_bytes);
  }
  if (t.lo > 0 && old < scale && scale != 255u) {
    const float less = older_factor(old, scale);
    uint2* older = reinterpret_cast<uint2*>(codes);
    for (int i = lane; i < t.lo * per; i += 32) {
      const uint2 q = older[i];
      put_at(older + i, make_uint2(scaled4(q.x, less), scaled4(q.y, less)), c.codes, c.codes_bytes);
    }
  }
  if (lane == 0) put_at(c.scales + block, (uint8_t)scale, c.scales, c.scales_bytes);
}

// How threads share blocks: `each` of them (whole warps) take a block, two vectors
// of sixteen elements a thread, `at_once` blocks of a slot at a time.
struct Share {
  int32_t each, at_once;
};

template <typename T, int kMost>
__global__ void __launch_bounds__(kMost) cache_append_kernel(CacheArgs c, Heads k, Heads v, Share sh) {
  __shared__ uint32_t most[2][32];
  ptx::launch_dependents();
  Slot t;
  if (!slot_of<2>(c, threadIdx.x & 31, &t)) return;
  const int mine = threadIdx.x / sh.each, in = threadIdx.x - mine * sh.each, per = c.head_dim >> 4;
  const int blocks = 2 * c.heads, stride = gridDim.y * sh.at_once;
  int token[2], d[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int at = in + i * sh.each;
    token[i] = at / per;
    d[i] = (at - token[i] * per) << 4;
  }
  const int64_t row0 = t.s.row + (t.at - t.s.pos);
  Vec16<T> ahead[2];
  uint32_t ahead_old = 0;
  auto fetch = [&](int task) {
    const int kind = task >= c.heads, h = task - kind * c.heads;
    const Heads& x = kind ? v : k;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (token[i] < t.lo || token[i] >= t.hi) continue;
      const T* p = static_cast<const T*>(x.p) + (row0 + token[i]) * x.ld_t + (int64_t)h * x.ld_h + d[i];
      load16e(p, on32(p), ahead[i]);
    }
    if (t.lo > 0) ahead_old = c.scales[(int64_t)t.page * blocks + task];
  };
  int task = blockIdx.y * sh.at_once + mine;
  if (task < blocks) fetch(task);
  // (all threads go round alike: a CTA's blocks end together)
  for (int round = 0; blockIdx.y * sh.at_once + round * stride < blocks; ++round, task += stride) {
    const bool some = task < blocks;
    const uint32_t old = ahead_old;
    const Vec16<T> now[2] = {ahead[0], ahead[1]};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (some && token[i] >= t.lo && token[i] < t.hi) m = max(m, most16(now[i]));
    if (task + stride < blocks) fetch(task + stride);
    const uint32_t bits = __reduce_max_sync(0xffffffffu, m);
    uint32_t all = bits;
    if (sh.each > 32) {
      uint32_t* slots = most[round & 1];
      if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = bits;
      __syncthreads();
      const int w0 = mine * sh.each >> 5;
      for (int w = 0; w < sh.each >> 5; ++w) all = max(all, slots[w0 + w]);
    }
    if (!some) continue;
    const int64_t block = (int64_t)t.page * blocks + task;
    uint8_t* codes = c.codes + block * c.page_tokens * c.head_dim;
    const uint32_t scale = max(scale_for(all), old);
    const float mul = scale_factor(scale);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint4* to = reinterpret_cast<uint4*>(codes + token[i] * c.head_dim + d[i]);
      if (token[i] >= t.lo && token[i] < t.hi) {
        float2 f[8];
        unpack16(now[i], f);
        uint4 q = make_uint4(0u, 0u, 0u, 0u);
        if (scale != 255u) {
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] = f2mul(f[j], make_float2(mul, mul));
          q = encode16_fp8(f, false);
        }
        put_at(to, q, c.codes, c.codes_bytes);
      } else if (token[i] < t.lo && old < scale && scale != 255u) {
        const float less = older_factor(old, scale);
        const uint4 q = *to;
        put_at(to, make_uint4(scaled4(q.x, less), scaled4(q.y, less), scaled4(q.z, less), scaled4(q.w, less)), c.codes,
               c.codes_bytes);
      }
    }
    if (in == 0) put_at(c.scales + block, (uint8_t)scale, c.scales, c.scales_bytes);
  }
}

template <typename T>
__global__ void __launch_bounds__(1024) cache_read_kernel(CacheArgs c, Heads k, Heads v, Share sh) {
  Slot t;
  if (!slot_of<1>(c, threadIdx.x & 31, &t)) return;
  const int mine = threadIdx.x / sh.each, in = threadIdx.x - mine * sh.each, per = c.head_dim >> 4;
  const int blocks = 2 * c.heads, stride = gridDim.y * sh.at_once;
  int token[2], d[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int at = in + i * sh.each;
    token[i] = at / per;
    d[i] = (at - token[i] * per) << 4;
  }
  uint4 ahead[2];
  uint32_t ahead_scale = 0;
  auto fetch = [&](int task) {
    const int64_t block = (int64_t)t.page * blocks + task;
    const uint8_t* codes = c.codes + block * c.page_tokens * c.head_dim;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (token[i] < t.hi) ahead[i] = load16(codes + token[i] * c.head_dim + d[i]);
    ahead_scale = c.scales[block];
  };
  int task = blockIdx.y * sh.at_once + mine;
  if (task < blocks) fetch(task);
  for (; task < blocks; task += stride) {
    const uint4 now[2] = {ahead[0], ahead[1]};
    const float mul = scale_value(ahead_scale);
    if (task + stride < blocks) fetch(task + stride);
    const int kind = task >= c.heads, h = task - kind * c.heads;
    const Heads& x = kind ? v : k;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (token[i] >= t.hi) continue;
      const uint32_t q[4] = {now[i].x, now[i].y, now[i].z, now[i].w};
      T* to = static_cast<T*>(x.p) + (int64_t)(t.s.row + t.at + token[i]) * x.ld_t + (int64_t)h * x.ld_h + d[i];
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        float a[4], b[4], f[8];
        values4(q[2 * z], a);
        values4(q[2 * z + 1], b);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f[j] = a[j] * mul;
          f[j + 4] = b[j] * mul;
        }
        Vec8<T> w;
        pack8(f, w);
        store8(to + 8 * z, w, x.p, x.bytes);
      }
    }
  }
}

// ----------------------------------------------------------------- attention ---
//
// With s_j a row's scores in log2 units and 2^ev_j the scale of token j's values,
//   out = (sum_j 2^s_j 2^ev_j code_j) / (sum_j 2^s_j)
// in one pass over the tokens with two running maxima, m = max s_j for the
// denominator and m + lift, lift = max (s_j - m + ev_j), for the numerator, whose
// weights are then at most one whatever the pages' scales are.
//
// The work is cut into units of 32 or 64 tokens of one sequence, one head of the cache
// and one tile of query rows (the rows of the query heads that share the head,
// over the sequence's new tokens), and every warp of the GPU takes an equal run of
// them, whatever the lengths: seven to fourteen warps of a CTA an SM that multiply, and
// one or two that fetch for them by TMA, keys and values apart, into a ring for each.
// A warp holds maxima and sums of its tile by itself; nothing in its loop waits for
// another. Codes become f16 in registers (exact), keys as the A operand of S^T = K
// Q^T, values, transposed as they are read, as that of O^T = V^T P^T: query rows
// are the instruction's N of eight. Tiles that several warps share are joined in
// the CTA when its runs end; those that several CTAs share leave their parts in
// the workspace for cache_join_kernel.
//
// One tile a head is bound by HBM from 96 channels on (1 x 131072 tokens, 8 heads of
// 128: 51 us, 77 % of a copy's rate), by the latency of scores and conversions
// at 64 (32 x 4096 tokens 32 us, 62 %; half of the issue slots are empty: what follows one
// another in a unit is not overlapped inside a warp); several tiles a head read again from L2 and
// convert again (16 sequences of 1000 to 16384 tokens, 16 rows a head: 53 us, 53 %). A
// call's least is its start and the join, about 6 us.

constexpr float kTop = 15.0f;                   // weights are held times 2^15: f16 keeps 2^-39 of the largest
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr int kMostWarps = 14, kMostStages = 8;
constexpr int kRows = 8;  // of a tile: sixteen, for half the conversions, gained 7 % at 16 rows and lost 20 % at 4 to 16

template <int D>
struct Attn {
  // Warps that multiply: as many as their registers (sums D / 4, queries D / 8 of
  // them) leave room for on the SM without spilling in earnest (at most 4 bytes, at 64
  // channels and for fp32 results at 192 and 256; 128 channels: 50.6 us at 131072
  // tokens with eleven, 57 with fifteen, which spill 180 and more, 58 with seven). Then those that
  // fetch for them, a lane for 16 tokens of a unit; a warp's copies go out one after
  // the other, and pages of 16 tokens of 64 channels need two (32 x 4096 tokens 33 us;
  // 48 with one).
  static constexpr int kWarps = D <= 64 ? 14 : D <= 128 ? 11 : 7;
  static constexpr int kFetch = D <= 64 ? 2 : 1;
  static constexpr int kFetched = kWarps / kFetch;  // warps that one fetches for
  static constexpr int kThreads = (kWarps + kFetch) * 32;
  // Bytes of a row in one slab, swizzled so that eight rows of 16 bytes lie in
  // different banks. 96 bytes are not swizzled: rows three apart meet in pairs, which
  // costs less than copies in slabs of 32 (32 x 4096 tokens: 43.8 us, 48.7).
  static constexpr int kBox = D == 96 ? 96 : D % 128 == 0 ? 128 : 64;
  // Tokens of a unit, in parts of 16 (64 channels: 200 sequences of 9 to 601 tokens 33 us
  // with 64, 39 with 32; more than 64 channels have no registers for 64).
  static constexpr int kChunk = D == 64 ? 64 : 32;
  static constexpr int kParts = kChunk / 16;
  static constexpr int kLanes = 32 / kParts;                               // of a fetching warp for one part
  static constexpr int kPart = 16 * D;                                     // a part's keys or values
  static constexpr int kStage = kChunk * D;                                // a unit's
  static constexpr int kQuads = D / 16 * 32;                               // of a tile's sums (below)
  static constexpr int kFixed = 2 * kWarps * 3 * kRows * 4 + 5120;
  static constexpr int kFit = (227 * 1024 - 1024 - kFixed) / (kWarps * kStage);
  static constexpr int kStages = kFit < kMostStages ? kFit : kMostStages;  // of a warp's ring
  static constexpr int kBytes = 1024 + kWarps * kStages * kStage + kFixed;
  // The warp that a fetching warp's lane fetches for.
  static __device__ __forceinline__ int fetched(int warp, int lane) {
    return (warp - kWarps) * kFetched + min(lane % kLanes, kFetched - 1);
  }
  static_assert(kStages >= 3 && kQuads * 16 <= kStages * kStage && kFetched <= kLanes, "ring");
};

// A tile: rows row0 .. row0 + rows - 1 of a sequence's (first token `token`), of one head.
struct Tile {
  int32_t token, row0, rows, head;
};

// Where a run begins: its sequence, as Walk has it, and the unit in that.
struct Start {
  int32_t b, n, row, len, tiles, units, at, unused;
};

struct AttnCtl {
  uint64_t full[kMostWarps][kMostStages], empty[kMostWarps][kMostStages];
  int32_t block[kMostWarps][kMostStages][4];  // of the keys in a stage's parts (-1: none)
  Tile head[kMostWarps], open[kMostWarps];       // tiles that a warp shares with the one before it, and behind it
  Start start[kMostWarps];               // of the warps' runs
  int32_t left[kMostWarps];                  // units of the open tile behind a warp's run, but for the spare one
  uint8_t has[kMostWarps];                   // kHead, kOpen, kBegan
  uint32_t abort;
};
static_assert(sizeof(AttnCtl) <= 5120, "control block");
// A warp's run ended a tile that began before it; it ends inside a tile; that tile began before it.
enum : uint8_t { kHead = 1, kOpen = 2, kBegan = 4 };

// A tile that goes on behind a CTA, for the join: over so many CTAs (0: none does).
struct Split {
  Tile tile;
  int32_t parts, unused[3];
};

// Floats of the workspace: a Split for each CTA, then two parts each (a tile
// that began before it, a tile that goes on behind it): maxima, lifts, sums and
// numerators; then the numerators of each warp's first tile.
__host__ __device__ constexpr int64_t part_floats(int D) { return (int64_t)kRows * D + 3 * kRows; }

// Bounded wait (about 2 s); the whole warp goes on or leaves together.
__device__ __forceinline__ bool wait_bar_warp(uint32_t bar, uint32_t parity, uint32_t* abort) {
  bool ok = ptx::mbar_try_wait(bar, parity);
  if (!ok) {
    const uint64_t t0 = ptx::globaltimer_ns();
    while (!(ok = ptx::mbar_try_wait_sleep(bar, parity, 100000u))) {
      if (*reinterpret_cast<volatile uint32_t*>(abort)) break;
      if (ptx::globaltimer_ns() - t0 > kWaitLimitNs) {
        *reinterpret_cast<volatile uint32_t*>(abort) = 1u;
        atomicExch(&g_cache_error, 6u);  // MXFP4_ERR_TIMEOUT
        break;
      }
    }
  }
  return __all_sync(0xffffffffu, ok);
}

// The same with a barrier for each lane that `need`s it.
__device__ __forceinline__ bool wait_bars(uint32_t bar, uint32_t parity, bool need, uint32_t* abort) {
  bool ok = !need || ptx::mbar_try_wait(bar, parity);
  if (__all_sync(0xffffffffu, ok)) return true;
  const uint64_t t0 = ptx::globaltimer_ns();
  for (;;) {
    if (!ok) ok = ptx::mbar_try_wait_sleep(bar, parity, 10000u);
    if (__all_sync(0xffffffffu, ok)) return true;
    bool out = *reinterpret_cast<volatile uint32_t*>(abort) != 0;
    if (ptx::globaltimer_ns() - t0 > kWaitLimitNs) {
      *reinterpret_cast<volatile uint32_t*>(abort) = 1u;
      atomicExch(&g_cache_error, 6u);  // MXFP4_ERR_TIMEOUT
      out = true;
    }
    if (__any_sync(0xffffffffu, out)) return false;
  }
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t f16x2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ void ldsm(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void tma_pages(uint32_t dst, const CUtensorMap* map, int32_t half, int32_t block, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %2, %2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(half), "r"(block), "r"(bar)
      : "memory");
}
template <int kWarps>
__device__ __forceinline__ void warps_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
}

// 2^e for a whole e, 0 below the smallest normal number.
__device__ __forceinline__ float pow2i(int e) { return e < -126 ? 0.0f : __uint_as_float((uint32_t)(min(e, 127) + 127) << 23); }

// r / G for a tile's rows: the multiplication for an invariant divisor of Granlund
// and Montgomery (1994), its numbers from the host.
__device__ __forceinline__ int32_t token_of(const AttentionArgs& a, int32_t r) {
  const uint32_t t = __umulhi(a.group_mul, (uint32_t)r);
  return (int32_t)((t + (((uint32_t)r - t) >> a.group_shift[0])) >> a.group_shift[1]);
}

// What a call says of one sequence, as it lies in memory. (This kernel starts while
// the one before it runs, which may write any of its inputs: ordinary loads, none
// by the path for data that stay as they are for a kernel's whole life.)
struct Said {
  int32_t row, end, len;
};
__device__ __forceinline__ Said said(const CacheArgs& c, int32_t b) {
  return Said{c.starts ? c.starts[b] : b, c.starts ? c.starts[b + 1] : b + 1, c.lens[b]};
}

// A place in the order of all units: sequences, their heads, their tiles of
// kRows query rows, kChunk tokens at a time. A sequence's tiles count alike (the
// longest's units): units that a tile has no tokens for are passed over. So is, where
// there are several sequences, one more of each tile (a.spare), which stands for what a
// tile costs by itself, its queries and results, about a unit's time: 200 sequences of 9
// to 601 tokens, 64 channels, 34.7 us, 37.9 without; 64 of 130 to 8192, 128 channels,
// 50.7 and 52.8; but 256 of 300 tokens each 53.8 and 51.4, and one of a single token
// would take 6.7 and takes 6.1.
template <int kChunk>
struct Walk {
  int32_t b, n, row, len, tiles, units;  // sequence: rows, first row, length, tiles, units of each
  int32_t head, tile, unit;
  int32_t row0, p0, lo, hi;  // tile: first row, its position, tokens [lo, hi) that a row attends; lo rounded down
  Said ahead;                // of sequence b + 1

  // Takes sequence s, of which the call says x; its number of units (below kMostUnits).
  __device__ __forceinline__ int32_t take(const AttentionArgs& a, int32_t s, const Said& x) {
    const int G = a.group;
    b = s;
    row = x.row;
    n = 0;
    if (x.row < 0 || x.end < x.row || x.end > a.c.tokens)
      index_fail();
    else
      n = x.end - x.row;
    if (n == 0) return 0;
    len = x.len;
    const int32_t most = a.c.max_pages * a.c.page_tokens;
    if (len < 0 || len > most) {
      index_fail();
      len = len < 0 ? 0 : most + 1;
    }
    tiles = (n * G + kRows - 1) / kRows;
    const int32_t tokens = (kRows + G - 2) / G + 1;  // that a tile's rows may belong to
    const int32_t span = a.window > 0 ? min(len, a.window + tokens + kChunk) : len;
    units = max(1, (span + kChunk - 1) / kChunk) + a.spare;
    return a.c.heads * tiles * units;
  }
  // Unit u of the sequence, where a run begins.
  __device__ __forceinline__ void place(const AttentionArgs& a, int32_t u) {
    ahead = said(a.c, min(b + 1, a.c.sequences - 1));
    const uint32_t t = (uint32_t)u / (uint32_t)units;
    unit = u - (int32_t)t * units;
    head = (int32_t)(t / (uint32_t)tiles);
    tile = (int32_t)t - head * tiles;
    set_tile(a);
  }
  __device__ __forceinline__ void begin(const AttentionArgs& a, const Start& x) {
    b = x.b;
    n = x.n;
    row = x.row;
    len = x.len;
    tiles = x.tiles;
    units = x.units;
    place(a, x.at);
  }
  __device__ __forceinline__ void set_tile(const AttentionArgs& a) {
    const int G = a.group;
    row0 = tile * kRows;
    p0 = len - n + token_of(a, row0);
    hi = max(0, len - n + token_of(a, min(row0 + kRows, n * G) - 1) + 1);
    lo = a.window > 0 ? max(0, p0 - a.window + 1) & -kChunk : 0;
  }
  __device__ __forceinline__ int32_t token() const { return lo + unit * kChunk; }
  // Whether this unit holds tokens to attend.
  __device__ __forceinline__ bool live() const { return token() < hi; }
  __device__ __forceinline__ bool last(const AttentionArgs& a) const { return unit == units - 1 - a.spare; }
  __device__ __forceinline__ bool spare(const AttentionArgs& a) const { return unit == units - a.spare; }
  __device__ __forceinline__ Tile rows(int G) const { return Tile{row, row0, min(n * G - row0, kRows), head}; }
  // The next unit (there is one).
  __device__ __forceinline__ void next(const AttentionArgs& a) {
    if (++unit < units) return;
    unit = 0;
    if (++tile == tiles) {
      tile = 0;
      if (++head == a.c.heads) {
        head = 0;
        bool some = false;
        while (!some && b + 1 < a.c.sequences) {
          some = take(a, b + 1, ahead) != 0;
          ahead = said(a.c, min(b + 1, a.c.sequences - 1));
        }
      }
    }
    set_tile(a);
  }
};

// All units in equal runs, one for each warp of the CTAs that work: warp i of
// them (CTA i / kWarps) begins at begin(i).
struct Cut {
  int32_t each, more, ctas;  // the first `more` runs have one more
  int32_t base;              // this CTA's first run
  __device__ __forceinline__ int32_t begin(int32_t i) const { return each * i + min(i, more); }
};
template <int kWarps>
__device__ __forceinline__ Cut cut(int32_t units) {
  Cut c;
  c.ctas = (int32_t)min(gridDim.x, ((uint32_t)units + kWarps - 1) / kWarps);
  const uint32_t runs = (uint32_t)max(c.ctas, 1) * kWarps;
  c.each = (int32_t)((uint32_t)units / runs);
  c.more = units - c.each * (int32_t)runs;
  c.base = (int32_t)blockIdx.x * kWarps;
  return c;
}

// Inclusive sums over a warp's lanes.
__device__ __forceinline__ int32_t warp_sums(int32_t v, int lane) {
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    const int32_t u = __shfl_up_sync(0xffffffffu, v, i);
    if (lane >= i) v += u;
  }
  return v;
}

// Row starts that fall may name rows twice, and more units than 32 bits count: such a
// call does nothing. Units are summed over 2^10 for this; what that rounds off (65535
// sequences) keeps the limit below 2^31, and the host's keeps right calls below the limit.
constexpr uint32_t kTooHigh = ((1u << 31) - (1u << 26)) >> 10;
static_assert(kMostUnits <= (1ll << 31) - (1 << 27), "limits");
__device__ __forceinline__ int32_t counted(int32_t units, uint32_t high) {
  if (high < kTooHigh) return units;
  index_fail();
  return 0;
}

// Where the runs of this CTA's warps begin. Up to 32 sequences every warp looks at
// them for itself, a lane at one, and has its run's first unit in w (lanes of the
// fetching warp: that of the warp they fetch for); more are the whole CTA's, a thread looks
// at one, and the runs' beginnings go to ctl. Ends with a barrier.
template <int D, int kChunk>
__device__ __forceinline__ Cut find_start(const AttentionArgs& a, int warp, int lane, AttnCtl* ctl, int32_t* sums,
                                          Walk<kChunk>* w) {
  using S = Attn<D>;
  constexpr int kWarps = S::kWarps;
  const bool few = a.c.sequences <= 32;
  const int32_t mine_at = few ? lane : (int32_t)threadIdx.x;
  Walk<kChunk> x{};
  const int32_t mine = mine_at < a.c.sequences ? x.take(a, mine_at, said(a.c, mine_at)) : 0;
  const int32_t upto = warp_sums(mine, lane);
  if (few) {
    const uint32_t high = __reduce_add_sync(0xffffffffu, (uint32_t)mine >> 10);
    Cut runs = cut<kWarps>(counted(__shfl_sync(0xffffffffu, upto, 31), high));
    const int32_t in = warp < kWarps ? warp : S::fetched(warp, lane);
    // No more tiles than CTAs, and no run longer for it: a CTA takes a tile, and no parts
    // are left to join (1 x 100 tokens 9.0 us without, 7.0; 16 x 700 12.6, 10.9).
    const int32_t tiles = mine ? a.c.heads * x.tiles : 0, tiles_upto = warp_sums(tiles, lane);
    const int32_t longest = __reduce_max_sync(0xffffffffu, mine ? x.units : 0) - a.spare;
    const bool whole = runs.ctas > 0 && (longest + kWarps - 1) / kWarps <= runs.each + (runs.more > 0) &&
                       __shfl_sync(0xffffffffu, tiles_upto, 31) <= (int32_t)gridDim.x;
    const int32_t begin = whole ? (int32_t)blockIdx.x : runs.begin(runs.base + in), ends = whole ? tiles_upto : upto;
    int32_t s = 0;  // sequences that end before
    for (int32_t i = 0; i < a.c.sequences; ++i) s += __shfl_sync(0xffffffffu, ends, i) <= begin;
    s = min(s, a.c.sequences - 1);
    Start y;
    y.b = s;
    y.n = __shfl_sync(0xffffffffu, x.n, s);
    y.row = __shfl_sync(0xffffffffu, x.row, s);
    y.len = __shfl_sync(0xffffffffu, x.len, s);
    y.tiles = __shfl_sync(0xffffffffu, x.tiles, s);
    y.units = __shfl_sync(0xffffffffu, x.units, s);
    y.at = begin - __shfl_sync(0xffffffffu, ends - (whole ? tiles : mine), s);
    if (whole) {
      const int32_t units = y.units - a.spare;
      runs.ctas = __shfl_sync(0xffffffffu, tiles_upto, 31);
      runs.base = 0;
      runs.each = units / kWarps;
      runs.more = units - runs.each * kWarps;
      y.at = y.at * y.units + runs.begin(in);
    }
    if (y.n > 0) w->begin(a, y);
    __syncthreads();
    return runs;
  }
  // all units, then the sequences again, as many at a time as there are threads
  constexpr int kThreads = S::kThreads;
  const bool once = a.c.sequences <= kThreads;
  uint32_t more = mine, high = more >> 10;
  for (int32_t s = mine_at + kThreads; s < a.c.sequences; s += kThreads) {
    const uint32_t units = x.take(a, s, said(a.c, s));
    more += units;
    high = min(high + (units >> 10), 1u << 22);  // (past the limit)
  }
  more = warp_sums(more, lane);
  high = __reduce_add_sync(0xffffffffu, high);
  if (lane == 31) {
    sums[warp] = more;
    sums[kThreads / 32 + warp] = high;
  }
  __syncthreads();
  uint32_t all = 0, all_high = 0;
  int32_t before = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    all += sums[i];
    all_high += sums[kThreads / 32 + i];
  }
  const Cut runs = cut<kWarps>(counted(all, all_high));
  for (int32_t from = 0; from < a.c.sequences; from += kThreads) {
    const int32_t s = from + mine_at;
    int32_t units = mine, within = upto;
    if (!once) {
      units = s < a.c.sequences ? x.take(a, s, said(a.c, s)) : 0;
      within = warp_sums(units, lane);
      __syncthreads();
      if (lane == 31) sums[warp] = within;
      __syncthreads();
    }
    int32_t at = before + within - units;  // units before this sequence
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
      if (i < warp) at += sums[i];
      before += sums[i];
    }
    for (int i = 0; i < kWarps; ++i) {
      const int32_t u = runs.begin(runs.base + i) - at;
      if (u >= 0 && u < units) ctl->start[i] = Start{s, x.n, x.row, x.len, x.tiles, x.units, u, 0};
    }
  }
  __syncthreads();
  return runs;
}

// Sums of a tile in the accumulators' order, four floats for each of 32 lanes:
// quad e belongs to rows 2 (lane % 4) (elements 0, 2) and the one behind (1, 3),
// channels 16 (e / 32) + 2 (lane / 4) and the one behind.
struct Quad {
  int row, d;
};
__device__ __forceinline__ Quad quad(int e) {
  const int lane = e & 31, i = e >> 5;
  return Quad{2 * (lane & 3), 16 * i + 2 * (lane >> 2)};
}

// Row r of a sequence's n * G rows: the tensors' row and the query head.
__device__ __forceinline__ int64_t row_of(const AttentionArgs& a, const Heads& x, int32_t token, int32_t head, int32_t r) {
  const int32_t i = token_of(a, r);
  return (int64_t)(token + i) * x.ld_t + (int64_t)(head * a.group + r - i * a.group) * x.ld_h;
}
__device__ __forceinline__ void put2(const AttentionArgs& a, int64_t at, float x, float y) {
  if (a.out_f32)
    put_at(static_cast<float*>(a.out.p) + at, make_float2(x, y), a.out.p, a.out.bytes);
  else
    put_at(static_cast<uint16_t*>(a.out.p) + at, bf16x2(x, y), a.out.p, a.out.bytes);
}
// What a numerator is multiplied by, one after the other (their product may leave
// fp32 where the result does not): 1 / sum out of the weights' units, and
// the values' scale. No token: 0.
__device__ __forceinline__ float2 last_factors(float lift, float sum) {
  float e;
  asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(lift));
  return sum == 0.0f ? make_float2(0.0f, 0.0f) : make_float2((1.0f / sum) * 0x1p-15f, e);
}
// The maximum of no scores: finite, so that differences with it are numbers.
constexpr float kLowest = -3.4e38f;
// A row's maximum, lift and sum of several parts.
struct Joined {
  float m, lift, sum;
};
__device__ __forceinline__ void put_lse(const AttentionArgs& a, int32_t token, int32_t head, int32_t r, float m, float sum) {
  const int32_t i = token_of(a, r);
  const int64_t at = (int64_t)(token + i) * a.q_heads + head * a.group + r - i * a.group;
  put_at(a.lse + at, sum == 0.0f ? -INFINITY : (m + lg2(sum)) * 0.693147180559945f, a.lse, a.lse_bytes);
}

template <int D, bool kExact>
__global__ void __launch_bounds__(Attn<D>::kThreads, 1)
    cache_attention_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ AttentionArgs a) {
  using S = Attn<D>;
  constexpr int kWarps = S::kWarps, kSegs = D / 16, kStages = S::kStages, kStat = 3 * kRows;
  constexpr int kChunk = S::kChunk, kParts = S::kParts;
  constexpr int kIn = S::kBox / 16;  // segments of 16 channels in a slab
  extern __shared__ uint8_t raw[];
  uint8_t* base = raw + ((1024u - (ptx::smem_u32(raw) & 1023u)) & 1023u);
  float* stats = reinterpret_cast<float*>(base + kWarps * kStages * S::kStage);  // of warps' open tiles, then of their heads
  AttnCtl* ctl = reinterpret_cast<AttnCtl*>(base + kWarps * kStages * S::kStage + S::kFixed - 5120);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = a.group;
  const uint32_t ring = ptx::smem_u32(base), full = ptx::smem_u32(ctl->full), empty = ptx::smem_u32(ctl->empty);

  if (warp == kWarps) {
    for (int i = lane; i < kWarps * kMostStages; i += 32) {
      ptx::mbar_init(full + 8 * i, 1);
      ptx::mbar_init(empty + 8 * i, 1);
    }
    if (lane == 0) {
      ctl->abort = 0;
      ptx::prefetch_tensormap(&map);
    }
    ptx::fence_mbar_init();
  }
  ptx::wait_prior_grid();  // (nothing of the call's is read or written before)
  ptx::launch_dependents();  // (only now: what starts next may count on all before this kernel)
  Walk<kChunk> w;
  const bool few = a.c.sequences <= 32;
  const Cut runs = find_start<D, kChunk>(a, warp, lane, ctl, reinterpret_cast<int32_t*>(stats), &w);
  if (blockIdx.x >= runs.ctas) {
    if (a.ws && threadIdx.x == 0) put_at(&reinterpret_cast<Split*>(a.ws)[blockIdx.x].parts, (int32_t)0, a.ws, a.ws_bytes);
    return;
  }

  if (warp >= kWarps) {
    // ------------------------------------------------------------ fetching ---
    // Lanes i, i + kLanes, .. walk warp i's run and fetch a part of its units each;
    // the table is read a unit ahead. A copy is of a page's tokens, or a unit's.
    const int i = S::fetched(warp, lane), part = lane / S::kLanes;
    const int32_t units = lane % S::kLanes < S::kFetched
                              ? runs.begin(runs.base + i + 1) - runs.begin(runs.base + i) : 0;
    const int32_t rounds = __reduce_max_sync(0xffffffffu, units);
    const int copy = min(a.c.page_tokens, kChunk);
    const bool leads = (16 * part & (copy - 1)) == 0;  // a copy begins with this part
    struct Page {
      int32_t page, head, place;  // page: -1 a wrong one, -2 none to load
      bool live;
    };
    auto page_at = [&]() {
      Page x{-2, w.head, 0, w.live()};
      const int32_t j = w.token() + 16 * part;
      // (pages that end before every row's window may be gone)
      if (j < w.hi && (a.window == 0 || (j | (a.c.page_tokens - 1)) > w.p0 - a.window)) {
        x.place = (j & (a.c.page_tokens - 1)) >> 4;
        x.page = j >> a.shift < a.c.max_pages ? a.c.table[(int64_t)w.b * a.c.ld_table + (j >> a.shift)] : -1;
      }
      return x;
    };
    Page ahead{-2, 0, 0, false};
    if (units > 0) {
      if (!few) w.begin(a, ctl->start[i]);
      ahead = page_at();
    }
    const uint32_t my_ring = ring + i * kStages * S::kStage, my_full = full + 8 * kMostStages * i, my_empty = empty + 8 * kMostStages * i;
    int32_t tiles = 0, stage = 0;
    uint32_t parity = 1;  // of the stage's reader
    bool go = true;
    for (int32_t round = 0; round < rounds && go; ++round) {
      const Page now = ahead;
      const bool mine = round < units && now.live;
      int32_t block = -1;
      if (mine) {
        if (now.page >= 0 && now.page < a.c.pages)
          block = now.page * 2 * a.c.heads + now.head;
        else if (now.page != -2)
          index_fail();
      }
      int32_t bytes = block >= 0 && leads ? copy * D : 0;
#pragma unroll
      for (int z = S::kLanes; z < 32; z <<= 1) bytes += __shfl_xor_sync(0xffffffffu, bytes, z);
#pragma unroll
      for (int kind = 0; kind < 2; ++kind) {
        go = go && wait_bars(my_empty + 8 * stage, parity, mine && tiles >= kStages, &ctl->abort);
        if (kind == 0 && mine && go) ctl->block[i][stage][part] = block;
        __syncwarp();
        if (mine && go) {
          const uint32_t bar = my_full + 8 * stage;
          if (part == 0) ptx::mbar_arrive_expect_tx(bar, bytes);
          if (block >= 0 && leads)
            tma_pages(my_ring + stage * S::kStage + part * S::kPart, &map, now.place, block + (kind ? a.c.heads : 0), bar);
          ++tiles;
          if (++stage == kStages) {
            stage = 0;
            parity ^= 1u;
          }
        }
      }
      if (round + 1 < units) {
        w.next(a);
        ahead = page_at();
      }
    }
    if (!go) {
      // the last load into each stage lands (bounded wait) before the CTA's memory goes
      const uint64_t t0 = ptx::globaltimer_ns();
      for (int32_t z = max(tiles - kStages, 0); z < tiles; ++z)
        while (!ptx::mbar_try_wait(my_full + 8 * (uint32_t)(z % kStages), (uint32_t)(z / kStages) & 1) &&
               ptx::globaltimer_ns() - t0 < kWaitLimitNs / 10) {
        }
    }
    return;
  }

  // ----------------------------------------------------------- multiplying ---
  const int g = lane >> 2, t = lane & 3;
  // ldmatrix rows: matrix lane / 8 holds tokens 8 (m % 2) .. of part m / 2 of two
  const int mrow = ((lane >> 3) & 1) * 8 + (lane & 7);
  const uint32_t swz = S::kBox == 128 ? mrow & 7 : S::kBox == 64 ? (mrow >> 1) & 3 : 0;
  auto segment = [](uint32_t at, int i) {
    return (S::kBox == 96 ? at + 16 * i : at ^ ((i % kIn) << 4)) + (i / kIn) * 16 * S::kBox;
  };
  const uint32_t my_ring = ring + warp * kStages * S::kStage;
  const uint32_t lane_at = my_ring + (lane >> 4) * S::kPart + mrow * S::kBox + (swz << 4);
  const uint32_t my_full = full + 8 * kMostStages * warp, my_empty = empty + 8 * kMostStages * warp;
  const float scale2 = a.scale * 1.44269504088896f, cap = a.softcap > 0.0f ? a.scale / a.softcap : 0.0f;
  float* heads = a.ws + gridDim.x * (sizeof(Split) / 4 + 2 * part_floats(D));  // (used with a workspace only)

  uint32_t qf[kSegs][2];
  float o[kSegs][4], m[2], lift[2], sum[2], unit_q[2];
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      m[i] = kLowest;
      lift[i] = sum[i] = 0.0f;
    }
#pragma unroll
    for (int s = 0; s < kSegs; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[s][i] = 0.0f;
  };
  clear();
  int32_t stage = 0;
  uint32_t parity = 0;
  bool go = true;
  uint8_t has = 0;
  const int32_t units = runs.begin(runs.base + warp + 1) - runs.begin(runs.base + warp);
  if (units && !few) w.begin(a, ctl->start[warp]);

  for (int32_t u = 0; u < units; ++u) {
    if (w.spare(a)) {
      if (u + 1 < units) w.next(a);
      continue;
    }
    if (u == 0 || w.unit == 0) {
      // queries of this tile, row by row times a power of two: the largest in [2^14, 2^15)
      uint2 x[kSegs];
      uint32_t top = 0;
#pragma unroll
      for (int s = 0; s < kSegs; ++s) x[s] = make_uint2(0u, 0u);
      if (w.row0 + g < w.n * G) {
        const uint16_t* q = static_cast<const uint16_t*>(a.q.p) + row_of(a, a.q, w.row, w.head, w.row0 + g) + 4 * t;
#pragma unroll
        for (int s = 0; s < kSegs; ++s) x[s] = *reinterpret_cast<const uint2*>(q + 16 * s);
      }
#pragma unroll
      for (int s = 0; s < kSegs; ++s)
        top = max(max(top, max((x[s].x << 16) & 0x7FFFFFFFu, x[s].x & 0x7FFF0000u)),
                  max((x[s].y << 16) & 0x7FFFFFFFu, x[s].y & 0x7FFF0000u));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = max((int)(top >> 23), 1);  // value = f16 * 2^(e - 141); 255: no number
      const float f1 = pow2i(min(141 - e, 126)), f2 = pow2i(max(141 - e - 126, 0));
#pragma unroll
      for (int s = 0; s < kSegs; ++s) {
        const float2 lo = unpack2(x[s].x), hi = unpack2(x[s].y);
        qf[s][0] = e == 255 ? 0u : f16x2(lo.x * f1 * f2, lo.y * f1 * f2);
        qf[s][1] = e == 255 ? 0u : f16x2(hi.x * f1 * f2, hi.y * f1 * f2);
      }
      // 2^(e - 141), down to 2^-140
      const float uq = e == 255 ? __uint_as_float(0x7FC00000u) : e > 14 ? pow2i(e - 141) : __uint_as_float(1u << (e + 8));
      // (the lanes' scores are of rows 2 t and 2 t + 1)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        unit_q[i] = __shfl_sync(0xffffffffu, uq, 8 * t + 4 * i);
      }
    }

    if (w.live() && go) go = wait_bar_warp(my_full + 8 * stage, parity, &ctl->abort);
    if (w.live() && go) {
      const int32_t c0 = w.token();
      // scales: a lane a part, the keys', then the values'
      const int32_t block = ctl->block[warp][stage][lane % kParts];
      uint32_t scale = 255u;
      if (block >= 0) scale = a.c.scales[block + (lane & kParts ? a.c.heads : 0)];
      float s[kParts][4];
#pragma unroll
      for (int h = 0; h < kParts; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[h][i] = 0.0f;
      {
        const uint32_t at = lane_at + stage * S::kStage;
#pragma unroll
        for (int i = 0; i < kSegs; ++i) {
#pragma unroll
          for (int h = 0; h < kParts; h += 2) {
            uint32_t r[4];
            ldsm(segment(at, i) + h * S::kPart, r);
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const uint32_t a0 = e4m3x2_f16x2(r[2 * z]), a2 = e4m3x2_f16x2(r[2 * z] >> 16);
              const uint32_t a1 = e4m3x2_f16x2(r[2 * z + 1]), a3 = e4m3x2_f16x2(r[2 * z + 1] >> 16);
              mma(s[h + z], a0, a1, a2, a3, qf[i][0], qf[i][1]);
            }
          }
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(my_empty + 8 * stage);
        if (++stage == kStages) {
          stage = 0;
          parity ^= 1u;
        }
      }

      // scores in log2 units; -infinity where a row does not attend
      // (a tile of one row: odd rows, which no lane needs, are left out. At 64 channels,
      // where scores are most of the work: 200 sequences 34.8 us without, 33.5 with; at 96,
      // 32 x 4096 tokens 42.3 and 42.8)
      const bool single = D == 64 && w.n * G - w.row0 == 1;
      const bool whole = c0 + kChunk <= w.p0 + 1 && (a.window == 0 || c0 > w.hi - 1 - a.window);
#pragma unroll
      for (int h = 0; h < kParts; ++h) {
        const float ks = scale_value(__shfl_sync(0xffffffffu, scale, h));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float f = unit_q[i] * ks;  // (a power of two)
          if (a.softcap > 0.0f) {
#pragma unroll
            for (int z = i; z < 4; z += 2) s[h][z] = a.softcap * 1.44269504088896f * tanhf(s[h][z] * (f * cap));
          } else {
            s[h][i] *= f * scale2;
            s[h][i + 2] *= f * scale2;
          }
        }
      }
      if (a.slopes || !whole) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (i == 1 && single) continue;
          const int32_t r = min(w.row0 + 2 * t + i, w.n * G - 1), token = token_of(a, r);
          const int32_t j0 = c0 + g - (w.len - w.n + token);  // the first token's position less the row's
          const float slope = a.slopes ? a.slopes[w.head * G + r - token * G] * 1.44269504088896f : 0.0f;
          const int32_t most = a.window > 0 ? a.window : 0x7FFFFFFF;
#pragma unroll
          for (int z = 0; z < 2 * kParts; ++z) {
            const int32_t j = j0 + 8 * z;
            float& x = s[z >> 1][i + 2 * (z & 1)];
            x += slope * (float)j;
            if (j > 0 || j <= -most) x = -INFINITY;
          }
        }
      }

      if (go) go = wait_bar_warp(my_full + 8 * stage, parity, &ctl->abort);
      float ev[kParts];
      bool one = true;  // all values under one scale
#pragma unroll
      for (int h = 0; h < kParts; ++h) {
        const uint32_t vs = __shfl_sync(0xffffffffu, scale, kParts + h);
        ev[h] = vs == 255u ? __uint_as_float(0x7FC00000u) : (float)((int)vs - 127);
        one = one && ev[h] == ev[0];
      }
      const uint32_t gone = __ballot_sync(0xffffffffu, block < 0);
      if (c0 + kChunk > w.hi || gone) {
        // tokens behind the last, parts without a page: whatever lies there must not
        // meet a weight of zero
        for (int i = lane; i < kChunk * kSegs; i += 32) {
          const int r = i / kSegs, seg = i % kSegs;
          if (c0 + r < w.hi && !(gone >> (r >> 4) & 1)) continue;
          const uint32_t at = my_ring + stage * S::kStage + (r >> 4) * S::kPart + (seg / kIn) * 16 * S::kBox +
                              (r & 15) * S::kBox + (seg % kIn) * 16;
          asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0) : "memory");
        }
        ptx::fence_proxy_async();
        __syncwarp();
      }

      // running maxima, and the weights
      uint32_t pf[kParts][2], pl[kParts][2];
      bool moved = false;
      float keep[2];
      float cm[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        cm[i] = m[i];
        keep[i] = 1.0f;
        if (i == 1 && single) continue;
        float part[kParts], x = -INFINITY;
#pragma unroll
        for (int h = 0; h < kParts; ++h) {
          part[h] = fmaxf(s[h][i], s[h][i + 2]);
          x = fmaxf(x, part[h]);
        }
#pragma unroll
        for (int z = 4; z < 32; z <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, z));
        cm[i] = fmaxf(m[i], x);
        float y = x - cm[i] + ev[0];
        if (!one) {
          y = -INFINITY;
#pragma unroll
          for (int h = 0; h < kParts; ++h) y = fmaxf(y, part[h] - cm[i] + ev[h]);
#pragma unroll
          for (int z = 4; z < 32; z <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, z));
        }
        const float down = m[i] - cm[i], was = down + lift[i], now = fmaxf(was, y);
        sum[i] *= ex2(down);
        keep[i] = ex2(was - now);
        moved |= was != now;
        m[i] = cm[i];
        lift[i] = now;
      }
#pragma unroll
      for (int h = 0; h < kParts; ++h) {
        const float c[2] = {ev[h] + kTop - lift[0], ev[h] + kTop - lift[1]};
        float p[4];
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          p[z] = 0.0f;
          if ((z & 1) && single) continue;
          const float x = s[h][z] - cm[z & 1];
          sum[z & 1] += ex2(x);
          p[z] = ex2(x + c[z & 1]);
        }
        if (ev[h] != ev[h]) {
          // values that are no numbers: where a row attends them
#pragma unroll
          for (int z = 0; z < 4; ++z) p[z] = s[h][z] == -INFINITY ? 0.0f : ev[h];
        }
        const uint32_t u0 = f16x2(p[0], p[1]), u1 = f16x2(p[2], p[3]);
        pf[h][0] = transposed(u0);
        pf[h][1] = transposed(u1);
        if (kExact) {
          const float2 q0 = f16x2_f32(u0), q1 = f16x2_f32(u1);
          pl[h][0] = transposed(f16x2(p[0] - q0.x, p[1] - q0.y));
          pl[h][1] = transposed(f16x2(p[2] - q1.x, p[3] - q1.y));
        }
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int i = 0; i < kSegs; ++i)
#pragma unroll
          for (int z = 0; z < 4; ++z) o[i][z] *= keep[z & 1];
      }
      // (the tensor core's sums round toward zero: for fp32 results a unit's are its own,
      // and join the tile's to nearest. 16 sequences of 1000 to 16384 tokens, 4 new: off by
      // 3.3e-7 of the result's norm at 52.9 us, by 1.5e-6 at 52.1 with one running sum)
      const uint32_t at = lane_at + stage * S::kStage;
#pragma unroll
      for (int i = 0; i < kSegs; ++i) {
        float own[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int h = 0; h < kParts; h += 2) {
          uint32_t r[4];
          ldsm_t(segment(at, i) + h * S::kPart, r);
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            // two tokens of a channel side by side, the even channel below
            const uint32_t x = __byte_perm(r[2 * z], 0, 0x3120), y = __byte_perm(r[2 * z + 1], 0, 0x3120);
            const uint32_t a0 = e4m3x2_f16x2(x), a1 = e4m3x2_f16x2(x >> 16), a2 = e4m3x2_f16x2(y), a3 = e4m3x2_f16x2(y >> 16);
            if (kExact) mma(own, a0, a1, a2, a3, pl[h + z][0], pl[h + z][1]);
            mma(kExact ? own : o[i], a0, a1, a2, a3, pf[h + z][0], pf[h + z][1]);
          }
        }
        if (kExact)
#pragma unroll
          for (int z = 0; z < 4; ++z) o[i][z] += own[z];
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(my_empty + 8 * stage);
      if (++stage == kStages) {
        stage = 0;
        parity ^= 1u;
      }
    }

    has = kOpen | (u < w.unit ? kBegan : 0) | (has & kHead);
    if (w.last(a)) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int z = 4; z < 32; z <<= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], z);
      const Tile tile = w.rows(G);
      if (u >= w.unit) {
        // a tile of this warp alone
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = 2 * t + i;
          if (r < tile.rows) {
            const float2 k = last_factors(lift[i], sum[i]);
            const int64_t at = row_of(a, a.out, tile.token, tile.head, tile.row0 + r) + 2 * g;
#pragma unroll
            for (int s = 0; s < kSegs; ++s) put2(a, at + 16 * s, o[s][i] * k.x * k.y, o[s][i + 2] * k.x * k.y);
            if (a.lse && g == 0) put_lse(a, tile.token, tile.head, tile.row0 + r, m[i], sum[i]);
          }
        }
        has &= kHead;
      } else {
        // the end of a tile that began before
        float4* to = reinterpret_cast<float4*>(heads) + ((int64_t)blockIdx.x * kWarps + warp) * S::kQuads + lane;
#pragma unroll
        for (int s = 0; s < kSegs; ++s) put_at(to + 32 * s, make_float4(o[s][0], o[s][1], o[s][2], o[s][3]), a.ws, a.ws_bytes);
        if (g == 0) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float* st = stats + (kWarps + warp) * kStat + 2 * t + i;
            st[0] = m[i];
            st[kRows] = lift[i];
            st[2 * kRows] = sum[i];
          }
        }
        if (lane == 0) ctl->head[warp] = tile;
        has = kHead;
      }
      clear();
    }
    if (u + 1 < units) w.next(a);
  }

  // ---------------------------------------------------- joining in the CTA ---
  if ((has & kOpen) || units == 0) {  // (an empty run adds nothing to the tile around it)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int z = 4; z < 32; z <<= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], z);
      if (g == 0) {
        float* st = stats + warp * kStat + 2 * t + i;
        st[0] = m[i];
        st[kRows] = lift[i];
        st[2 * kRows] = sum[i];
      }
    }
    // (this warp's ring: its loads have all been read)
    float4* to = reinterpret_cast<float4*>(base + warp * kStages * S::kStage) + lane;
    __syncwarp();
#pragma unroll
    for (int s = 0; s < kSegs; ++s) to[32 * s] = make_float4(o[s][0], o[s][1], o[s][2], o[s][3]);
  }
  if (lane == 0) {
    ctl->has[warp] = has;
    if (has & kOpen) {
      ctl->open[warp] = w.rows(G);
      ctl->left[warp] = w.units - 1 - a.spare - w.unit;
    }
  }
  warps_sync<kWarps>();

  // Tiles that warps share, all of them at once. Warps first .. last have one: open
  // in all but the last, which ends it, or open to the CTA's end. `before`: it
  // began before this CTA.
  const uint8_t h = lane < kWarps ? ctl->has[lane] : 0;
  const uint32_t heads_in = __ballot_sync(0xffffffffu, h & kHead), open_in = __ballot_sync(0xffffffffu, h & kOpen);
  const uint32_t begun_in = open_in & ~__ballot_sync(0xffffffffu, h & kBegan);
  // (a warp ends a tile before it leaves one open)
  const int ended = __popc(heads_in), groups = ended + (open_in != 0 && open_in >= 1u << max(31 - __clz(heads_in), 0));
  struct Group {
    int first, last;
    bool closed, before;
  };
  auto group = [&](int i) {
    Group x{0, kWarps - 1, i < ended, false};
    uint32_t up_to = 0xffffffffu;  // warps in which the tile may have begun
    if (x.closed) {
      uint32_t left = heads_in;
      for (int z = 0; z < i; ++z) left &= left - 1;
      x.last = __ffs(left) - 1;
      up_to = (1u << x.last) - 1;
    }
    const uint32_t in = begun_in & up_to, ends = heads_in & up_to;
    const int at = 31 - __clz(in);  // -1: none
    x.before = at < 31 - __clz(ends) || !in;
    x.first = x.before ? 0 : at;
    return x;
  };
  // a warp a tile, and nothing waits for another from here on
#pragma unroll 1
  for (int i = warp; i < groups; i += kWarps) {
    const Group x = group(i);
    const bool final = x.closed && !x.before;
    const int opens = x.last + !x.closed;  // members that have it open: first .. opens - 1
    const float4* ending = reinterpret_cast<const float4*>(heads) + ((int64_t)blockIdx.x * kWarps + x.last) * S::kQuads + lane;
    float4 sums[kSegs];
#pragma unroll
    for (int s = 0; s < kSegs; ++s) sums[s] = x.closed ? ending[32 * s] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    // statistics: a lane a row, four lanes take its members in turn
    const int r = lane & 7;
    auto stat = [&](int z) { return stats + ((z == opens ? kWarps : 0) + z) * kStat + r; };
    Joined j = {kLowest, -INFINITY, 0.0f};
    for (int z = x.first + (lane >> 3); z <= x.last; z += 4) j.m = fmaxf(j.m, stat(z)[0]);
#pragma unroll
    for (int d = 8; d < 32; d <<= 1) j.m = fmaxf(j.m, __shfl_xor_sync(0xffffffffu, j.m, d));
    for (int z = x.first + (lane >> 3); z <= x.last; z += 4) {
      const float* st = stat(z);
      const float down = st[0] - j.m;
      j.lift = fmaxf(j.lift, down + st[kRows]);
      j.sum += st[2 * kRows] * ex2(down);
    }
#pragma unroll
    for (int d = 8; d < 32; d <<= 1) {
      j.lift = fmaxf(j.lift, __shfl_xor_sync(0xffffffffu, j.lift, d));
      j.sum += __shfl_xor_sync(0xffffffffu, j.sum, d);
    }
    for (int z = x.first + (lane >> 3); z <= x.last; z += 4) {
      // (a member's maximum has done its part: its factor takes the place)
      float* st = stat(z);
      st[0] = ex2(st[0] - j.m + st[kRows] - j.lift);
    }
    __syncwarp();
    // numerators: this lane's quads
    float2 f;
    if (x.closed) {
      f = *reinterpret_cast<const float2*>(stats + (kWarps + x.last) * kStat + 2 * t);
#pragma unroll
      for (int s = 0; s < kSegs; ++s) sums[s] = make_float4(sums[s].x * f.x, sums[s].y * f.y, sums[s].z * f.x, sums[s].w * f.y);
    }
    for (int z = x.first; z < opens; ++z) {
      f = *reinterpret_cast<const float2*>(stats + z * kStat + 2 * t);
      const float4* from = reinterpret_cast<const float4*>(base + z * kStages * S::kStage) + lane;
#pragma unroll
      for (int s = 0; s < kSegs; ++s) {
        const float4 y = from[32 * s];
        sums[s] = make_float4(fmaf(y.x, f.x, sums[s].x), fmaf(y.y, f.y, sums[s].y), fmaf(y.z, f.x, sums[s].z),
                              fmaf(y.w, f.y, sums[s].w));
      }
    }
    if (final) {
      const Tile tile = ctl->head[x.last];
      const float2 k = last_factors(j.lift, j.sum);
      if (a.lse && lane < tile.rows && lane < kRows) put_lse(a, tile.token, tile.head, tile.row0 + r, j.m, j.sum);
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const float k1 = __shfl_sync(0xffffffffu, k.x, 2 * t + z), k2 = __shfl_sync(0xffffffffu, k.y, 2 * t + z);
        if (2 * t + z >= tile.rows) continue;
        const int64_t at = row_of(a, a.out, tile.token, tile.head, tile.row0 + 2 * t + z) + 2 * g;
#pragma unroll
        for (int s = 0; s < kSegs; ++s)
          put2(a, at + 16 * s, (z ? sums[s].y : sums[s].x) * k1 * k2, (z ? sums[s].w : sums[s].z) * k1 * k2);
      }
    } else {
      float* ws = a.ws + gridDim.x * (sizeof(Split) / 4) + (2 * (int64_t)blockIdx.x + !x.before) * part_floats(D);
      if (lane < kRows) {
        put_at(ws + r, j.m, a.ws, a.ws_bytes);
        put_at(ws + kRows + r, j.lift, a.ws, a.ws_bytes);
        put_at(ws + 2 * kRows + r, j.sum, a.ws, a.ws_bytes);
      }
#pragma unroll
      for (int s = 0; s < kSegs; ++s) put_at(reinterpret_cast<float4*>(ws + 3 * kRows) + 32 * s + lane, sums[s], a.ws, a.ws_bytes);
    }
  }
  if (threadIdx.x == 0 && a.ws) {
    Split sp = {{0, 0, 0, 0}, 0, {0, 0, 0}};
    const Group x = group(ended);
    if (groups > ended && !x.before) {
      // the CTAs up to the tile's last unit
      const int32_t at = runs.begin((blockIdx.x + 1) * kWarps) - 1 + ctl->left[31 - __clz(open_in)];
      int32_t c = blockIdx.x + 1;
      while (c < runs.ctas && runs.begin(c * kWarps) <= at) ++c;
      sp.tile = ctl->open[x.first];
      sp.parts = c - (int32_t)blockIdx.x;
    }
    put_at(reinterpret_cast<Split*>(a.ws) + blockIdx.x, sp, a.ws, a.ws_bytes);
  }
}

// Joins the parts of the tile that goes on behind CTA blockIdx.x: a warp for a
// row's statistics, a lane for a part; then as many groups of threads as fit take
// every so many-th part each. How many parts there are is known only when the first
// load is back: statistics of 32 parts and the first numerators are asked for
// beside it, whatever they hold.
constexpr int kJoinThreads = 512;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) cache_join_kernel(const __grid_constant__ AttentionArgs a) {
  constexpr int kQuads = Attn<D>::kQuads, kGroups = kJoinThreads / kQuads, kEarly = 4;
  static_assert(kGroups >= 1, "a quad a thread");
  __shared__ float factors[kSms][kRows];
  __shared__ float2 last[kRows];
  __shared__ float4 sums[kGroups > 1 ? kJoinThreads : 1];
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5, group = threadIdx.x / kQuads, e = threadIdx.x % kQuads;
  // part 0 is this CTA's second, the others the first of the CTAs behind it
  const float* parts = a.ws + gridDim.x * (sizeof(Split) / 4) + 2 * (int64_t)blockIdx.x * part_floats(D);
  auto part = [&](int i) { return parts + (2 * i + (i == 0)) * part_floats(D); };
  const int behind = gridDim.x - blockIdx.x;  // parts that the workspace has room for
  ptx::wait_prior_grid();
  ptx::launch_dependents();
  const Split sp = reinterpret_cast<const Split*>(a.ws)[blockIdx.x];
  constexpr int kMost = (kSms + 31) / 32;
  float m[kMost], lift[kMost], sum[kMost];
  auto statistics = [&](int i, int count) {
    const bool some = 32 * i + lane < count;
    const float* p = part(some ? 32 * i + lane : 0) + (row < kRows ? row : 0);
    m[i] = p[0];
    lift[i] = p[kRows];
    sum[i] = p[2 * kRows];
  };
  statistics(0, behind);
  float4 early[kEarly];
#pragma unroll
  for (int k = 0; k < kEarly; ++k) {
    const int i = group + k * kGroups;
    early[k] = *reinterpret_cast<const float4*>(part(i < behind ? i : 0) + 3 * kRows + 4 * e);
  }
  if (sp.parts == 0) return;
  if (row < kRows) {
    float top = kLowest, high = -INFINITY, all = 0.0f;
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      if (i > 0 && 32 * i < sp.parts) statistics(i, sp.parts);
      if (32 * i + lane >= sp.parts) {
        m[i] = kLowest;
        lift[i] = sum[i] = 0.0f;
      }
      top = fmaxf(top, m[i]);
    }
    for (int z = 16; z; z >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, z));
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      high = fmaxf(high, m[i] - top + lift[i]);
      all += sum[i] * ex2(m[i] - top);
    }
    for (int z = 16; z; z >>= 1) {
      high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, z));
      all += __shfl_xor_sync(0xffffffffu, all, z);
    }
#pragma unroll
    for (int i = 0; i < kMost; ++i)
      if (32 * i + lane < sp.parts) factors[32 * i + lane][row] = ex2(m[i] - top + lift[i] - high);
    if (lane == 0) {
      last[row] = last_factors(high, all);
      if (a.lse && row < sp.tile.rows) put_lse(a, sp.tile.token, sp.tile.head, sp.tile.row0 + row, top, all);
    }
  }
  __syncthreads();
  const Quad qd = quad(e);
  float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  auto add = [&](int i, const float4& y) {
    const float f0 = factors[i][qd.row], f1 = factors[i][qd.row + 1];
    x = make_float4(fmaf(y.x, f0, x.x), fmaf(y.y, f1, x.y), fmaf(y.z, f0, x.z), fmaf(y.w, f1, x.w));
  };
  if (group < kGroups) {
#pragma unroll
    for (int k = 0; k < kEarly; ++k)
      if (group + k * kGroups < sp.parts) add(group + k * kGroups, early[k]);
#pragma unroll 8
    for (int i = group + kEarly * kGroups; i < sp.parts; i += kGroups)
      add(i, *reinterpret_cast<const float4*>(part(i) + 3 * kRows + 4 * e));
  }
  if (kGroups > 1) {
    sums[threadIdx.x] = x;
    __syncthreads();
  }
  if (group > 0) return;
#pragma unroll
  for (int i = 1; i < kGroups; ++i) {
    const float4 y = sums[i * kQuads + e];
    x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = qd.row + i;
    if (r < sp.tile.rows)
      put2(a, row_of(a, a.out, sp.tile.token, sp.tile.head, sp.tile.row0 + r) + qd.d,
           (i ? x.y : x.x) * last[r].x * last[r].y, (i ? x.w : x.z) * last[r].x * last[r].y);
  }
}

}  // namespace

namespace {
// A block's threads, blocks at once and a slot's CTAs: about 256 threads to a CTA,
// which goes round at most four times (the lookups before a CTA's first load cost as
// much as a round: 15503 tokens in bf16 24.7 us with one round, 21.7 with two, 20.6
// with four; read back, 63622 tokens, 81, 76 and 73, and 79 with sixteen, whose CTAs
// end unevenly), and fewer times where there are not six CTAs an SM otherwise.
struct Launch {
  Share share;
  dim3 grid, block;
};
Launch launch_shape(const CacheArgs& c, int64_t slots) {
  Launch l;
  l.share.each = (c.page_tokens * c.head_dim / 32 + 31) / 32 * 32;
  l.share.at_once = l.share.each < 256 ? 256 / l.share.each : 1;
  const int blocks = 2 * c.heads, threads = l.share.each * l.share.at_once, most = (blocks + l.share.at_once - 1) / l.share.at_once;
  const int64_t fill = ((int64_t)kSms * 6 * 256 + slots * threads - 1) / (slots * threads), four = (most + 3) / 4;
  const int64_t want = fill > four ? fill : four;
  l.grid = dim3((unsigned)slots, (unsigned)(want < most ? want : most));
  l.block = dim3((unsigned)threads);
  return l;
}
}  // namespace

cudaError_t launch_cache_append(const CacheArgs& c, const Heads& k, const Heads& v, bool f32, cudaStream_t st) {
  if (c.tokens == 0 || c.sequences == 0) return cudaSuccess;
  (void)cudaGetLastError();
  const int64_t slots = c.starts ? c.tokens / c.page_tokens + 2 * (int64_t)c.sequences : c.sequences;
  // A warp a block while it holds a sequence's new elements in registers: 1024 (heads of
  // 128: 256 sequences of 8 tokens 6.1 us, 14.1 by whole CTAs; 8 of them 3.2 and 3.1),
  // or 2048 where there are blocks enough (32 sequences of 16 tokens on 8 heads 4.2 and 5.0,
  // 256 of them 8.7 and 15.4; but 16 of them 4.1 and 3.5). One row each is 256 at most.
  const int64_t elems = (int64_t)c.tokens * c.head_dim, blocks = 2 * (int64_t)c.heads * c.sequences;
  const bool held4 = elems <= 1024 * (int64_t)c.sequences, held8 = elems <= 2048 * (int64_t)c.sequences && blocks >= 512;
  if (!c.starts || held4 || held8) {
    const dim3 grid((unsigned)slots, (unsigned)((2 * c.heads + 7) / 8));
    (f32 ? !c.starts ? cache_append_few_kernel<float, 1>
           : held4 ? cache_append_few_kernel<float, 4> : cache_append_few_kernel<float, 8>
         : !c.starts ? cache_append_few_kernel<uint16_t, 1>
           : held4 ? cache_append_few_kernel<uint16_t, 4> : cache_append_few_kernel<uint16_t, 8>)
        <<<grid, 256, 0, st>>>(c, k, v);
    return cudaGetLastError();
  }
  const Launch l = launch_shape(c, slots);
  // (fp32 in blocks of more than 512 threads, pages of 128 tokens of 192 and 256 channels, spills 104 bytes:
  // 8 prompts of 2048 tokens, 256 channels, 52 % of a copy's rate; 76 % at 128)
  (f32 ? l.block.x <= 512 ? cache_append_kernel<float, 512> : cache_append_kernel<float, 1024>
       : l.block.x <= 512 ? cache_append_kernel<uint16_t, 512> : cache_append_kernel<uint16_t, 1024>)
      <<<l.grid, l.block, 0, st>>>(c, k, v, l.share);
  return cudaGetLastError();
}

cudaError_t launch_cache_read(const CacheArgs& c, const Heads& k, const Heads& v, bool f32, cudaStream_t st) {
  if (c.tokens == 0 || c.sequences == 0) return cudaSuccess;
  (void)cudaGetLastError();
  const Launch l = launch_shape(c, c.tokens / c.page_tokens + (int64_t)c.sequences);
  (f32 ? cache_read_kernel<float> : cache_read_kernel<uint16_t>)<<<l.grid, l.block, 0, st>>>(c, k, v, l.share);
  return cudaGetLastError();
}

namespace {
// How a call is cut, by what the host knows of it: warps of a CTA, CTAs, whether a
// tile may be split, units at most.
struct AttnShape {
  int warps, ctas;
  bool split;
  int64_t units;
};
template <int D>
AttnShape attn_shape(const AttentionArgs& a) {
  using S = Attn<D>;
  const int64_t G = a.group, rows = a.c.tokens * G, tiles = rows / kRows + a.c.sequences;
  const int64_t most = (int64_t)a.c.max_pages * a.c.page_tokens + 1, windowed = a.window + (kRows + G - 2) / G + 1 + S::kChunk;
  const int64_t span = a.window > 0 && windowed < most ? windowed : most;
  const int64_t units = (span + S::kChunk - 1) / S::kChunk, all = tiles * a.c.heads * (units + a.spare), runs = (all + S::kWarps - 1) / S::kWarps;
  const int64_t ctas = tiles * a.c.heads > runs ? tiles * a.c.heads : runs;  // (a tile a CTA, at most)
  return AttnShape{S::kWarps, (int)(ctas < kSms ? ctas : kSms), units > 1, all};
}
AttnShape attn_shape(const AttentionArgs& a) {
  switch (a.c.head_dim) {
    case 64: return attn_shape<64>(a);
    case 96: return attn_shape<96>(a);
    case 128: return attn_shape<128>(a);
    case 192: return attn_shape<192>(a);
    default: return attn_shape<256>(a);
  }
}

// The pages' codes as [blocks, page_tokens / 16, head_dim / box, 16, box] bytes, copied a page's tokens at a time, or
// `chunk`: 16 tokens lie in shared memory as slabs of `box` bytes a token, swizzled.
// (A cache without pages, whose pages are never looked at, borrows an address.)
bool pages_map(CUtensorMap* m, const CacheArgs& c, const void* any, int box, int chunk) {
  auto fn = tma_encode_fn();
  if (!fn) return false;
  ensure_context();
  const uint64_t D = c.head_dim, P = c.page_tokens;
  const cuuint64_t dims[5] = {(cuuint64_t)box, 16, D / box, P / 16, (cuuint64_t)(c.pages ? c.pages : 1) * 2 * c.heads};
  const cuuint64_t strides[4] = {D, (cuuint64_t)box, 16 * D, P * D};
  const cuuint32_t boxes[5] = {(cuuint32_t)box, 16, (cuuint32_t)(D / box), (cuuint32_t)(c.page_tokens < chunk ? P / 16 : chunk / 16), 1};
  const cuuint32_t es[5] = {1, 1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, c.pages ? c.codes : const_cast<void*>(any), dims, strides, boxes, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            box == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : box == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool kExact>
cudaError_t attend(const AttentionArgs& a, const AttnShape& sh, cudaStream_t st) {
  using S = Attn<D>;
  static bool set[kMaxDevices] = {};
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!set[dev]) {
      e = cudaFuncSetAttribute(cache_attention_kernel<D, kExact>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
      if (e != cudaSuccess) return e;
      set[dev] = true;
    }
  }
  CUtensorMap map;
  if (!pages_map(&map, a.c, a.q.p, S::kBox, S::kChunk)) return cudaErrorInvalidValue;
  // Both kernels are launched while the one before them drains, and wait for its
  // end themselves.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)sh.ctas);
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = S::kBytes;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, cache_attention_kernel<D, kExact>, map, a)) != cudaSuccess || !sh.split) return e;
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, cache_join_kernel<D>, a);
}
template <int D>
cudaError_t attend(const AttentionArgs& a, const AttnShape& sh, cudaStream_t st) {
  return a.out_f32 ? attend<D, true>(a, sh, st) : attend<D, false>(a, sh, st);
}
}  // namespace

int64_t cache_attention_units(const AttentionArgs& a) { return attn_shape(a).units; }

int64_t cache_attention_workspace_bytes(const AttentionArgs& a) {
  const AttnShape s = attn_shape(a);
  if (!s.split) return 0;
  return s.ctas * ((int64_t)sizeof(Split) + 8 * part_floats(a.c.head_dim) + (int64_t)s.warps * kRows * a.c.head_dim * 4);
}

cudaError_t launch_cache_attention(const AttentionArgs& a, cudaStream_t st) {
  if (a.c.tokens == 0 || a.c.sequences == 0) return cudaSuccess;
  (void)cudaGetLastError();
  const AttnShape sh = attn_shape(a);
  switch (a.c.head_dim) {
    case 64: return attend<64>(a, sh, st);
    case 96: return attend<96>(a, sh, st);
    case 128: return attend<128>(a, sh, st);
    case 192: return attend<192>(a, sh, st);
    default: return attend<256>(a, sh, st);
  }
}

namespace {
// Both waits on barriers that nothing signals: the first warp as a warp that multiplies,
// the second with one lane in need as a warp that fetches. Each runs out by its limit and
// says so to all of its lanes; the word is kErrIndex instead where one of them was told
// otherwise.
__global__ void __launch_bounds__(64) cache_wait_probe_kernel() {
  __shared__ uint64_t bars[2];
  __shared__ uint32_t abort[2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bar = ptx::smem_u32(bars + warp);
  if (lane == 0) {
    ptx::mbar_init(bar, 1);
    abort[warp] = 0;
    ptx::fence_mbar_init();
  }
  __syncthreads();
  bool ok = warp == 0 ? wait_bar_warp(bar, 0, abort) : wait_bars(bar, 0, lane == 3, abort + 1);
  // (once the flag is up they give up without a limit's wait, and one that is over still goes on)
  ok |= warp == 0 ? wait_bar_warp(bar, 0, abort) : wait_bars(bar, 0, lane == 30, abort + 1);
  ok |= warp == 0 ? !wait_bar_warp(bar, 1, abort) : !wait_bars(bar, 1, true, abort + 1);
  __syncthreads();
  if (ok || abort[warp] != 1u) index_fail();
}
}  // namespace

cudaError_t launch_cache_wait_probe(cudaStream_t st) {
  (void)cudaGetLastError();
  cache_wait_probe_kernel<<<1, 64, 0, st>>>();
  return cudaGetLastError();
}

cudaError_t read_cache_error(uint32_t* err) {
  cudaError_t e = cudaMemcpyFromSymbol(err, g_cache_error, sizeof(uint32_t));
  if (e == cudaSuccess && *err) {
    const uint32_t zero = 0;
    e = cudaMemcpyToSymbol(g_cache_error, &zero, sizeof(uint32_t));
  }
  return e;
}

}  // namespace mx
