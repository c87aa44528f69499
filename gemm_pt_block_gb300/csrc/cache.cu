// cache.cu -- keys and values in 8 bits (sm_103a): quantization as they are
// written, reading them back, and attention over them.
#include <cstdint>
#include <cuda_runtime.h>

#include "internal.h"
#include "mx_device.cuh"
#include "ptx.cuh"

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

// The last sequence b with start(b) <= slot, start being monotonic (where it is
// not, some sequence). start(0) <= slot.
template <typename F>
__device__ __forceinline__ int32_t find(int32_t count, int64_t slot, F start) {
  int32_t lo = 0, hi = count;
  while (hi - lo > 1) {
    const int32_t mid = (lo + hi) >> 1;
    if (start(mid) <= slot)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
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

// A block of threads takes one page, one head, keys or values: 32 elements a
// thread, four vectors of eight.
constexpr int kPerThread = 32;

// Where each sequence's slots of the grid begin: one for each page that its n
// rows may touch. Rows that go on inside a page (kExtra 2) touch at most
// floor(n / P) + 2 pages, rows from a page's start (kExtra 1) floor(n / P) + 1,
// and floor(end / P) - floor(begin / P) >= floor(n / P).
template <int kExtra>
__device__ __forceinline__ int64_t first_slot(const CacheArgs& c, int32_t b, int shift) {
  return c.starts ? (int64_t)(__ldg(c.starts + b) >> shift) + (int64_t)kExtra * b : b;
}

// The page a block works on: sequence, page number in it, tokens [lo, hi) of the page.
struct Task {
  Seq s;
  int32_t page, at, lo, hi;
};
template <int kExtra>
__device__ __forceinline__ bool task(const CacheArgs& c, Task* t) {
  const int shift = 31 - __clz(c.page_tokens);
  const int64_t slot = blockIdx.x;
  const int32_t b = find(c.sequences, slot, [&](int32_t i) { return first_slot<kExtra>(c, i, shift); });
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
  const int64_t k = slot - first_slot<kExtra>(c, b, shift);
  const int32_t first = t->s.pos >> shift;
  if (t->s.n == 0 || k < 0 || first + k > (t->s.len - 1) >> shift) return false;
  t->at = (first + (int32_t)k) << shift;
  t->page = page_of(c, b, first + (int32_t)k);
  if (t->page < 0) return false;
  t->lo = max(t->s.pos - t->at, 0);
  t->hi = min(t->s.len - t->at, c.page_tokens);
  return true;
}

template <typename T>
__global__ void __launch_bounds__(1024) cache_append_kernel(CacheArgs c, Heads k, Heads v) {
  __shared__ uint32_t most[32];
  Task t;
  if (!task<2>(c, &t)) return;
  const int h = blockIdx.y >> 1, kind = blockIdx.y & 1, per = c.head_dim >> 3;
  const Heads& x = kind ? v : k;
  const int64_t block = ((int64_t)t.page * 2 + kind) * c.heads + h;
  uint8_t* codes = c.codes + block * c.page_tokens * c.head_dim;
  float f[kPerThread / 8][8];
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < kPerThread / 8; ++i) {
    const int at = i * blockDim.x + threadIdx.x, token = at / per, d = (at - token * per) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) f[i][j] = 0.0f;
    if (token >= t.lo && token < t.hi) {
      const int64_t row = t.s.row + (t.at + token - t.s.pos);
      Vec8<T> w;
      load8(static_cast<const T*>(x.p) + row * x.ld_t + (int64_t)h * x.ld_h + d, w);
      unpack8(w, f[i]);
      m = absmax3_nan(m, absmax3_nan(f[i][0], f[i][1], f[i][2]),
                      absmax3_nan(absmax3_nan(f[i][3], f[i][4], f[i][5]), f[i][6], f[i][7]));
    }
  }
  // as whole numbers: magnitudes, then infinity, then NaN
  uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(m) & 0x7FFFFFFFu);
  if ((threadIdx.x & 31) == 0) most[threadIdx.x >> 5] = bits;
  const uint32_t old = t.lo > 0 ? c.scales[block] : 0u;
  __syncthreads();
  bits = 0;
  for (int w = 0; w < (int)(blockDim.x + 31) >> 5; ++w) bits = max(bits, most[w]);
  // 448 = 1.75 * 2^8: one more where the fraction passes it
  uint32_t scale = bits >= 0x7F800000u ? 255u : (uint32_t)max((int)(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u), 0);
  scale = max(scale, old);
  const float mul = scale == 255u ? 0.0f : __uint_as_float((254u - scale) << 23);
  const bool shrink = t.lo > 0 && old < scale && scale != 255u;
  // (below 2^-30 every older code rounds to zero)
  const float less = __uint_as_float((127u - min(scale - old, 64u)) << 23);
#pragma unroll
  for (int i = 0; i < kPerThread / 8; ++i) {
    const int at = i * blockDim.x + threadIdx.x, token = at / per, d = (at - token * per) * 8;
    uint2* to = reinterpret_cast<uint2*>(codes + token * c.head_dim + d);
    if (token >= t.lo && token < t.hi) {
      uint2 q = make_uint2(e4m3x4(f[i][0] * mul, f[i][1] * mul, f[i][2] * mul, f[i][3] * mul),
                           e4m3x4(f[i][4] * mul, f[i][5] * mul, f[i][6] * mul, f[i][7] * mul));
      if (scale == 255u) q = make_uint2(0u, 0u);
      put_at(to, q, c.codes, c.codes_bytes);
    } else if (shrink && token < t.lo) {
      const uint2 q = *to;
      float a[4], b[4];
      values4(q.x, a);
      values4(q.y, b);
      put_at(to, make_uint2(e4m3x4(a[0] * less, a[1] * less, a[2] * less, a[3] * less),
                            e4m3x4(b[0] * less, b[1] * less, b[2] * less, b[3] * less)),
             c.codes, c.codes_bytes);
    }
  }
  if (threadIdx.x == 0) put_at(c.scales + block, (uint8_t)scale, c.scales, c.scales_bytes);
}

template <typename T>
__global__ void __launch_bounds__(1024) cache_read_kernel(CacheArgs c, Heads k, Heads v) {
  Task t;
  if (!task<1>(c, &t)) return;
  const int h = blockIdx.y >> 1, kind = blockIdx.y & 1, per = c.head_dim >> 3;
  const Heads& x = kind ? v : k;
  const int64_t block = ((int64_t)t.page * 2 + kind) * c.heads + h;
  const uint8_t* codes = c.codes + block * c.page_tokens * c.head_dim;
  const float mul = scale_value(c.scales[block]);
#pragma unroll
  for (int i = 0; i < kPerThread / 8; ++i) {
    const int at = i * blockDim.x + threadIdx.x, token = at / per, d = (at - token * per) * 8;
    if (token < t.hi) {
      const uint2 q = *reinterpret_cast<const uint2*>(codes + token * c.head_dim + d);
      float a[4], b[4];
      values4(q.x, a);
      values4(q.y, b);
      float f[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[j] = a[j] * mul;
        f[j + 4] = b[j] * mul;
      }
      Vec8<T> w;
      pack8(f, w);
      store8(static_cast<T*>(x.p) + (int64_t)(t.s.row + t.at + token) * x.ld_t + (int64_t)h * x.ld_h + d, w, x.p, x.bytes);
    }
  }
}

// ----------------------------------------------------------------- attention ---

// A warp takes one query row: a token a lane for the scores, channels a lane
// for the values.
template <int D>
__global__ void __launch_bounds__(32) cache_attention_kernel(AttentionArgs a) {
  constexpr int kChannels = D / 32;
  __shared__ float qs[D];
  const CacheArgs& c = a.c;
  const int lane = threadIdx.x, shift = 31 - __clz(c.page_tokens);
  const int32_t t = blockIdx.x, hq = blockIdx.y, h = hq / (a.q_heads / c.heads);
  int32_t b = t;
  if (c.starts) b = find(c.sequences, t, [&](int32_t i) { return (int64_t)__ldg(c.starts + i); });
  Seq s;
  if (!rows_of(c, b, &s) || t < s.row || t >= s.row + s.n) return;
  const int32_t most = c.max_pages << shift;
  s.len = __ldg(c.lens + b);
  if (s.len < 0 || s.len > most) {
    index_fail();
    s.len = s.len < 0 ? 0 : most + 1;
  }
  const int32_t p = s.len - s.n + (t - s.row), lo = a.window > 0 ? max(0, p - a.window + 1) : 0;
  const uint16_t* q = static_cast<const uint16_t*>(a.q.p) + t * a.q.ld_t + hq * a.q.ld_h;
  for (int d = lane; d < D; d += 32) qs[d] = __uint_as_float((uint32_t)q[d] << 16);
  __syncwarp();
  float m = -INFINITY, sum = 0.0f, o[kChannels] = {};
  const float slope = a.slopes ? __ldg(a.slopes + hq) : 0.0f;
  for (int32_t j0 = lo; j0 <= p; j0 += 32) {
    const int32_t j = j0 + lane;
    float z = -INFINITY, vs = 0.0f;
    const uint8_t* vrow = nullptr;
    if (j <= p) {
      const int32_t page = page_of(c, b, j >> shift);
      z = __uint_as_float(0x7FC00000u);
      if (page >= 0) {
        const int64_t kb = (int64_t)page * 2 * c.heads + h;
        const int64_t at = (j & (c.page_tokens - 1)) * D;
        const uint8_t* krow = c.codes + kb * c.page_tokens * D + at;
        vrow = c.codes + (kb + c.heads) * c.page_tokens * D + at;
        vs = scale_value(c.scales[kb + c.heads]);
        float dot = 0.0f;
        for (int d = 0; d < D; d += 16) {
          const uint4 w = *reinterpret_cast<const uint4*>(krow + d);
          const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float f[4];
            values4(x[i], f);
#pragma unroll
            for (int e = 0; e < 4; ++e) dot = fmaf(f[e], qs[d + 4 * i + e], dot);
          }
        }
        z = dot * (scale_value(c.scales[kb]) * a.scale);
        if (a.softcap > 0.0f) z = a.softcap * tanhf(z / a.softcap);
        z += slope * (float)(j - p);
      }
    }
    float top = z;
    for (int i = 16; i; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
    const float now = fmaxf(m, top), keep = m == now ? 1.0f : expf(m - now);
    const float e = j <= p ? expf(z - now) : 0.0f;
    float es = e;
    for (int i = 16; i; i >>= 1) es += __shfl_xor_sync(0xffffffffu, es, i);
    sum = sum * keep + es;
    m = now;
#pragma unroll
    for (int i = 0; i < kChannels; ++i) o[i] *= keep;
    const int count = min(32, p - j0 + 1);
    for (int i = 0; i < count; ++i) {
      const float w = __shfl_sync(0xffffffffu, e * vs, i);
      const uint8_t* row = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, (unsigned long long)vrow, i));
#pragma unroll
      for (int ch = 0; ch < kChannels; ++ch) {
        const float x = row ? f16x2_f32(e4m3x2_f16x2(row[lane + 32 * ch])).x : __uint_as_float(0x7FC00000u);
        o[ch] = fmaf(w, x, o[ch]);
      }
    }
  }
  const int64_t at = t * a.out.ld_t + hq * a.out.ld_h;
#pragma unroll
  for (int ch = 0; ch < kChannels; ++ch) {
    const float y = p < 0 ? 0.0f : o[ch] / sum;
    if (a.out_f32)
      put_at(static_cast<float*>(a.out.p) + at + lane + 32 * ch, y, a.out.p, a.out.bytes);
    else
      put_at(static_cast<uint16_t*>(a.out.p) + at + lane + 32 * ch, (uint16_t)bf16x2(y, 0.0f), a.out.p, a.out.bytes);
  }
  if (a.lse && lane == 0)
    put_at(a.lse + (int64_t)t * a.q_heads + hq, p < 0 ? -INFINITY : m + logf(sum), a.lse, a.lse_bytes);
}

}  // namespace

cudaError_t launch_cache_append(const CacheArgs& c, const Heads& k, const Heads& v, bool f32, cudaStream_t st) {
  if (c.tokens == 0 || c.sequences == 0) return cudaSuccess;
  (void)cudaGetLastError();
  const int64_t slots = c.starts ? c.tokens / c.page_tokens + 2 * (int64_t)c.sequences : c.sequences;
  const dim3 grid((unsigned)slots, (unsigned)(2 * c.heads));
  const int threads = c.page_tokens * c.head_dim / kPerThread;
  if (f32)
    cache_append_kernel<float><<<grid, threads, 0, st>>>(c, k, v);
  else
    cache_append_kernel<uint16_t><<<grid, threads, 0, st>>>(c, k, v);
  return cudaGetLastError();
}

cudaError_t launch_cache_read(const CacheArgs& c, const Heads& k, const Heads& v, bool f32, cudaStream_t st) {
  if (c.tokens == 0 || c.sequences == 0) return cudaSuccess;
  (void)cudaGetLastError();
  const dim3 grid((unsigned)(c.tokens / c.page_tokens + (int64_t)c.sequences), (unsigned)(2 * c.heads));
  const int threads = c.page_tokens * c.head_dim / kPerThread;
  if (f32)
    cache_read_kernel<float><<<grid, threads, 0, st>>>(c, k, v);
  else
    cache_read_kernel<uint16_t><<<grid, threads, 0, st>>>(c, k, v);
  return cudaGetLastError();
}

int64_t cache_attention_workspace_bytes(const AttentionArgs&) { return 0; }

cudaError_t launch_cache_attention(const AttentionArgs& a, cudaStream_t st) {
  if (a.c.tokens == 0 || a.c.sequences == 0 || a.q_heads == 0) return cudaSuccess;
  (void)cudaGetLastError();
  const dim3 grid((unsigned)a.c.tokens, (unsigned)a.q_heads);
  switch (a.c.head_dim) {
    case 64: cache_attention_kernel<64><<<grid, 32, 0, st>>>(a); break;
    case 96: cache_attention_kernel<96><<<grid, 32, 0, st>>>(a); break;
    case 128: cache_attention_kernel<128><<<grid, 32, 0, st>>>(a); break;
    case 192: cache_attention_kernel<192><<<grid, 32, 0, st>>>(a); break;
    default: cache_attention_kernel<256><<<grid, 32, 0, st>>>(a); break;
  }
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
