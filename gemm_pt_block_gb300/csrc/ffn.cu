// ffn.cu -- the operators around a feed-forward block's products (sm_103a):
// residual addition + root-mean-square norm + quantization, SwiGLU +
// quantization, and their gradients. All are bound by HBM traffic.
#include <cstdint>
#include <mutex>

#include "internal.h"
#include "mx_device.cuh"
#include "ptx.cuh"

namespace mx {
namespace {
__device__ uint32_t g_ffn_error;
}  // namespace
}  // namespace mx
#define MX_BOUNDS_FAIL() atomicExch(&::mx::g_ffn_error, ::mx::kErrBounds)

#include "row_device.cuh"

namespace mx {
namespace {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, d));
  return v;
}

// Sum over the CTA's `warps` warps, the same bits in every thread (fixed
// order, a tree: rounding errors grow with the logarithm of the row's length).
__device__ __forceinline__ float block_sum(float v, float* part, int warps) {
  v = warp_sum(v);
  if (warps == 1) return v;
  const int lane = threadIdx.x & 31;
  if (lane == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum(lane < warps ? part[lane] : 0.0f);
}

__device__ __forceinline__ float sum8(const float (&f)[8]) {
  return __fadd_rn(__fadd_rn(__fadd_rn(f[0], f[1]), __fadd_rn(f[2], f[3])),
                   __fadd_rn(__fadd_rn(f[4], f[5]), __fadd_rn(f[6], f[7])));
}

// ------------------------------------------------------------------ norm ---
// h = x + r, rounded to the stream's type T (what the next layer reads); the
// norm is taken of the rounded h, so that the backward pass, which reads it
// back, differentiates the same function:
//   y_i = (h_i w_i) rstd,   rstd = 1 / sqrt(sum h^2 / D + eps).
// bf16 products h_i w_i are exact in fp32, so y has two roundings.
//
// A row stays in registers between the sum of squares and the output, so that
// each input is read once: one warp a row up to 1024 columns, a CTA a row above
// (up to 32 columns a thread), two passes over rows that registers do not hold.
// Bound by HBM: 16384 x 8192 bf16 with residual, E4M3 codes, 152 us (6.2 TB/s,
// 93 % of a copy); few rows by latency (1 x 8192: 2.9 us, a launch is two).
template <typename T>
__device__ __forceinline__ void add_stream(Vec8<T>& x, const Vec8<T>& r, float (&h)[8]) {
  float f[8];
  unpack8(x, h);
  unpack8(r, f);
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = __fadd_rn(h[i], f[i]);
  pack8(h, x);
  unpack8(x, h);
}

__device__ __forceinline__ float reciprocal_rms(float sum, const NormArgs& a) {
  return __frsqrt_rn(__fadd_rn(__fdiv_rn(sum, (float)a.cols), a.eps));
}

// Eight outputs of a row whose norm is known: y and the quantized y.
template <typename T, typename W>
__device__ __forceinline__ void norm_out8(const NormArgs& a, const Vec8<T>& raw, bool live, int64_t row, int64_t c,
                                          float rstd, const RowOut& out) {
  float f[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (live) {
    float h[8];
    unpack8(raw, h);
    if (a.w) {
      Vec8<W> wv;
      load8_cached(static_cast<const W*>(a.w) + c, wv);
      unpack8(wv, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = __fmul_rn(__fmul_rn(h[i], f[i]), rstd);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = __fmul_rn(h[i], rstd);
    }
    if (a.y) store8_as(a.y, a.y_f32, row * a.ld_y + c, f, a.y_bytes);
  }
  if (a.quant.fmt != RowQuant::kNone) quantize8(a.quant, f, live, out, (uint32_t)c);
}

// A row in registers: kChunks vectors of eight elements to a thread, all loads
// in flight at once, one pass over HBM. Rows of one warp (blockDim.x = 32)
// share a CTA (blockDim.y of them), longer ones have a CTA each; several CTAs
// an SM keep its loads going through one another's sums.
template <typename T, typename W, int kChunks, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads) norm_rows_kernel(const NormArgs a) {
  __shared__ float part[32];
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (row >= a.rows) return;  // whole warps: only one-warp rows share a CTA
  const T* x = static_cast<const T*>(a.x) + row * a.ld_x;
  const T* r = static_cast<const T*>(a.r) + row * a.ld_r;
  Vec8<T> v[kChunks], u[kChunks];
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int64_t c = (int64_t)(i * blockDim.x + threadIdx.x) * 8;
    v[i] = Vec8<T>{};
    if (c < a.cols) load8(x + c, v[i]);
  }
  if (a.r) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int64_t c = (int64_t)(i * blockDim.x + threadIdx.x) * 8;
      u[i] = Vec8<T>{};
      if (c < a.cols) load8(r + c, u[i]);
    }
  }
  float s[kChunks];
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int64_t c = (int64_t)(i * blockDim.x + threadIdx.x) * 8;
    float h[8];
    if (a.r)
      add_stream(v[i], u[i], h);
    else
      unpack8(v[i], h);
    if (a.h && c < a.cols) store8(static_cast<T*>(a.h) + row * a.ld_h + c, v[i], a.h, a.h_bytes);
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = __fmul_rn(h[j], h[j]);
    s[i] = sum8(h);
  }
#pragma unroll
  for (int d = 1; d < kChunks; d *= 2)
#pragma unroll
    for (int i = 0; i < kChunks; i += 2 * d) s[i] = __fadd_rn(s[i], s[i + d]);
  const float rstd = reciprocal_rms(block_sum(s[0], part, blockDim.x >> 5), a);
  if (a.rstd && threadIdx.x == 0) put_at(a.rstd + row, rstd, a.rstd, a.rows * sizeof(float));
  if (!a.y && a.quant.fmt == RowQuant::kNone) return;
  const RowOut out = row_out(a.quant, row, a.cols);
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    if ((int64_t)i * blockDim.x * 8 >= a.cols) break;  // (the same in the whole CTA)
    const int64_t c = (int64_t)(i * blockDim.x + threadIdx.x) * 8;
    norm_out8<T, W>(a, v[i], c < a.cols, row, c, rstd, out);
  }
}

// Rows longer than a CTA's registers hold: two passes, the second one reading
// x and r again (out of L2 for all but the longest).
constexpr int kRowThreads = 1024;

template <typename T, typename W>
__global__ void __launch_bounds__(kRowThreads) norm_long_rows_kernel(const NormArgs a) {
  __shared__ float part[32];
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.ld_x;
  const T* r = static_cast<const T*>(a.r) + row * a.ld_r;
  float sum = 0.0f, h[8];
  Vec8<T> v, u;
  for (int64_t c = threadIdx.x * 8; c < a.cols; c += kRowThreads * 8) {
    load8(x + c, v);
    if (a.r) {
      load8(r + c, u);
      add_stream(v, u, h);
    } else {
      unpack8(v, h);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = __fmul_rn(h[i], h[i]);
    sum = __fadd_rn(sum, sum8(h));
  }
  const float rstd = reciprocal_rms(block_sum(sum, part, kRowThreads / 32), a);
  if (a.rstd && threadIdx.x == 0) put_at(a.rstd + row, rstd, a.rstd, a.rows * sizeof(float));
  const RowOut out = row_out(a.quant, row, a.cols);
  for (int64_t c0 = 0; c0 < a.cols; c0 += kRowThreads * 8) {
    const int64_t c = c0 + threadIdx.x * 8;
    v = Vec8<T>{};
    if (c < a.cols) {
      load8(x + c, v);
      if (a.r) {
        load8(r + c, u);
        add_stream(v, u, h);
      }
      if (a.h) store8(static_cast<T*>(a.h) + row * a.ld_h + c, v, a.h, a.h_bytes);
    }
    norm_out8<T, W>(a, v, c < a.cols, row, c, rstd, out);
  }
}

// Gradients. With n = h rstd and dn = dy w:
//   dx = (dn - n mean(dn n)) rstd + dh,   dw = sum over rows of dy n
// (dh: what reaches h past the norm, through the residual stream).
//
// One kernel reads dy, h and dh once: one persistent CTA an SM, whose threads
// form up to twelve groups that take rows in turn. Whole rows come by bulk copies
// into the group's ring of shared memory, a few rows ahead, and every thread keeps
// its columns' part of dw in registers over all of its group's rows. The groups'
// parts are added in shared memory, the CTAs' parts go to the workspace and a
// second kernel sums them, all in order (no atomics: dw has the same bits on
// every call). Bound by HBM: 16384 x 8192 bf16 157 us (6.8 TB/s, a copy's rate);
// 1001 x 4096 11.3 us, bound by the two launches and the first rows' way in.
constexpr int kGradChunks = 2;
constexpr int kGradSmem = 192 << 10;    // of the SM's 228 KB
constexpr int kGradMaxStages = 8;
constexpr int kGradMaxGroups = 12;      // (a hardware barrier each; 16384 x 1024: 8 groups 29 us, 12 26, 15 27)
constexpr int kSms = 152;
constexpr uint64_t kWaitLimitNs = 2000000000ull;

// Bounded wait (about 2 s) of one thread; on expiry the device error word is set.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer_ns();
  while (!ptx::mbar_try_wait_sleep(bar, parity, 100000u)) {
    if (ptx::globaltimer_ns() - t0 > kWaitLimitNs) {
      atomicExch(&g_ffn_error, 6u);  // MXFP4_ERR_TIMEOUT
      return false;
    }
  }
  return true;
}

template <typename T>
__device__ __forceinline__ void load8_shared(const uint8_t* row, int64_t c, float (&f)[8]) {
  Vec8<T> v = *reinterpret_cast<const Vec8<T>*>(row + c * sizeof(T));
  unpack8(v, f);
}

// Barrier and sum over the threads of one group (full warps); `part` has a place
// for each of the CTA's warps.
__device__ __forceinline__ void group_barrier(uint32_t group, uint32_t threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(threads) : "memory");
}
__device__ __forceinline__ float group_sum(float v, float* part, uint32_t group, uint32_t threads) {
  const uint32_t lane = threadIdx.x & 31, warps = threads >> 5;
  part += group * warps;
  v = warp_sum(v);
  if (lane == 0) part[threadIdx.x >> 5] = v;
  group_barrier(group, threads);
  return warp_sum(lane < warps ? part[lane] : 0.0f);
}

// Keeps bf16 weights packed in their registers: unpacked ahead of the loop they
// would take twice as many.
__device__ __forceinline__ void hold(Vec8<uint16_t>& v) {
  asm volatile("" : "+r"(v.a.x), "+r"(v.a.y), "+r"(v.a.z), "+r"(v.a.w));
}
__device__ __forceinline__ void hold(Vec8<float>&) {}

// (what every thread would otherwise hold in registers)
struct GradRing {
  uint32_t stages, stage_bytes, dy_bytes, h_bytes, step;  // step: rows between a group's rows
};

template <typename T, typename G, typename W>
__global__ void __launch_bounds__(1024) norm_grad_kernel(const NormGradArgs a, const GradRing r) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float part[32];
  __shared__ uint64_t full[kGradMaxGroups * kGradMaxStages];
  __shared__ volatile uint32_t abort[kGradMaxGroups];
  const uint32_t tid = threadIdx.x, group = threadIdx.y, cols = (uint32_t)a.cols, rows = (uint32_t)a.rows;
  const uint32_t bars = ptx::smem_u32(full) + 8 * kGradMaxStages * group;
  const uint32_t first = group * gridDim.x + blockIdx.x, slots = group * r.stages * r.stage_bytes;
  if (tid == 0) {
    for (uint32_t i = 0; i < r.stages; ++i) ptx::mbar_init(bars + 8 * i, 1);
    abort[group] = 0;
    ptx::fence_mbar_init();
  }
  __syncthreads();
  auto fetch = [&](int64_t row, uint32_t slot) {
    const uint32_t dst = ptx::smem_u32(ring) + slots + slot * r.stage_bytes, bar = bars + 8 * slot;
    ptx::mbar_arrive_expect_tx(bar, r.stage_bytes);
    ptx::bulk_load(dst, static_cast<const G*>(a.dy) + row * a.ld_dy, r.dy_bytes, bar);
    ptx::bulk_load(dst + r.dy_bytes, static_cast<const T*>(a.h) + row * a.ld_h, r.h_bytes, bar);
    if (a.dh)
      ptx::bulk_load(dst + r.dy_bytes + r.h_bytes, static_cast<const T*>(a.dh) + row * a.ld_dh, r.h_bytes, bar);
  };
  if (tid == 0)
    for (uint32_t i = 0; i < r.stages && first + i * r.step < rows; ++i) fetch(first + i * r.step, i);

  Vec8<W> wv[kGradChunks];
  float acc[kGradChunks][8];
#pragma unroll
  for (int i = 0; i < kGradChunks; ++i) {
    const uint32_t c = (i * blockDim.x + tid) * 8;
    if (a.w && c < cols) load8_cached(static_cast<const W*>(a.w) + c, wv[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.0f;
  }
  uint32_t slot = 0, parity = 0;
  float rstd = first < rows ? __ldg(a.rstd + first) : 0.0f;
  for (uint32_t row = first; row < rows; row += r.step) {
    const float next = row + r.step < rows ? __ldg(a.rstd + row + r.step) : 0.0f;
    if (!wait_bar(bars + 8 * slot, parity)) abort[group] = 1u;
    const uint8_t* dy = ring + slots + slot * r.stage_bytes;
    // the row is read twice from shared memory: kept in registers between the
    // passes, its values would leave too few for 1024 threads an SM
    float n[8], d[8], f[8], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kGradChunks; ++i) {
      hold(wv[i]);
      const uint32_t c = (i * blockDim.x + tid) * 8;
      if (c < cols) {
        load8_shared<G>(dy, c, d);
        load8_shared<T>(dy + r.dy_bytes, c, n);
        if (a.w) unpack8(wv[i], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          n[j] = __fmul_rn(n[j], rstd);
          acc[i][j] = __fmaf_rn(d[j], n[j], acc[i][j]);
          sum = __fmaf_rn(a.w ? __fmul_rn(d[j], f[j]) : d[j], n[j], sum);
        }
      }
    }
    const float mean = __fdiv_rn(group_sum(sum, part, group, blockDim.x), (float)cols);
    if (abort[group]) {  // past the barrier: the whole group leaves, or none of it
      // the copies in flight land (bounded wait) before the CTA's memory goes
      if (tid == 0)
        for (uint32_t i = 0; i < r.stages && row + i * r.step < rows; ++i) {
          const uint64_t t0 = ptx::globaltimer_ns();
          while (!ptx::mbar_try_wait(bars + 8 * slot, parity) && ptx::globaltimer_ns() - t0 < kWaitLimitNs / 10) {
          }
          if (++slot == r.stages) {
            slot = 0;
            parity ^= 1u;
          }
        }
      break;
    }
#pragma unroll
    for (int i = 0; i < kGradChunks; ++i) {
      const uint32_t c = (i * blockDim.x + tid) * 8;
      if (c < cols) {
        load8_shared<G>(dy, c, d);
        load8_shared<T>(dy + r.dy_bytes, c, n);
        if (a.w) {
          unpack8(wv[i], f);
#pragma unroll
          for (int j = 0; j < 8; ++j) d[j] = __fmul_rn(d[j], f[j]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = __fmul_rn(__fmaf_rn(-__fmul_rn(n[j], rstd), mean, d[j]), rstd);
        if (a.dh) {
          load8_shared<T>(dy + r.dy_bytes + r.h_bytes, c, f);
#pragma unroll
          for (int j = 0; j < 8; ++j) d[j] = __fadd_rn(d[j], f[j]);
        }
        Vec8<T> o;
        pack8(d, o);
        store8(static_cast<T*>(a.dx) + row * a.ld_dx + c, o, a.dx, a.dx_bytes);
      }
    }
    rstd = next;
    // the slot's next row at once, for the price of a barrier: past the next
    // row's own barrier instead, a ring of two slots would have no copy in flight
    // while that row is read (16384 x 8192: 168 us; this way 157)
    group_barrier(group, blockDim.x);
    const uint32_t ahead = row + r.stages * r.step;
    if (tid == 0 && ahead < rows) fetch(ahead, slot);
    if (++slot == r.stages) {
      slot = 0;
      parity ^= 1u;
    }
  }
  if (!a.dw) return;
  if (blockDim.y == 1) {
#pragma unroll
    for (int i = 0; i < kGradChunks; ++i) {
      const uint32_t c = (i * blockDim.x + tid) * 8;
      if (c < cols) store8_as(a.ws, true, (int64_t)blockIdx.x * cols + c, acc[i], a.ws_bytes);
    }
    return;
  }
  // the ring holds no row any more; a slot is at least as large as a row of sums
  __syncthreads();
  float* sums = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int i = 0; i < kGradChunks; ++i) {
    const uint32_t c = (i * blockDim.x + tid) * 8;
    if (c < cols) {
      float4* to = reinterpret_cast<float4*>(sums + group * cols + c);
      to[0] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
      to[1] = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
    }
  }
  __syncthreads();
  for (uint32_t c = (group * blockDim.x + tid) * 4; c < cols; c += blockDim.x * blockDim.y * 4) {
    float4 t = *reinterpret_cast<const float4*>(sums + c);
    for (uint32_t g = 1; g < blockDim.y; ++g) {
      const float4 v = *reinterpret_cast<const float4*>(sums + g * cols + c);
      t = make_float4(__fadd_rn(t.x, v.x), __fadd_rn(t.y, v.y), __fadd_rn(t.z, v.z), __fadd_rn(t.w, v.w));
    }
    put_at(reinterpret_cast<float4*>(a.ws + (int64_t)blockIdx.x * cols + c), t, a.ws, a.ws_bytes);
  }
}

// Short rows: a warp each, straight from HBM (eight warps a CTA, each with a
// row's loads in flight), dw of the CTA's warps summed in order at the end
// (16384 x 512: 15 us, 4.4 TB/s; the ring takes 23 there, and less from 544
// columns on: 25 and 27 at 16384 x 640).
template <typename T, typename G, typename W, int kChunks>
__global__ void __launch_bounds__(256, 2) norm_short_grad_kernel(const NormGradArgs a) {
  __shared__ float part[8][kChunks * 256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Vec8<W> wv[kChunks];
  float acc[kChunks][8];
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int64_t c = (i * 32 + lane) * 8;
    if (a.w && c < a.cols) load8_cached(static_cast<const W*>(a.w) + c, wv[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.0f;
  }
  for (int64_t row = (int64_t)blockIdx.x * 8 + warp; row < a.rows; row += (int64_t)gridDim.x * 8) {
    Vec8<T> hv[kChunks], sv[kChunks];
    Vec8<G> dv[kChunks];
    const float rstd = __ldg(a.rstd + row);
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int64_t c = (i * 32 + lane) * 8;
      if (c < a.cols) {
        load8_apart(static_cast<const T*>(a.h) + row * a.ld_h + c, hv[i]);
        load8_apart(static_cast<const G*>(a.dy) + row * a.ld_dy + c, dv[i]);
        if (a.dh) load8_apart(static_cast<const T*>(a.dh) + row * a.ld_dh + c, sv[i]);
      }
    }
    float n[8], d[8], f[8], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      if ((i * 32 + lane) * 8 < a.cols) {
        unpack8(hv[i], n);
        unpack8(dv[i], d);
        if (a.w) unpack8(wv[i], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          n[j] = __fmul_rn(n[j], rstd);
          acc[i][j] = __fmaf_rn(d[j], n[j], acc[i][j]);
          sum = __fmaf_rn(a.w ? __fmul_rn(d[j], f[j]) : d[j], n[j], sum);
        }
      }
    }
    const float mean = __fdiv_rn(warp_sum(sum), (float)a.cols);
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int64_t c = (i * 32 + lane) * 8;
      if (c < a.cols) {
        unpack8(hv[i], n);
        unpack8(dv[i], d);
        if (a.w) {
          unpack8(wv[i], f);
#pragma unroll
          for (int j = 0; j < 8; ++j) d[j] = __fmul_rn(d[j], f[j]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = __fmul_rn(__fmaf_rn(-__fmul_rn(n[j], rstd), mean, d[j]), rstd);
        if (a.dh) {
          unpack8(sv[i], f);
#pragma unroll
          for (int j = 0; j < 8; ++j) d[j] = __fadd_rn(d[j], f[j]);
        }
        Vec8<T> o;
        pack8(d, o);
        store8(static_cast<T*>(a.dx) + row * a.ld_dx + c, o, a.dx, a.dx_bytes);
      }
    }
  }
  if (!a.dw) return;
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    float4* p = reinterpret_cast<float4*>(&part[warp][(i * 32 + lane) * 8]);
    p[0] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
    p[1] = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
  }
  __syncthreads();
  for (int c = threadIdx.x; c < a.cols; c += 256) {
    float v = part[0][c];
#pragma unroll
    for (int i = 1; i < 8; ++i) v = __fadd_rn(v, part[i][c]);
    put_at(a.ws + (int64_t)blockIdx.x * a.cols + c, v, a.ws, a.ws_bytes);
  }
}

// Rows too long for that ring: dx in two passes over the row, and dw from a
// second reading of dy and h by columns.
template <typename T, typename G, typename W>
__global__ void __launch_bounds__(kRowThreads) norm_long_dx_kernel(const NormGradArgs a) {
  __shared__ float part[32];
  const int64_t row = blockIdx.x;
  const T* hp = static_cast<const T*>(a.h) + row * a.ld_h;
  const G* dp = static_cast<const G*>(a.dy) + row * a.ld_dy;
  const float rstd = a.rstd[row];
  float h[8], d[8], w[8], sum = 0.0f, mean = 0.0f;
  for (int pass = 0; pass < 2; ++pass) {
    if (pass) mean = __fdiv_rn(block_sum(sum, part, kRowThreads / 32), (float)a.cols);
    for (int64_t c = threadIdx.x * 8; c < a.cols; c += kRowThreads * 8) {
      Vec8<T> hv;
      Vec8<G> dv;
      load8(hp + c, hv);
      load8(dp + c, dv);
      unpack8(hv, h);
      unpack8(dv, d);
      if (a.w) {
        Vec8<W> wv;
        load8_cached(static_cast<const W*>(a.w) + c, wv);
        unpack8(wv, w);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        h[i] = __fmul_rn(h[i], rstd);
        if (a.w) d[i] = __fmul_rn(d[i], w[i]);
        if (!pass) sum = __fmaf_rn(d[i], h[i], sum);
      }
      if (pass) {
        if (a.dh) {
          load8(static_cast<const T*>(a.dh) + row * a.ld_dh + c, hv);
          unpack8(hv, w);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          d[i] = __fmul_rn(__fmaf_rn(-h[i], mean, d[i]), rstd);
          if (a.dh) d[i] = __fadd_rn(d[i], w[i]);
        }
        pack8(d, hv);
        store8(static_cast<T*>(a.dx) + row * a.ld_dx + c, hv, a.dx, a.dx_bytes);
      }
    }
  }
}

constexpr int kColThreads = 256;

template <typename T, typename G>
__global__ void __launch_bounds__(kColThreads) norm_long_dw_kernel(const NormGradArgs a) {
  const int64_t c = ((int64_t)blockIdx.x * kColThreads + threadIdx.x) * 8;
  if (c >= a.cols) return;
  float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0}, h[8], d[8];
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    Vec8<T> hv;
    Vec8<G> dv;
    load8(static_cast<const T*>(a.h) + row * a.ld_h + c, hv);
    load8(static_cast<const G*>(a.dy) + row * a.ld_dy + c, dv);
    unpack8(hv, h);
    unpack8(dv, d);
    const float rstd = a.rstd[row];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = __fmaf_rn(d[i], __fmul_rn(h[i], rstd), acc[i]);
  }
  store8_as(a.ws, true, (int64_t)blockIdx.y * a.cols + c, acc, a.ws_bytes);
}

// dw from the partial sums: a CTA takes 32 columns, its warps every kSumWarps'th
// slice, and the warps' sums are added in order.
constexpr int kSumWarps = 16;
template <typename W>
__global__ void __launch_bounds__(kSumWarps * 32) norm_dw_sum_kernel(const float* ws, int slices, int64_t cols, W* dw) {
  __shared__ float part[kSumWarps][32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.0f;
#pragma unroll 8
  for (int i = warp; i < slices; i += kSumWarps) s = __fadd_rn(s, ws[i * cols + c]);
  part[warp][lane] = s;
  __syncthreads();
  if (warp) return;
#pragma unroll
  for (int i = 1; i < kSumWarps; ++i) s = __fadd_rn(s, part[i][lane]);
  if (sizeof(W) == 4)
    put_at(dw + c, s, dw, cols * sizeof(W));
  else
    put_at(dw + c, (uint16_t)bf16x2(s, 0.0f), dw, cols * sizeof(W));
}

// ---------------------------------------------------------------- SwiGLU ---
// a = silu(g) u with silu(g) = g / (1 + e^-g).
constexpr int kActThreads = 256;

// g / (1 + e^-g) and 1 / (1 + e^-g) of a pair, in fp32 throughout and without a
// case for the sign: with t = 2^-24 e^-g the second is 2^-24 / (2^-24 + t),
// where t spans all that fp32 needs (e^-g up to 2^150, past which the quotient
// is below every fp32; g counts between -105 and 200). The exponential comes in
// two steps: -g / ln 2 is rounded to a multiple z of 2^-14 (as z + 768, whose
// binade has that step), the hardware takes 2^(z - 24), and what z misses, d =
// -g - z ln 2 (ln 2 in two parts, |d| < 2^-15), enters as the factor 1 + d
// (d^2 / 2 stays below 2^-31). All but the clamps, the powers and the
// reciprocals works on packed pairs: the forward kernel is bound by issue.
__device__ __forceinline__ float ex2(float z) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(z));
  return r;
}
__device__ __forceinline__ float rcp(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float2 pair(float v) { return make_float2(v, v); }
// 2^24 / (1 + e^-g)
__device__ __forceinline__ float2 sigmoid2_24(float2 g) {
  const float2 m = make_float2(fmaxf(fminf(-g.x, 105.0f), -200.0f), fmaxf(fminf(-g.y, 105.0f), -200.0f));
  const float2 s = f2fma(m, pair(1.44269504088896341f), pair(768.0f));
  const float2 z = f2sub(s, pair(768.0f));
  const float2 d = f2fma(z, pair(1.90465429995776804e-9f), f2fma(z, pair(-0.693147182464599609375f), m));
  const float2 z24 = f2sub(s, pair(792.0f));
  const float2 e = make_float2(ex2(z24.x), ex2(z24.y));
  const float2 q = f2add(f2fma(e, d, e), pair(0x1p-24f));
  return make_float2(rcp(q.x), rcp(q.y));
}

// A thread takes sixteen columns of one row after another (blockDim.y and the
// grid's height apart), the next row's loads in flight meanwhile: what a thread
// works out once is spread over many rows. Short rows (blockDim.x below 32)
// share a warp. Bound by HBM and issue alike (IPC 3.2): 8192 x 28672 bf16 to
// E4M3 codes 186.5 us (6.3 TB/s, 95 % of a copy); fp32 2048 x 28672 80 us (98 %).
// `wide`: 32-byte loads where every row allows them (191 us, 193 without).
template <typename T>
// bf16: three CTAs an SM (80 registers) measured 191 us at 8192 x 28672 where
// 126 registers took 225 and 64 (four CTAs) 207; fp32 is at HBM's rate with two.
__global__ void __launch_bounds__(kActThreads, sizeof(T) == 2 ? 3 : 1) swiglu_kernel(const SwigluArgs a, const bool wide) {
  const int64_t c = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * 16, step = (int64_t)gridDim.y * blockDim.y;
  const bool in_row = c < a.cols;
  int64_t row = (int64_t)blockIdx.y * blockDim.y + threadIdx.y;
  const T* g = static_cast<const T*>(a.g) + row * a.ld_g + c;
  const T* u = static_cast<const T*>(a.u) + row * a.ld_u + c;
  Vec16<T> gv = {}, uv = {};
  if (in_row && row < a.rows) {
    load16e(g, wide, gv);
    load16e(u, wide, uv);
  }
  for (int64_t left = a.rows - (int64_t)blockIdx.y * blockDim.y; left > 0; left -= step) {  // the same in the whole CTA
    const bool live = in_row && row < a.rows;
    float2 x[8], y[8];
    unpack16(gv, x);
    unpack16(uv, y);
    g += step * a.ld_g;
    u += step * a.ld_u;
    if (in_row && row + step < a.rows) {
      load16e(g, wide, gv);
      load16e(u, wide, uv);
    }
    // (the sigmoid takes the 2^-24: a tiny g, brought down by it, would lose bits from 2^-102 on)
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = f2mul(f2mul(f2mul(sigmoid2_24(x[i]), pair(0x1p-24f)), x[i]), y[i]);
    if (a.y && live) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float f[8] = {y[4 * i].x,     y[4 * i].y,     y[4 * i + 1].x, y[4 * i + 1].y,
                            y[4 * i + 2].x, y[4 * i + 2].y, y[4 * i + 3].x, y[4 * i + 3].y};
        store8_as(a.y, a.y_f32, row * a.ld_y + c + 8 * i, f, a.y_bytes);
      }
    }
    if (a.quant.fmt != RowQuant::kNone) quantize16(a.quant, y, live, row_out(a.quant, row, a.cols), (uint32_t)c);
    row += step;
  }
}

// With s = 1 / (1 + e^-g): dg = dy u s (1 + g (1 - s)), du = dy g s. Eight
// columns of one row a thread; bound by HBM: 4096 x 28672 bf16 169 us (7.0 TB/s,
// a copy's rate).
template <typename T, typename G>
__global__ void __launch_bounds__(kActThreads) swiglu_grad_kernel(const SwigluGradArgs a) {
  const int64_t c = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * 8;
  if (c >= a.cols) return;
  for (int64_t row = (int64_t)blockIdx.y * blockDim.y + threadIdx.y; row < a.rows;
       row += (int64_t)gridDim.y * blockDim.y) {
    float g[8], u[8], d[8];
    Vec8<T> gv, uv;
    Vec8<G> dv;
    load8(static_cast<const T*>(a.g) + row * a.ld_g + c, gv);
    load8(static_cast<const T*>(a.u) + row * a.ld_u + c, uv);
    load8(static_cast<const G*>(a.dy) + row * a.ld_dy + c, dv);
    unpack8(gv, g);
    unpack8(uv, u);
    unpack8(dv, d);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float2 x = make_float2(g[i], g[i + 1]), s = f2mul(sigmoid2_24(x), pair(0x1p-24f));
      const float2 ds = f2mul(make_float2(d[i], d[i + 1]), s);
      const float2 p = f2fma(x, f2sub(pair(1.0f), s), pair(1.0f));
      const float2 q = f2mul(f2mul(ds, make_float2(u[i], u[i + 1])), p), v = f2mul(ds, x);
      u[i] = q.x;
      u[i + 1] = q.y;
      d[i] = v.x;
      d[i + 1] = v.y;
    }
    pack8(u, gv);
    pack8(d, uv);
    store8(static_cast<T*>(a.dg) + row * a.ld_dg + c, gv, a.dg, a.dg_bytes);
    store8(static_cast<T*>(a.du) + row * a.ld_du + c, uv, a.du, a.du_bytes);
  }
}

// Block and grid of the activation kernels for rows of per_row threads: CTAs of
// up to 256 threads, a row cut into equal parts of whole warps; rows that leave
// more than a tenth of those lanes empty (and short rows) in parts of 16, 8 or
// fewer, side by side (SwiGLU, 4096 x 4480: 28.8 us in parts of 256 lanes, 20.5
// in two of 160, 18.6 in 18 of 16; 9879 x 1056: 15.9 in 96 lanes, 12.9 in nine
// times 8); at most `ctas` CTAs.
void act_shape(int64_t rows, int64_t per_row, int64_t ctas, dim3* grid, dim3* block) {
  int64_t wide = (per_row + kActThreads - 1) / kActThreads;
  unsigned x = (unsigned)((per_row + 32 * wide - 1) / (32 * wide) * 32);
  while (per_row <= x / 2 && x <= 32) x /= 2;
  for (unsigned c = 16; c >= 8 && c < x; c /= 2)
    if ((per_row + c - 1) / c * c * 10 < wide * x * 9) {
      x = c;
      wide = (per_row + c - 1) / c;
    }
  const unsigned y = kActThreads / x;
  int64_t tall = (rows + y - 1) / y, most = (ctas + wide - 1) / wide;
  if (most > 65535) most = 65535;
  *block = dim3(x, y);
  *grid = dim3((unsigned)wide, (unsigned)(tall < most ? tall : most));
}

bool aligned32(const void* p, int64_t ld_bytes) { return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)ld_bytes) & 31u) == 0; }

// Rows of one warp; the CTAs that take them.
constexpr int64_t kShortCols = 512;
int64_t short_ctas(int64_t rows) {
  const int64_t ctas = (rows + 7) / 8;
  return ctas < 2 * kSms ? ctas : 2 * kSms;
}

// The ring kernel's threads for a row of `cols` (kGradChunks vectors each).
int grad_threads(int64_t cols) { return (int)((cols / 8 + 32 * kGradChunks - 1) / (32 * kGradChunks) * 32); }

}  // namespace

// Rows of partial sums that the workspace holds, for either way of taking dw.
int norm_dw_slices(int64_t rows) { return (int)(rows < 2 * kSms ? rows : 2 * kSms); }

namespace {
template <typename T, typename W>
void launch_norm(const NormArgs& a, cudaStream_t st) {
  const int64_t vecs = a.cols / 8;
  const unsigned rows = (unsigned)a.rows;
  if (vecs <= 128) {
    // one warp a row, eight rows a CTA; as many vectors to a lane as the row needs
    // (16384 x 512: 11.4 us with two, 16.2 with four of which two hold nothing)
    const dim3 grid((unsigned)((a.rows + 7) / 8)), block(32, 8);
    if (vecs <= 32)
      norm_rows_kernel<T, W, 1, 256><<<grid, block, 0, st>>>(a);
    else if (vecs <= 64)
      norm_rows_kernel<T, W, 2, 256><<<grid, block, 0, st>>>(a);
    else
      norm_rows_kernel<T, W, 4, 256><<<grid, block, 0, st>>>(a);
  } else if (vecs <= 1024 && a.rows <= kSms) {
    // an SM or more to each row: the widest CTA has the shortest way through it
    // (152 x 8192: 3.7 us, 5.0 the other way; 400 x 8192: 7.5 and 6.9)
    norm_rows_kernel<T, W, 1, 1024><<<rows, (unsigned)((vecs + 31) / 32 * 32), 0, st>>>(a);
  } else if (vecs <= 1024) {
    norm_rows_kernel<T, W, 4, 256><<<rows, (unsigned)((vecs + 127) / 128 * 32), 0, st>>>(a);
  } else if (vecs <= 2048) {
    norm_rows_kernel<T, W, 4, 512><<<rows, (unsigned)((vecs + 127) / 128 * 32), 0, st>>>(a);
  } else {
    if constexpr (sizeof(T) == 2)
      if (vecs <= 4096) {
        norm_rows_kernel<T, W, 4, 1024><<<rows, (unsigned)((vecs + 127) / 128 * 32), 0, st>>>(a);
        return;
      }
    norm_long_rows_kernel<T, W><<<rows, kRowThreads, 0, st>>>(a);
  }
}
}  // namespace

cudaError_t launch_rmsnorm(const NormArgs& a, bool x_f32, bool w_f32, cudaStream_t st) {
  if (a.rows == 0 || a.cols == 0) return cudaSuccess;
  (void)cudaGetLastError();  // drop a stale error left by an earlier call
  if (x_f32 && w_f32)
    launch_norm<float, float>(a, st);
  else if (x_f32)
    launch_norm<float, uint16_t>(a, st);
  else if (w_f32)
    launch_norm<uint16_t, float>(a, st);
  else
    launch_norm<uint16_t, uint16_t>(a, st);
  return cudaGetLastError();
}

namespace {
template <typename T, typename G, typename W>
cudaError_t norm_grad(const NormGradArgs& a, cudaStream_t st) {
  int slices = 0;
  const int64_t stage = a.cols * (int64_t)(sizeof(G) + sizeof(T) * (a.dh ? 2 : 1));
  if (a.cols <= kShortCols) {
    slices = (int)short_ctas(a.rows);
    if (slices && a.cols <= 256)
      norm_short_grad_kernel<T, G, W, 1><<<slices, 256, 0, st>>>(a);
    else if (slices)
      norm_short_grad_kernel<T, G, W, 2><<<slices, 256, 0, st>>>(a);
  } else if (a.cols <= 1024 * 8 * kGradChunks && 2 * stage <= kGradSmem) {
    if (a.rows > 0) {
      int dev = 0;
      cudaError_t e = cudaGetDevice(&dev);
      if (e != cudaSuccess) return e;
      if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
      {
        static bool set[kMaxDevices] = {};
        static std::mutex mu;
        std::lock_guard<std::mutex> lock(mu);
        if (!set[dev]) {
          e = cudaFuncSetAttribute(norm_grad_kernel<T, G, W>, cudaFuncAttributeMaxDynamicSharedMemorySize, kGradSmem);
          if (e != cudaSuccess) return e;
          set[dev] = true;
        }
      }
      // groups: as many as there are threads, slots (two each) and rows for
      const int threads = grad_threads(a.cols);
      slices = (int)(a.rows < kSms ? a.rows : kSms);
      int64_t groups = 1024 / threads, fit = kGradSmem / (2 * stage), each = (a.rows + kSms - 1) / kSms;
      if (groups > kGradMaxGroups) groups = kGradMaxGroups;
      if (groups > fit) groups = fit;
      if (groups > each) groups = each;
      fit = kGradSmem / (stage * groups);
      const int stages = (int)(fit < kGradMaxStages ? fit : kGradMaxStages);
      const GradRing r = {(uint32_t)stages, (uint32_t)stage, (uint32_t)(a.cols * sizeof(G)),
                          (uint32_t)(a.cols * sizeof(T)), (uint32_t)(slices * groups)};
      norm_grad_kernel<T, G, W><<<slices, dim3(threads, (unsigned)groups), stages * groups * stage, st>>>(a, r);
    }
  } else if (a.rows > 0) {
    norm_long_dx_kernel<T, G, W><<<(unsigned)a.rows, kRowThreads, 0, st>>>(a);
    if (cudaError_t e = cudaGetLastError()) return e;
    if (a.dw) {
      slices = (int)(a.rows < 256 ? a.rows : 256);
      norm_long_dw_kernel<T, G><<<dim3((unsigned)((a.cols / 8 + kColThreads - 1) / kColThreads), slices), kColThreads,
                                  0, st>>>(a);
    }
  }
  if (cudaError_t e = cudaGetLastError()) return e;
  if (!a.dw) return cudaSuccess;
  // launched while the kernel before it drains; it waits for that kernel's sums itself
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.cols / 32));
  cfg.blockDim = dim3(kSumWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_dw_sum_kernel<W>, static_cast<const float*>(a.ws), slices, a.cols,
                            static_cast<W*>(a.dw));
}
}  // namespace

cudaError_t launch_rmsnorm_grad(const NormGradArgs& a, bool h_f32, bool dy_f32, bool w_f32, cudaStream_t st) {
  if (a.cols == 0) return cudaSuccess;
  (void)cudaGetLastError();
  using B = uint16_t;
  switch ((h_f32 ? 4 : 0) | (dy_f32 ? 2 : 0) | (w_f32 ? 1 : 0)) {
    case 0: return norm_grad<B, B, B>(a, st);
    case 1: return norm_grad<B, B, float>(a, st);
    case 2: return norm_grad<B, float, B>(a, st);
    case 3: return norm_grad<B, float, float>(a, st);
    case 4: return norm_grad<float, B, B>(a, st);
    case 5: return norm_grad<float, B, float>(a, st);
    case 6: return norm_grad<float, float, B>(a, st);
    default: return norm_grad<float, float, float>(a, st);
  }
}

cudaError_t launch_swiglu(const SwigluArgs& a, bool f32, cudaStream_t st) {
  if (a.rows == 0 || a.cols == 0) return cudaSuccess;
  (void)cudaGetLastError();
  dim3 grid, block;
  // four rows to a thread, between one round of CTAs (4 an SM) and 32 an SM (8192 x
  // 28672: 275 us with 4, 196 with 16, 191 with 32; 2048 x 4096: 10.6 us with 4, 12.7 with 12)
  const int64_t want = a.rows * (a.cols / 16) / (4 * kActThreads);
  act_shape(a.rows, a.cols / 16, want < 4 * kSms ? 4 * kSms : want > 32 * kSms ? 32 * kSms : want, &grid, &block);
  const int64_t es = f32 ? 4 : 2;
  const bool wide = aligned32(a.g, a.ld_g * es) && aligned32(a.u, a.ld_u * es);
  if (f32)
    swiglu_kernel<float><<<grid, block, 0, st>>>(a, wide);
  else
    swiglu_kernel<uint16_t><<<grid, block, 0, st>>>(a, wide);
  return cudaGetLastError();
}

cudaError_t launch_swiglu_grad(const SwigluGradArgs& a, bool f32, bool dy_f32, cudaStream_t st) {
  if (a.rows == 0 || a.cols == 0) return cudaSuccess;
  (void)cudaGetLastError();
  dim3 grid, block;
  act_shape(a.rows, a.cols / 8, INT64_MAX / 2, &grid, &block);
  if (f32 && dy_f32)
    swiglu_grad_kernel<float, float><<<grid, block, 0, st>>>(a);
  else if (f32)
    swiglu_grad_kernel<float, uint16_t><<<grid, block, 0, st>>>(a);
  else if (dy_f32)
    swiglu_grad_kernel<uint16_t, float><<<grid, block, 0, st>>>(a);
  else
    swiglu_grad_kernel<uint16_t, uint16_t><<<grid, block, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t read_ffn_error(uint32_t* err) {
  cudaError_t e = cudaMemcpyFromSymbol(err, g_ffn_error, sizeof(uint32_t));
  if (e == cudaSuccess && *err) {
    const uint32_t zero = 0;
    e = cudaMemcpyToSymbol(g_ffn_error, &zero, sizeof(uint32_t));
  }
  return e;
}

}  // namespace mx
