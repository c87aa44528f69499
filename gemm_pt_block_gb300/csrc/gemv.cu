// gemv.cu -- products of a few activation rows with a 4-bit weight matrix
// (sm_103a): the single-token form of the block-scaled GEMM.
//   y[m, n] = sum_k x[m, k] W[n, k]
// The weights' codes and scales are all of the traffic (N K (1/2 + 1/32)
// bytes against M K + M N values), so the kernel is built around streaming
// them once:
//  * a CTA owns 128 rows of W and a slice of K; one thread streams the codes
//    by TMA, 256 of K a stage, into a ring of shared memory (128-byte swizzle);
//  * converter warps bring x into the same ring as f16, 32 elements under one
//    power-of-two factor (bf16 is divided by 2^(E - 14), E the exponent of its
//    block's largest magnitude: exact down to 2^-31 of that magnitude, and off
//    by at most 2^-39 of it below; MXFP8 codes are f16 values as they are and
//    bring their own factor);
//  * eight warps multiply on the tensor cores: E2M1 codes become f16 exactly
//    (one conversion per two codes), a 16-row x 32-deep block of W meets eight
//    rows of x in two m16n8k16 instructions with fp32 sums that start at zero,
//    and the block's sum enters the running fp32 sum times (factor of W) x
//    (factor of x). NVFP4's E4M3 scales are multiplied into the f16 weights
//    instead (4 + 2 significant bits: exact).
// tcgen05 is not used: its 4-bit operands would need x in 8 or 4 bits, and at
// up to 32 rows the loads, not the products, are what costs.
// Few CTAs: K is split over a cluster of 2, 4 or 8 CTAs, whose sums are added
// in rank order through distributed shared memory, so results do not depend
// on timing.
#include <cuda.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <mutex>

#include "internal.h"
#include "mx_device.cuh"
#include "ptx.cuh"

namespace mx {
namespace {
__device__ uint32_t g_gemv_error;
}  // namespace
}  // namespace mx
#define MX_BOUNDS_FAIL() atomicExch(&::mx::g_gemv_error, ::mx::kErrBounds)

#include "row_device.cuh"
#include "tma_host.h"

namespace mx {
namespace {

constexpr int kRows = 128;                 // rows of W per CTA
constexpr int kStageK = 256;               // K per stage
constexpr int kRowBytes = kStageK / 2;     // code bytes per row and stage
constexpr int kMmaWarps = 8;               // 4 groups of 32 rows x 2 halves of a stage
constexpr int kConvWarps = 4;
constexpr int kThreads = (kMmaWarps + 1 + kConvWarps) * 32;
constexpr int kWBytes = kRows * kRowBytes;
constexpr int kMaxTokens = 32;
#ifndef GEMV_WANT
#define GEMV_WANT 456
#define GEMV_MAX_SPLITS 8
#endif
constexpr uint64_t kWaitLimitNs = 2000000000ull;

// Shared memory of one CTA for tiles of TT rows of x.
template <int TT, bool NV>
struct Smem {
  static constexpr int kX = TT * kStageK * 2;            // f16 [block][token][32]
  static constexpr int kSw = kRows * kStageK / (NV ? 16 : 32);
  static constexpr int kSx = TT * (kStageK / 32) * 4;    // float [block][token]
  static constexpr int kStage = kWBytes + kX + kSw + kSx;
  static constexpr int kStages = TT == 32 ? 6 : TT == 16 ? 4 : 5;
  static constexpr int kCtl = 256;
  static constexpr int kBytes = kStages * kStage + kCtl + 1024;
  static constexpr int kRed = 132 * TT * 4;              // partial sums, in place of the first W stages
  static_assert(kRed <= kWBytes * 2, "partial sums fit the ring");
};

struct Ctl {
  uint64_t full_w[8], full_x[8], empty[8];
  uint32_t abort;
};
static_assert(sizeof(Ctl) <= 256, "control block");

// Bounded wait (about 2 s): on expiry the CTA stops issuing work and the
// library's device error word is set.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, Ctl* ctl) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer_ns();
  while (!ptx::mbar_try_wait_sleep(bar, parity, 100000u)) {
    if (*reinterpret_cast<volatile uint32_t*>(&ctl->abort)) return false;
    if (ptx::globaltimer_ns() - t0 > kWaitLimitNs) {
      *reinterpret_cast<volatile uint32_t*>(&ctl->abort) = 1u;
      atomicExch(&g_gemv_error, 6u);  // MXFP4_ERR_TIMEOUT
      return false;
    }
  }
  return true;
}

// Two codes (low 16 bits) to f16, exact.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t v) {
  uint32_t r;
  asm("{.reg .b16 t, u;\n\tmov.b32 {t, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;}" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t e5m2x2_f16x2(uint32_t v) {
  uint32_t r;
  asm("{.reg .b16 t, u;\n\tmov.b32 {t, u}, %1;\n\tcvt.rn.f16x2.e5m2x2 %0, t;}" : "=r"(r) : "r"(v));
  return r;
}
// Eight E2M1 codes to four f16 pairs (code 0 in the low half of r[0]).
__device__ __forceinline__ void e2m1x8_f16(uint32_t v, uint32_t (&r)[4]) {
  asm("{.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(v));
}
// Two E8M0 bytes (low 16 bits) to bf16, exact (0xFF: NaN).
__device__ __forceinline__ uint32_t e8m0x2_bf16x2(uint32_t v) {
  uint32_t r;
  asm("{.reg .b16 t, u;\n\tmov.b32 {t, u}, %1;\n\tcvt.rn.bf16x2.ue8m0x2 %0, t;}" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t f16x2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
  return r;
}
__device__ __forceinline__ float2 lds64f(uint32_t a) {
  float2 r;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(r.x), "=f"(r.y) : "r"(a));
  return r;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ void stsf(uint32_t a, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
__device__ __forceinline__ float lds_cluster(uint32_t a) {
  float r;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(r) : "r"(a));
  return r;
}

// One stage of x rows m0 .. m0 + tokens - 1, K from k0: lane 4 b + t brings
// elements 8 t .. 8 t + 7 of block b, a row at a time.
template <int TT>
__device__ __forceinline__ void convert_x(const GemvArgs& a, int64_t m0, int tokens, int64_t k0, int lane,
                                          uint32_t xs, uint32_t sxs) {
  const int b = lane >> 2, t = lane & 3;
  const int64_t k = k0 + b * 32 + t * 8;
  const bool live = k < a.K;
  const uint32_t dst = xs + b * (TT * 64) + t * 16, sdst = sxs + b * (TT * 4);
  if (a.x_kind == GemvArgs::kXBf16) {
    const uint16_t* p = static_cast<const uint16_t*>(a.x) + m0 * a.ld_x + k;
#pragma unroll 1
    for (int m = 0; m < tokens; m += 4) {
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = live && m + i < tokens ? __ldg(reinterpret_cast<const uint4*>(p + (m + i) * a.ld_x))
                                      : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (m + i >= tokens) break;
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        uint32_t top = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                                __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
        top = max(top >> 16, top & 0xFFFFu);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // E the exponent field of the block's largest magnitude: times 2^(14 - (E - 127))
        // (at most 2^127) on the way in, its inverse as the factor
        const uint32_t E = max(top >> 7, 14u);
        const float f = __uint_as_float((268u - E) << 23);
        uint32_t h[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          h[j] = f16x2(__fmul_rn(__uint_as_float(w[j] << 16), f), __fmul_rn(__uint_as_float(w[j] & 0xFFFF0000u), f));
        sts128(dst + (m + i) * 64, make_uint4(h[0], h[1], h[2], h[3]));
        if (t == 0) stsf(sdst + (m + i) * 4, E == 14u ? __uint_as_float(0x00400000u) : __uint_as_float((E - 14u) << 23));
      }
    }
  } else {
    const uint8_t* p = static_cast<const uint8_t*>(a.x) + m0 * a.ld_x + k;
    const uint8_t* sp = a.sx + m0 * (a.K >> 5) + (k0 >> 5) + b;
    const bool e5 = a.x_kind == GemvArgs::kXE5m2;
#pragma unroll 1
    for (int m = 0; m < tokens; m += 4) {
      uint2 v[4];
      uint32_t s[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool on = live && m + i < tokens;
        v[i] = on ? __ldg(reinterpret_cast<const uint2*>(p + (m + i) * a.ld_x)) : make_uint2(0, 0);
        s[i] = on && t == 0 ? __ldg(sp + (m + i) * (a.K >> 5)) : 0u;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (m + i >= tokens) break;
        const uint4 h = e5 ? make_uint4(e5m2x2_f16x2(v[i].x), e5m2x2_f16x2(v[i].x >> 16), e5m2x2_f16x2(v[i].y),
                                        e5m2x2_f16x2(v[i].y >> 16))
                           : make_uint4(e4m3x2_f16x2(v[i].x), e4m3x2_f16x2(v[i].x >> 16), e4m3x2_f16x2(v[i].y),
                                        e4m3x2_f16x2(v[i].y >> 16));
        sts128(dst + (m + i) * 64, h);
        if (t == 0) stsf(sdst + (m + i) * 4, __uint_as_float(e8m0x2_bf16x2(s[i]) << 16));
      }
    }
  }
}

// One stage of row-major weight scales, rearranged into the tensor-core tiles
// (128 rows x 4 columns, 512 bytes) that the multiplying warps read: lane l
// brings rows l, l + 32, l + 64, l + 96. Rows past N repeat the last one.
template <bool NV>
__device__ __forceinline__ void convert_sw(const GemvArgs& a, int64_t n0, int64_t k0, int lane, uint32_t sws) {
  constexpr int kCols = kStageK / (NV ? 16 : 32);
  const int64_t cols = a.K / (NV ? 16 : 32), c0 = k0 / (NV ? 16 : 32);
  uint32_t v[kCols / 4][4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint8_t* p = a.sw + min(n0 + lane + 32 * j, a.N - 1) * cols + c0;
    if ((cols & 3) == 0) {
#pragma unroll
      for (int c = 0; c < kCols / 4; ++c)
        v[c][j] = c0 + 4 * c < cols ? __ldg(reinterpret_cast<const uint32_t*>(p) + c) : 0u;
    } else {
#pragma unroll
      for (int c = 0; c < kCols / 4; ++c) {
        v[c][j] = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c0 + 4 * c + i < cols) v[c][j] |= (uint32_t)__ldg(p + 4 * c + i) << (8 * i);
      }
    }
  }
#pragma unroll
  for (int c = 0; c < kCols / 4; ++c) sts128(sws + c * 512 + lane * 16, make_uint4(v[c][0], v[c][1], v[c][2], v[c][3]));
}

template <int NT, bool NV>
__global__ void __launch_bounds__(kThreads, NT == 4 ? 1 : 2)
gemv_kernel(const __grid_constant__ CUtensorMap tm, const GemvArgs a, const int splits) {
  constexpr int TT = 8 * NT;
  using S = Smem<TT, NV>;
  constexpr int ST = S::kStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (ptx::smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t ws = base, xs = ws + ST * kWBytes, sws = xs + ST * S::kX, sxs = sws + ST * S::kSw,
                 ctls = sxs + ST * S::kSx;
  Ctl* ctl = reinterpret_cast<Ctl*>(smem_raw + (ctls - ptx::smem_u32(smem_raw)));
  const uint32_t full_w = ptx::smem_u32(ctl->full_w), full_x = ptx::smem_u32(ctl->full_x),
                 empty = ptx::smem_u32(ctl->empty);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)(blockIdx.x % splits);
  const int64_t n0 = (int64_t)(blockIdx.x / splits) * kRows, m0 = (int64_t)blockIdx.y * kMaxTokens;
  const int tokens = (int)min((int64_t)TT, a.M - m0);
  const int64_t stages = (a.K + kStageK - 1) / kStageK;
  const int64_t s0 = stages * rank / splits, s1 = stages * (rank + 1) / splits;

  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      ptx::mbar_init(full_w + 8 * i, 1);
      ptx::mbar_init(full_x + 8 * i, 1);
      ptx::mbar_init(empty + 8 * i, kMmaWarps);
    }
    ctl->abort = 0;
    ptx::fence_mbar_init();
  }
  __syncthreads();

  float acc[2][NT][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[i][n][c] = 0.0f;
  const int g = lane >> 2, t = lane & 3, wr = warp & 3, half = (warp >> 2) & 1;

  if (warp == kMmaWarps) {
    // ---- producer: codes by TMA, tensor-core scales as they lie in memory
    if (lane == 0) {
      ptx::prefetch_tensormap(&tm);
      int64_t done = s0;
      for (int64_t s = s0; s < s1; ++s, ++done) {
        const int i = (int)((s - s0) % ST);
        const uint32_t round = (uint32_t)((s - s0) / ST);
        if (round && !wait_bar(empty + 8 * i, (round - 1) & 1, ctl)) break;
        uint32_t bytes = kWBytes;
        const int64_t cols = a.K / (NV ? 16 : 32), c0 = s * (kStageK / (NV ? 16 : 32));
        uint32_t sb = 0;
        if (a.mma) {
          sb = (uint32_t)min((int64_t)S::kSw, (cols - c0) * kRows);
          bytes += sb;
        }
        ptx::mbar_arrive_expect_tx(full_w + 8 * i, bytes);
        ptx::tma_load_2d(ws + i * kWBytes, &tm, (int32_t)(s * kRowBytes), (int32_t)n0, full_w + 8 * i);
        if (a.mma) ptx::bulk_load(sws + i * S::kSw, a.sw + n0 * cols + c0 * kRows, sb, full_w + 8 * i);
      }
      // after an abort: the last load into each slot lands (bounded wait) before the CTA's memory goes
      if (*reinterpret_cast<volatile uint32_t*>(&ctl->abort)) {
        const int64_t issued = done - s0;
        for (int64_t r = issued > ST ? issued - ST : 0; r < issued; ++r) {
          const uint64_t t0 = ptx::globaltimer_ns();
          while (!ptx::mbar_try_wait(full_w + 8 * (uint32_t)(r % ST), (uint32_t)(r / ST) & 1) &&
                 ptx::globaltimer_ns() - t0 < kWaitLimitNs / 10) {
          }
        }
      }
    }
    __syncwarp();
  } else if (warp > kMmaWarps) {
    // ---- converters: whole stages in turn
    for (int64_t s = s0 + (warp - kMmaWarps - 1); s < s1; s += kConvWarps) {
      const int i = (int)((s - s0) % ST);
      const uint32_t round = (uint32_t)((s - s0) / ST);
      if (round && !wait_bar(empty + 8 * i, (round - 1) & 1, ctl)) break;
      if (!a.mma) convert_sw<NV>(a, n0, s * kStageK, lane, sws + i * S::kSw);
      convert_x<TT>(a, m0, tokens, s * kStageK, lane, xs + i * S::kX, sxs + i * S::kSx);
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(full_x + 8 * i);
    }
  } else {
    // ---- multiplying warps: rows 32 wr .. 32 wr + 31, four 32-blocks of every stage
    uint32_t chunk[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) chunk[b] = (uint32_t)((((4 * half + b) ^ g) << 4) + 4 * t + (32 * wr + g) * kRowBytes);
    const uint32_t xoff = half * 4 * (TT * 64) + g * 64 + t * 16, sxoff = half * 4 * (TT * 4) + 8 * t,
                   swoff = (NV ? half * 1024 : half * 512) + g * 16 + wr * 4;
    for (int64_t s = s0; s < s1; ++s) {
      const int i = (int)((s - s0) % ST);
      const uint32_t parity = (uint32_t)((s - s0) / ST) & 1;
      if (!wait_bar(full_w + 8 * i, parity, ctl) || !wait_bar(full_x + 8 * i, parity, ctl)) break;
      const int blocks = (int)min((int64_t)4, (a.K - s * kStageK) / 32 - 4 * half);
      const uint32_t w = ws + i * kWBytes, x = xs + i * S::kX + xoff, sx = sxs + i * S::kSx + sxoff,
                     sw = sws + i * S::kSw + swoff;
      uint32_t sc[4][2];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t v = lds32(sw + j * 128);
        if (NV) {
          sc[j][0] = v;
          sc[j][1] = lds32(sw + 512 + j * 128);
        } else {
          sc[j][0] = e8m0x2_bf16x2(v);
          sc[j][1] = e8m0x2_bf16x2(v >> 16);
        }
      }
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        if (b >= blocks) break;
        uint32_t q[4][4];
        float f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          e2m1x8_f16(lds32(w + chunk[b] + j * 8 * kRowBytes), q[j]);
          if (NV) {
            // this lane's eight elements lie in 16-block t / 2 of the run
            const uint32_t d = __byte_perm(sc[j][b >> 1], 0, (2 * (b & 1) + (t >> 1)) * 0x11);
            const uint32_t h = e4m3x2_f16x2(d);
#pragma unroll
            for (int e = 0; e < 4; ++e) q[j][e] = hmul2(q[j][e], h);
          } else {
            f[j] = __uint_as_float((b & 1) ? sc[j][b >> 1] & 0xFFFF0000u : sc[j][b >> 1] << 16);
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint4 v = lds128(x + b * (TT * 64) + n * 512);
          const float2 fx = lds64f(sx + b * (TT * 4) + n * 32);
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            mma16816(c, q[2 * r][0], q[2 * r + 1][0], q[2 * r][1], q[2 * r + 1][1], v.x, v.y);
            mma16816(c, q[2 * r][2], q[2 * r + 1][2], q[2 * r][3], q[2 * r + 1][3], v.z, v.w);
            const float2 p0 = NV ? fx : f2mul(fx, make_float2(f[2 * r], f[2 * r]));
            const float2 p1 = NV ? fx : f2mul(fx, make_float2(f[2 * r + 1], f[2 * r + 1]));
            float2 u = f2fma(make_float2(c[0], c[1]), p0, make_float2(acc[r][n][0], acc[r][n][1]));
            acc[r][n][0] = u.x;
            acc[r][n][1] = u.y;
            u = f2fma(make_float2(c[2], c[3]), p1, make_float2(acc[r][n][2], acc[r][n][3]));
            acc[r][n][2] = u.x;
            acc[r][n][3] = u.y;
          }
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(empty + 8 * i);
    }
  }

  // ---- sums of the two halves, then of the cluster's slices, in fixed order
  __syncthreads();  // every load has landed and been read (or the CTA has aborted)
  const bool ok = *reinterpret_cast<volatile uint32_t*>(&ctl->abort) == 0;
  const uint32_t red = ws;  // float [token][132]
  for (int h = 1; h >= 0; --h) {
    if (ok && warp < kMmaWarps && half == h) {
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t at = red + (uint32_t)((8 * n + 2 * t + (c & 1)) * 132 + 32 * wr + 16 * r + 8 * (c >> 1) + g) * 4;
            float v = acc[r][n][c];
            if (h == 0) v = __fadd_rn(v, __uint_as_float(lds32(at)));
            stsf(at, v);
          }
    }
    __syncthreads();
  }
  if (splits > 1) ptx::cluster_sync();
  if (ok) {
    const int rows = kRows / splits;
    for (int e = threadIdx.x; e < tokens * rows; e += kThreads) {
      const int m = e / rows, r = rank * rows + e % rows;
      const int64_t n = n0 + r;
      if (n >= a.N) continue;
      const uint32_t at = red + (uint32_t)(m * 132 + r) * 4;
      float v = 0.0f;
      if (splits == 1) {
        v = __uint_as_float(lds32(at));
      } else {
        for (int c = 0; c < splits; ++c) v = __fadd_rn(v, lds_cluster(ptx::mapa(at, (uint32_t)c)));
      }
      if (NV) v = __fmul_rn(v, a.p2k);
      const int64_t o = (m0 + m) * a.ld_y + n;
      if (a.y_f32)
        put_at(static_cast<float*>(a.y) + o, v, a.y, a.y_bytes);
      else
        put_at(static_cast<uint16_t*>(a.y) + o, (uint16_t)bf16x2(v, 0.0f), a.y, a.y_bytes);
    }
  }
  __syncwarp();
  if (splits > 1) ptx::cluster_sync();  // peers read this CTA's sums until here
}

template <int NT, bool NV>
cudaError_t launch(const CUtensorMap& tm, const GemvArgs& a, int splits, cudaStream_t st) {
  constexpr int bytes = Smem<8 * NT, NV>::kBytes;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  {
    static bool set[kMaxDevices] = {};
    static std::mutex mu;
    std::lock_guard<std::mutex> lock(mu);
    if (!set[dev]) {
      e = cudaFuncSetAttribute(gemv_kernel<NT, NV>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
      if (e != cudaSuccess) return e;
      set[dev] = true;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.N + kRows - 1) / kRows) * (unsigned)splits,
                     (unsigned)((a.M + kMaxTokens - 1) / kMaxTokens));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)splits;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, gemv_kernel<NT, NV>, tm, a, splits);
}

}  // namespace

cudaError_t launch_gemv(const GemvArgs& a, cudaStream_t st) {
  if (a.M == 0 || a.N == 0) return cudaSuccess;
  (void)cudaGetLastError();  // drop a stale error left by an earlier call
  if (a.K == 0) {
    const size_t es = a.y_f32 ? 4 : 2;
    return cudaMemset2DAsync(a.y, a.ld_y * es, 0, a.N * es, a.M, st);
  }
  CUtensorMap tm;
  if (!make_tma_2d(&tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.qw, a.N, a.K / 2, a.K / 2, kRows, kRowBytes))
    return cudaErrorInvalidValue;
  // K is split until there are about three CTAs an SM.
  const int64_t tiles = (a.N + kRows - 1) / kRows * ((a.M + kMaxTokens - 1) / kMaxTokens);
  const int64_t stages = (a.K + kStageK - 1) / kStageK;
  int splits = 1;
  while (splits < GEMV_MAX_SPLITS && tiles * splits < GEMV_WANT && 2 * splits <= stages) splits *= 2;
  const int nt = a.M <= 8 ? 1 : a.M <= 16 ? 2 : 4;
  if (a.nv)
    return nt == 1 ? launch<1, true>(tm, a, splits, st)
                   : nt == 2 ? launch<2, true>(tm, a, splits, st) : launch<4, true>(tm, a, splits, st);
  return nt == 1 ? launch<1, false>(tm, a, splits, st)
                 : nt == 2 ? launch<2, false>(tm, a, splits, st) : launch<4, false>(tm, a, splits, st);
}

cudaError_t read_gemv_error(uint32_t* err) {
  cudaError_t e = cudaMemcpyFromSymbol(err, g_gemv_error, sizeof(uint32_t));
  if (e == cudaSuccess && *err) {
    const uint32_t zero = 0;
    e = cudaMemcpyToSymbol(g_gemv_error, &zero, sizeof(uint32_t));
  }
  return e;
}

}  // namespace mx
