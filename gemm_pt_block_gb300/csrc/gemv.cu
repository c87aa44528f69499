// gemv.cu -- products of a few activation rows with a 4-bit weight matrix
// (sm_103a): the single-token form of the block-scaled GEMM.
//   y[m, n] = sum_k x[m, k] W[n, k]
// The weights' codes and scales are all of the traffic (N K (1/2 + 1/32)
// bytes, NVFP4 1/2 + 1/16, against M K + M N values), so every kernel here
// streams them once. launch_gemv chooses:
//  * gemv_mx_kernel: MXFP4 weights, K a multiple of 128, a workspace: the
//    tensor cores' MXFP8 products take the codes as they lie in memory;
//  * gemv_kernel: up to eight rows of x otherwise: codes become f16 in
//    registers for mma.sync. One launch and no workspace, so also the faster
//    one for small weights (one row, 8192 x 8192: 12 us against 15);
//  * gemv_tc_kernel: more rows otherwise: codes become bf16 or f16 in tensor
//    memory, once for up to 32 rows.
// Sums are fp32 throughout and added in a fixed order. What each form keeps of x
// stands at its kernel; the call's choice of one by size changes that.
//
// ------------------------------------------------------- up to eight rows ---
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
// K is split over a cluster of up to 16 CTAs (k_splits) where there are few
// row tiles; their sums are added in rank order through distributed shared
// memory.
// Bound by the time to fill and empty two CTAs' rings an SM, then by the
// conversions: 14336 x 4096, one row, 11.7 us (tiled scales; 2.7 TB/s of HBM's
// 6.7), 13.3 with row-major ones; 1000 x 1024 4.2 us, of which a launch is two.
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
constexpr int kBlocks = kStageK / 32;
constexpr int kRowBytes = kStageK / 2;     // code bytes per row and stage
constexpr int kParts = 2;                  // parts of a stage's blocks, each a warp's
constexpr int kMmaWarps = 8;               // four groups of 32 rows x kParts
constexpr int kConvWarps = 4;
constexpr int kThreads = (kMmaWarps + 1 + kConvWarps) * 32;
constexpr int kWBytes = kRows * kRowBytes;
constexpr int kTokens = 8;                 // rows of x: the N of one product
constexpr int kSms = 152, kMostSplits = 16;
constexpr uint64_t kWaitLimitNs = 2000000000ull;

// Shared memory of one CTA.
template <bool NV>
struct Smem {
  static constexpr int kX = kTokens * kStageK * 2;            // f16 [block][token][32]
  static constexpr int kSw = kRows * kStageK / (NV ? 16 : 32);  // scales, as tensor-core tiles
  static constexpr int kSx = kTokens * kBlocks * 4;           // float [block][token]
  static constexpr int kStages = NV ? 4 : 5;
  static constexpr int kBytes = kStages * (kWBytes + kX + kSw + kSx) + 256 + 1024;
  // partial sums [part][token][rows + 4] in place of the W stages
  static_assert(kParts * (kRows + 4) * kTokens * 4 <= kStages * kWBytes, "partial sums fit the ring");
};

struct Ctl {
  uint64_t full_w[8], full_x[8], empty[8];
  uint32_t abort;
};
static_assert(sizeof(Ctl) <= 256, "control block");

// Bounded wait (about 2 s): on expiry the CTA stops issuing work and the
// library's device error word is set. kLong: the first look already lets the
// hardware suspend the thread, for roles that usually have to wait and must not
// take issue slots from the others (MXFP8 form, 28672 x 8192, one row: 27.0 us,
// 28.6 without; the converting form 51 us, 49 without; loops that only look: 35).
template <bool kLong = false>
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, uint32_t* abort) {
  if (kLong ? ptx::mbar_try_wait_sleep(bar, parity, 100000u) : ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer_ns();
  while (!ptx::mbar_try_wait_sleep(bar, parity, 100000u)) {
    if (*reinterpret_cast<volatile uint32_t*>(abort)) return false;
    if (ptx::globaltimer_ns() - t0 > kWaitLimitNs) {
      *reinterpret_cast<volatile uint32_t*>(abort) = 1u;
      atomicExch(&g_gemv_error, 6u);  // MXFP4_ERR_TIMEOUT
      return false;
    }
  }
  return true;
}

// The same for a whole warp, which goes on or leaves together: lanes that saw the phase end and lanes that saw
// the abort flag would otherwise wait for one another at the warp's and the CTA's barriers, without a limit.
template <bool kLong = false>
__device__ __forceinline__ bool wait_bar_warp(uint32_t bar, uint32_t parity, uint32_t* abort) {
  return __all_sync(0xffffffffu, wait_bar<kLong>(bar, parity, abort));
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
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float lds_cluster(uint32_t a) {
  float r;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(r) : "r"(a) : "memory");
  return r;
}

// One stage of x rows 0 .. tokens - 1, K from k0: lane 4 b + t brings
// elements 8 t .. 8 t + 7 of block b, a row at a time.
__device__ __forceinline__ void convert_x(const GemvArgs& a, int tokens, int64_t k0, int lane,
                                          uint8_t* xs, float* sxs) {
  const int b = lane >> 2, t = lane & 3;
  const int64_t k = k0 + b * 32 + t * 8;
  const bool live = k < a.K;
  uint8_t* dst = xs + b * (kTokens * 64) + t * 16;
  float* sdst = sxs + b * kTokens;
  if (a.x_kind == GemvArgs::kXBf16) {
    const uint16_t* p = static_cast<const uint16_t*>(a.x) + k;
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
        *reinterpret_cast<uint4*>(dst + (m + i) * 64) = make_uint4(h[0], h[1], h[2], h[3]);
        if (t == 0) sdst[m + i] = E == 14u ? __uint_as_float(0x00400000u) : __uint_as_float((E - 14u) << 23);
      }
    }
  } else {
    const uint8_t* p = static_cast<const uint8_t*>(a.x) + k;
    const uint8_t* sp = a.sx + (k0 >> 5) + b;
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
        *reinterpret_cast<uint4*>(dst + (m + i) * 64) = h;
        if (t == 0) sdst[m + i] = __uint_as_float(e8m0x2_bf16x2(s[i]) << 16);
      }
    }
  }
}

// Row-major weight scales of one row and stage: kCols consecutive bytes, which
// start at any address. Byte loads of them, each lane another row, filled the L1
// (14336 x 4128, 12 rows: 28 us, and 16 at K = 4096); here the aligned words of
// kCols bytes that hold them are loaded whole.
template <bool NV>
struct RowScales {
  static constexpr int kCols = kStageK / (NV ? 16 : 32), kWords = kCols / 4;
  const uint8_t *p, *end;  // the aligned word of the first stage's scales; the end of the array
  uint32_t off;            // of the scales in the word
  int64_t cols;
  __device__ __forceinline__ RowScales(const GemvArgs& a, int64_t n) : cols(a.K / (NV ? 16 : 32)) {
    const uint8_t* row = a.sw + min(n, a.N - 1) * cols;  // rows past N repeat the last one
    off = (uint32_t)reinterpret_cast<uintptr_t>(row) & (kCols - 1);
    p = row - off;
    end = a.sw + a.N * cols;
  }
  // Word s of the row (the array starts on a multiple of 16 bytes: none begins before it).
  __device__ __forceinline__ void load(int s, uint32_t (&w)[kWords]) const {
    const uint8_t* q = p + (int64_t)s * kCols;
    if (q + kCols <= end) {
      if (NV) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(q));
        w[0] = v.x;
        w[1] = v.y;
        w[2 % kWords] = v.z;
        w[3 % kWords] = v.w;
      } else {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(q));
        w[0] = v.x;
        w[1] = v.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        if ((i & 3) == 0) w[i >> 2] = 0;
        if (q + i < end) w[i >> 2] |= (uint32_t)__ldg(q + i) << (8 * (i & 3));
      }
    }
  }
  // Stage s's scales out of words s and s + 1 (not looked at when `off` is 0); zero bytes past K.
  __device__ __forceinline__ void take(int s, const uint32_t (&lo)[kWords], const uint32_t (&hi)[kWords],
                                       uint32_t (&out)[kWords]) const {
    uint32_t w[2 * kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      w[i] = lo[i];
      w[kWords + i] = hi[i];
    }
    if (NV && (off & 8)) {
#pragma unroll
      for (int i = 0; i + 2 < 2 * kWords; ++i) w[i] = w[i + 2];
    }
    if (off & 4) {
#pragma unroll
      for (int i = 0; i + 1 < 2 * kWords; ++i) w[i] = w[i + 1];
    }
    const int64_t left = cols - (int64_t)s * kCols;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      out[i] = __funnelshift_r(w[i], w[i + 1], 8 * (off & 3));
      if (left < 4 * i + 4) out[i] &= left <= 4 * i ? 0u : 0xFFFFFFFFu >> (32 - 8 * (int)(left - 4 * i));
    }
  }
};

// One stage of row-major weight scales, rearranged into the tensor-core tiles
// (128 rows x 4 columns, 512 bytes) that the multiplying warps read: lane l
// brings rows l, l + 32, l + 64, l + 96.
template <bool NV>
__device__ __forceinline__ void convert_sw(const GemvArgs& a, int64_t n0, int s, int lane, uint8_t* sws) {
  using R = RowScales<NV>;
  constexpr int kWords = R::kWords;
  const int64_t cols = a.K / (NV ? 16 : 32), c0 = (int64_t)s * R::kCols;
  uint32_t v[4][kWords];
  if ((cols & 3) == 0) {
    // rows of whole 4-byte words need no shifts (14336 x 4160, one row, NVFP4: 15.6 us, 16.8 below)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (cols % R::kCols == 0) {
        R(a, n0 + lane + 32 * j).load(s, v[j]);
      } else {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(a.sw + min(n0 + lane + 32 * j, a.N - 1) * cols + c0);
#pragma unroll
        for (int c = 0; c < kWords; ++c) v[j][c] = c0 + 4 * c < cols ? __ldg(p + c) : 0u;
      }
    }
#pragma unroll
    for (int c = 0; c < kWords; ++c)
      *reinterpret_cast<uint4*>(sws + c * 512 + lane * 16) = make_uint4(v[0][c], v[1][c], v[2][c], v[3][c]);
    return;
  }
#pragma unroll
  for (int h = 0; h < 4; h += 2) {  // two rows at a time: four take too many registers
    uint32_t lo[2][kWords], hi[2][kWords];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const R row(a, n0 + lane + 32 * (h + j));
      row.load(s, lo[j]);
      row.load(s + 1, hi[j]);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) R(a, n0 + lane + 32 * (h + j)).take(s, lo[j], hi[j], v[j]);
#pragma unroll
    for (int c = 0; c < kWords; ++c)
      *reinterpret_cast<uint2*>(sws + c * 512 + lane * 16 + 4 * h) = make_uint2(v[0][c], v[1][c]);
  }
}

// The producer thread: stages s0 .. s1 - 1 of the codes of the CTA's 128 rows by
// TMA, and tensor-core scale tiles as they lie in memory, into rings of ST slots.
template <bool NV, int ST>
__device__ void produce(const CUtensorMap& tm, const GemvArgs& a, int64_t n0, int s0, int s1, uint8_t* ws, uint8_t* sws,
                        uint32_t full, uint32_t empty, uint32_t* abort) {
  constexpr int kPer = NV ? 16 : 32, kTile = kRows * kStageK / kPer;
  const int64_t cols = a.K / kPer;
  int i = 0, s = s0;
  uint32_t round = 0;
  for (; s < s1; ++s) {
    if (round && !wait_bar(empty + 8 * i, (round - 1) & 1, abort)) break;
    const int64_t c0 = (int64_t)s * (kStageK / kPer);
    const uint32_t sb = a.mma ? (uint32_t)min((int64_t)kTile, (cols - c0) * kRows) : 0u;
    ptx::mbar_arrive_expect_tx(full + 8 * i, kWBytes + sb);
    ptx::tma_load_2d(ptx::smem_u32(ws + i * kWBytes), &tm, s * kRowBytes, (int32_t)n0, full + 8 * i);
    if (a.mma) ptx::bulk_load(ptx::smem_u32(sws + i * kTile), a.sw + n0 * cols + c0 * kRows, sb, full + 8 * i);
    if (++i == ST) {
      i = 0;
      ++round;
    }
  }
  // after an abort: the last load into each slot lands (bounded wait) before the CTA's memory goes
  if (*reinterpret_cast<volatile uint32_t*>(abort)) {
    const int issued = s - s0;
    for (int r = issued > ST ? issued - ST : 0; r < issued; ++r) {
      const uint64_t t0 = ptx::globaltimer_ns();
      while (!ptx::mbar_try_wait(full + 8 * (uint32_t)(r % ST), (uint32_t)(r / ST) & 1) &&
             ptx::globaltimer_ns() - t0 < kWaitLimitNs / 10) {
      }
    }
  }
}

// The CTA's sums, `planes` of them [token][ld] a plane apart in its shared
// memory, and those of the cluster's other slices of K, added in fixed order
// and stored. Every thread of the CTA calls it, the planes written and visible.
__device__ __forceinline__ void finish(const GemvArgs& a, float* red, int ld, int plane, int planes, int tokens,
                                       int rank, int splits, int64_t n0, int64_t m0, float factor,
                                       const float* per_token, bool ok) {
  const int total = tokens * kRows;
  if (splits > 1) {
    if (ok && planes > 1)
      for (int e = threadIdx.x; e < total; e += blockDim.x) {
        float* d = red + e / kRows * ld + e % kRows;
        *d = __fadd_rn(d[0], d[plane]);
      }
    __syncwarp();
    ptx::cluster_sync();
  }
  if (ok) {
    for (int e = total * rank / splits + threadIdx.x; e < total * (rank + 1) / splits; e += blockDim.x) {
      const int m = e / kRows, r = e % kRows;
      const int64_t n = n0 + r;
      if (n >= a.N) continue;
      const float* d = red + m * ld + r;
      float v = 0.0f;
      if (splits == 1) {
        v = planes > 1 ? __fadd_rn(d[0], d[plane]) : d[0];
      } else {
        const uint32_t at = ptx::smem_u32(d);
        for (int c = 0; c < splits; ++c) v = __fadd_rn(v, lds_cluster(ptx::mapa(at, (uint32_t)c)));
      }
      // (in units of x first: 2^tensor_exp may be 2^100 either way)
      if (per_token) v = __fmul_rn(v, __ldcg(per_token + m0 + m));
      v = __fmul_rn(v, factor);
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

template <bool NV>
__global__ void __launch_bounds__(kThreads, 2)
gemv_kernel(const __grid_constant__ CUtensorMap tm, const GemvArgs a, const int splits) {
  constexpr int groups = kRows / 32;
  using S = Smem<NV>;
  constexpr int ST = S::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const base = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t *const ws = base, *const xs = ws + ST * kWBytes, *const sws = xs + ST * S::kX;
  float* const sxs = reinterpret_cast<float*>(sws + ST * S::kSw);
  Ctl* const ctl = reinterpret_cast<Ctl*>(sws + ST * (S::kSw + S::kSx));
  const uint32_t full_w = ptx::smem_u32(ctl->full_w), full_x = ptx::smem_u32(ctl->full_x),
                 empty = ptx::smem_u32(ctl->empty);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)(blockIdx.x % (unsigned)splits);
  const int64_t n0 = (int64_t)(blockIdx.x / (unsigned)splits) * kRows;
  const int tokens = (int)a.M;
  const int stages = (int)((a.K + kStageK - 1) / kStageK);
  const int s0 = (int)((int64_t)stages * rank / splits), s1 = (int)((int64_t)stages * (rank + 1) / splits);

  if (threadIdx.x == 0) {
    ptx::prefetch_tensormap(&tm);
    for (int i = 0; i < ST; ++i) {
      ptx::mbar_init(full_w + 8 * i, 1);
      ptx::mbar_init(full_x + 8 * i, 1);
      ptx::mbar_init(empty + 8 * i, kMmaWarps);
    }
    ctl->abort = 0;
    ptx::fence_mbar_init();
  }
  __syncthreads();

  float2 acc[2][2];
#pragma unroll
  for (int r = 0; r < 2; ++r) acc[r][0] = acc[r][1] = make_float2(0.0f, 0.0f);
  const int g = lane >> 2, t = lane & 3, part = warp / groups, wr = warp - part * groups;

  if (warp == kMmaWarps) {
    if (lane == 0) produce<NV, ST>(tm, a, n0, s0, s1, ws, sws, full_w, empty, &ctl->abort);
    __syncwarp();
  } else if (warp > kMmaWarps) {
    // ---- converters: whole stages in turn
    for (int s = s0 + (warp - kMmaWarps - 1); s < s1; s += kConvWarps) {
      const int i = (s - s0) % ST;
      const uint32_t round = (uint32_t)((s - s0) / ST);
      if (round && !wait_bar_warp(empty + 8 * i, (round - 1) & 1, &ctl->abort)) break;
      const int64_t k0 = (int64_t)s * kStageK;
      if (!a.mma) convert_sw<NV>(a, n0, s, lane, sws + i * S::kSw);
      convert_x(a, tokens, k0, lane, xs + i * S::kX, sxs + i * (S::kSx / 4));
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(full_x + 8 * i);
    }
  } else {
    // ---- multiplying warps: rows 32 wr .. 32 wr + 31, 32-blocks 4 part .. 4 part + 3 of every stage.
    // Blocks past K need no case of their own: their codes (TMA's fill), their x and its factor are
    // finite (zeros), and their scales are taken as zero bytes.
    uint32_t chunk[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) chunk[b] = (uint32_t)(((4 * part + b) ^ g) << 4) + 4 * t + (32 * wr + g) * kRowBytes;
    const uint32_t swoff = part * (NV ? 1024 : 512) + g * 16 + wr * 4;
    const uint32_t xoff = 4 * part * (kTokens * 64) + g * 64 + t * 16, sxoff = 4 * part * kTokens + 2 * t;
    int i = 0;
    uint32_t parity = 0;
    for (int s = s0; s < s1; ++s) {
      if (!wait_bar_warp(full_w + 8 * i, parity, &ctl->abort) || !wait_bar_warp(full_x + 8 * i, parity, &ctl->abort)) break;
      const bool live = s * kBlocks + 4 * part < (int)(a.K >> 5);
      const uint8_t *w = ws + i * kWBytes, *x = xs + i * S::kX + xoff, *sw = sws + i * S::kSw + swoff;
      const float* sx = sxs + i * (S::kSx / 4) + sxoff;
      uint32_t sc[4][2];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t v = live ? *reinterpret_cast<const uint32_t*>(sw + j * 128) : 0u;
        if (NV) {
          sc[j][0] = v;
          sc[j][1] = live ? *reinterpret_cast<const uint32_t*>(sw + 512 + j * 128) : 0u;
        } else {
          sc[j][0] = e8m0x2_bf16x2(v);
          sc[j][1] = e8m0x2_bf16x2(v >> 16);
        }
      }
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        uint32_t q[4][4];
        float f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          e2m1x8_f16(*reinterpret_cast<const uint32_t*>(w + chunk[b] + j * 8 * kRowBytes), q[j]);
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
        const uint4 v = *reinterpret_cast<const uint4*>(x + b * (kTokens * 64));
        const float2 fx = *reinterpret_cast<const float2*>(sx + b * kTokens);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          mma16816(c, q[2 * r][0], q[2 * r + 1][0], q[2 * r][1], q[2 * r + 1][1], v.x, v.y);
          mma16816(c, q[2 * r][2], q[2 * r + 1][2], q[2 * r][3], q[2 * r + 1][3], v.z, v.w);
          float2 c0 = make_float2(c[0], c[1]), c1 = make_float2(c[2], c[3]), w0 = fx, w1 = fx;
          if (!NV) {
            // the block's sum in units of x first, then times the weights' factor: the product of the two
            // factors may pass fp32 (2^100 by 2^30) where the sum times both does not
            c0 = f2mul(c0, fx);
            c1 = f2mul(c1, fx);
            w0 = make_float2(f[2 * r], f[2 * r]);
            w1 = make_float2(f[2 * r + 1], f[2 * r + 1]);
          }
          acc[r][0] = f2fma(c0, w0, acc[r][0]);
          acc[r][1] = f2fma(c1, w1, acc[r][1]);
        }
      }
      // The loads above have to be done before the slot goes back to the producer. The arrival alone
      // did not keep the last block's behind it in compiled code (slots were refilled under them).
      __threadfence_block();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(empty + 8 * i);
      if (++i == ST) {
        i = 0;
        parity ^= 1u;
      }
    }
  }

  // ---- sums of the parts, then of the cluster's slices, in fixed order
  __syncthreads();  // every load has landed and been read (or the CTA has aborted)
  const bool ok = *reinterpret_cast<volatile uint32_t*>(&ctl->abort) == 0;
  float* const red = reinterpret_cast<float*>(ws);  // [part][token][rows + 4]
  constexpr int ld = kRows + 4, plane = kTokens * ld;
  if (ok && warp < kMmaWarps) {
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float* d = red + part * plane + 2 * t * ld + 32 * wr + 16 * r + 8 * c + g;
        d[0] = acc[r][c].x;
        d[ld] = acc[r][c].y;
      }
  }
  __syncthreads();
  finish(a, red, ld, plane, kParts, tokens, rank, splits, n0, 0, NV ? a.p2k : 1.0f, nullptr, ok);
}

// ---------------------------------------------------- more rows of x ---
// Above eight rows the products of mma.sync and their operands' reads grow with
// the rows; here the weights become bf16 once, in tensor memory, and tcgen05
// multiplies them with up to 32 rows of x for one instruction's issue:
//  * 128 rows of W are the M of the instruction, the rows of x its N; x goes in
//    as bf16 (E4M3 and E5M2 codes times their factor are exact in bf16 down to
//    its smallest step, 2^-133), so both operands are exact and the sums fp32, in
//    tensor memory;
//  * eight warps turn codes into bf16: a code's three magnitude bits, moved to
//    bits 8..6 of a bf16 word, are the subnormal that is 2^-126 times its value
//    (zero and the half included), so one packed product with 2^126 times the
//    block's scale gives code x scale exactly. Scales above 2 (E8M0) take a
//    second product; NVFP4's scales go in 2^-8 smaller, which the end undoes (as
//    little as their largest allows: sums of tiny x stay above the subnormals);
//  * the pairs that one word of codes gives are elements (i, i + 4) of its
//    eight: x is laid down in the same order instead of reordering W.
// Two CTAs an SM, so that one converts while the other starts or ends. Bound by
// the hand-over of buffers between the roles (store to tensor memory, barrier,
// issue, barrier), which the number of rows does not change: without conversions
// and products 43 of 52 us remained. NVFP4, tiled scales, 28672 x 8192, 32 rows
// 49 us (23 rows, 14336 x 4096: 21 us); MXFP4 without the workspace, 16 rows,
// 58 us. Tried without gain: waiting for a buffer's store only after the next
// one's conversion, buffers handed over in pairs, twice the converting warps (28
// us where eight take 22), one issuing thread (26) or four (21.6 against 20.9),
// a deeper ring of x, byte-permute tables in place of some conversions.
constexpr int kTcTokens = 32;
constexpr int kTcStages = 3;                // of kStageK
constexpr int kTcK = 64;                    // K per tensor-core buffer
constexpr int kTcBufs = 4, kTcBufsX = 4;    // of the weights (tensor memory), of x (shared memory)
constexpr int kTcDeq = 8;                   // warps that convert weights
// Sums kept in tensor memory, two to an issuing thread, in turn, added at the
// end: the tensor cores round every K = 16 step of a sum toward zero, so
// one sum over all of K drifts by up to K / 16 units of its last place
// (measured: 1.1e-5 of sum |x w| at K = 16384), and four by a quarter of that.
constexpr int kTcSums = 4;
// tensor-memory columns: the sums, then the buffers of the weights
constexpr uint32_t kTcA = kTcSums * kTcTokens, kTcACols = kTcK / 2, kTcTmem = kTcA + kTcBufs * kTcACols;
static_assert(kTcTmem == 256, "two CTAs an SM");
constexpr int kTcIss = 2;                   // threads that issue products: the even and the odd buffers
// Warps that convert x, or (kF16) the one that loads it: fewer threads leave the others more registers (NVFP4, 32
// rows, 28672 x 8192: 49 us with 80, 52 with 64).
template <bool kF16>
struct TcRoles {
  static constexpr int kConv = kF16 ? 1 : 4, kThreads = (kTcDeq + 1 + kTcIss + kConv) * 32;
};
constexpr int kTcB = kTcTokens * kTcK * 2;

struct TcCtl {
  uint64_t full_w[kTcStages], empty_w[kTcStages], full_a[kTcBufs], empty_a[kTcBufs], full_b[kTcBufsX],
      empty_b[kTcBufsX], acc_full;
  uint32_t tmem, abort;
};

template <bool NV>
constexpr int tc_smem() {
  return kTcBufsX * kTcB + kTcStages * (kWBytes + kRows * kStageK / (NV ? 16 : 32)) + (int)sizeof(TcCtl) + 1024;
}

__device__ __forceinline__ uint32_t hmul2_bf16(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Eight codes to bf16 pairs (0, 4), (1, 5), (2, 6), (3, 7) of 2^-126 times their values.
__device__ __forceinline__ void e2m1x8_bf16_tiny(uint32_t v, uint32_t (&r)[4]) {
  r[0] = ((v << 12) & 0x80008000u) | ((v << 6) & 0x01C001C0u);
  r[1] = ((v << 8) & 0x80008000u) | ((v << 2) & 0x01C001C0u);
  r[2] = ((v << 4) & 0x80008000u) | ((v >> 2) & 0x01C001C0u);
  r[3] = (v & 0x80008000u) | ((v >> 6) & 0x01C001C0u);
}

// f16 x of the NVFP4 form: rows [tile][n][K] and a factor for each token, in the workspace.
struct TcX {
  int tiles, n;
  int64_t factors, bytes;
};
TcX tc_x(const GemvArgs& a) {
  TcX x;
  const int tokens = (int)(a.M < kTcTokens ? a.M : kTcTokens);
  x.tiles = (int)((a.M + kTcTokens - 1) / kTcTokens);
  x.n = (tokens + 15) & ~15;
  x.factors = (int64_t)x.tiles * x.n * a.K * 2;
  x.bytes = x.factors + a.M * 4;
  return x;
}

// One CTA a token: the largest magnitude's exponent E, x 2^(14 - E) as f16, and 2^(E - 14). (As in the
// conversion for few rows, with one factor for the whole row: exact down to 2^-31 of the row's largest
// magnitude, off by at most 2^-39 of it below.)
constexpr int kF16Threads = 512;
__global__ void __launch_bounds__(kF16Threads) gemv_f16_rows_kernel(const GemvArgs a, const TcX s) {
  ptx::launch_dependents();
  __shared__ uint32_t part[kF16Threads / 32];
  const int64_t m = blockIdx.x, nkb = a.K >> 5;
  uint8_t* const out = a.ws + ((m / kTcTokens) * s.n + m % kTcTokens) * a.K * 2;
  const bool codes = a.x_kind != GemvArgs::kXBf16, e5 = a.x_kind == GemvArgs::kXE5m2;
  auto load = [&](int64_t k, float (&f)[8]) {
    if (!codes) {
      Vec8<uint16_t> v{__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + m * a.ld_x + k))};
      unpack8(v, f);
      return;
    }
    const uint2 q = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.x) + m * a.ld_x + k));
    const float sx = __uint_as_float(e8m0x2_bf16x2(__ldg(a.sx + m * nkb + (k >> 5))) << 16);
    const uint32_t c[4] = {q.x, q.x >> 16, q.y, q.y >> 16};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t h = e5 ? e5m2x2_f16x2(c[j]) : e4m3x2_f16x2(c[j]);
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
      f[2 * j] = __fmul_rn(v.x, sx);
      f[2 * j + 1] = __fmul_rn(v.y, sx);
    }
  };
  uint32_t top = 0;
  float f[8];
  for (int64_t k = threadIdx.x * 8; k < a.K; k += kF16Threads * 8) {
    load(k, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(f[j]) & 0x7FFFFFFFu);
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
  __syncthreads();
  top = __reduce_max_sync(0xffffffffu, part[threadIdx.x % (kF16Threads / 32)]);
  const uint32_t E = max(top >> 23, 15u);
  const float scale = __uint_as_float((268u - E) << 23);
  if (threadIdx.x == 0)
    put_at(reinterpret_cast<float*>(a.ws + s.factors) + m, __uint_as_float((E - 14u) << 23), a.ws, a.ws_bytes);
  for (int64_t k = threadIdx.x * 8; k < a.K; k += kF16Threads * 8) {
    load(k, f);
    put_at(out + 2 * k, make_uint4(f16x2(f[0] * scale, f[1] * scale), f16x2(f[2] * scale, f[3] * scale),
                                   f16x2(f[4] * scale, f[5] * scale), f16x2(f[6] * scale, f[7] * scale)),
           a.ws, a.ws_bytes);
  }
}

// kF16: NVFP4 weights with x as f16 in the workspace. E2M1 codes become f16 by
// conversion, two an instruction, and one packed product with their E4M3 scale
// (six significant bits: exact) finishes them; x comes by TMA.
template <bool NV, bool kF16>
__global__ void __launch_bounds__(TcRoles<kF16>::kThreads, 2)
gemv_tc_kernel(const __grid_constant__ CUtensorMap tm, const __grid_constant__ CUtensorMap tm_x, const GemvArgs a,
               const TcX sx, const int splits) {
  static_assert(NV || !kF16, "E8M0 scales are beyond f16");
  constexpr int kPer = NV ? 16 : 32, kTile = kRows * kStageK / kPer;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const base = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t *const ws = base, *const bs = ws + kTcStages * kWBytes, *const sws = bs + kTcBufsX * kTcB;
  TcCtl* const ctl = reinterpret_cast<TcCtl*>(sws + kTcStages * kTile);
  const uint32_t full_w = ptx::smem_u32(ctl->full_w), empty_w = ptx::smem_u32(ctl->empty_w),
                 full_a = ptx::smem_u32(ctl->full_a), empty_a = ptx::smem_u32(ctl->empty_a),
                 full_b = ptx::smem_u32(ctl->full_b), empty_b = ptx::smem_u32(ctl->empty_b),
                 acc_full = ptx::smem_u32(&ctl->acc_full);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)(blockIdx.x % (unsigned)splits);
  const int64_t n0 = (int64_t)(blockIdx.x / (unsigned)splits) * kRows, m0 = (int64_t)blockIdx.y * kTcTokens;
  const int tokens = (int)min((int64_t)kTcTokens, a.M - m0), cols_n = (tokens + 15) & ~15;
  const int stages = (int)((a.K + kStageK - 1) / kStageK);
  const int s0 = (int)((int64_t)stages * rank / splits), s1 = (int)((int64_t)stages * (rank + 1) / splits);
  // buffers of kTcK that hold anything (the last stage may be short)
  const int bufs = (int)min((int64_t)(s1 - s0) * (kStageK / kTcK), (a.K - (int64_t)s0 * kStageK + kTcK - 1) / kTcK);

  if (threadIdx.x == 0) {
    ptx::prefetch_tensormap(&tm);
    for (int i = 0; i < kTcStages; ++i) {
      ptx::mbar_init(full_w + 8 * i, 1);
      ptx::mbar_init(empty_w + 8 * i, kTcDeq);
    }
    for (int i = 0; i < kTcBufs; ++i) {
      ptx::mbar_init(full_a + 8 * i, kTcDeq);
      ptx::mbar_init(empty_a + 8 * i, 1);
    }
    for (int i = 0; i < kTcBufsX; ++i) {
      ptx::mbar_init(full_b + 8 * i, 1);
      ptx::mbar_init(empty_b + 8 * i, 1);
    }
    ptx::mbar_init(acc_full, kTcIss);
    ctl->abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == kTcDeq + 1) {
    ptx::tmem_alloc(ptx::smem_u32(&ctl->tmem), kTcTmem);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = ctl->tmem;

  if (warp == kTcDeq) {
    if (lane == 0) produce<NV, kTcStages>(tm, a, n0, s0, s1, ws, sws, full_w, empty_w, &ctl->abort);
    __syncwarp();
  } else if (warp > kTcDeq && warp <= kTcDeq + kTcIss) {
    // ---- the threads that issue the products; a slot of the rings is always the same one's
    if (lane == 0) {
      // bf16 operands (1 at bits 7 and 10; f16: 0), fp32 sums (1 at bit 4), K-major, N / 8 and M / 16
      const uint32_t idesc = (1u << 4) | (kF16 ? 0u : (1u << 7) | (1u << 10)) | ((uint32_t)(cols_n >> 3) << 17) | ((kRows >> 4) << 24);
      const int me = warp - kTcDeq - 1;
      const uint64_t b0 = ptx::smem_desc(ptx::smem_u32(bs), 16, 1024, 2);
      for (int b = me; b < bufs; b += kTcIss) {
        const int i = b % kTcBufs, ix = b % kTcBufsX;
        if (!wait_bar(full_a + 8 * i, (uint32_t)(b / kTcBufs) & 1, &ctl->abort) ||
            !wait_bar(full_b + 8 * ix, (uint32_t)(b / kTcBufsX) & 1, &ctl->abort))
          break;
        ptx::tc_fence_after();
        const uint64_t bd = b0 + (uint32_t)ix * (kTcB >> 4);
#pragma unroll
        for (int k = 0; k < kTcK / 16; ++k)
          ptx::mma_f16_ta(tmem + (2 * me + (k & 1)) * kTcTokens, tmem + kTcA + i * kTcACols + k * 8, bd + 2 * k, idesc,
                          b != me || k > 1);
        ptx::tc_commit(empty_a + 8 * i);
        ptx::tc_commit(empty_b + 8 * ix);
      }
      // completes when the products issued so far have: nothing reads shared or
      // writes tensor memory past it, after an abort either (bounded wait there)
      ptx::tc_commit(acc_full);
      const uint64_t t0 = ptx::globaltimer_ns();
      while (!ptx::mbar_try_wait(acc_full, 0) && ptx::globaltimer_ns() - t0 < kWaitLimitNs / 10) {
      }
    }
    __syncwarp();
  } else if (kF16 && warp > kTcDeq + kTcIss) {
    // ---- x by TMA, once the rows are written
    if (lane == 0) {
      ptx::wait_prior_grid();
      for (int b = 0; b < bufs; ++b) {
        const int i = b % kTcBufsX;
        if (b >= kTcBufsX && !wait_bar(empty_b + 8 * i, (uint32_t)(b / kTcBufsX - 1) & 1, &ctl->abort)) break;
        ptx::mbar_arrive_expect_tx(full_b + 8 * i, (uint32_t)sx.n * kTcK * 2);
        ptx::tma_load_2d(ptx::smem_u32(bs + i * kTcB), &tm_x, s0 * kStageK + b * kTcK, (int)blockIdx.y * sx.n, full_b + 8 * i);
      }
      if (*reinterpret_cast<volatile uint32_t*>(&ctl->abort)) {  // loads in flight land before the CTA's memory goes
        const uint64_t t0 = ptx::globaltimer_ns();
        while (ptx::globaltimer_ns() - t0 < kWaitLimitNs / 100) {
        }
      }
    }
    __syncwarp();
  } else if (warp > kTcDeq + kTcIss) {
    // ---- x: whole buffers in turn, a lane eight elements (16 bytes of bf16) of every fourth row,
    // in the weights' order. A buffer's loads are all in flight before its slot is waited for.
    const int c = lane & 7;
    const int64_t x_bytes = a.x_kind == GemvArgs::kXBf16 ? 2 : 1, x_step = 4 * a.ld_x * x_bytes, s_step = 4 * (a.K >> 5);
    const uint8_t* const x_rows = static_cast<const uint8_t*>(a.x) + (m0 + (lane >> 3)) * a.ld_x * x_bytes;
    const uint8_t* const s_rows = a.sx + (m0 + (lane >> 3)) * (a.K >> 5);
    for (int b = warp - kTcDeq - kTcIss - 1; b < bufs; b += TcRoles<kF16>::kConv) {
      const int i = b % kTcBufsX;
      const uint32_t round = (uint32_t)(b / kTcBufsX);
      const int64_t k = (int64_t)s0 * kStageK + (int64_t)b * kTcK + 8 * c;
      const bool live = k < a.K;
      uint4 w[kTcTokens / 4];  // bf16 pairs (0, 1), (2, 3), (4, 5), (6, 7); or codes and their scale
      const uint8_t* px = x_rows + k * x_bytes;
      const uint8_t* ps = s_rows + (k >> 5);
#pragma unroll
      for (int e = 0; e < kTcTokens / 4; ++e) {
        w[e] = make_uint4(0, 0, 0, 0);
        if (live && 4 * e + (lane >> 3) < tokens) {
          if (a.x_kind == GemvArgs::kXBf16) {
            w[e] = __ldg(reinterpret_cast<const uint4*>(px));
          } else {
            const uint2 q = __ldg(reinterpret_cast<const uint2*>(px));
            w[e] = make_uint4(q.x, q.y, __ldg(ps), 0);
          }
        }
        px += x_step;
        ps += s_step;
      }
      if (round && !wait_bar_warp(empty_b + 8 * i, (round - 1) & 1, &ctl->abort)) break;
#pragma unroll
      for (int e = 0; e < kTcTokens / 4; ++e) {
        const int m = 4 * e + (lane >> 3);
        if (4 * e >= tokens) break;
        if (a.x_kind != GemvArgs::kXBf16) {
          const float f = __uint_as_float(e8m0x2_bf16x2(w[e].z) << 16);
          const bool e5 = a.x_kind == GemvArgs::kXE5m2;
          uint32_t h[4] = {w[e].x, w[e].x >> 16, w[e].y, w[e].y >> 16};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            h[j] = e5 ? e5m2x2_f16x2(h[j]) : e4m3x2_f16x2(h[j]);
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
            h[j] = bf16x2(__fmul_rn(v.x, f), __fmul_rn(v.y, f));
          }
          w[e] = make_uint4(h[0], h[1], h[2], h[3]);
        }
        *reinterpret_cast<uint4*>(bs + i * kTcB + m * 128 + ((c ^ (m & 7)) << 4)) =
            make_uint4(__byte_perm(w[e].x, w[e].z, 0x5410), __byte_perm(w[e].x, w[e].z, 0x7632),
                       __byte_perm(w[e].y, w[e].w, 0x5410), __byte_perm(w[e].y, w[e].w, 0x7632));
      }
      ptx::fence_proxy_async();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(full_b + 8 * i);
    }
  } else {
    // ---- weights: a thread has one row and one of a buffer's two 32-blocks
    constexpr int kWords = NV ? 4 : 2;  // of a row's scales in a stage
    const int r = threadIdx.x & 127, half = threadIdx.x >> 7;
    const int64_t cols = a.K / kPer;
    const RowScales<NV> row(a, n0 + r);  // row-major scales: words of this stage and of the next
    uint32_t sc[kWords] = {}, now[kWords] = {}, ahead[kWords] = {};
    if (!a.mma && s0 < s1) {
      row.load(s0, now);
      if (row.off || s0 + 1 < s1) row.load(s0 + 1, ahead);
    }
    bool go = true;
    for (int st = 0; go && st < s1 - s0; ++st) {
      const int slot = st % kTcStages;
      if (!a.mma) {
        row.take(s0 + st, now, ahead, sc);
#pragma unroll
        for (int e = 0; e < kWords; ++e) now[e] = ahead[e];
        if (st + 1 < s1 - s0 && (row.off || st + 2 < s1 - s0)) row.load(s0 + st + 2, ahead);
      }
      if (!wait_bar_warp(full_w + 8 * slot, (uint32_t)(st / kTcStages) & 1, &ctl->abort)) break;
      if (a.mma) {
        const int live = (int)min((int64_t)kWords, (cols - (int64_t)(s0 + st) * (kStageK / kPer)) / 4);
#pragma unroll
        for (int e = 0; e < kWords; ++e)  // words past K were not copied
          sc[e] = e < live ? *reinterpret_cast<const uint32_t*>(sws + slot * kTile + e * 512 + (r & 31) * 16 + (r >> 5) * 4)
                           : 0u;
      }
#pragma unroll
      for (int j = 0; j < kStageK / kTcK; ++j) {
        const int b = st * (kStageK / kTcK) + j, i = j % kTcBufs;
        if (b >= bufs) break;
        const uint32_t round = (uint32_t)(b / kTcBufs);
        const uint4 v = *reinterpret_cast<const uint4*>(ws + slot * kWBytes + r * kRowBytes + (((2 * j + half) ^ (r & 7)) << 4));
        uint32_t f0, f1, g = 0;  // factors of the two halves of the block; second factor (E8M0 above 2)
        if (kF16) {
          const uint32_t h = e4m3x2_f16x2(sc[j] >> (16 * half));
          f0 = __byte_perm(h, 0, 0x1010);
          f1 = __byte_perm(h, 0, 0x3232);
        } else if (NV) {
          const uint32_t h = e4m3x2_f16x2(sc[j] >> (16 * half));
          const float2 q = __half22float2(*reinterpret_cast<const __half2*>(&h));
          f0 = bf16x2(q.x * 0x1p118f, q.x * 0x1p118f);  // (up to 1.75 2^126)
          f1 = bf16x2(q.y * 0x1p118f, q.y * 0x1p118f);
        } else {
          // 2^126 2^(c - 127), in two factors above 2^127
          const uint32_t c = (sc[j >> 1] >> (16 * (j & 1) + 8 * half)) & 0xFFu;
          f0 = c <= 128u ? (c + 126u) << 7 : c == 255u ? 0x7FC0u : 254u << 7;
          g = c <= 128u || c == 255u ? 0u : (c - 1u) << 7;
          f0 |= f0 << 16;
          g |= g << 16;
          f1 = f0;
        }
        uint32_t out[16];
        const uint32_t words[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t q[4];
          if (kF16)
            e2m1x8_f16(words[w], q);
          else
            e2m1x8_bf16_tiny(words[w], q);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            out[4 * w + e] = kF16 ? hmul2(q[e], w < 2 ? f0 : f1) : hmul2_bf16(q[e], w < 2 ? f0 : f1);
        }
        if (!NV && g) {
#pragma unroll
          for (int e = 0; e < 16; ++e) out[e] = hmul2_bf16(out[e], g);
        }
        // the warp stores together
        if (round && !(go = wait_bar_warp(empty_a + 8 * i, (round - 1) & 1, &ctl->abort))) break;
        ptx::tc_fence_after();
        ptx::tmem_st_32x32b_x16(tmem + ((uint32_t)(r & ~31) << 16) + kTcA + i * kTcACols + 16 * half, out);
        ptx::tc_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(full_a + 8 * i);
      }
      // (the loads from this stage's slot are done: what they read has been stored)
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(empty_w + 8 * slot);
    }
  }

  // ---- the sums leave tensor memory: warp w has rows 32 w .. 32 w + 31
  float* const red = reinterpret_cast<float*>(ws);  // [token][132], in place of the codes
  constexpr int ld = kRows + 4;
  __syncthreads();  // the issuing thread has seen its last product complete (or the CTA has aborted)
  const bool ok = *reinterpret_cast<volatile uint32_t*>(&ctl->abort) == 0;
  ptx::tc_fence_after();
  if (warp < 4) {
    for (int c = 0; c < cols_n; c += 16) {
      float f[16] = {};
      for (int j = 0; j < min(bufs, kTcIss) * (kTcSums / kTcIss); ++j) {
        uint32_t v[16];
        ptx::tmem_ld_32x32b_x16(tmem + ((uint32_t)(32 * warp) << 16) + j * kTcTokens + c, v);
        ptx::tc_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) f[e] = __fadd_rn(f[e], __uint_as_float(v[e]));
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) red[(c + e) * ld + 32 * warp + lane] = f[e];
    }
    ptx::tc_fence_before();
  }
  __syncthreads();
  if (warp == kTcDeq + 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTcTmem);
  }
  if (kF16) ptx::wait_prior_grid();  // (the tokens' factors)
  finish(a, red, ld, 0, 1, tokens, rank, splits, n0, m0, kF16 ? a.p2k : NV ? a.p2k * 0x1p8f : 1.0f,
         kF16 ? reinterpret_cast<const float*>(a.ws + sx.factors) : nullptr, ok);
}

// ------------------------------------- MXFP4 weights on the MXFP8 products ---
// kind::mxf8f6f4 multiplies E2M1 by E4M3 or E5M2, each side with its E8M0 scale
// per 32: the weights go in as they lie in memory and nothing is converted per
// weight. x comes as MXFP8 codes, or is written as a sum of MXFP8 vectors:
// digit 1 is bf16 x rounded to E4M3 under its block's scale 2^e, digit 2 what
// that leaves under 2^(e - 4), digit 3 what is left then under 2^(e - 8). Each
// digit is a row of the instruction's N, and a token's digits are added at the
// end. E4M3 keeps four significant bits and bf16 has eight, so the digits are
// exact for magnitudes down to 2^-17 of their block's largest, and off by at
// most 2^-25 of it below: the last digit ends at 2^-17 steps, half of one is
// 2^-18, and the block's largest is above 224 (two digits: 2^-21, which an outlier
// in a block of small values shows: measured 4.6e-5 of sum |x w|). Scales end at
// 2^-127, so a block below 2^-111 is off by up to 2^-137. A block that holds an
// infinity or a NaN has the NaN scale: its token's sums are NaN.
//
// A small kernel makes the digits and their scale tiles once, in the caller's
// workspace; the product's CTAs start under it (programmatic launch) and have
// their first weights in flight when it ends. They stream 128 rows of W, 128 of
// K a stage: TMA spreads the codes into the 8-bit containers that the
// instruction reads, two threads issue the products in turn, and the row-major
// scales, where W has those, are arranged into tiles by four warps.
//
// 28672 x 8192 (125 MB) takes 27 us at one row, 4.6 TB/s or 69 % of a copy's
// rate: of the other 8 us about one is the digits' kernel and two are the join of
// shared tiles; the rest is not shown (a plain read of as many bytes, 28.5 us, has
// the same start and end of every SM's stream, and is no bound: this kernel is
// faster). 30 us at 12 rows, 37 at 32 (three digits of each row are 96 of the
// instruction's N, and leave a ring of six stages).
//
// One CTA an SM takes an equal run of all (row tile, stage) units, its ring
// going on from one tile to the next, so that every SM streams to the end
// (28672 x 8192 has 224 tiles: a CTA each on 152 SMs took 32 us). A tile
// that several CTAs share goes to the workspace in parts; the CTA that adds the
// last part sums them in CTA order, so the result does not depend on timing.
constexpr int kMxN = 96;                    // most digit rows per CTA
constexpr int kMxK = 128;
constexpr int kMxA = kRows * kMxK, kMxTile = 512;
// threads that issue products; warps: sums out of tensor memory, row-major scales
constexpr int kMxIss = 2, kMxEpi = 4, kMxConv = 4;
constexpr int kMxThreads = (2 + kMxIss + kMxEpi + kMxConv) * 32;
template <int kN>
struct MxRing {
  static constexpr int kB = kN * kMxK;
  static constexpr int kStages = kN <= 32 ? 10 : kN <= 64 ? 8 : 6;
  static_assert(kStages % kMxIss == 0 && kStages >= kMxConv, "a slot is always the same issuing thread's");
  static constexpr int kBytes = kStages * (kMxA + kB + 2 * kMxTile) + 1024 + 512;
};
// Tensor-memory columns: two buffers of sums (one filled while the other leaves), and for each issuing thread a
// slot of scales (A's four columns, then B's), so that one thread's copies do not wait for the other's products.
constexpr uint32_t kMxTmem = 512, kMxBuf = 240, kMxSf = 480;
static_assert(2 * kMxBuf <= kMxSf && kMxSf + 8 * kMxIss <= kMxTmem, "columns");

struct MxCtl {
  uint64_t full[10], empty[10], acc_full[2], acc_empty[2], drain[kMxIss];
  uint32_t tmem, abort, last;
};
static_assert(sizeof(MxCtl) <= 512, "control block");

// How x is spread over the N of the instruction (`digits` rows a token,
// `tokens` tokens a tile, `tiles` of them; n the rows rounded up to 16), and the
// work over `ctas` CTAs.
struct MxShape {
  int digits, tokens, tiles, n, ctas;
  int64_t stages, units;  // stages of K; (row tile, token tile, stage) units
};
MxShape mx_shape(const GemvArgs& a) {
  MxShape s;
  s.digits = a.x_kind != GemvArgs::kXBf16 ? 1 : 3;
  const int most = s.digits == 3 ? kMxN / 3 : 64;
  s.tokens = (int)(a.M < most ? a.M : most);
  s.tiles = (int)((a.M + s.tokens - 1) / s.tokens);
  s.n = (s.digits * s.tokens + 15) & ~15;
  s.stages = a.K / kMxK;
  s.units = (a.N + kRows - 1) / kRows * s.tiles * s.stages;
  // eight stages to a CTA at least: shorter runs lose more to filling the ring and adding parts
  const int64_t want = (s.units + 7) / 8;
  s.ctas = (int)(want < kSms ? want : kSms);
  return s;
}
// The workspace: codes [tile][n][K], scale tiles [tile][K / 128][512], parts
// [cta][2][token][128] of fp32, a counter for each row and token tile.
struct MxSpace {
  int64_t scales, parts, counters, bytes;
};
__host__ __device__ inline MxSpace mx_space(const MxShape& s) {
  MxSpace w;
  w.scales = (int64_t)s.tiles * s.n * s.stages * kMxK;
  w.parts = w.scales + s.tiles * s.stages * kMxTile;
  w.counters = w.parts + (int64_t)s.ctas * 2 * s.tokens * kRows * 4;
  w.bytes = w.counters + s.units / s.stages * 4;
  return w;
}

// x to digit codes [tile][n][K] and scale tiles [tile][K / 128][512]; four lanes
// a 32-block.
__global__ void __launch_bounds__(256) gemv_digits_kernel(const GemvArgs a, const MxShape s) {
  ptx::launch_dependents();
  const MxSpace w = mx_space(s);
  uint8_t *const codes = a.ws, *const scales = a.ws + w.scales;
  if (blockIdx.y == 0)
    for (int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x; c < s.units / s.stages; c += (int64_t)gridDim.x * 256)
      put_at(reinterpret_cast<uint32_t*>(a.ws + w.counters) + c, 0u, a.ws, a.ws_bytes);
  const int64_t nkb = a.K >> 5, i = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 2;
  const int64_t m = blockIdx.y, kb = i;
  const int t = threadIdx.x & 3;
  const bool live = kb < nkb;
  const int64_t k = live ? kb * 32 + 8 * t : 0;
  const int tile = (int)(m / s.tokens), row = (int)(m % s.tokens) * s.digits;
  uint8_t* q = codes + ((int64_t)tile * s.n + row) * a.K + k;
  uint8_t* f = scales + ((int64_t)tile * (a.K / kMxK) + kb / 4) * kMxTile + kb % 4;
  auto put_scale = [&](int r, uint32_t c) {
    if (live && t == 0) put_at(f + (r & 31) * 16 + (r >> 5) * 4, (uint8_t)c, a.ws, a.ws_bytes);
  };
  if (a.x_kind != GemvArgs::kXBf16) {
    if (!live) return;
    put_at(q, __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.x) + m * a.ld_x + k)), a.ws, a.ws_bytes);
    put_scale(row, __ldg(a.sx + m * nkb + kb));
    return;
  }
  const uint4 v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + m * a.ld_x + k));
  Vec8<uint16_t> raw{v};
  float x[8];
  unpack8(raw, x);
  float top = absmax3_nan(absmax3_nan(x[0], x[1], x[2]), absmax3_nan(x[3], x[4], x[5]), absmax3_nan(x[6], x[7], 0.0f));
  top = absmax3_nan(top, __shfl_xor_sync(0xffffffffu, top, 1), 0.0f);
  top = absmax3_nan(top, __shfl_xor_sync(0xffffffffu, top, 2), 0.0f);
  const bool bad = __float_as_uint(top) >= 0x7F800000u;
  // the smallest scale under which nothing saturates (448 = 1.75 2^8), kept so that the last digit has one too
  const int e = max(scale_exponent(top, true, true), -127 + 4 * (s.digits - 1));
  float2 r[4];
  const float2 inv = make_float2(inv_scale(e), inv_scale(e));
#pragma unroll
  for (int j = 0; j < 4; ++j) r[j] = bad ? make_float2(0.0f, 0.0f) : f2mul(make_float2(x[2 * j], x[2 * j + 1]), inv);
  for (int d = 0; d < s.digits; ++d) {
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      asm("{.reg .b16 t;\n\tcvt.rn.satfinite.e4m3x2.f32 t, %2, %1;\n\tcvt.u32.u16 %0, t;}"
          : "=r"(c[j]) : "f"(r[j].x), "f"(r[j].y));
      const uint32_t h = e4m3x2_f16x2(c[j]);
      const float2 got = __half22float2(*reinterpret_cast<const __half2*>(&h));
      r[j] = f2mul(f2sub(r[j], got), make_float2(16.0f, 16.0f));  // exact: what this digit leaves, 2^4 finer
    }
    if (live)
      put_at(q + (int64_t)d * a.K, make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16)), a.ws, a.ws_bytes);
    put_scale(row + d, bad ? 255u : (uint32_t)(e - 4 * d + 127));
  }
}

template <int kN>
__global__ void __launch_bounds__(kMxThreads, 1)
gemv_mx_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x, const GemvArgs a,
               const MxShape sh) {
  constexpr int ST = MxRing<kN>::kStages, kB = MxRing<kN>::kB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const base = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
  // A of all stages, then B (both 1024-byte aligned), then the scale tiles
  uint8_t *const as = base, *const bs = as + ST * kMxA, *const sfa = bs + ST * kB, *const sfb = sfa + ST * kMxTile;
  MxCtl* const ctl = reinterpret_cast<MxCtl*>(sfb + ST * kMxTile);
  const uint32_t full = ptx::smem_u32(ctl->full), empty = ptx::smem_u32(ctl->empty),
                 acc_full = ptx::smem_u32(ctl->acc_full), acc_empty = ptx::smem_u32(ctl->acc_empty);
  const MxSpace space = mx_space(sh);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t u0 = sh.units * blockIdx.x / sh.ctas, u1 = sh.units * (blockIdx.x + 1) / sh.ctas;
  const int per = 2 * kMxIss * sh.n <= (int)kMxBuf ? 2 : 1;  // sums of each issuing thread

  if (threadIdx.x == 0) {
    ptx::prefetch_tensormap(&tm_w);
    ptx::prefetch_tensormap(&tm_x);
    for (int i = 0; i < ST; ++i) {
      ptx::mbar_init(full + 8 * i, a.mma ? 2 : 3);
      ptx::mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(acc_full + 8 * i, kMxIss);
      ptx::mbar_init(acc_empty + 8 * i, kMxEpi);
    }
    for (int i = 0; i < kMxIss; ++i) ptx::mbar_init(ptx::smem_u32(&ctl->drain[i]), 1);
    ctl->abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(&ctl->tmem), kMxTmem);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = ctl->tmem;

  // The roles of one thread each run on the latency of their instructions, so
  // what they do per unit is kept short: addresses go on by additions (64-bit
  // divisions here took 64 us, and one thread for both kinds of load, with
  // descriptors made anew, 44 us, at one row of x and 28672 x 8192).
  if (warp == 0 || warp == kMxThreads / 32 - 1) {
    // ---- producers: the weights (and their scales where those lie in tiles), and the digits of x
    if (lane == 0) {
      const bool w = warp == 0;
      const int last = (int)sh.stages, tiles = sh.tiles;
      const int64_t t0 = u0 / sh.stages;
      int64_t row = t0 / tiles;
      int tile = (int)(t0 % tiles), s = (int)(u0 - t0 * sh.stages);
      const uint8_t* from = w ? a.sw + (row * last + s) * kMxTile : a.ws + space.scales + ((int64_t)tile * last + s) * kMxTile;
      const uint32_t big = ptx::smem_u32(w ? as : bs), small = ptx::smem_u32(w ? sfa : sfb), step = w ? kMxA : kB;
      // the spread codes count with the bytes they have in memory, half of what they take here
      const bool scales = !w || a.mma;
      const uint32_t bytes = (w ? kMxA / 2 : (uint32_t)sh.n * kMxK) + (scales ? kMxTile : 0);
      const CUtensorMap* tm = w ? &tm_w : &tm_x;
      if (!w) ptx::wait_prior_grid();  // the weights start before the digits are written
      int64_t left = u1 - u0, issued = 0;
      int i = 0, y = w ? (int)(row * kRows) : tile * sh.n;
      uint32_t parity = 1;  // the first round finds the slots empty
      for (; left; --left, ++issued) {
        if (!wait_bar<true>(empty + 8 * i, parity, &ctl->abort)) break;
        ptx::mbar_arrive_expect_tx(full + 8 * i, bytes);
        ptx::tma_load_2d(big + i * step, tm, s * kMxK, y, full + 8 * i);
        if (scales) ptx::bulk_load(small + i * kMxTile, from, kMxTile, full + 8 * i);
        from += kMxTile;
        if (++i == ST) {
          i = 0;
          parity ^= 1u;
        }
        if (++s == last) {  // the next token tile, or the next row tile
          s = 0;
          if (++tile == tiles) {
            tile = 0;
            ++row;
          }
          y = w ? (int)(row * kRows) : tile * sh.n;
          from = w ? a.sw + row * last * kMxTile : a.ws + space.scales + (int64_t)tile * last * kMxTile;
        }
      }
      // after an abort: the last load into each slot lands (bounded wait) before the CTA's memory goes
      if (*reinterpret_cast<volatile uint32_t*>(&ctl->abort)) {
        for (int64_t r = issued > ST ? issued - ST : 0; r < issued; ++r) {
          const uint64_t t = ptx::globaltimer_ns();
          while (!ptx::mbar_try_wait(full + 8 * (uint32_t)(r % ST), (uint32_t)(r / ST) & 1) &&
                 ptx::globaltimer_ns() - t < kWaitLimitNs / 10) {
          }
        }
      }
    }
    __syncwarp();
  } else if (warp <= kMxIss) {
    // ---- two threads issue the products, the even and the odd units of the run, each into sums of its
    // own: four products and two copies of scales to a unit take one thread longer than their loads
    // (42 us where two take 28, at one row of x and 28672 x 8192). The ring has an even number of slots,
    // so a slot is always the same thread's, which sees every phase of its barrier.
    if (lane == 0) {
      const uint32_t xfmt = a.x_kind == GemvArgs::kXE5m2 ? 1u : 0u;
      // A E2M1 (5 at bits 7-9), B E4M3 (0) or E5M2 (1 at bits 10-12), E8M0 scales (bit 23), N / 8, M / 16;
      // which byte of a row's scale word: bits 4-5 (B) and 29-30 (A)
      const uint32_t idesc = (5u << 7) | (xfmt << 10) | ((uint32_t)(sh.n >> 3) << 17) | (1u << 23) | ((kRows >> 4) << 24);
      const uint64_t a0 = ptx::smem_desc(ptx::smem_u32(as), 16, 1024, 2), b0 = ptx::smem_desc(ptx::smem_u32(bs), 16, 1024, 2),
                     fa0 = ptx::smem_desc(ptx::smem_u32(sfa), 0, 128, 0), fb0 = ptx::smem_desc(ptx::smem_u32(sfb), 0, 128, 0);
      const int me = warp - 1;
      const uint32_t mine = (uint32_t)(me * per) * sh.n, other = per == 2 ? (uint32_t)sh.n : 0u;
      int i = me, seg = 0;
      uint32_t parity = 0;
      const uint32_t f = tmem + kMxSf + (uint32_t)me * 8;
      int64_t u = u0 + me;
      bool go = true;
      for (int64_t begin = u0; go && begin < u1; ++seg) {
        const int64_t end = min(u1, (begin / sh.stages + 1) * sh.stages);
        const int buf = seg & 1;
        if (seg >= 2 && !wait_bar<true>(acc_empty + 8 * buf, (uint32_t)(seg / 2 - 1) & 1, &ctl->abort)) break;
        ptx::tc_fence_after();
        const uint32_t d = tmem + buf * kMxBuf + mine;
        bool begun = false;
        for (; u < end; u += kMxIss) {
          if (!(go = wait_bar<true>(full + 8 * i, parity, &ctl->abort))) break;
          ptx::tc_fence_after();
          ptx::tc_cp_32x128b_warpx4(f, fa0 + (uint32_t)i * (kMxTile >> 4));
          ptx::tc_cp_32x128b_warpx4(f + 4, fb0 + (uint32_t)i * (kMxTile >> 4));
          const uint64_t ad = a0 + (uint32_t)i * (kMxA >> 4), bd = b0 + (uint32_t)i * (kB >> 4);
#pragma unroll
          for (int k = 0; k < kMxK / 32; ++k)
            ptx::mma_mxf8f6f4(d + (k & 1) * other, ad + 2 * k, bd + 2 * k, idesc | (k << 4) | (k << 29), f, f + 4,
                              begun || k >= per);
          ptx::tc_commit(empty + 8 * i);
          begun = true;
          i += kMxIss;
          if (i >= ST) {
            i -= ST;
            parity ^= 1u;
          }
        }
        ptx::tc_commit(acc_full + 8 * buf);
        begin = end;
      }
      // the products issued so far complete before the CTA's memory goes (bounded wait; after an abort too)
      ptx::tc_commit(ptx::smem_u32(&ctl->drain[me]));
      const uint64_t t0 = ptx::globaltimer_ns();
      while (!ptx::mbar_try_wait(ptx::smem_u32(&ctl->drain[me]), 0) && ptx::globaltimer_ns() - t0 < kWaitLimitNs / 10) {
      }
    }
    __syncwarp();
  } else if (warp < 1 + kMxIss + kMxEpi) {
    // ---- sums out of tensor memory: a warp may read the 32 rows of its index modulo four
    const int quarter = warp & 3, r = 32 * quarter + lane, tid = threadIdx.x - 32 * (1 + kMxIss);
    ptx::wait_prior_grid();  // the counters are zero from here on
    float* const parts = reinterpret_cast<float*>(a.ws + space.parts);
    const int64_t plane = (int64_t)sh.tokens * kRows;
    int seg = 0;
    for (int64_t u = u0; u < u1; ++seg) {
      const int64_t t = u / sh.stages, first = t * sh.stages, end = min(u1, first + sh.stages);
      const int buf = seg & 1;
      // fewer units than issuing threads: the others' sums hold nothing of this tile
      const int units = (int)min((int64_t)kMxIss, end - u), from = (int)((u - u0) % kMxIss);
      const bool whole = end - u == sh.stages;
      const int64_t n = t / sh.tiles * kRows + r, m0 = t % sh.tiles * sh.tokens;
      const int tokens = (int)min((int64_t)sh.tokens, a.M - m0);
      // slot 0: the run's first tile, slot 1: its last one
      float* const part = parts + (2 * (int64_t)blockIdx.x + (u == u0 ? 0 : 1)) * plane + r;
      // after an abort the warps still go through the barriers below together, moving nothing
      const bool ok = wait_bar_warp<true>(acc_full + 8 * buf, (uint32_t)(seg / 2) & 1, &ctl->abort);
      ptx::tc_fence_after();
      auto store = [&](int m, float v) {
        if (n >= a.N) return;
        const int64_t o = (m0 + m) * a.ld_y + n;
        if (a.y_f32)
          put_at(static_cast<float*>(a.y) + o, v, a.y, a.y_bytes);
        else
          put_at(static_cast<uint16_t*>(a.y) + o, (uint16_t)bf16x2(v, 0.0f), a.y, a.y_bytes);
      };
      const uint32_t src = tmem + ((uint32_t)(32 * quarter) << 16) + buf * kMxBuf;
      for (int m = 0; ok && m < tokens; m += 16) {
        float f[16] = {};
        for (int q = 0; q < units * per; ++q) {
          const int j = (from * per + q) % (kMxIss * per);
          if (sh.digits == 1) {
            uint32_t v[16];
            ptx::tmem_ld_32x32b_x16(src + j * sh.n + m, v);
            ptx::tc_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) f[e] = __fadd_rn(f[e], __uint_as_float(v[e]));
          } else {
            // 16 tokens' digits, three to each
            uint32_t v[3][16];
#pragma unroll
            for (int d = 0; d < 3; ++d) ptx::tmem_ld_32x32b_x16(src + j * sh.n + 3 * m + 16 * d, v[d]);
            ptx::tc_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float a0 = __uint_as_float(v[3 * e / 16][3 * e % 16]);
              const float a1 = __uint_as_float(v[(3 * e + 1) / 16][(3 * e + 1) % 16]);
              const float a2 = __uint_as_float(v[(3 * e + 2) / 16][(3 * e + 2) % 16]);
              f[e] = __fadd_rn(f[e], __fadd_rn(a0, __fadd_rn(a1, a2)));
            }
          }
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          if (m + e >= tokens) break;
          if (whole)
            store(m + e, f[e]);
          else
            put_at(part + (m + e) * kRows, f[e], a.ws, a.ws_bytes);
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(acc_empty + 8 * buf);
      if (!whole) {
        // the tile's CTAs are those that have its first and its last unit, and all between
        const int64_t c0 = ((first + 1) * sh.ctas - 1) / sh.units, c1 = ((first + sh.stages) * sh.ctas - 1) / sh.units;
        __threadfence();
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (tid == 0)
          ctl->last = ok && atomicAdd(reinterpret_cast<uint32_t*>(a.ws + space.counters) + t, 1u) == (uint32_t)(c1 - c0);
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (ok && *reinterpret_cast<volatile uint32_t*>(&ctl->last)) {
          __threadfence();
          // sixteen tokens' loads of a part in flight together
          for (int m = 0; m < tokens; m += 16) {
            float v[16] = {};
            for (int64_t c = c0; c <= c1; ++c) {
              const int slot = sh.units * c / sh.ctas >= first ? 0 : 1;
              const float* from = parts + (2 * c + slot) * plane + m * kRows + r;
              float w[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e] = m + e < tokens ? __ldcg(from + e * kRows) : 0.0f;
#pragma unroll
              for (int e = 0; e < 16; ++e) v[e] = __fadd_rn(v[e], w[e]);
            }
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (m + e < tokens) store(m + e, v[e]);
          }
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");  // ctl->last is read before the next tile writes it
      }
      u = end;
    }
  } else if (!a.mma) {
    // ---- row-major weight scales into tiles, whole stages in turn: lane l brings rows l, l + 32, l + 64, l + 96
    const int64_t nkb = a.K >> 5;  // a multiple of four: words
    int64_t t = -1, begin = 0, end = 0;  // the tile at hand and its units
    const uint32_t* row[4];
    for (int64_t u = u0 + warp - 1 - kMxIss - kMxEpi; u < u1; u += kMxConv) {
      if (u >= end) {
        t = u / sh.stages;
        begin = t * sh.stages;
        end = begin + sh.stages;
        const int64_t n0 = t / sh.tiles * kRows;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          row[j] = reinterpret_cast<const uint32_t*>(a.sw + min(n0 + lane + 32 * j, a.N - 1) * nkb);
      }
      const int c = (int)(u - u0), i = c % ST;
      uint32_t v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = __ldg(row[j] + (u - begin));
      if (c >= ST && !wait_bar_warp<true>(empty + 8 * i, (uint32_t)(c / ST - 1) & 1, &ctl->abort)) break;
      *reinterpret_cast<uint4*>(sfa + i * kMxTile + lane * 16) = make_uint4(v[0], v[1], v[2], v[3]);
      ptx::fence_proxy_async();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(full + 8 * i);
    }
  }
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kMxTmem);
  }
}

template <typename... P, typename... Q>
cudaError_t launch_cluster(void (*kernel)(P...), dim3 grid, int threads, int bytes, int splits, bool under_prior,
                           cudaStream_t st, Q... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  unsigned n = 0;
  if (splits > 1) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = (unsigned)splits;
    at[n].val.clusterDim.y = 1;
    at[n++].val.clusterDim.z = 1;
  }
  if (under_prior) {
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = at;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Lets a kernel use `bytes` of dynamic shared memory and clusters above the
// portable size, once per device.
template <typename K>
cudaError_t allow_smem(K kernel, int bytes, bool (&set)[kMaxDevices]) {
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (set[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  set[dev] = e == cudaSuccess;
  return e;
}

bool codes_map(CUtensorMap* tm, const GemvArgs& a) {
  return make_tma_2d(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.qw, a.N, a.K / 2, a.K / 2, kRows, kRowBytes);
}

template <bool NV>
cudaError_t launch_few(const GemvArgs& a, int splits, cudaStream_t st) {
  constexpr int bytes = Smem<NV>::kBytes;
  static bool set[kMaxDevices] = {};
  if (cudaError_t e = allow_smem(gemv_kernel<NV>, bytes, set)) return e;
  CUtensorMap tm;
  if (!codes_map(&tm, a)) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)((a.N + kRows - 1) / kRows) * (unsigned)splits);
  return launch_cluster(gemv_kernel<NV>, grid, kThreads, bytes, splits, false, st, tm, a, splits);
}

template <bool NV, bool kF16>
cudaError_t launch_tc(const GemvArgs& a, int splits, cudaStream_t st) {
  constexpr int bytes = tc_smem<NV>();
  static bool set[kMaxDevices] = {};
  if (cudaError_t e = allow_smem(gemv_tc_kernel<NV, kF16>, bytes, set)) return e;
  CUtensorMap tm, tx;
  if (!codes_map(&tm, a)) return cudaErrorInvalidValue;
  const TcX x = tc_x(a);
  if (kF16) {
    if (!make_tma_2d(&tx, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, a.ws, (int64_t)x.tiles * x.n, a.K, a.K, x.n, kTcK))
      return cudaErrorInvalidValue;
    gemv_f16_rows_kernel<<<(unsigned)a.M, kF16Threads, 0, st>>>(a, x);
    if (cudaError_t e = cudaGetLastError()) return e;
  } else {
    tx = tm;  // not used
  }
  const dim3 grid((unsigned)((a.N + kRows - 1) / kRows) * (unsigned)splits,
                  (unsigned)((a.M + kTcTokens - 1) / kTcTokens));
  return launch_cluster(gemv_tc_kernel<NV, kF16>, grid, TcRoles<kF16>::kThreads, bytes, splits, kF16, st, tm, tx, a, x, splits);
}

template <int kN>
cudaError_t launch_mx(const GemvArgs& a, const MxShape& sh, cudaStream_t st) {
  static bool set[kMaxDevices] = {};
  if (cudaError_t e = allow_smem(gemv_mx_kernel<kN>, MxRing<kN>::kBytes, set)) return e;
  CUtensorMap tw, tx;
  if (!make_tma_4bit(&tw, a.qw, a.N, a.K, kRows) ||
      !make_tma_2d(&tx, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.ws, (int64_t)sh.tiles * sh.n, a.K, a.K, sh.n, kMxK))
    return cudaErrorInvalidValue;
  gemv_digits_kernel<<<dim3((unsigned)((a.K / 32 + 63) / 64), (unsigned)a.M), 256, 0, st>>>(a, sh);
  if (cudaError_t e = cudaGetLastError()) return e;
  return launch_cluster(gemv_mx_kernel<kN>, dim3((unsigned)sh.ctas), kMxThreads, MxRing<kN>::kBytes, 1, true, st, tw, tx,
                        a, sh);
}

cudaError_t launch_mx(const GemvArgs& a, cudaStream_t st) {
  const MxShape sh = mx_shape(a);
  return sh.n <= 32 ? launch_mx<32>(a, sh, st) : sh.n <= 64 ? launch_mx<64>(a, sh, st) : launch_mx<kMxN>(a, sh, st);
}

}  // namespace

namespace {

// Whether the MXFP8 products can take it: whole 128-deep steps of MXFP4 weights.
bool mx_fits(const GemvArgs& a) {
  return !a.nv && a.M > 0 && a.M <= 32768 && a.N > 0 && a.K >= kMxK && a.K % kMxK == 0 &&
         (reinterpret_cast<uintptr_t>(a.qw) & 31u) == 0;
}

// K is split over a cluster so that all CTAs (two an SM) end together: what counts is the rounds of CTAs
// times a CTA's stages and what it costs besides them, about six (64 tiles of 32 stages, 23 rows: 32 us in one
// slice, 19 in four, 24 in eight; 224 tiles: 50 us in one, 58 in three). Clusters above eight, the portable
// size, only where they leave an SM to each CTA: past that they wait for one another's places (16384 of K, 12
// rows: 256 of N 15.8 us in eight slices, 10.4 in sixteen; 4096 of K, one row: 2048 of N 5.6 and 8.9).
int k_splits(const GemvArgs& a, int tokens) {
  const int64_t tiles = (a.N + kRows - 1) / kRows * ((a.M + tokens - 1) / tokens), stages = (a.K + kStageK - 1) / kStageK;
  int splits = 1;
  int64_t best = INT64_MAX;
  for (int n = 1; n <= (tiles * n <= kSms ? kMostSplits : 8) && n <= stages; ++n) {
    const int64_t cost = (tiles * n + 2 * kSms - 1) / (2 * kSms) * ((stages + n - 1) / n + 6);
    if (cost < best) {
      best = cost;
      splits = n;
    }
  }
  return splits;
}

}  // namespace

int64_t gemv_workspace_bytes(const GemvArgs& a) {
  if (mx_fits(a)) return mx_space(mx_shape(a)).bytes;
  return a.nv && a.M > kTokens && a.N > 0 && a.K > 0 ? tc_x(a).bytes : 0;
}

cudaError_t launch_gemv(const GemvArgs& a, cudaStream_t st) {
  if (a.M == 0 || a.N == 0) return cudaSuccess;
  (void)cudaGetLastError();  // drop a stale error left by an earlier call
  if (a.K == 0) {
    const size_t es = a.y_f32 ? 4 : 2;
    return cudaMemset2DAsync(a.y, a.ld_y * es, 0, a.N * es, a.M, st);
  }
  const bool space = a.ws && a.ws_bytes >= (uint64_t)gemv_workspace_bytes(a);
  if (space && mx_fits(a)) return launch_mx(a, st);
  // One N of the products for up to eight rows of x (4096 x 4096: 7 us, 11 in tensor memory); from nine on the
  // weights are converted once for all of them (16 rows, 28672 x 8192: 58 us and 75; with the workspace 31).
  if (a.M <= kTokens) {
    const int splits = k_splits(a, kTokens);
    return a.nv ? launch_few<true>(a, splits, st) : launch_few<false>(a, splits, st);
  }
  const int splits = k_splits(a, kTcTokens);
  if (!a.nv) return launch_tc<false, false>(a, splits, st);
  return space ? launch_tc<true, true>(a, splits, st) : launch_tc<true, false>(a, splits, st);
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
