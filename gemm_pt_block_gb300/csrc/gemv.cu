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

constexpr int kRows = 128;                 // most rows of W per CTA
constexpr int kStageK = 256;               // K per stage
constexpr int kBlocks = kStageK / 32;
constexpr int kRowBytes = kStageK / 2;     // code bytes per row and stage
constexpr int kParts = 2;                  // parts of a stage's blocks, each a warp's
constexpr int kMmaWarps = 8;               // (up to four) groups of 32 rows x kParts
constexpr int kConvWarps = 4;
constexpr int kThreads = (kMmaWarps + 1 + kConvWarps) * 32;
constexpr int kWBytes = kRows * kRowBytes;
constexpr int kMaxTokens = 32;
constexpr int kSms = 152;
constexpr uint64_t kWaitLimitNs = 2000000000ull;

// Shared memory of one CTA for tiles of TT rows of x.
template <int TT, bool NV>
struct Smem {
  static constexpr int kX = TT * kStageK * 2;            // f16 [block][token][32]
  static constexpr int kSw = 2 * kRows * kStageK / (NV ? 16 : 32);  // two 128-row tiles of scales
  static constexpr int kSx = TT * (kStageK / 32) * 4;    // float [block][token]
  static constexpr int kStage = kWBytes + kX + kSw + kSx;
  static constexpr int kStages = TT == 32 ? 5 : TT == 16 ? 4 : NV ? 4 : 5;
  static constexpr int kCtl = 256;
  static constexpr int kBytes = kStages * kStage + kCtl + 1024;
  // partial sums [part][token][rows + 4] in place of the W stages
  static_assert(kParts * (kRows + 4) * TT * 4 <= kStages * kWBytes, "partial sums fit the ring");
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

// One stage of x rows m0 .. m0 + tokens - 1, K from k0: lane 4 b + t brings
// elements 8 t .. 8 t + 7 of block b, a row at a time.
template <int TT>
__device__ __forceinline__ void convert_x(const GemvArgs& a, int64_t m0, int tokens, int64_t k0, int lane,
                                          uint8_t* xs, float* sxs) {
  const int b = lane >> 2, t = lane & 3;
  const int64_t k = k0 + b * 32 + t * 8;
  const bool live = k < a.K;
  uint8_t* dst = xs + b * (TT * 64) + t * 16;
  float* sdst = sxs + b * TT;
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
        *reinterpret_cast<uint4*>(dst + (m + i) * 64) = make_uint4(h[0], h[1], h[2], h[3]);
        if (t == 0) sdst[m + i] = E == 14u ? __uint_as_float(0x00400000u) : __uint_as_float((E - 14u) << 23);
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
        *reinterpret_cast<uint4*>(dst + (m + i) * 64) = h;
        if (t == 0) sdst[m + i] = __uint_as_float(e8m0x2_bf16x2(s[i]) << 16);
      }
    }
  }
}

// One stage of row-major weight scales, rearranged into the tensor-core tiles
// (128 rows x 4 columns, 512 bytes) that the multiplying warps read: lane l
// brings rows l, l + 32, l + 64, l + 96. Rows past N repeat the last one.
template <bool NV>
__device__ __forceinline__ void convert_sw(const GemvArgs& a, int groups, int64_t n0, int64_t k0, int lane,
                                           uint8_t* sws) {
  constexpr int kCols = kStageK / (NV ? 16 : 32);
  const int64_t cols = a.K / (NV ? 16 : 32), c0 = k0 / (NV ? 16 : 32);
  uint32_t v[kCols / 4][4] = {};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (j >= groups) break;
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
  for (int c = 0; c < kCols / 4; ++c)
    *reinterpret_cast<uint4*>(sws + c * 512 + lane * 16) = make_uint4(v[c][0], v[c][1], v[c][2], v[c][3]);
}

template <int NT, bool NV>
__global__ void __launch_bounds__(kThreads, NT == 4 ? 1 : 2)
gemv_kernel(const __grid_constant__ CUtensorMap tm, const GemvArgs a, const int groups, const int splits) {
  constexpr int TT = 8 * NT;
  using S = Smem<TT, NV>;
  constexpr int ST = S::kStages;
  constexpr int kPer = NV ? 16 : 32;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const base = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t *const ws = base, *const xs = ws + ST * kWBytes, *const sws = xs + ST * S::kX;
  float* const sxs = reinterpret_cast<float*>(sws + ST * S::kSw);
  Ctl* const ctl = reinterpret_cast<Ctl*>(sws + ST * (S::kSw + S::kSx));
  const uint32_t full_w = ptx::smem_u32(ctl->full_w), full_x = ptx::smem_u32(ctl->full_x),
                 empty = ptx::smem_u32(ctl->empty);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int mma_warps = groups * kParts, rows = 32 * groups;
  const int rank = (int)(blockIdx.x % (unsigned)splits);
  const int64_t n0 = (int64_t)(blockIdx.x / (unsigned)splits) * rows, m0 = (int64_t)blockIdx.y * kMaxTokens;
  const int tokens = (int)min((int64_t)TT, a.M - m0);
  const int stages = (int)((a.K + kStageK - 1) / kStageK);
  const int s0 = (int)((int64_t)stages * rank / splits), s1 = (int)((int64_t)stages * (rank + 1) / splits);

  if (threadIdx.x == 0) {
    ptx::prefetch_tensormap(&tm);
    for (int i = 0; i < ST; ++i) {
      ptx::mbar_init(full_w + 8 * i, 1);
      ptx::mbar_init(full_x + 8 * i, 1);
      ptx::mbar_init(empty + 8 * i, mma_warps);
    }
    ctl->abort = 0;
    ptx::fence_mbar_init();
  }
  __syncthreads();

  float2 acc[2][NT][2];
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[r][n][0] = acc[r][n][1] = make_float2(0.0f, 0.0f);
  const int g = lane >> 2, t = lane & 3, part = warp / groups, wr = warp - part * groups;

  if (warp == kMmaWarps) {
    // ---- producer: codes by TMA, tensor-core scales as they lie in memory
    if (lane == 0) {
      const int64_t cols = a.K / kPer, tile0 = n0 >> 7, tiles = ((n0 + rows - 1) >> 7) - tile0 + 1;
      const int64_t last = (a.N >> 7) - 1;               // the scale array's last row tile
      int i = 0, s = s0;
      uint32_t round = 0;
      for (; s < s1; ++s) {
        if (round && !wait_bar(empty + 8 * i, (round - 1) & 1, ctl)) break;
        uint32_t bytes = (uint32_t)rows * kRowBytes, sb = 0;
        const int64_t c0 = (int64_t)s * (kStageK / kPer);
        if (a.mma) {
          sb = (uint32_t)min((int64_t)(S::kSw / 2), (cols - c0) * kRows);
          bytes += sb * (uint32_t)tiles;
        }
        ptx::mbar_arrive_expect_tx(full_w + 8 * i, bytes);
        ptx::tma_load_2d(ptx::smem_u32(ws + i * kWBytes), &tm, s * kRowBytes, (int32_t)n0, full_w + 8 * i);
        if (a.mma)
          for (int64_t j = 0; j < tiles; ++j)
            ptx::bulk_load(ptx::smem_u32(sws + i * S::kSw + j * (S::kSw / 2)),
                           a.sw + min(tile0 + j, last) * 128 * cols + c0 * kRows, sb, full_w + 8 * i);
        if (++i == ST) {
          i = 0;
          ++round;
        }
      }
      // after an abort: the last load into each slot lands (bounded wait) before the CTA's memory goes
      if (*reinterpret_cast<volatile uint32_t*>(&ctl->abort)) {
        const int issued = s - s0;
        for (int r = issued > ST ? issued - ST : 0; r < issued; ++r) {
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
    for (int s = s0 + (warp - kMmaWarps - 1); s < s1; s += kConvWarps) {
      const int i = (s - s0) % ST;
      const uint32_t round = (uint32_t)((s - s0) / ST);
      if (round && !wait_bar(empty + 8 * i, (round - 1) & 1, ctl)) break;
      const int64_t k0 = (int64_t)s * kStageK;
      if (!a.mma) convert_sw<NV>(a, groups, n0, k0, lane, sws + i * S::kSw);
      convert_x<TT>(a, m0, tokens, k0, lane, xs + i * S::kX, sxs + i * (S::kSx / 4));
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(full_x + 8 * i);
    }
  } else if (warp < mma_warps) {
    // ---- multiplying warps: rows 32 wr .. 32 wr + 31, 32-blocks 4 part .. 4 part + 3 of every stage.
    // Blocks past K need no case of their own: their codes (TMA's fill), their x and its factor are
    // finite (zeros), and their scales are taken as zero bytes.
    uint32_t chunk[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) chunk[b] = (uint32_t)(((4 * part + b) ^ g) << 4) + 4 * t + (32 * wr + g) * kRowBytes;
    // where this warp's 32 rows stand among the 128-row tiles of scales
    const int64_t nw = n0 + 32 * wr;
    const uint32_t tile = a.mma ? (uint32_t)((nw >> 7) - (n0 >> 7)) : 0u, quarter = a.mma ? (uint32_t)(nw >> 5) & 3u : wr;
    const uint32_t swoff = tile * (S::kSw / 2) + part * (NV ? 1024 : 512) + g * 16 + quarter * 4;
    const uint32_t xoff = 4 * part * (TT * 64) + g * 64 + t * 16, sxoff = 4 * part * TT + 2 * t;
    int i = 0;
    uint32_t parity = 0;
    for (int s = s0; s < s1; ++s) {
      if (!wait_bar(full_w + 8 * i, parity, ctl) || !wait_bar(full_x + 8 * i, parity, ctl)) break;
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
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint4 v = *reinterpret_cast<const uint4*>(x + b * (TT * 64) + n * 512);
          const float2 fx = *reinterpret_cast<const float2*>(sx + b * TT + n * 8);
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            mma16816(c, q[2 * r][0], q[2 * r + 1][0], q[2 * r][1], q[2 * r + 1][1], v.x, v.y);
            mma16816(c, q[2 * r][2], q[2 * r + 1][2], q[2 * r][3], q[2 * r + 1][3], v.z, v.w);
            const float2 p0 = NV ? fx : f2mul(fx, make_float2(f[2 * r], f[2 * r]));
            const float2 p1 = NV ? fx : f2mul(fx, make_float2(f[2 * r + 1], f[2 * r + 1]));
            acc[r][n][0] = f2fma(make_float2(c[0], c[1]), p0, acc[r][n][0]);
            acc[r][n][1] = f2fma(make_float2(c[2], c[3]), p1, acc[r][n][1]);
          }
        }
      }
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
  const int ld = rows + 4, plane = TT * ld;
  if (ok && warp < mma_warps) {
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float* d = red + part * plane + (8 * n + 2 * t) * ld + 32 * wr + 16 * r + 8 * c + g;
          d[0] = acc[r][n][c].x;
          d[ld] = acc[r][n][c].y;
        }
  }
  __syncthreads();
  const int total = tokens * rows;
  if (splits > 1) {
    if (ok)
      for (int e = threadIdx.x; e < total; e += kThreads) {
        float* d = red + e / rows * ld + e % rows;
        *d = __fadd_rn(d[0], d[plane]);
      }
    __syncwarp();
    ptx::cluster_sync();
  }
  if (ok) {
    for (int e = total * rank / splits + threadIdx.x; e < total * (rank + 1) / splits; e += kThreads) {
      const int m = e / rows, r = e % rows;
      const int64_t n = n0 + r;
      if (n >= a.N) continue;
      const float* d = red + m * ld + r;
      float v = 0.0f;
      if (splits == 1) {
        v = __fadd_rn(d[0], d[plane]);
      } else {
        const uint32_t at = ptx::smem_u32(d);
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
cudaError_t launch(const GemvArgs& a, int groups, int splits, cudaStream_t st) {
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
  CUtensorMap tm;
  if (!make_tma_2d(&tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.qw, a.N, a.K / 2, a.K / 2, 32 * groups, kRowBytes))
    return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.N + 32 * groups - 1) / (32 * groups)) * (unsigned)splits,
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
  cfg.numAttrs = splits > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, gemv_kernel<NT, NV>, tm, a, groups, splits);
}

}  // namespace

cudaError_t launch_gemv(const GemvArgs& a, cudaStream_t st) {
  if (a.M == 0 || a.N == 0) return cudaSuccess;
  (void)cudaGetLastError();  // drop a stale error left by an earlier call
  if (a.K == 0) {
    const size_t es = a.y_f32 ? 4 : 2;
    return cudaMemset2DAsync(a.y, a.ld_y * es, 0, a.N * es, a.M, st);
  }
  const int nt = a.M <= 8 ? 1 : a.M <= 16 ? 2 : 4;
  // K is split until two thirds of the SMs have a CTA (a CTA alone on its SM is
  // bound by its own latency), and on to three CTAs an SM where each keeps 16
  // stages to itself (shorter ones lose more to filling and emptying the ring).
  const int64_t tiles = (a.N + kRows - 1) / kRows * ((a.M + kMaxTokens - 1) / kMaxTokens);
  const int64_t stages = (a.K + kStageK - 1) / kStageK;
  int groups = 4, splits = 1;
  while (splits < 8 && ((3 * tiles * splits < 2 * kSms && 2 * splits <= stages) ||
                        (2 * tiles * splits <= 3 * kSms && 32 * splits <= stages)))
    splits *= 2;
#ifdef GEMV_TUNE
  if (getenv("GEMV_R")) groups = atoi(getenv("GEMV_R"));
  if (getenv("GEMV_S")) splits = atoi(getenv("GEMV_S"));
#endif
  if (a.nv)
    return nt == 1 ? launch<1, true>(a, groups, splits, st)
                   : nt == 2 ? launch<2, true>(a, groups, splits, st) : launch<4, true>(a, groups, splits, st);
  return nt == 1 ? launch<1, false>(a, groups, splits, st)
                 : nt == 2 ? launch<2, false>(a, groups, splits, st) : launch<4, false>(a, groups, splits, st);
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
