// gemv.cu -- products of a few activation rows with a 4-bit weight matrix
// (sm_103a): the single-token form of the block-scaled GEMM.
//   y[m, n] = sum_k x[m, k] W[n, k]
// The weights' codes and scales are read once (per tile of rows of x); at
// these sizes they are all of the traffic.
#include <cstdint>
#include <cuda_fp16.h>

#include "internal.h"
#include "mx_device.cuh"

namespace mx {
namespace {
__device__ uint32_t g_gemv_error;
}  // namespace
}  // namespace mx
#define MX_BOUNDS_FAIL() atomicExch(&::mx::g_gemv_error, ::mx::kErrBounds)

#include "row_device.cuh"

namespace mx {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 4;

__device__ __forceinline__ float e8m0_value(uint32_t b) {
  return b == 255u ? __uint_as_float(0x7FC00000u) : b ? __uint_as_float(b << 23) : __uint_as_float(0x00400000u);
}

// Two E4M3 codes (low 16 bits) to f16, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {
  uint32_t r;
  asm("{.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;}" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t e5m2x2_to_f16x2(uint32_t v) {
  uint32_t r;
  asm("{.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e5m2x2 %0, t;}" : "=r"(r) : "r"(v));
  return r;
}

// One warp per output column n; each lane takes whole 32-blocks of K.
__global__ void __launch_bounds__(kThreads) gemv_kernel(const GemvArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t n = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (n >= a.N) return;
  const int64_t nkb = a.K >> 5, m0 = (int64_t)blockIdx.y * kTokens;
  const int tokens = (int)min((int64_t)kTokens, a.M - m0);
  float acc[kTokens] = {0, 0, 0, 0};
  for (int64_t kb = lane; kb < nkb; kb += 32) {
    const uint4 q = load16(a.qw + n * (a.K >> 1) + kb * 16);
    const uint32_t words[4] = {q.x, q.y, q.z, q.w};
    float w[32];
    float s0, s1;
    if (a.nv) {
      const int64_t b0 = 2 * kb, nb = a.K >> 4;
      const uint8_t c0 = a.sw[a.mma ? mma_scale_offset(n, b0, nb) : n * nb + b0];
      const uint8_t c1 = a.sw[a.mma ? mma_scale_offset(n, b0 + 1, nb) : n * nb + b0 + 1];
      const uint32_t h = e4m3x2_to_f16x2(c0 | ((uint32_t)c1 << 8));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      s0 = f.x * a.p2k;
      s1 = f.y * a.p2k;
    } else {
      s0 = s1 = e8m0_value(a.sw[a.mma ? mma_scale_offset(n, kb, nkb) : n * nkb + kb]);
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const uint32_t c = words[i >> 3] >> (4 * (i & 7));
      const float v = e2m1_magnitude(c & 7u) * (i < 16 ? s0 : s1);
      w[i] = (c & 8u) ? -v : v;
    }
    for (int t = 0; t < tokens; ++t) {
      const int64_t at = (m0 + t) * a.ld_x + kb * 32;
      float x[32];
      if (a.x_kind == GemvArgs::kXBf16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          Vec8<uint16_t> v;
          float f[8];
          load8_cached(static_cast<const uint16_t*>(a.x) + at + 8 * i, v);
          unpack8(v, f);
#pragma unroll
          for (int j = 0; j < 8; ++j) x[8 * i + j] = f[j];
        }
      } else {
        const float sx = e8m0_value(a.sx[(m0 + t) * nkb + kb]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.x) + at) + i);
          const uint32_t c[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t p = (c[j >> 1] >> (16 * (j & 1))) & 0xFFFFu;
            const uint32_t h = a.x_kind == GemvArgs::kXE4m3 ? e4m3x2_to_f16x2(p) : e5m2x2_to_f16x2(p);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
            x[16 * i + 2 * j] = f.x * sx;
            x[16 * i + 2 * j + 1] = f.y * sx;
          }
        }
      }
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < 32; ++i) s = __fmaf_rn(x[i], w[i], s);
#pragma unroll
      for (int u = 0; u < kTokens; ++u)
        if (u == t) acc[u] += s;
    }
  }
#pragma unroll
  for (int t = 0; t < kTokens; ++t) {
    float s = acc[t];
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    if (lane == 0 && t < tokens) {
      if (a.y_f32)
        put_at(static_cast<float*>(a.y) + (m0 + t) * a.ld_y + n, s, a.y, a.y_bytes);
      else
        put_at(static_cast<uint16_t*>(a.y) + (m0 + t) * a.ld_y + n, (uint16_t)bf16x2(s, 0.0f), a.y, a.y_bytes);
    }
  }
}

}  // namespace

cudaError_t launch_gemv(const GemvArgs& a, cudaStream_t st) {
  if (a.M == 0 || a.N == 0) return cudaSuccess;
  (void)cudaGetLastError();  // drop a stale error left by an earlier call
  const dim3 grid((unsigned)((a.N + kThreads / 32 - 1) / (kThreads / 32)), (unsigned)((a.M + kTokens - 1) / kTokens));
  gemv_kernel<<<grid, kThreads, 0, st>>>(a);
  return cudaGetLastError();
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
