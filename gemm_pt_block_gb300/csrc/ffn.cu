// ffn.cu -- the operators around a feed-forward block's products (sm_103a):
// residual addition + root-mean-square norm + quantization, SwiGLU +
// quantization, and their gradients. All are bound by HBM traffic.
#include <cstdint>
#include <mutex>

#include "internal.h"
#include "mx_device.cuh"

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

// Sum over the CTA, the same bits in every thread (fixed order).
template <int kThreads>
__device__ __forceinline__ float block_sum(float v, float* part) {
  v = warp_sum(v);
  if (kThreads == 32) return v;
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) s = __fadd_rn(s, part[i]);
  __syncthreads();
  return s;
}

// ------------------------------------------------------------------ norm ---
// h = x + r, rounded to the stream's type T (what the next layer reads); the
// norm is taken of the rounded h, so that the backward pass, which reads it
// back, differentiates the same function:
//   y_i = (h_i w_i) rstd,   rstd = 1 / sqrt(sum h^2 / D + eps).
// bf16 products h_i w_i are exact in fp32, so y has two roundings. One CTA per
// row, two passes over it; the second reads h back (from x and r, out of L2).
constexpr int kRowThreads = 256;

template <typename T>
__device__ __forceinline__ void stream_of(const NormArgs& a, const T* x, const T* r, int64_t c, float (&h)[8],
                                          Vec8<T>& raw) {
  load8(x + c, raw);
  unpack8(raw, h);
  if (r) {
    float f[8];
    load8(r + c, raw);
    unpack8(raw, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = __fadd_rn(h[i], f[i]);
    pack8(h, raw);
    unpack8(raw, h);
  }
}

template <typename T, typename W>
__global__ void __launch_bounds__(kRowThreads) norm_rows_kernel(const NormArgs a) {
  __shared__ float part[kRowThreads / 32];
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.ld_x;
    const T* r = a.r ? static_cast<const T*>(a.r) + row * a.ld_r : nullptr;
    float sum = 0.0f, h[8];
    Vec8<T> raw;
    for (int64_t c = threadIdx.x * 8; c < a.cols; c += kRowThreads * 8) {
      stream_of(a, x, r, c, h, raw);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = __fmaf_rn(h[i], h[i], sum);
    }
    const float rstd = __frsqrt_rn(__fadd_rn(__fdiv_rn(block_sum<kRowThreads>(sum, part), (float)a.cols), a.eps));
    if (a.rstd && threadIdx.x == 0) put_at(a.rstd + row, rstd, a.rstd, a.rows * sizeof(float));
    for (int64_t c0 = 0; c0 < a.cols; c0 += kRowThreads * 8) {
      const int64_t c = c0 + threadIdx.x * 8;
      const bool live = c < a.cols;
      float f[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (live) {
        stream_of(a, x, r, c, h, raw);
        if (a.h) store8(static_cast<T*>(a.h) + row * a.ld_h + c, raw, a.h, a.h_bytes);
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
      if (a.quant.fmt != RowQuant::kNone) quantize8(a.quant, f, live, row, c, a.cols);
    }
  }
}

// Gradients. With n = h rstd and dn = dy w:
//   dx = (dn - n mean(dn n)) rstd + dh,   dw = sum over rows of dy n
// (dh: what reaches h past the norm, through the residual stream).
template <typename T, typename G, typename W>
__global__ void __launch_bounds__(kRowThreads) norm_dx_kernel(const NormGradArgs a) {
  __shared__ float part[kRowThreads / 32];
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* hp = static_cast<const T*>(a.h) + row * a.ld_h;
    const G* dp = static_cast<const G*>(a.dy) + row * a.ld_dy;
    const float rstd = a.rstd[row];
    float h[8], d[8], w[8], sum = 0.0f;
    for (int pass = 0; pass < 2; ++pass) {
      const float mean = pass ? __fdiv_rn(block_sum<kRowThreads>(sum, part), (float)a.cols) : 0.0f;
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
}

// dw: every CTA row slice (blockIdx.y) sums its rows into one row of the
// workspace, in order; the sum over slices follows in the next kernel, so dw
// has the same bits on every call.
template <typename T, typename G>
__global__ void __launch_bounds__(kRowThreads) norm_dw_kernel(const NormGradArgs a) {
  const int64_t c = ((int64_t)blockIdx.x * kRowThreads + threadIdx.x) * 8;
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

template <typename W>
__global__ void __launch_bounds__(kRowThreads) norm_dw_sum_kernel(const float* __restrict__ ws, int slices,
                                                                  int64_t cols, W* dw) {
  const int64_t c = (int64_t)blockIdx.x * kRowThreads + threadIdx.x;
  if (c >= cols) return;
  float s = 0.0f;
  for (int i = 0; i < slices; ++i) s = __fadd_rn(s, ws[i * cols + c]);
  if (sizeof(W) == 4)
    put_at(dw + c, s, dw, cols * sizeof(W));
  else
    put_at(dw + c, (uint16_t)bf16x2(s, 0.0f), dw, cols * sizeof(W));
}

// ---------------------------------------------------------------- SwiGLU ---
// a = silu(g) u with silu(g) = g / (1 + e^-g). Each thread takes eight
// elements of a row.
constexpr int kActThreads = 256;

// 1 / (1 + e^-g) as t / (1 + t) or 1 / (1 + t) with t = e^-|g| <= 1: nothing
// overflows, and the quotient's denominator lies in [1, 2], where the fast
// division is within 2 ulp.
__device__ __forceinline__ float sigmoid(float g) {
  const float t = expf(-fabsf(g));
  return __fdividef(g < 0.0f ? t : 1.0f, __fadd_rn(1.0f, t));
}

template <typename T>
__global__ void __launch_bounds__(kActThreads) swiglu_kernel(const SwigluArgs a) {
  const int64_t vecs = a.cols >> 3, total = a.rows * vecs;
  for (int64_t v0 = (int64_t)blockIdx.x * kActThreads; v0 < total; v0 += (int64_t)gridDim.x * kActThreads) {
    const int64_t v = v0 + threadIdx.x;
    const bool live = v < total;
    const int64_t row = live ? v / vecs : 0, c = live ? (v - row * vecs) * 8 : 0;
    float g[8] = {0, 0, 0, 0, 0, 0, 0, 0}, u[8];
    if (live) {
      Vec8<T> gv, uv;
      load8(static_cast<const T*>(a.g) + row * a.ld_g + c, gv);
      load8(static_cast<const T*>(a.u) + row * a.ld_u + c, uv);
      unpack8(gv, g);
      unpack8(uv, u);
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = __fmul_rn(__fmul_rn(g[i], sigmoid(g[i])), u[i]);
      if (a.y) store8_as(a.y, a.y_f32, row * a.ld_y + c, g, a.y_bytes);
    }
    if (a.quant.fmt != RowQuant::kNone) quantize8(a.quant, g, live, row, c, a.cols);
  }
}

// With s = 1 / (1 + e^-g): dg = dy u s (1 + g (1 - s)), du = dy g s.
template <typename T, typename G>
__global__ void __launch_bounds__(kActThreads) swiglu_grad_kernel(const SwigluGradArgs a) {
  const int64_t vecs = a.cols >> 3, total = a.rows * vecs;
  for (int64_t v = (int64_t)blockIdx.x * kActThreads + threadIdx.x; v < total;
       v += (int64_t)gridDim.x * kActThreads) {
    const int64_t row = v / vecs, c = (v - row * vecs) * 8;
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
    for (int i = 0; i < 8; ++i) {
      const float s = sigmoid(g[i]);
      const float ds = __fmul_rn(d[i], s);
      u[i] = __fmul_rn(__fmul_rn(ds, u[i]), __fmaf_rn(g[i], 1.0f - s, 1.0f));
      d[i] = __fmul_rn(ds, g[i]);
    }
    pack8(u, gv);
    pack8(d, uv);
    store8(static_cast<T*>(a.dg) + row * a.ld_dg + c, gv, a.dg, a.dg_bytes);
    store8(static_cast<T*>(a.du) + row * a.ld_du + c, uv, a.du, a.du_bytes);
  }
}

unsigned grid_for(int64_t items) { return (unsigned)(items < (1 << 20) ? items : (1 << 20)); }

}  // namespace

int norm_dw_slices(int64_t rows) { return (int)(rows < 256 ? rows : 256); }

cudaError_t launch_rmsnorm(const NormArgs& a, bool x_f32, bool w_f32, cudaStream_t st) {
  if (a.rows == 0 || a.cols == 0) return cudaSuccess;
  (void)cudaGetLastError();  // drop a stale error left by an earlier call
  const unsigned grid = grid_for(a.rows);
  if (x_f32 && w_f32)
    norm_rows_kernel<float, float><<<grid, kRowThreads, 0, st>>>(a);
  else if (x_f32)
    norm_rows_kernel<float, uint16_t><<<grid, kRowThreads, 0, st>>>(a);
  else if (w_f32)
    norm_rows_kernel<uint16_t, float><<<grid, kRowThreads, 0, st>>>(a);
  else
    norm_rows_kernel<uint16_t, uint16_t><<<grid, kRowThreads, 0, st>>>(a);
  return cudaGetLastError();
}

namespace {
template <typename T, typename G, typename W>
void norm_grad(const NormGradArgs& a, cudaStream_t st) {
  if (a.rows > 0) norm_dx_kernel<T, G, W><<<grid_for(a.rows), kRowThreads, 0, st>>>(a);
  if (!a.dw) return;
  const int slices = norm_dw_slices(a.rows);
  if (slices)
    norm_dw_kernel<T, G><<<dim3((unsigned)((a.cols / 8 + kRowThreads - 1) / kRowThreads), slices), kRowThreads, 0,
                           st>>>(a);
  norm_dw_sum_kernel<W><<<(unsigned)((a.cols + kRowThreads - 1) / kRowThreads), kRowThreads, 0, st>>>(
      a.ws, slices, a.cols, static_cast<W*>(a.dw));
}
}  // namespace

cudaError_t launch_rmsnorm_grad(const NormGradArgs& a, bool h_f32, bool dy_f32, bool w_f32, cudaStream_t st) {
  if (a.cols == 0) return cudaSuccess;
  (void)cudaGetLastError();
  using B = uint16_t;
  switch ((h_f32 ? 4 : 0) | (dy_f32 ? 2 : 0) | (w_f32 ? 1 : 0)) {
    case 0: norm_grad<B, B, B>(a, st); break;
    case 1: norm_grad<B, B, float>(a, st); break;
    case 2: norm_grad<B, float, B>(a, st); break;
    case 3: norm_grad<B, float, float>(a, st); break;
    case 4: norm_grad<float, B, B>(a, st); break;
    case 5: norm_grad<float, B, float>(a, st); break;
    case 6: norm_grad<float, float, B>(a, st); break;
    default: norm_grad<float, float, float>(a, st);
  }
  return cudaGetLastError();
}

cudaError_t launch_swiglu(const SwigluArgs& a, bool f32, cudaStream_t st) {
  if (a.rows == 0 || a.cols == 0) return cudaSuccess;
  (void)cudaGetLastError();
  const unsigned grid = grid_for((a.rows * (a.cols / 8) + kActThreads - 1) / kActThreads);
  if (f32)
    swiglu_kernel<float><<<grid, kActThreads, 0, st>>>(a);
  else
    swiglu_kernel<uint16_t><<<grid, kActThreads, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_swiglu_grad(const SwigluGradArgs& a, bool f32, bool dy_f32, cudaStream_t st) {
  if (a.rows == 0 || a.cols == 0) return cudaSuccess;
  (void)cudaGetLastError();
  const unsigned grid = grid_for((a.rows * (a.cols / 8) + kActThreads - 1) / kActThreads);
  if (f32 && dy_f32)
    swiglu_grad_kernel<float, float><<<grid, kActThreads, 0, st>>>(a);
  else if (f32)
    swiglu_grad_kernel<float, uint16_t><<<grid, kActThreads, 0, st>>>(a);
  else if (dy_f32)
    swiglu_grad_kernel<uint16_t, float><<<grid, kActThreads, 0, st>>>(a);
  else
    swiglu_grad_kernel<uint16_t, uint16_t><<<grid, kActThreads, 0, st>>>(a);
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
