// api.cu -- the extern "C" entry points declared in include/mxfp4.h:
// argument validation, status codes and the thread-local error detail; the
// work itself is enqueued by the launchers in quant.cu, gemm.cu, ffn.cu, gemv.cu and cache.cu.
#include <cstdarg>
#include <cstdint>
#include <cmath>
#include <cstdio>

#include "../../include/mxfp4.h"
#include "internal.h"

namespace {

thread_local char g_last_error[512] = "";
// Bounds-checking builds: bytes taken off every output extent this thread's
// later calls check against (mxfp4_bounds_check_shrink).
thread_local int64_t g_extent_shrink = 0;

mxfp4_status fail(mxfp4_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
  va_end(ap);
  return s;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

mxfp4_status from_cuda(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return MXFP4_OK;
  return fail(MXFP4_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// Validates one orientation's parameters and fills the launcher's view.
mxfp4_status check_params(const mxfp4_quant_params* p, uint8_t* q, uint8_t* s, int64_t out_rows,
                          int64_t k, const char* name, mx::OrientArgs* o) {
  if ((!q || !s) && out_rows * k > 0)
    return fail(MXFP4_ERR_INVALID_ARG, "%s: output pointers must be non-NULL", name);
  if (!aligned16(q)) return fail(MXFP4_ERR_ALIGN, "%s: codes pointer not 16-byte aligned", name);
  if (p->block != MXFP4_BLOCK_1X32 && p->block != MXFP4_BLOCK_32X32 &&
      p->block != MXFP4_BLOCK_64X64 && p->block != MXFP4_BLOCK_1X16)
    return fail(MXFP4_ERR_INVALID_ARG, "%s: bad block %d", name, p->block);
  const bool nv = p->block == MXFP4_BLOCK_1X16;
  if (nv && (p->tensor_exp < -100 || p->tensor_exp > 100))
    return fail(MXFP4_ERR_INVALID_ARG, "%s: tensor_exp %d outside [-100, 100]", name, p->tensor_exp);
  if (!nv && p->tensor_exp != 0)
    return fail(MXFP4_ERR_INVALID_ARG, "%s: tensor_exp is for 1x16 (NVFP4) blocks only", name);
  if (nv && p->elem_format != MXFP4_FORMAT_E2M1)
    return fail(MXFP4_ERR_UNSUPPORTED, "%s: 1x16 blocks take E2M1 elements", name);
  if (p->block == MXFP4_BLOCK_64X64 && (out_rows % 64 != 0 || k % 64 != 0))
    return fail(MXFP4_ERR_SHAPE, "%s: 64x64 blocks need rows %% 64 == 0 and K %% 64 == 0 (got %lld x %lld)",
                name, (long long)out_rows, (long long)k);
  if (p->scale_mode != MXFP4_SCALE_FLOOR && p->scale_mode != MXFP4_SCALE_ROUNDUP)
    return fail(MXFP4_ERR_INVALID_ARG, "%s: bad scale_mode %d", name, p->scale_mode);
  if (p->rounding != MXFP4_ROUND_RTN && p->rounding != MXFP4_ROUND_SR)
    return fail(MXFP4_ERR_INVALID_ARG, "%s: bad rounding %d", name, p->rounding);
  if (p->scale_layout != MXFP4_LAYOUT_ROWMAJOR && p->scale_layout != MXFP4_LAYOUT_MMA)
    return fail(MXFP4_ERR_INVALID_ARG, "%s: bad scale_layout %d", name, p->scale_layout);
  if (p->wht != 0 && p->wht != 1) return fail(MXFP4_ERR_INVALID_ARG, "%s: wht must be 0/1", name);
  if (p->elem_format != MXFP4_FORMAT_E2M1 && p->elem_format != MXFP4_FORMAT_E4M3 &&
      p->elem_format != MXFP4_FORMAT_E5M2)
    return fail(MXFP4_ERR_INVALID_ARG, "%s: bad elem_format %u", name, p->elem_format);
  if (p->elem_format != MXFP4_FORMAT_E2M1 && p->rounding == MXFP4_ROUND_SR)
    return fail(MXFP4_ERR_UNSUPPORTED, "%s: stochastic rounding is available for E2M1 only", name);
  if (p->scale_layout == MXFP4_LAYOUT_MMA && (out_rows % 128 != 0 || k % 128 != 0))
    return fail(MXFP4_ERR_SHAPE,
                "%s: tensor-core scale layout needs rows %% 128 == 0 and K %% 128 == 0 (got %lld x %lld)",
                name, (long long)out_rows, (long long)k);
  o->block = nv ? 0 : p->block;
  o->nv = nv;
  o->nv_p2k = nv ? ldexpf(1.0f, p->tensor_exp) : 1.0f;
  o->nv_zmul = nv ? (float)(ldexp(1.0, -p->tensor_exp) / 6.0) : 1.0f;
  o->roundup = p->scale_mode == MXFP4_SCALE_ROUNDUP;
  o->sr = p->rounding == MXFP4_ROUND_SR;
  o->mma_layout = p->scale_layout == MXFP4_LAYOUT_MMA;
  o->wht = p->wht;
  o->e4m3 = p->elem_format == MXFP4_FORMAT_E4M3 || p->elem_format == MXFP4_FORMAT_E5M2;
  o->e5m2 = p->elem_format == MXFP4_FORMAT_E5M2;
  o->sign_mask = p->wht_sign_mask;
  o->seed = p->seed;
  o->stream = p->sr_stream;
  o->q = q;
  o->s = s;
  const int64_t qb = out_rows * (o->e4m3 ? k : k / 2), sb = out_rows * (nv ? k / 16 : k / 32);
  o->q_bytes = (uint64_t)(qb > g_extent_shrink ? qb - g_extent_shrink : 0);
  o->s_bytes = (uint64_t)(sb > g_extent_shrink ? sb - g_extent_shrink : 0);
  mx::prepare_orient(o);
  return MXFP4_OK;
}

// Element counts above 2^40 (2 TB of bf16) cannot be resident on one GPU;
// rejecting them first keeps every size product below int64's range.
constexpr int64_t kMaxElems = (int64_t)1 << 40;

bool too_large(int64_t rows, int64_t cols) { return rows > 0 && cols > kMaxElems / rows; }

mxfp4_status check_input(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t ld) {
  if (dtype != MXFP4_DTYPE_BF16 && dtype != MXFP4_DTYPE_F32)
    return fail(MXFP4_ERR_INVALID_ARG, "bad x_dtype %d", dtype);
  if (rows < 0 || cols < 0) return fail(MXFP4_ERR_SHAPE, "negative dimension");
  if (too_large(rows, cols)) return fail(MXFP4_ERR_SHAPE, "tensor too large (more than 2^40 elements)");
  if (!x && rows * cols > 0) return fail(MXFP4_ERR_INVALID_ARG, "x is NULL");
  if (cols % 32 != 0) return fail(MXFP4_ERR_SHAPE, "cols (%lld) must be a multiple of 32", (long long)cols);
  if (ld < cols) return fail(MXFP4_ERR_SHAPE, "ld_x (%lld) < cols (%lld)", (long long)ld, (long long)cols);
  if (!aligned16(x) || ld % 8 != 0)
    return fail(MXFP4_ERR_ALIGN, "x must be 16-byte aligned with ld_x %% 8 == 0");
  return MXFP4_OK;
}

}  // namespace

extern "C" {

const char* mxfp4_status_string(mxfp4_status s) {
  switch (s) {
    case MXFP4_OK: return "MXFP4_OK";
    case MXFP4_ERR_INVALID_ARG: return "MXFP4_ERR_INVALID_ARG";
    case MXFP4_ERR_SHAPE: return "MXFP4_ERR_SHAPE";
    case MXFP4_ERR_ALIGN: return "MXFP4_ERR_ALIGN";
    case MXFP4_ERR_UNSUPPORTED: return "MXFP4_ERR_UNSUPPORTED";
    case MXFP4_ERR_CUDA: return "MXFP4_ERR_CUDA";
    case MXFP4_ERR_TIMEOUT: return "MXFP4_ERR_TIMEOUT";
    case MXFP4_ERR_BOUNDS: return "MXFP4_ERR_BOUNDS";
  }
  return "MXFP4_ERR_UNKNOWN";
}

const char* mxfp4_last_error(void) { return g_last_error; }

mxfp4_status mxfp4_quantize(const void* x, int32_t x_dtype, int64_t rows, int64_t cols,
                            int64_t ld_x, const mxfp4_quant_params* row, uint8_t* q_row,
                            uint8_t* s_row, const mxfp4_quant_params* col, uint8_t* q_col,
                            uint8_t* s_col, void* stream) {
  if (!row && !col) return fail(MXFP4_ERR_INVALID_ARG, "at least one of row / col params is required");
  mxfp4_status st = check_input(x, x_dtype, rows, cols, ld_x);
  if (st) return st;
  // The row kernel counts 16-element units in 32 bits: units < 2^31 plus a
  // grid stride < 2^31 keeps every index it forms below 2^32.
  if (rows > 0 && cols / 16 > (int64_t)0x7FFFFFFF / rows)
    return fail(MXFP4_ERR_SHAPE, "tensor too large: rows * cols / 16 must be below 2^31");
  const bool need_rows32 =
      col || (row && row->block != MXFP4_BLOCK_1X32 && row->block != MXFP4_BLOCK_1X16);
  if (need_rows32 && rows % 32 != 0)
    return fail(MXFP4_ERR_SHAPE, "rows (%lld) must be a multiple of 32 for column-wise or 32x32 output",
                (long long)rows);
  mx::OrientArgs ro{}, co{};
  if (row && (st = check_params(row, q_row, s_row, rows, cols, "row", &ro))) return st;
  if (col && (st = check_params(col, q_col, s_col, cols, rows, "col", &co))) return st;
  return from_cuda(mx::launch_quantize(x, x_dtype == MXFP4_DTYPE_F32, rows, cols, ld_x,
                                       row ? &ro : nullptr, col ? &co : nullptr,
                                       static_cast<cudaStream_t>(stream)),
                   "mxfp4_quantize launch");
}

namespace {
mxfp4_status dequantize_common(const char* name, const uint8_t* q, const uint8_t* s,
                               int32_t scale_layout, int fmt, int32_t tensor_exp, int64_t rows,
                               int64_t cols, float* out, void* stream) {
  if (scale_layout != MXFP4_LAYOUT_ROWMAJOR && scale_layout != MXFP4_LAYOUT_MMA)
    return fail(MXFP4_ERR_INVALID_ARG, "%s: bad scale_layout %d", name, scale_layout);
  if (rows < 0 || cols < 0 || cols % 32 != 0)
    return fail(MXFP4_ERR_SHAPE, "%s: cols (%lld) must be a non-negative multiple of 32", name,
                (long long)cols);
  if (too_large(rows, cols)) return fail(MXFP4_ERR_SHAPE, "%s: tensor too large (more than 2^40 elements)", name);
  if ((!q || !s || !out) && rows * cols > 0) return fail(MXFP4_ERR_INVALID_ARG, "%s: NULL pointer", name);
  if (scale_layout == MXFP4_LAYOUT_MMA && (rows % 128 != 0 || cols % 128 != 0))
    return fail(MXFP4_ERR_SHAPE, "%s: tensor-core scale layout needs rows and cols %% 128 == 0", name);
  if (!aligned16(q) || !aligned16(out))
    return fail(MXFP4_ERR_ALIGN, "%s: q / out must be 16-byte aligned", name);
  return from_cuda(mx::launch_dequantize(q, s, scale_layout == MXFP4_LAYOUT_MMA, rows, cols, fmt,
                                         ldexpf(1.0f, tensor_exp), out,
                                         static_cast<cudaStream_t>(stream)),
                   name);
}
}  // namespace

mxfp4_status mxfp4_dequantize(const uint8_t* q, const uint8_t* s, int32_t scale_layout,
                              int64_t rows, int64_t cols, float* out, void* stream) {
  return dequantize_common("mxfp4_dequantize", q, s, scale_layout, 0, 0, rows, cols, out, stream);
}

mxfp4_status mxfp4_dequantize_ex(const uint8_t* q, const uint8_t* s, int32_t scale_layout,
                                 int32_t block, uint32_t elem_format, int32_t tensor_exp,
                                 int64_t rows, int64_t cols, float* out, void* stream) {
  if (block != MXFP4_BLOCK_1X32 && block != MXFP4_BLOCK_32X32 && block != MXFP4_BLOCK_64X64 &&
      block != MXFP4_BLOCK_1X16)
    return fail(MXFP4_ERR_INVALID_ARG, "mxfp4_dequantize_ex: bad block %d", block);
  if (elem_format != MXFP4_FORMAT_E2M1 && elem_format != MXFP4_FORMAT_E4M3 &&
      elem_format != MXFP4_FORMAT_E5M2)
    return fail(MXFP4_ERR_INVALID_ARG, "mxfp4_dequantize_ex: bad elem_format %u", elem_format);
  const bool nv = block == MXFP4_BLOCK_1X16;
  if (nv && elem_format != MXFP4_FORMAT_E2M1)
    return fail(MXFP4_ERR_UNSUPPORTED, "mxfp4_dequantize_ex: 1x16 blocks take E2M1 elements");
  if (nv ? (tensor_exp < -100 || tensor_exp > 100) : tensor_exp != 0)
    return fail(MXFP4_ERR_INVALID_ARG, "mxfp4_dequantize_ex: bad tensor_exp %d", tensor_exp);
  const int fmt = nv ? 2 : (elem_format == MXFP4_FORMAT_E4M3 ? 1 : (elem_format == MXFP4_FORMAT_E5M2 ? 3 : 0));
  return dequantize_common("mxfp4_dequantize_ex", q, s, scale_layout, fmt, tensor_exp, rows, cols,
                           out, stream);
}

namespace {
// Shape rules of the GEMM entry points (MXFP4, MXFP8, NVFP4).
mxfp4_status gemm_shape(const char* name, int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K <= 0 || M % 128 != 0 || N % 128 != 0 || K % 128 != 0)
    return fail(MXFP4_ERR_SHAPE, "%s needs M, N, K positive multiples of 128 (got %lld, %lld, %lld)",
                name, (long long)M, (long long)N, (long long)K);
  if (M > (1ll << 30) || N > (1ll << 30) || K > (1ll << 30) || (M / 128) * (N / 128) > (1ll << 30))
    return fail(MXFP4_ERR_SHAPE, "%s dimensions too large", name);
  return MXFP4_OK;
}

mxfp4_status gemm_common(const char* name, const uint8_t* qa, const uint8_t* sa, const uint8_t* qb,
                         const uint8_t* sb, int64_t M, int64_t N, int64_t K, void* c,
                         int32_t c_dtype, int64_t ldc, const mx::OrientArgs* qout,
                         const mx::OrientArgs* qcol, void* ws, size_t ws_bytes, void* stream) {
  if (!qa || !sa || !qb || !sb || (!c && !qout && !qcol))
    return fail(MXFP4_ERR_INVALID_ARG, "%s: NULL pointer", name);
  if (c_dtype != MXFP4_DTYPE_BF16 && c_dtype != MXFP4_DTYPE_F32)
    return fail(MXFP4_ERR_INVALID_ARG, "%s: bad c_dtype %d", name, c_dtype);
  if (mxfp4_status st = gemm_shape(name, M, N, K)) return st;
  if (c && ldc < N) return fail(MXFP4_ERR_SHAPE, "ldc (%lld) < N (%lld)", (long long)ldc, (long long)N);
  if (!aligned16(qa) || !aligned16(qb) || !aligned16(sa) || !aligned16(sb) || !aligned16(c) ||
      (c && ldc % 8 != 0))
    return fail(MXFP4_ERR_ALIGN, "operands must be 16-byte aligned and ldc %% 8 == 0");
  if (ws && !aligned16(ws)) return fail(MXFP4_ERR_ALIGN, "%s: workspace must be 16-byte aligned", name);
  const char* why = "";
  cudaError_t e = mx::launch_gemm(qa, sa, qb, sb, M, N, K, c, c_dtype == MXFP4_DTYPE_BF16, ldc,
                                  qout, qcol, ws, ws_bytes, static_cast<cudaStream_t>(stream), &why);
  if (e == cudaErrorNotSupported) return fail(MXFP4_ERR_UNSUPPORTED, "%s", why);
  if (e == cudaErrorInvalidValue && why[0]) return fail(MXFP4_ERR_ALIGN, "%s", why);
  return from_cuda(e, name);
}
}  // namespace

mxfp4_status mxfp4_gemm(const uint8_t* qa, const uint8_t* sa, const uint8_t* qb,
                        const uint8_t* sb, int64_t M, int64_t N, int64_t K, float* c,
                        int64_t ldc, void* stream) {
  if (!c) return fail(MXFP4_ERR_INVALID_ARG, "NULL pointer");
  return gemm_common("mxfp4_gemm", qa, sa, qb, sb, M, N, K, c, MXFP4_DTYPE_F32, ldc, nullptr,
                     nullptr, nullptr, 0, stream);
}

mxfp4_status mxfp4_gemm_noalloc(const uint8_t* qa, const uint8_t* sa, const uint8_t* qb,
                                const uint8_t* sb, int64_t M, int64_t N, int64_t K, float* c,
                                int64_t ldc, void* stream) {
  if (!c) return fail(MXFP4_ERR_INVALID_ARG, "NULL pointer");
  if (mxfp4_status st = gemm_shape("mxfp4_gemm_noalloc", M, N, K)) return st;
  // Only the CTA-pair kernel (M % 256 == 0) reads scale images; the dimensions
  // are validated above, so the image size cannot overflow.
  if (M % 256 == 0 && mx::workspace_bytes(M, N, K, false) > (int64_t)mx::kStaticScratchBytes)
    return fail(MXFP4_ERR_SHAPE,
                "mxfp4_gemm_noalloc: scale images of %lld x %lld x %lld exceed the static scratch (%zu bytes)",
                (long long)M, (long long)N, (long long)K, mx::kStaticScratchBytes);
  void* ws = nullptr;
  const cudaError_t e = mx::static_scratch(&ws);
  if (e != cudaSuccess) return from_cuda(e, "mxfp4_gemm_noalloc: static scratch");
  return gemm_common("mxfp4_gemm_noalloc", qa, sa, qb, sb, M, N, K, c, MXFP4_DTYPE_F32, ldc, nullptr,
                     nullptr, ws, mx::kStaticScratchBytes, stream);
}

size_t mxfp4_gemm_workspace_size(int64_t M, int64_t N, int64_t K, int32_t scale_block) {
  if (M <= 0 || N <= 0 || K <= 0 || (scale_block != 32 && scale_block != 16)) return 0;
  return (size_t)mx::workspace_bytes(M, N, K, scale_block == 16);
}

mxfp4_status mxfp4_gemm_ex(const uint8_t* qa, const uint8_t* sa, const uint8_t* qb,
                           const uint8_t* sb, int64_t M, int64_t N, int64_t K, void* c,
                           int32_t c_dtype, int64_t ldc, void* workspace, size_t workspace_bytes,
                           void* stream) {
  if (!c) return fail(MXFP4_ERR_INVALID_ARG, "NULL pointer");
  return gemm_common("mxfp4_gemm_ex", qa, sa, qb, sb, M, N, K, c, c_dtype, ldc, nullptr, nullptr,
                     workspace, workspace_bytes, stream);
}

namespace {
mxfp4_status mxfp8_common(const uint8_t* qa, const uint8_t* sa, const uint8_t* qb,
                          const uint8_t* sb, int64_t M, int64_t N, int64_t K, uint32_t elem_format,
                          void* c, int32_t c_dtype, int64_t ldc, void* stream) {
  if (!qa || !sa || !qb || !sb || !c) return fail(MXFP4_ERR_INVALID_ARG, "mxfp8_gemm: NULL pointer");
  if (elem_format != MXFP4_FORMAT_E4M3 && elem_format != MXFP4_FORMAT_E5M2)
    return fail(MXFP4_ERR_INVALID_ARG, "mxfp8_gemm: elem_format %u is not E4M3 or E5M2", elem_format);
  if (c_dtype != MXFP4_DTYPE_BF16 && c_dtype != MXFP4_DTYPE_F32)
    return fail(MXFP4_ERR_INVALID_ARG, "mxfp8_gemm: bad c_dtype %d", c_dtype);
  if (mxfp4_status st = gemm_shape("mxfp8_gemm", M, N, K)) return st;
  if (ldc < N) return fail(MXFP4_ERR_SHAPE, "ldc (%lld) < N (%lld)", (long long)ldc, (long long)N);
  if (!aligned16(qa) || !aligned16(qb) || !aligned16(sa) || !aligned16(sb) || !aligned16(c) || ldc % 8 != 0)
    return fail(MXFP4_ERR_ALIGN, "operands must be 16-byte aligned and ldc %% 8 == 0");
  const char* why = "";
  cudaError_t e = mx::launch_gemm_f8(qa, sa, qb, sb, M, N, K, elem_format == MXFP4_FORMAT_E5M2, c,
                                     c_dtype == MXFP4_DTYPE_BF16, ldc,
                                     static_cast<cudaStream_t>(stream), &why);
  if (e == cudaErrorNotSupported) return fail(MXFP4_ERR_UNSUPPORTED, "%s", why);
  if (e == cudaErrorInvalidValue && why[0]) return fail(MXFP4_ERR_ALIGN, "%s", why);
  return from_cuda(e, "mxfp8_gemm");
}
}  // namespace

mxfp4_status mxfp8_gemm(const uint8_t* qa, const uint8_t* sa, const uint8_t* qb,
                        const uint8_t* sb, int64_t M, int64_t N, int64_t K, void* c,
                        int32_t c_dtype, int64_t ldc, void* stream) {
  return mxfp8_common(qa, sa, qb, sb, M, N, K, MXFP4_FORMAT_E4M3, c, c_dtype, ldc, stream);
}

mxfp4_status mxfp8_gemm_ex(const uint8_t* qa, const uint8_t* sa, const uint8_t* qb,
                           const uint8_t* sb, int64_t M, int64_t N, int64_t K,
                           uint32_t elem_format, void* c, int32_t c_dtype, int64_t ldc,
                           void* stream) {
  return mxfp8_common(qa, sa, qb, sb, M, N, K, elem_format, c, c_dtype, ldc, stream);
}

mxfp4_status nvfp4_gemm(const uint8_t* qa, const uint8_t* sa, int32_t ka, const uint8_t* qb,
                        const uint8_t* sb, int32_t kb, int64_t M, int64_t N, int64_t K, void* c,
                        int32_t c_dtype, int64_t ldc, void* workspace, size_t workspace_bytes,
                        void* stream) {
  if (!qa || !sa || !qb || !sb || !c) return fail(MXFP4_ERR_INVALID_ARG, "nvfp4_gemm: NULL pointer");
  if (c_dtype != MXFP4_DTYPE_BF16 && c_dtype != MXFP4_DTYPE_F32)
    return fail(MXFP4_ERR_INVALID_ARG, "nvfp4_gemm: bad c_dtype %d", c_dtype);
  if (ka < -100 || ka > 100 || kb < -100 || kb > 100 || ka + kb < -126 || ka + kb > 126)
    return fail(MXFP4_ERR_INVALID_ARG, "nvfp4_gemm: tensor exponents %d, %d out of range", ka, kb);
  if (mxfp4_status st = gemm_shape("nvfp4_gemm", M, N, K)) return st;
  if (ldc < N) return fail(MXFP4_ERR_SHAPE, "ldc (%lld) < N (%lld)", (long long)ldc, (long long)N);
  if (!aligned16(qa) || !aligned16(qb) || !aligned16(sa) || !aligned16(sb) || !aligned16(c) || ldc % 8 != 0)
    return fail(MXFP4_ERR_ALIGN, "operands must be 16-byte aligned and ldc %% 8 == 0");
  if (workspace && !aligned16(workspace))
    return fail(MXFP4_ERR_ALIGN, "nvfp4_gemm: workspace must be 16-byte aligned");
  const char* why = "";
  cudaError_t e = mx::launch_gemm_nv(qa, sa, qb, sb, M, N, K, ldexpf(1.0f, ka + kb), c,
                                     c_dtype == MXFP4_DTYPE_BF16, ldc, workspace, workspace_bytes,
                                     static_cast<cudaStream_t>(stream), &why);
  if (e == cudaErrorNotSupported) return fail(MXFP4_ERR_UNSUPPORTED, "%s", why);
  if (e == cudaErrorInvalidValue && why[0]) return fail(MXFP4_ERR_ALIGN, "%s", why);
  return from_cuda(e, "nvfp4_gemm");
}

mxfp4_status mxfp4_gemm_quantize(const uint8_t* qa, const uint8_t* sa, const uint8_t* qb,
                                 const uint8_t* sb, int64_t M, int64_t N, int64_t K, void* c,
                                 int32_t c_dtype, int64_t ldc, const mxfp4_quant_params* row,
                                 uint8_t* q_row, uint8_t* s_row, const mxfp4_quant_params* col,
                                 uint8_t* q_col, uint8_t* s_col, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  if (!row && !col)
    return fail(MXFP4_ERR_INVALID_ARG, "mxfp4_gemm_quantize: row or col params are required");
  for (const mxfp4_quant_params* p : {row, col}) {
    if (p && p->block == MXFP4_BLOCK_64X64)
      return fail(MXFP4_ERR_UNSUPPORTED,
                  "mxfp4_gemm_quantize: 64x64 blocks span two epilogue warps; quantize C separately");
    if (p && p->block == MXFP4_BLOCK_1X16)
      return fail(MXFP4_ERR_UNSUPPORTED,
                  "mxfp4_gemm_quantize: 1x16 (NVFP4) output is not fused; quantize C separately");
  }
  mx::OrientArgs ro{}, co{};
  if (M > 0 && N > 0) {
    mxfp4_status st;
    if (row && (st = check_params(row, q_row, s_row, M, N, "row", &ro))) return st;
    if (col && (st = check_params(col, q_col, s_col, N, M, "col", &co))) return st;
  }
  return gemm_common("mxfp4_gemm_quantize", qa, sa, qb, sb, M, N, K, c, c_dtype, ldc,
                     row ? &ro : nullptr, col ? &co : nullptr, workspace, workspace_bytes, stream);
}

mxfp4_status hadamard32(const void* x, int32_t x_dtype, int64_t rows, int64_t cols,
                        int64_t ld_x, uint32_t sign_mask, int32_t inverse, float* y,
                        void* stream) {
  mxfp4_status st = check_input(x, x_dtype, rows, cols, ld_x);
  if (st) return st;
  if (!y && rows * cols > 0) return fail(MXFP4_ERR_INVALID_ARG, "y is NULL");
  if (!aligned16(y)) return fail(MXFP4_ERR_ALIGN, "y must be 16-byte aligned");
  if (inverse != 0 && inverse != 1) return fail(MXFP4_ERR_INVALID_ARG, "inverse must be 0/1");
  return from_cuda(mx::launch_hadamard32(x, x_dtype == MXFP4_DTYPE_F32, rows, cols, ld_x, sign_mask,
                                         inverse != 0, y, static_cast<cudaStream_t>(stream)),
                   "hadamard32 launch");
}

mxfp4_status mxfp4_tensor_amax(const void* x, int32_t x_dtype, int64_t rows, int64_t cols,
                               int64_t ld_x, float* amax, int32_t* tensor_exp, void* stream) {
  mxfp4_status st = check_input(x, x_dtype, rows, cols, ld_x);
  if (st) return st;
  if (!amax) return fail(MXFP4_ERR_INVALID_ARG, "mxfp4_tensor_amax: amax is NULL");
  if ((reinterpret_cast<uintptr_t>(amax) & 3u) || (reinterpret_cast<uintptr_t>(tensor_exp) & 3u))
    return fail(MXFP4_ERR_ALIGN, "mxfp4_tensor_amax: amax / tensor_exp must be 4-byte aligned");
  return from_cuda(mx::launch_amax(x, x_dtype == MXFP4_DTYPE_F32, rows, cols, ld_x, amax, tensor_exp,
                                   static_cast<cudaStream_t>(stream)),
                   "mxfp4_tensor_amax launch");
}

namespace {
// A [rows, cols] matrix operand of the norm, activation and few-row calls.
mxfp4_status check_matrix(const char* fn, const char* name, const void* p, int32_t dtype, int64_t rows,
                          int64_t cols, int64_t ld) {
  if (dtype != MXFP4_DTYPE_BF16 && dtype != MXFP4_DTYPE_F32)
    return fail(MXFP4_ERR_INVALID_ARG, "%s: bad dtype %d of %s", fn, dtype, name);
  if (!p && rows * cols > 0) return fail(MXFP4_ERR_INVALID_ARG, "%s: %s is NULL", fn, name);
  if (ld < cols || ld > kMaxElems)
    return fail(MXFP4_ERR_SHAPE, "%s: leading dimension %lld of %s (cols %lld)", fn, (long long)ld, name,
                (long long)cols);
  if (rows > 1 && too_large(rows, ld)) return fail(MXFP4_ERR_SHAPE, "%s: %s too large (more than 2^40 elements)", fn, name);
  if (!aligned16(p) || ld % 8 != 0)
    return fail(MXFP4_ERR_ALIGN, "%s: %s must be 16-byte aligned with a leading dimension %% 8 == 0", fn, name);
  return MXFP4_OK;
}

mxfp4_status check_dims(const char* fn, int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0 || cols % 32 != 0)
    return fail(MXFP4_ERR_SHAPE, "%s: rows (%lld) must be >= 0 and cols (%lld) a non-negative multiple of 32", fn,
                (long long)rows, (long long)cols);
  if (cols >= ((int64_t)1 << 31) || too_large(rows, cols))
    return fail(MXFP4_ERR_SHAPE, "%s: tensor too large (cols below 2^31, at most 2^40 elements)", fn);
  return MXFP4_OK;
}

int64_t elem_bytes(int32_t dtype) { return dtype == MXFP4_DTYPE_F32 ? 4 : 2; }

// Bytes from the first to the last element of a [rows, cols] output (what a
// bounds-checking build lets a call store to).
uint64_t extent(int64_t rows, int64_t cols, int64_t ld, int32_t dtype) {
  if (rows == 0 || cols == 0) return 0;
  const int64_t n = ((rows - 1) * ld + cols) * elem_bytes(dtype);
  return (uint64_t)(n > g_extent_shrink ? n - g_extent_shrink : 0);
}

// The quantized output of the norm and activation calls: 1x32 or 1x16 blocks,
// nearest-even, no rotation.
mxfp4_status check_row_quant(const char* fn, const mxfp4_quant_params* p, uint8_t* q, uint8_t* s, int64_t rows,
                             int64_t cols, mx::RowQuant* o) {
  *o = mx::RowQuant{};
  if (!p) return MXFP4_OK;
  if (p->block != MXFP4_BLOCK_1X32 && p->block != MXFP4_BLOCK_1X16)
    return fail(MXFP4_ERR_UNSUPPORTED, "%s: output blocks are 1x32 or 1x16", fn);
  if (p->rounding == MXFP4_ROUND_SR || p->wht)
    return fail(MXFP4_ERR_UNSUPPORTED, "%s: stochastic rounding and rotation are mxfp4_quantize's", fn);
  mx::OrientArgs a{};
  if (mxfp4_status st = check_params(p, q, s, rows, cols, fn, &a)) return st;
  o->fmt = a.nv ? mx::RowQuant::kNvfp4
                : a.e5m2 ? mx::RowQuant::kE5m2 : a.e4m3 ? mx::RowQuant::kE4m3 : mx::RowQuant::kE2m1;
  o->roundup = a.roundup;
  o->emax = a.e5m2 ? 15 : a.e4m3 ? 8 : 2;
  o->over = !a.roundup ? 0x7FFFFFu : a.e4m3 ? 0x600000u : 0x400000u;  // 1.75 2^emax, E2M1 1.5 2^emax
  o->mma = a.mma_layout;
  o->packed = cols % (a.nv ? 64 : 128) == 0 && (reinterpret_cast<uintptr_t>(s) & 3u) == 0;
  o->p2k = a.nv_p2k;
  o->zmul = a.nv_zmul;
  o->q = q;
  o->s = s;
  o->q_bytes = a.q_bytes;
  o->s_bytes = a.s_bytes;
  return MXFP4_OK;
}

mxfp4_status check_vector(const char* fn, const char* name, const void* p, int32_t dtype) {
  if (dtype != MXFP4_DTYPE_BF16 && dtype != MXFP4_DTYPE_F32)
    return fail(MXFP4_ERR_INVALID_ARG, "%s: bad dtype %d of %s", fn, dtype, name);
  if (!aligned16(p)) return fail(MXFP4_ERR_ALIGN, "%s: %s must be 16-byte aligned", fn, name);
  return MXFP4_OK;
}
}  // namespace

mxfp4_status mxfp4_rmsnorm_quantize(const void* x, int32_t x_dtype, int64_t rows, int64_t cols, int64_t ld_x,
                                    const void* residual, int64_t ld_residual, const void* weight,
                                    int32_t weight_dtype, float eps, void* h, int64_t ld_h, void* y,
                                    int32_t y_dtype, int64_t ld_y, float* rstd, const mxfp4_quant_params* row,
                                    uint8_t* q, uint8_t* s, void* stream) {
  const char* fn = "mxfp4_rmsnorm_quantize";
  mxfp4_status st = check_dims(fn, rows, cols);
  if (st) return st;
  if ((st = check_matrix(fn, "x", x, x_dtype, rows, cols, ld_x))) return st;
  if (residual && (st = check_matrix(fn, "residual", residual, x_dtype, rows, cols, ld_residual))) return st;
  if (h && (st = check_matrix(fn, "h", h, x_dtype, rows, cols, ld_h))) return st;
  if (y && (st = check_matrix(fn, "y", y, y_dtype, rows, cols, ld_y))) return st;
  if (weight && (st = check_vector(fn, "weight", weight, weight_dtype))) return st;
  if (reinterpret_cast<uintptr_t>(rstd) & 3u) return fail(MXFP4_ERR_ALIGN, "%s: rstd must be 4-byte aligned", fn);
  if (!(eps >= 0.0f && eps <= 1.0e30f)) return fail(MXFP4_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", fn);
  if (!row && !y && !h && !rstd) return fail(MXFP4_ERR_INVALID_ARG, "%s: no output is asked for", fn);
  mx::NormArgs a{};
  if ((st = check_row_quant(fn, row, q, s, rows, cols, &a.quant))) return st;
  a.x = x;
  a.r = residual;
  a.w = weight;
  a.h = h;
  a.y = y;
  a.rstd = rstd;
  a.rows = rows;
  a.cols = cols;
  a.ld_x = ld_x;
  a.ld_r = ld_residual;
  a.ld_h = ld_h;
  a.ld_y = ld_y;
  a.h_bytes = h ? extent(rows, cols, ld_h, x_dtype) : 0;
  a.y_bytes = y ? extent(rows, cols, ld_y, y_dtype) : 0;
  a.eps = eps;
  a.y_f32 = y_dtype == MXFP4_DTYPE_F32;
  return from_cuda(mx::launch_rmsnorm(a, x_dtype == MXFP4_DTYPE_F32, weight && weight_dtype == MXFP4_DTYPE_F32,
                                      static_cast<cudaStream_t>(stream)),
                   fn);
}

size_t mxfp4_rmsnorm_backward_workspace_size(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0 || cols >= ((int64_t)1 << 31)) return 0;
  return (size_t)mx::norm_dw_slices(rows) * (size_t)cols * sizeof(float);
}

mxfp4_status mxfp4_rmsnorm_backward(const void* dy, int32_t dy_dtype, int64_t ld_dy, const void* h, int32_t h_dtype,
                                    int64_t ld_h, const void* weight, int32_t weight_dtype, const float* rstd,
                                    const void* dh, int64_t ld_dh, int64_t rows, int64_t cols, void* dx,
                                    int64_t ld_dx, void* dw, void* workspace, size_t workspace_bytes,
                                    void* stream) {
  const char* fn = "mxfp4_rmsnorm_backward";
  mxfp4_status st = check_dims(fn, rows, cols);
  if (st) return st;
  if ((st = check_matrix(fn, "dy", dy, dy_dtype, rows, cols, ld_dy))) return st;
  if ((st = check_matrix(fn, "h", h, h_dtype, rows, cols, ld_h))) return st;
  if (dh && (st = check_matrix(fn, "dh", dh, h_dtype, rows, cols, ld_dh))) return st;
  if ((st = check_matrix(fn, "dx", dx, h_dtype, rows, cols, ld_dx))) return st;
  if ((weight || dw) && (st = check_vector(fn, "weight", weight, weight_dtype))) return st;
  if ((st = check_vector(fn, "dw", dw, MXFP4_DTYPE_F32))) return st;
  if (!rstd && rows > 0) return fail(MXFP4_ERR_INVALID_ARG, "%s: rstd is NULL", fn);
  if (reinterpret_cast<uintptr_t>(rstd) & 3u) return fail(MXFP4_ERR_ALIGN, "%s: rstd must be 4-byte aligned", fn);
  const size_t need = dw ? mxfp4_rmsnorm_backward_workspace_size(rows, cols) : 0;
  if (need && !workspace) return fail(MXFP4_ERR_INVALID_ARG, "%s: workspace is NULL", fn);
  if (need && workspace_bytes < need)
    return fail(MXFP4_ERR_INVALID_ARG, "%s: workspace of %zu bytes, %zu are needed", fn, workspace_bytes, need);
  if (!aligned16(workspace)) return fail(MXFP4_ERR_ALIGN, "%s: workspace must be 16-byte aligned", fn);
  mx::NormGradArgs a{};
  a.dy = dy;
  a.h = h;
  a.w = weight;
  a.dh = dh;
  a.rstd = rstd;
  a.dx = dx;
  a.dw = dw;
  a.ws = static_cast<float*>(workspace);
  a.rows = rows;
  a.cols = cols;
  a.ld_dy = ld_dy;
  a.ld_h = ld_h;
  a.ld_dh = ld_dh;
  a.ld_dx = ld_dx;
  a.dx_bytes = extent(rows, cols, ld_dx, h_dtype);
  a.ws_bytes = need;
  return from_cuda(mx::launch_rmsnorm_grad(a, h_dtype == MXFP4_DTYPE_F32, dy_dtype == MXFP4_DTYPE_F32,
                                           (weight || dw) && weight_dtype == MXFP4_DTYPE_F32,
                                           static_cast<cudaStream_t>(stream)),
                   fn);
}

mxfp4_status mxfp4_swiglu_quantize(const void* gate, int64_t ld_gate, const void* up, int64_t ld_up, int32_t dtype,
                                   int64_t rows, int64_t cols, void* y, int32_t y_dtype, int64_t ld_y,
                                   const mxfp4_quant_params* row, uint8_t* q, uint8_t* s, void* stream) {
  const char* fn = "mxfp4_swiglu_quantize";
  mxfp4_status st = check_dims(fn, rows, cols);
  if (st) return st;
  if ((st = check_matrix(fn, "gate", gate, dtype, rows, cols, ld_gate))) return st;
  if ((st = check_matrix(fn, "up", up, dtype, rows, cols, ld_up))) return st;
  if (y && (st = check_matrix(fn, "y", y, y_dtype, rows, cols, ld_y))) return st;
  if (!row && !y) return fail(MXFP4_ERR_INVALID_ARG, "%s: no output is asked for", fn);
  mx::SwigluArgs a{};
  if ((st = check_row_quant(fn, row, q, s, rows, cols, &a.quant))) return st;
  a.g = gate;
  a.u = up;
  a.y = y;
  a.rows = rows;
  a.cols = cols;
  a.ld_g = ld_gate;
  a.ld_u = ld_up;
  a.ld_y = ld_y;
  a.y_bytes = y ? extent(rows, cols, ld_y, y_dtype) : 0;
  a.y_f32 = y_dtype == MXFP4_DTYPE_F32;
  return from_cuda(mx::launch_swiglu(a, dtype == MXFP4_DTYPE_F32, static_cast<cudaStream_t>(stream)), fn);
}

mxfp4_status mxfp4_swiglu_backward(const void* dy, int32_t dy_dtype, int64_t ld_dy, const void* gate,
                                   int64_t ld_gate, const void* up, int64_t ld_up, int32_t dtype, int64_t rows,
                                   int64_t cols, void* dgate, int64_t ld_dgate, void* dup, int64_t ld_dup,
                                   void* stream) {
  const char* fn = "mxfp4_swiglu_backward";
  mxfp4_status st = check_dims(fn, rows, cols);
  if (st) return st;
  if ((st = check_matrix(fn, "dy", dy, dy_dtype, rows, cols, ld_dy))) return st;
  if ((st = check_matrix(fn, "gate", gate, dtype, rows, cols, ld_gate))) return st;
  if ((st = check_matrix(fn, "up", up, dtype, rows, cols, ld_up))) return st;
  if ((st = check_matrix(fn, "dgate", dgate, dtype, rows, cols, ld_dgate))) return st;
  if ((st = check_matrix(fn, "dup", dup, dtype, rows, cols, ld_dup))) return st;
  mx::SwigluGradArgs a{};
  a.dy = dy;
  a.g = gate;
  a.u = up;
  a.dg = dgate;
  a.du = dup;
  a.rows = rows;
  a.cols = cols;
  a.ld_dy = ld_dy;
  a.ld_g = ld_gate;
  a.ld_u = ld_up;
  a.ld_dg = ld_dgate;
  a.ld_du = ld_dup;
  a.dg_bytes = extent(rows, cols, ld_dgate, dtype);
  a.du_bytes = extent(rows, cols, ld_dup, dtype);
  return from_cuda(mx::launch_swiglu_grad(a, dtype == MXFP4_DTYPE_F32, dy_dtype == MXFP4_DTYPE_F32,
                                          static_cast<cudaStream_t>(stream)),
                   fn);
}

mxfp4_status mxfp4_gemv(const void* x, int32_t x_kind, int64_t ld_x, const uint8_t* sx, const uint8_t* qw,
                        const uint8_t* sw, int32_t block, int32_t scale_layout, int32_t tensor_exp, int64_t M,
                        int64_t N, int64_t K, void* y, int32_t y_dtype, int64_t ld_y, void* stream) {
  return mxfp4_gemv_ex(x, x_kind, ld_x, sx, qw, sw, block, scale_layout, tensor_exp, M, N, K, y, y_dtype, ld_y,
                       nullptr, 0, stream);
}

size_t mxfp4_gemv_workspace_size(int32_t x_kind, int32_t block, int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K <= 0 || M > 65536 || N > (1ll << 30) || K > (1ll << 30)) return 0;
  mx::GemvArgs a{};
  a.x_kind = x_kind;
  a.nv = block == MXFP4_BLOCK_1X16;
  a.M = M;
  a.N = N;
  a.K = K;
  return (size_t)mx::gemv_workspace_bytes(a);
}

mxfp4_status mxfp4_gemv_ex(const void* x, int32_t x_kind, int64_t ld_x, const uint8_t* sx, const uint8_t* qw,
                           const uint8_t* sw, int32_t block, int32_t scale_layout, int32_t tensor_exp, int64_t M,
                           int64_t N, int64_t K, void* y, int32_t y_dtype, int64_t ld_y, void* workspace,
                           size_t workspace_bytes, void* stream) {
  const char* fn = "mxfp4_gemv";
  if (x_kind != MXFP4_GEMV_X_BF16 && x_kind != MXFP4_GEMV_X_E4M3 && x_kind != MXFP4_GEMV_X_E5M2)
    return fail(MXFP4_ERR_INVALID_ARG, "%s: bad x_kind %d", fn, x_kind);
  if (y_dtype != MXFP4_DTYPE_BF16 && y_dtype != MXFP4_DTYPE_F32)
    return fail(MXFP4_ERR_INVALID_ARG, "%s: bad y_dtype %d", fn, y_dtype);
  if (block != MXFP4_BLOCK_1X32 && block != MXFP4_BLOCK_32X32 && block != MXFP4_BLOCK_64X64 &&
      block != MXFP4_BLOCK_1X16)
    return fail(MXFP4_ERR_INVALID_ARG, "%s: bad block %d", fn, block);
  if (scale_layout != MXFP4_LAYOUT_ROWMAJOR && scale_layout != MXFP4_LAYOUT_MMA)
    return fail(MXFP4_ERR_INVALID_ARG, "%s: bad scale_layout %d", fn, scale_layout);
  const bool nv = block == MXFP4_BLOCK_1X16;
  if (nv ? (tensor_exp < -100 || tensor_exp > 100) : tensor_exp != 0)
    return fail(MXFP4_ERR_INVALID_ARG, "%s: bad tensor_exp %d", fn, tensor_exp);
  if (M < 0 || N < 0 || K < 0 || K % 32 != 0)
    return fail(MXFP4_ERR_SHAPE, "%s: M, N >= 0 and K a non-negative multiple of 32 (got %lld, %lld, %lld)", fn,
                (long long)M, (long long)N, (long long)K);
  if (M > 65536 || N > (1ll << 30) || K > (1ll << 30) || too_large(N, K))
    return fail(MXFP4_ERR_SHAPE, "%s: dimensions too large (M up to 65536, N and K up to 2^30, N K up to 2^40)", fn);
  if (scale_layout == MXFP4_LAYOUT_MMA && (N % 128 != 0 || K % 128 != 0))
    return fail(MXFP4_ERR_SHAPE, "%s: tensor-core scale layout needs N %% 128 == 0 and K %% 128 == 0", fn);
  const bool codes = x_kind != MXFP4_GEMV_X_BF16;
  if (ld_x < K || ld_y < N || ld_x > kMaxElems || ld_y > kMaxElems || (M > 1 && (too_large(M, ld_x) || too_large(M, ld_y))))
    return fail(MXFP4_ERR_SHAPE, "%s: ld_x (%lld) < K or ld_y (%lld) < N, or too large", fn, (long long)ld_x,
                (long long)ld_y);
  if (M * N > 0) {
    if (!y) return fail(MXFP4_ERR_INVALID_ARG, "%s: y is NULL", fn);
    if (K > 0 && (!x || !qw || !sw || (codes && !sx)))
      return fail(MXFP4_ERR_INVALID_ARG, "%s: x, qw, sw (and sx with one-byte x) must be non-NULL", fn);
  }
  if (!aligned16(x) || !aligned16(qw) || !aligned16(sw) || ld_x % (codes ? 16 : 8) != 0)
    return fail(MXFP4_ERR_ALIGN, "%s: x, qw and sw must be 16-byte aligned, rows of x multiples of 16 bytes", fn);
  if (reinterpret_cast<uintptr_t>(y) % elem_bytes(y_dtype))
    return fail(MXFP4_ERR_ALIGN, "%s: y must be aligned to its element", fn);
  if (!aligned16(workspace)) return fail(MXFP4_ERR_ALIGN, "%s: workspace must be 16-byte aligned", fn);
  mx::GemvArgs a{};
  a.ws = static_cast<uint8_t*>(workspace);
  a.ws_bytes = workspace ? workspace_bytes : 0;
  a.x = x;
  a.sx = sx;
  a.qw = qw;
  a.sw = sw;
  a.y = y;
  a.M = M;
  a.N = N;
  a.K = K;
  a.ld_x = ld_x;
  a.ld_y = ld_y;
  a.y_bytes = extent(M, N, ld_y, y_dtype);
  a.p2k = nv ? ldexpf(1.0f, tensor_exp) : 1.0f;
  a.x_kind = x_kind;
  a.nv = nv;
  a.mma = scale_layout == MXFP4_LAYOUT_MMA;
  a.y_f32 = y_dtype == MXFP4_DTYPE_F32;
  return from_cuda(mx::launch_gemv(a, static_cast<cudaStream_t>(stream)), fn);
}

namespace {
constexpr int64_t kMaxBlocks = (int64_t)1 << 31;  // pages * 2 * heads

mxfp4_status check_cache(const char* fn, const mxfp8_cache* c, const mxfp8_cache_batch* b, bool lens, mx::CacheArgs* o) {
  if (!c || !b) return fail(MXFP4_ERR_INVALID_ARG, "%s: cache and batch must be non-NULL", fn);
  if (c->page_tokens != 16 && c->page_tokens != 32 && c->page_tokens != 64 && c->page_tokens != 128)
    return fail(MXFP4_ERR_SHAPE, "%s: page_tokens (%d) must be 16, 32, 64 or 128", fn, c->page_tokens);
  if (c->head_dim != 64 && c->head_dim != 96 && c->head_dim != 128 && c->head_dim != 192 && c->head_dim != 256)
    return fail(MXFP4_ERR_SHAPE, "%s: head_dim (%d) must be 64, 96, 128, 192 or 256", fn, c->head_dim);
  if (c->heads < 1 || c->heads > 32767)
    return fail(MXFP4_ERR_SHAPE, "%s: heads (%d) must be 1 to 32767", fn, c->heads);
  if (c->pages < 0 || c->pages >= kMaxBlocks / (2 * c->heads))
    return fail(MXFP4_ERR_SHAPE, "%s: pages (%lld) must be >= 0 with fewer than 2^31 blocks", fn, (long long)c->pages);
  if (b->sequences < 0 || b->sequences > 65535)
    return fail(MXFP4_ERR_SHAPE, "%s: sequences (%lld) must be 0 to 65535", fn, (long long)b->sequences);
  if (b->tokens < 0 || b->tokens >= (1 << 24))
    return fail(MXFP4_ERR_SHAPE, "%s: tokens (%lld) must be >= 0 and below 2^24", fn, (long long)b->tokens);
  if (b->max_pages < 0 || b->max_pages >= (1 << 30) / c->page_tokens)
    return fail(MXFP4_ERR_SHAPE, "%s: max_pages (%lld) * page_tokens must be below 2^30", fn, (long long)b->max_pages);
  if (b->ld_table < b->max_pages || b->ld_table > kMaxElems)
    return fail(MXFP4_ERR_SHAPE, "%s: ld_table (%lld) < max_pages, or too large", fn, (long long)b->ld_table);
  if (!b->starts && b->tokens != b->sequences)
    return fail(MXFP4_ERR_SHAPE, "%s: without starts tokens (%lld) must equal sequences (%lld)", fn, (long long)b->tokens,
                (long long)b->sequences);
  const int64_t blocks = c->pages * 2 * c->heads;
  if (blocks > 0 && (!c->codes || !c->scales))
    return fail(MXFP4_ERR_INVALID_ARG, "%s: codes and scales must be non-NULL", fn);
  if (b->sequences > 0 && ((b->max_pages > 0 && !b->page_table) || (lens && !b->lens)))
    return fail(MXFP4_ERR_INVALID_ARG, "%s: page_table and lens must be non-NULL", fn);
  if (!aligned16(c->codes)) return fail(MXFP4_ERR_ALIGN, "%s: codes must be 16-byte aligned", fn);
  if ((reinterpret_cast<uintptr_t>(b->page_table) | reinterpret_cast<uintptr_t>(b->lens) |
       reinterpret_cast<uintptr_t>(b->starts)) & 3u)
    return fail(MXFP4_ERR_ALIGN, "%s: page_table, lens and starts must be 4-byte aligned", fn);
  o->codes = c->codes;
  o->scales = c->scales;
  o->table = b->page_table;
  o->lens = b->lens;
  o->starts = b->starts;
  o->ld_table = b->ld_table;
  o->pages = (int32_t)c->pages;
  o->heads = c->heads;
  o->page_tokens = c->page_tokens;
  o->head_dim = c->head_dim;
  o->max_pages = (int32_t)b->max_pages;
  o->sequences = (int32_t)b->sequences;
  o->tokens = (int32_t)b->tokens;
  const int64_t cb = blocks * c->page_tokens * c->head_dim;
  o->codes_bytes = (uint64_t)(cb > g_extent_shrink ? cb - g_extent_shrink : 0);
  o->scales_bytes = (uint64_t)(blocks > g_extent_shrink ? blocks - g_extent_shrink : 0);
  return MXFP4_OK;
}

// A [tokens, heads, head_dim] tensor; an output's rows may not overlap.
mxfp4_status check_heads(const char* fn, const char* name, const mxfp8_heads* t, int64_t tokens, int32_t heads,
                         int32_t head_dim, bool out, mx::Heads* o) {
  if (!t) return fail(MXFP4_ERR_INVALID_ARG, "%s: %s is NULL", fn, name);
  if (t->dtype != MXFP4_DTYPE_BF16 && t->dtype != MXFP4_DTYPE_F32)
    return fail(MXFP4_ERR_INVALID_ARG, "%s: bad dtype %d of %s", fn, t->dtype, name);
  if (!t->p && tokens > 0) return fail(MXFP4_ERR_INVALID_ARG, "%s: %s is NULL", fn, name);
  // (the stride of a single head or a single row is not used)
  const int64_t ld_h = heads > 1 ? t->ld_head : head_dim, ld_t = tokens > 1 ? t->ld_token : 0;
  if (ld_h < head_dim || ld_h > kMaxElems || ld_t < 0 || ld_t > kMaxElems || (heads > 1 && too_large(heads, ld_h)) ||
      (tokens > 1 && ld_t > 0 && too_large(tokens, ld_t)))
    return fail(MXFP4_ERR_SHAPE, "%s: strides (%lld, %lld) of %s out of range (head_dim %d)", fn, (long long)t->ld_token,
                (long long)t->ld_head, name, head_dim);
  // disjoint: rows behind one another's heads, or heads behind one another's rows
  if (tokens > 1 && (out ? ld_t < (heads - 1) * ld_h + head_dim && (ld_t < head_dim || ld_h < (tokens - 1) * ld_t + head_dim)
                         : false))
    return fail(MXFP4_ERR_SHAPE, "%s: rows of %s overlap (strides %lld, %lld)", fn, name, (long long)t->ld_token,
                (long long)t->ld_head);
  if (!aligned16(t->p) || ld_h % 8 != 0 || ld_t % 8 != 0)
    return fail(MXFP4_ERR_ALIGN, "%s: %s must be 16-byte aligned with strides %% 8 == 0", fn, name);
  o->p = t->p;
  o->ld_t = ld_t;
  o->ld_h = ld_h;
  const int64_t n = tokens > 0 ? ((tokens - 1) * ld_t + (heads - 1) * ld_h + head_dim) * elem_bytes(t->dtype) : 0;
  o->bytes = (uint64_t)(n > g_extent_shrink ? n - g_extent_shrink : 0);
  return MXFP4_OK;
}

// Keys and values, in one dtype.
mxfp4_status check_pair(const char* fn, const mxfp8_heads* k, const mxfp8_heads* v, const mx::CacheArgs& c, bool out,
                        mx::Heads* ok, mx::Heads* ov) {
  mxfp4_status st = check_heads(fn, "k", k, c.tokens, c.heads, c.head_dim, out, ok);
  if (!st) st = check_heads(fn, "v", v, c.tokens, c.heads, c.head_dim, out, ov);
  if (!st && k->dtype != v->dtype) return fail(MXFP4_ERR_INVALID_ARG, "%s: k and v must have one dtype", fn);
  return st;
}
}  // namespace

mxfp4_status mxfp8_cache_append(const mxfp8_cache* cache, const mxfp8_cache_batch* batch, const mxfp8_heads* k,
                                const mxfp8_heads* v, void* stream) {
  const char* fn = "mxfp8_cache_append";
  mx::CacheArgs c{};
  mx::Heads hk{}, hv{};
  mxfp4_status st = check_cache(fn, cache, batch, true, &c);
  if (!st) st = check_pair(fn, k, v, c, false, &hk, &hv);
  if (st) return st;
  return from_cuda(mx::launch_cache_append(c, hk, hv, k->dtype == MXFP4_DTYPE_F32, static_cast<cudaStream_t>(stream)), fn);
}

mxfp4_status mxfp8_cache_read(const mxfp8_cache* cache, const mxfp8_cache_batch* batch, const mxfp8_heads* k,
                              const mxfp8_heads* v, void* stream) {
  const char* fn = "mxfp8_cache_read";
  mx::CacheArgs c{};
  mx::Heads hk{}, hv{};
  mxfp4_status st = check_cache(fn, cache, batch, false, &c);
  if (st) return st;
  if (!c.starts && c.sequences > 0) return fail(MXFP4_ERR_INVALID_ARG, "%s: starts is NULL", fn);
  if ((st = check_pair(fn, k, v, c, true, &hk, &hv))) return st;
  return from_cuda(mx::launch_cache_read(c, hk, hv, k->dtype == MXFP4_DTYPE_F32, static_cast<cudaStream_t>(stream)), fn);
}

namespace {
mxfp4_status check_q_heads(const char* fn, mx::AttentionArgs* a, int32_t q_heads, int32_t window) {
  const mx::CacheArgs& c = a->c;
  if (q_heads < 1 || q_heads > 65535 || q_heads % c.heads != 0)
    return fail(MXFP4_ERR_SHAPE, "%s: q_heads (%d) must be a multiple of heads (%d), 1 to 65535", fn, q_heads, c.heads);
  if ((int64_t)c.tokens * q_heads >= (int64_t)1 << 30)
    return fail(MXFP4_ERR_SHAPE, "%s: tokens (%d) * q_heads (%d) must be below 2^30", fn, c.tokens, q_heads);
  a->q_heads = q_heads;
  a->group = q_heads / c.heads;
  // l = ceil(log2 group), floor(2^32 (2^l - group) / group) + 1
  const int l = a->group > 1 ? 32 - __builtin_clz((unsigned)a->group - 1) : 0;
  a->group_mul = (uint32_t)(((((uint64_t)1 << l) - (uint64_t)a->group) << 32) / (uint64_t)a->group + 1);
  a->group_shift[0] = l < 1 ? 0 : 1;
  a->group_shift[1] = (uint8_t)(l > 1 ? l - 1 : 0);
  a->spare = c.sequences > 1;
  a->shift = c.page_tokens == 16 ? 4 : c.page_tokens == 32 ? 5 : c.page_tokens == 64 ? 6 : 7;
  a->window = window < (1 << 30) ? window : 1 << 30;  // (no length passes it)
  return MXFP4_OK;
}
}  // namespace

size_t mxfp8_cache_attention_workspace_size(const mxfp8_cache* cache, const mxfp8_cache_batch* batch, int32_t q_heads) {
  const char* fn = "mxfp8_cache_attention_workspace_size";
  mx::AttentionArgs a{};
  // (sizes alone count: no pointer is looked at)
  if (!cache || !batch) return 0;
  mxfp8_cache c = *cache;
  mxfp8_cache_batch b = *batch;
  c.codes = c.scales = reinterpret_cast<uint8_t*>(16);
  b.page_table = b.lens = reinterpret_cast<const int32_t*>(16);
  if (check_cache(fn, &c, &b, true, &a.c) || check_q_heads(fn, &a, q_heads, 0)) return 0;
  return (size_t)mx::cache_attention_workspace_bytes(a);
}

mxfp4_status mxfp8_cache_attention(const mxfp8_cache* cache, const mxfp8_cache_batch* batch, const mxfp8_heads* q,
                                   int32_t q_heads, const mxfp8_attention_params* params, const mxfp8_heads* out,
                                   float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "mxfp8_cache_attention";
  mx::AttentionArgs a{};
  mxfp4_status st = check_cache(fn, cache, batch, true, &a.c);
  if (st) return st;
  if (!params) return fail(MXFP4_ERR_INVALID_ARG, "%s: params is NULL", fn);
  if (params->window < 0) return fail(MXFP4_ERR_INVALID_ARG, "%s: window (%d) must be >= 0", fn, params->window);
  if ((st = check_q_heads(fn, &a, q_heads, params->window))) return st;
  if (mx::cache_attention_units(a) >= mx::kMostUnits)
    return fail(MXFP4_ERR_SHAPE, "%s: too many tokens (%d) of %d heads over %d pages for one call", fn, a.c.tokens, q_heads,
                a.c.max_pages);
  if (!(params->scale >= -1.0e30f && params->scale <= 1.0e30f))
    return fail(MXFP4_ERR_INVALID_ARG, "%s: scale must be finite", fn);
  if (!(params->softcap == 0.0f || (params->softcap >= 1.0e-30f && params->softcap <= 1.0e30f)))
    return fail(MXFP4_ERR_INVALID_ARG, "%s: softcap must be 0 or a positive number", fn);
  // (what the kernel multiplies by; an infinity would make scores of 0 no numbers)
  if (params->softcap > 0.0f && std::fabs((double)params->scale) > 1.0e30 * (double)params->softcap)
    return fail(MXFP4_ERR_INVALID_ARG, "%s: scale / softcap must be at most 1e30 (got %g / %g)", fn, params->scale,
                params->softcap);
  if ((reinterpret_cast<uintptr_t>(params->slopes) | reinterpret_cast<uintptr_t>(lse)) & 3u)
    return fail(MXFP4_ERR_ALIGN, "%s: slopes and lse must be 4-byte aligned", fn);
  if ((st = check_heads(fn, "q", q, a.c.tokens, q_heads, a.c.head_dim, false, &a.q))) return st;
  if (q->dtype != MXFP4_DTYPE_BF16) return fail(MXFP4_ERR_INVALID_ARG, "%s: q must be bf16", fn);
  if ((st = check_heads(fn, "out", out, a.c.tokens, q_heads, a.c.head_dim, true, &a.out))) return st;
  if (!aligned16(workspace)) return fail(MXFP4_ERR_ALIGN, "%s: workspace must be 16-byte aligned", fn);
  const size_t need = (size_t)mx::cache_attention_workspace_bytes(a);
  if (need && (!workspace || workspace_bytes < need))
    return fail(MXFP4_ERR_INVALID_ARG, "%s: workspace of %zu bytes, %zu are needed", fn, workspace ? workspace_bytes : 0,
                need);
  a.ws = need ? static_cast<float*>(workspace) : nullptr;  // (one that no call asked for is not written)
  a.ws_bytes = need;
  a.lse = lse;
  const int64_t n = (int64_t)a.c.tokens * q_heads * 4;
  a.lse_bytes = (uint64_t)(n > g_extent_shrink ? n - g_extent_shrink : 0);
  a.slopes = params->slopes;
  a.scale = params->scale;
  a.softcap = params->softcap;
  a.out_f32 = out->dtype == MXFP4_DTYPE_F32;
  return from_cuda(mx::launch_cache_attention(a, static_cast<cudaStream_t>(stream)), fn);
}

mxfp4_status mxfp4_device_status(void* stream) {
  uint32_t err = 0;
  cudaError_t e = mx::read_device_error(static_cast<cudaStream_t>(stream), &err);
  if (e != cudaSuccess) return from_cuda(e, "mxfp4_device_status");
  if (err == MXFP4_ERR_TIMEOUT)
    return fail(MXFP4_ERR_TIMEOUT, "a bounded device-side wait ran out");
  if (err == MXFP4_ERR_BOUNDS)
    return fail(MXFP4_ERR_BOUNDS, "a kernel store fell outside its output (skipped)");
  if (err == MXFP4_ERR_INVALID_ARG)
    return fail(MXFP4_ERR_INVALID_ARG, "a cache call met a page, a length or a row start outside its range (skipped)");
  return err ? fail(static_cast<mxfp4_status>(err), "device error word %u", err) : MXFP4_OK;
}

mxfp4_status mxfp4_bounds_check_shrink(int64_t bytes) {
#ifdef MXFP4_BOUNDS_CHECK
  if (bytes < 0) return fail(MXFP4_ERR_INVALID_ARG, "mxfp4_bounds_check_shrink: negative bytes");
  g_extent_shrink = bytes;
  return MXFP4_OK;
#else
  (void)bytes;
  return fail(MXFP4_ERR_UNSUPPORTED, "mxfp4_bounds_check_shrink: not a bounds-checking build");
#endif
}

mxfp4_status mxfp4_selftest_wait_timeout(void* stream) {
  cudaError_t e = mx::launch_wait_probe(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return from_cuda(e, "mxfp4_selftest_wait_timeout");
  return MXFP4_OK;
}

mxfp4_status mxfp8_selftest_cache_wait_timeout(void* stream) {
  return from_cuda(mx::launch_cache_wait_probe(static_cast<cudaStream_t>(stream)), "mxfp8_selftest_cache_wait_timeout");
}

}  // extern "C"
