// row_device.cuh -- eight-element vectors and row-wise quantization of values
// held eight to a lane (the norm and activation kernels, sm_103a).
#pragma once
#include <cstdint>

#include "internal.h"
#include "mx_device.cuh"

#ifndef MX_BOUNDS_FAIL
#error "define MX_BOUNDS_FAIL() before including row_device.cuh"
#endif

namespace mx {

// Eight consecutive elements as they lie in memory: bf16 (uint16_t) 16 bytes,
// fp32 32 bytes.
template <typename T>
struct Vec8;
template <>
struct Vec8<uint16_t> {
  uint4 a;
};
template <>
struct Vec8<float> {
  uint4 a, b;
};

// Loads of data that the kernel reads once. Not the read-only path: an output
// may lie in place of an input.
__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void load8(const uint16_t* p, Vec8<uint16_t>& v) { v.a = load16(p); }
// Sixteen bf16 or fp32 elements of a row, 16 (or, where `wide`, 32) bytes at a
// time; p 16-byte (32-byte) aligned.
struct Vec16B {
  uint4 a, b;
};
__device__ __forceinline__ Vec16B load32(const void* p, bool wide) {
  Vec16B v;
  if (wide) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v.a.x), "=r"(v.a.y), "=r"(v.a.z), "=r"(v.a.w), "=r"(v.b.x), "=r"(v.b.y), "=r"(v.b.z),
                   "=r"(v.b.w)
                 : "l"(p)
                 : "memory");
  } else {
    v.a = load16(p);
    v.b = load16(static_cast<const uint8_t*>(p) + 16);
  }
  return v;
}
// Eight fp32 elements at once where they lie on a 32-byte boundary: the two halves
// of a sector loaded (or stored) apart move it twice (SwiGLU's gradient, fp32
// 4452 x 13184: 251 us apart, 165 at once; norm, 4096 x 8192: 75 and 69).
__device__ __forceinline__ bool on32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }
__device__ __forceinline__ void load8(const float* p, Vec8<float>& v) {
  const Vec16B w = load32(p, on32(p));
  v.a = w.a;
  v.b = w.b;
}
// The same without the case: a lane with many loads to issue has the second halves
// close enough behind the first to find their sectors, and the cases between them
// cost more (norm gradient, fp32 16384 x 512: 20 us, 24.6 with load8).
__device__ __forceinline__ void load8_apart(const uint16_t* p, Vec8<uint16_t>& v) { load8(p, v); }
__device__ __forceinline__ void load8_apart(const float* p, Vec8<float>& v) {
  v.a = load16(p);
  v.b = load16(p + 4);
}
template <typename T>
struct Vec16;
template <>
struct Vec16<uint16_t> {
  Vec16B v;
};
template <>
struct Vec16<float> {
  Vec16B v[2];
};
__device__ __forceinline__ void load16e(const uint16_t* p, bool wide, Vec16<uint16_t>& o) { o.v = load32(p, wide); }
__device__ __forceinline__ void load16e(const float* p, bool wide, Vec16<float>& o) {
  o.v[0] = load32(p, wide);
  o.v[1] = load32(p + 8, wide);
}
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ void unpack16(const Vec16<uint16_t>& o, float2 (&f)[8]) {
  const uint32_t w[8] = {o.v.a.x, o.v.a.y, o.v.a.z, o.v.a.w, o.v.b.x, o.v.b.y, o.v.b.z, o.v.b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = unpack2(w[i]);
}
__device__ __forceinline__ void unpack16(const Vec16<float>& o, float2 (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const Vec16B& v = o.v[i];
    f[4 * i] = make_float2(__uint_as_float(v.a.x), __uint_as_float(v.a.y));
    f[4 * i + 1] = make_float2(__uint_as_float(v.a.z), __uint_as_float(v.a.w));
    f[4 * i + 2] = make_float2(__uint_as_float(v.b.x), __uint_as_float(v.b.y));
    f[4 * i + 3] = make_float2(__uint_as_float(v.b.z), __uint_as_float(v.b.w));
  }
}

// Loads of data that other rows read again (weights).
__device__ __forceinline__ void load8_cached(const uint16_t* p, Vec8<uint16_t>& v) {
  v.a = __ldg(reinterpret_cast<const uint4*>(p));
}
__device__ __forceinline__ void load8_cached(const float* p, Vec8<float>& v) {
  v.a = __ldg(reinterpret_cast<const uint4*>(p));
  v.b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
}

__device__ __forceinline__ void unpack8(const Vec8<uint16_t>& v, float (&f)[8]) {
  const uint32_t w[4] = {v.a.x, v.a.y, v.a.z, v.a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void unpack8(const Vec8<float>& v, float (&f)[8]) {
  const uint32_t w[8] = {v.a.x, v.a.y, v.a.z, v.a.w, v.b.x, v.b.y, v.b.z, v.b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
}

// Two fp32 values to a bf16 pair, nearest-even (a in the low half).
__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ void pack8(const float (&f)[8], Vec8<uint16_t>& v) {
  v.a = make_uint4(bf16x2(f[0], f[1]), bf16x2(f[2], f[3]), bf16x2(f[4], f[5]), bf16x2(f[6], f[7]));
}
__device__ __forceinline__ void pack8(const float (&f)[8], Vec8<float>& v) {
  v.a = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  v.b = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
}

// Stores v at p; bounds-checking builds skip and report a store outside the
// `bytes` bytes at base.
template <typename V>
__device__ __forceinline__ void put_at(void* p, const V& v, const void* base, uint64_t bytes) {
#ifdef MXFP4_BOUNDS_CHECK
  const uint8_t *b = static_cast<const uint8_t*>(base), *a = static_cast<const uint8_t*>(p);
  if (a < b || a + sizeof(V) > b + bytes) {
    MX_BOUNDS_FAIL();
    return;
  }
#else
  (void)base;
  (void)bytes;
#endif
  *static_cast<V*>(p) = v;
}
__device__ __forceinline__ void store8(uint16_t* p, const Vec8<uint16_t>& v, const void* base, uint64_t bytes) {
  put_at(p, v.a, base, bytes);
}
__device__ __forceinline__ void store8(float* p, const Vec8<float>& v, const void* base, uint64_t bytes) {
#ifndef MXFP4_BOUNDS_CHECK
  if (on32(p)) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v.a.x), "r"(v.a.y), "r"(v.a.z),
                 "r"(v.a.w), "r"(v.b.x), "r"(v.b.y), "r"(v.b.z), "r"(v.b.w)
                 : "memory");
    return;
  }
#endif
  put_at(p, v.a, base, bytes);
  put_at(p + 4, v.b, base, bytes);
}
// Eight fp32 values to a matrix of bf16 or fp32 elements.
__device__ __forceinline__ void store8_as(void* base, bool f32, int64_t at, const float (&f)[8], uint64_t bytes) {
  if (f32) {
    Vec8<float> v;
    pack8(f, v);
    store8(static_cast<float*>(base) + at, v, base, bytes);
  } else {
    Vec8<uint16_t> v;
    pack8(f, v);
    store8(static_cast<uint16_t*>(base) + at, v, base, bytes);
  }
}

// Largest of three magnitudes; NaN if one of them is.
__device__ __forceinline__ float absmax3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)), "f"(fabsf(c)));
  return r;
}

// Where the codes and scales of one output row lie.
struct RowOut {
  uint8_t *q, *s;
};
__device__ __forceinline__ RowOut row_out(const RowQuant& o, int64_t row, int64_t cols) {
  RowOut r;
  const int64_t nkb = o.fmt == RowQuant::kNvfp4 ? cols >> 4 : cols >> 5;
  r.q = o.q + (o.fmt == RowQuant::kE4m3 || o.fmt == RowQuant::kE5m2 ? row * cols : (row * cols) >> 1);
  r.s = o.s + (o.mma ? mma_scale_offset(row, 0, nkb) : row * nkb);
  return r;
}

// The scale of a block with max-abs m (NaN or infinity: the format's NaN):
// its code and the factor that brings the block into the elements' range.
struct BlockScale {
  uint32_t code;
  float mul;
  bool bad;
};
__device__ __forceinline__ BlockScale block_scale(const RowQuant& o, float m) {
  BlockScale r;
  const uint32_t b = __float_as_uint(m);
  r.bad = b >= 0x7F800000u;
  if (o.fmt == RowQuant::kNvfp4) {
    const NvScale s = nv_scale(r.bad ? 0.0f : m, o.roundup, o.p2k, o.zmul);
    r.code = r.bad ? 0x7Fu : s.code;
    r.mul = s.rcp;
  } else {
    // scale_exponent() with the format's constants at hand: the exponent field
    // less emax, one more where the fraction passes the format's largest value
    const int e = max((int)(b >> 23) - o.emax + ((b & 0x7FFFFFu) > o.over ? 1 : 0), 0);
    r.code = r.bad ? 0xFFu : (uint32_t)e;
    r.mul = __uint_as_float((uint32_t)(254 - e) << 23);
  }
  return r;
}

// Stores the scale of the block at column col, held by lane 0 of its `lanes`
// lanes; with o.packed four neighbouring blocks' scales as one word.
__device__ __forceinline__ void store_scale(const RowQuant& o, const RowOut& out, uint32_t code, int lanes,
                                            uint32_t col, bool live) {
  const bool nv = o.fmt == RowQuant::kNvfp4;
  const uint32_t kb = nv ? col >> 4 : col >> 5, at = o.mma ? ((kb >> 2) << 9) + (kb & 3) : kb;
  live = live && (col & (nv ? 15 : 31)) == 0;
  if (o.packed) {
    code |= __shfl_down_sync(0xffffffffu, code, lanes) << 8;
    code |= __shfl_down_sync(0xffffffffu, code, 2 * lanes) << 16;
    if (live && (kb & 3) == 0) put_at(out.s + at, code, o.s, o.s_bytes);
  } else if (live) {
    put_at(out.s + at, (uint8_t)code, o.s, o.s_bytes);
  }
}

// Quantizes the eight values f that this lane holds of one output row, columns
// col .. col + 7, and stores codes and scales. Lanes 4 i .. 4 i + 3 of the warp
// hold one 32-run (columns of a multiple of 32 first), so a block's max-abs is
// two exchanges away (one for 1x16 blocks). Every lane of the warp calls this;
// one with `live` false holds zeros and stores nothing. The maximum keeps a
// NaN: a block that holds an infinity or a NaN gets the scale format's NaN as
// its scale and zero codes, and so dequantizes to NaN.
__device__ __forceinline__ void quantize8(const RowQuant& o, float (&f)[8], bool live, const RowOut& out,
                                          uint32_t col) {
  const bool nv = o.fmt == RowQuant::kNvfp4;
  float m = absmax3_nan(absmax3_nan(f[0], f[1], f[2]), absmax3_nan(f[3], f[4], f[5]), absmax3_nan(f[6], f[7], 0.0f));
  m = absmax3_nan(m, __shfl_xor_sync(0xffffffffu, m, 1), 0.0f);
  if (!nv) m = absmax3_nan(m, __shfl_xor_sync(0xffffffffu, m, 2), 0.0f);
  const BlockScale s = block_scale(o, m);
  if (s.bad) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 0.0f;
  }
  const float2 mm = make_float2(s.mul, s.mul);
  const float2 a = f2mul(make_float2(f[0], f[1]), mm), b = f2mul(make_float2(f[2], f[3]), mm),
               c = f2mul(make_float2(f[4], f[5]), mm), d = f2mul(make_float2(f[6], f[7]), mm);
  if (live) {
    if (o.fmt == RowQuant::kE4m3)
      put_at(out.q + col, make_uint2(e4m3x4(a.x, a.y, b.x, b.y), e4m3x4(c.x, c.y, d.x, d.y)), o.q, o.q_bytes);
    else if (o.fmt == RowQuant::kE5m2)
      put_at(out.q + col, make_uint2(e5m2x4(a.x, a.y, b.x, b.y), e5m2x4(c.x, c.y, d.x, d.y)), o.q, o.q_bytes);
    else
      put_at(out.q + (col >> 1), e2m1x8(a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y), o.q, o.q_bytes);
  }
  store_scale(o, out, s.code, nv ? 2 : 4, col, live);
}

// The same for sixteen values a lane (columns col .. col + 15, as pairs): two
// lanes a 32-run, one a 1x16 block. Half the scale arithmetic and stores per
// element.
__device__ __forceinline__ void quantize16(const RowQuant& o, float2 (&f)[8], bool live, const RowOut& out,
                                           uint32_t col) {
  const bool nv = o.fmt == RowQuant::kNvfp4;
  float m = absmax3_nan(f[7].y, f[0].x, f[0].y);
#pragma unroll
  for (int i = 1; i < 7; ++i) m = absmax3_nan(m, f[i].x, f[i].y);
  m = absmax3_nan(m, f[7].x, nv ? 0.0f : __shfl_xor_sync(0xffffffffu, absmax3_nan(m, f[7].x, 0.0f), 1));
  const BlockScale s = block_scale(o, m);
  if (s.bad) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = make_float2(0.0f, 0.0f);
  }
  const float2 mm = make_float2(s.mul, s.mul);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = f2mul(f[i], mm);
  if (live) {
    if (o.fmt == RowQuant::kE4m3 || o.fmt == RowQuant::kE5m2)
      put_at(out.q + col, encode16_fp8(f, o.fmt == RowQuant::kE5m2), o.q, o.q_bytes);
    else
      put_at(out.q + (col >> 1), encode16(f), o.q, o.q_bytes);
  }
  store_scale(o, out, s.code, nv ? 1 : 2, col, live);
}

}  // namespace mx
