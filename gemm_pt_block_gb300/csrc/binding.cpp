// binding.cpp -- the norm, activation and few-row calls from Python: checks of
// tensors, outputs and workspaces that the caller did not pass, and the call of
// the C ABI, in one C++ function each. These calls are small (a decode step
// makes several a layer), and the same work in Python took 15 to 35 us, more
// than most of their kernels. Nothing here computes; the library's functions
// come as a table of addresses, so that any build of it can be called.
#include "binding_util.h"

namespace {

// The library's functions.
struct Table {
  decltype(&mxfp4_rmsnorm_quantize) norm;
  decltype(&mxfp4_rmsnorm_backward) norm_backward;
  decltype(&mxfp4_rmsnorm_backward_workspace_size) norm_workspace;
  decltype(&mxfp4_swiglu_quantize) swiglu;
  decltype(&mxfp4_swiglu_backward) swiglu_backward;
  decltype(&mxfp4_gemv_ex) gemv;
  decltype(&mxfp4_gemv_workspace_size) gemv_workspace;
};
constexpr int kFunctions = sizeof(Table) / sizeof(void*);
const Table& table(PyObject* o) { return table_at<Table>(o); }

// The attributes of QuantParams, as the interpreter's own strings.
enum Field { kBlock, kScaleMode, kRounding, kScaleLayout, kWht, kSignMask, kSeed, kSrStream, kElemFormat, kTensorExp, kFields };
const char* const field_names[kFields] = {"block",         "scale_mode", "rounding",  "scale_layout", "wht",
                                          "wht_sign_mask", "seed",       "sr_stream", "elem_format",  "tensor_exp"};
PyObject* fields[kFields];

int64_t field(PyObject* o, Field f) {
  PyObject* v = PyObject_GetAttr(o, fields[f]);
  if (!v) throw Raised{};
  const unsigned long long n = PyLong_AsUnsignedLongLongMask(v);
  Py_DECREF(v);
  if (n == (unsigned long long)-1 && PyErr_Occurred()) throw Raised{};
  return (int64_t)n;
}

mxfp4_quant_params params(PyObject* o) {
  mxfp4_quant_params p{};
  p.block = (int32_t)field(o, kBlock);
  p.scale_mode = (int32_t)field(o, kScaleMode);
  p.rounding = (int32_t)field(o, kRounding);
  p.scale_layout = (int32_t)field(o, kScaleLayout);
  p.wht = field(o, kWht) != 0;
  p.wht_sign_mask = (uint32_t)field(o, kSignMask);
  p.seed = (uint64_t)field(o, kSeed);
  p.sr_stream = (uint32_t)field(o, kSrStream);
  p.elem_format = (uint32_t)field(o, kElemFormat);
  p.tensor_exp = (int32_t)field(o, kTensorExp);
  return p;
}

int64_t scale_cols(int32_t block, int64_t k) { return block == MXFP4_BLOCK_1X16 ? k / 16 : k / 32; }

// The quantized output (None: not asked for): its parameters, and its codes and
// scales allocated or checked.
struct Quantized {
  bool on = false;
  mxfp4_quant_params p{};
  at::Tensor q, s;
  const mxfp4_quant_params* params() const { return on ? &p : nullptr; }
  uint8_t* codes() { return on ? static_cast<uint8_t*>(q.data_ptr()) : nullptr; }
  uint8_t* scales() { return on ? static_cast<uint8_t*>(s.data_ptr()) : nullptr; }
};
Quantized quantized(PyObject* row, PyObject* q, PyObject* s, const Shape& sh, const at::Tensor& like) {
  Quantized r;
  if (!given(row)) return r;
  r.on = true;
  r.p = params(row);
  const bool bytes = r.p.elem_format == MXFP4_FORMAT_E4M3 || r.p.elem_format == MXFP4_FORMAT_E5M2;
  const int64_t qc = bytes ? sh.cols : sh.cols / 2, sc = scale_cols(r.p.block, sh.cols);
  if (given(q)) {
    r.q = tensor(q, "q");
    dense(r.q, "q", sh.rows * qc, at::kByte, sh.dev);
  } else {
    r.q = empty({sh.rows, qc}, at::kByte, like);
  }
  if (given(s)) {
    r.s = tensor(s, "s");
    dense(r.s, "s", sh.rows * sc, at::kByte, sh.dev);
  } else if (r.p.scale_layout == MXFP4_LAYOUT_MMA) {
    r.s = empty({sh.rows * sc}, at::kByte, like);
  } else {
    r.s = empty({sh.rows, sc}, at::kByte, like);
  }
  return r;
}

// An optional matrix output: given, wanted in a type, or absent.
struct Out {
  at::Tensor t;
  int64_t ld = 0;
  void* ptr() { return t.defined() ? t.data_ptr() : nullptr; }
};

// (table, x, weight, row, residual, eps, y_dtype, with_rstd, h, y, rstd, q, s)
// -> (q, s, y, h, rstd), or the status of a refused call
PyObject* norm(PyObject* const* a) {
  const Table& lib = table(a[0]);
  const at::Tensor& x = tensor(a[1], "x");
  const Shape sh = shape_of(x, "x");
  const OnDevice current(static_cast<c10::DeviceIndex>(sh.dev));
  const int64_t ldx = rows_ld(x, "x", sh.rows, sh.cols, sh.dev);
  const int32_t dt = dtype_code(x, "x");
  const double eps = PyFloat_AsDouble(a[5]);
  if (eps == -1.0 && PyErr_Occurred()) throw Raised{};
  const void *pw = nullptr, *pr = nullptr;
  int32_t wdt = MXFP4_DTYPE_F32, ydt = MXFP4_DTYPE_F32;
  int64_t ldr = sh.cols;
  Out h, y;
  h.ld = y.ld = sh.cols;
  if (given(a[2])) {
    const at::Tensor& w = tensor(a[2], "weight");
    vector(w, "weight", sh.cols, sh.dev);
    wdt = dtype_code(w, "weight");
    pw = w.data_ptr();
  }
  if (given(a[4])) {
    const at::Tensor& r = tensor(a[4], "residual");
    if (r.scalar_type() != x.scalar_type())
      throw Raise(PyExc_TypeError, "residual must have x's type (got %s)", c10::toString(r.scalar_type()));
    ldr = rows_ld(r, "residual", sh.rows, sh.cols, sh.dev);
    pr = r.data_ptr();
  }
  if (given(a[8])) {
    h.t = tensor(a[8], "h");
    if (h.t.scalar_type() != x.scalar_type())
      throw Raise(PyExc_TypeError, "h must have x's type (got %s)", c10::toString(h.t.scalar_type()));
    h.ld = rows_ld(h.t, "h", sh.rows, sh.cols, sh.dev);
  } else if (given(a[4])) {
    h.t = empty({sh.rows, sh.cols}, x.scalar_type(), x);
  }
  if (given(a[9])) {
    y.t = tensor(a[9], "y");
    y.ld = rows_ld(y.t, "y", sh.rows, sh.cols, sh.dev);
  } else if (given(a[6])) {
    const at::ScalarType t = scalar_type(a[6], "y_dtype");
    dtype_code(t, "y");
    y.t = empty({sh.rows, sh.cols}, t, x);
  }
  if (y.t.defined()) ydt = dtype_code(y.t, "y");
  at::Tensor rstd;
  if (given(a[10])) {
    rstd = tensor(a[10], "rstd");
    dense(rstd, "rstd", sh.rows, at::kFloat, sh.dev);
  } else if (truth(a[7])) {
    rstd = empty({sh.rows}, at::kFloat, x);
  }
  Quantized z = quantized(a[3], a[11], a[12], sh, x);
  const mxfp4_status st =
      call(lib.norm, x.data_ptr(), dt, sh.rows, sh.cols, ldx, pr, ldr, pw, wdt, (float)eps, h.ptr(), h.ld, y.ptr(), ydt,
           y.ld, rstd.defined() ? static_cast<float*>(rstd.data_ptr()) : nullptr, z.params(), z.codes(), z.scales(),
           stream_of(sh.dev));
  if (st) return PyLong_FromLong(st);
  return tuple({&z.q, &z.s, &y.t, &h.t, &rstd});
}

// (table, dy, h, weight, rstd, dh, dx, dw, with_dw, workspace) -> (dx, dw)
PyObject* norm_backward(PyObject* const* a) {
  const Table& lib = table(a[0]);
  const at::Tensor& h = tensor(a[2], "h");
  const Shape sh = shape_of(h, "h");
  const OnDevice current(static_cast<c10::DeviceIndex>(sh.dev));
  const int64_t ldh = rows_ld(h, "h", sh.rows, sh.cols, sh.dev);
  const int32_t hdt = dtype_code(h, "h");
  const at::Tensor& dy = tensor(a[1], "dy");
  const int64_t ldy = rows_ld(dy, "dy", sh.rows, sh.cols, sh.dev);
  const int32_t ydt = dtype_code(dy, "dy");
  const at::Tensor& rstd = tensor(a[4], "rstd");
  dense(rstd, "rstd", sh.rows, at::kFloat, sh.dev);
  auto of_h = [&](const at::Tensor& t, const char* name) {
    if (t.scalar_type() != h.scalar_type())
      throw Raise(PyExc_TypeError, "%s must have h's type (got %s)", name, c10::toString(t.scalar_type()));
    return rows_ld(t, name, sh.rows, sh.cols, sh.dev);
  };
  const void *pd = nullptr, *pw = nullptr;
  int64_t ldd = sh.cols;
  if (given(a[5])) {
    const at::Tensor& dh = tensor(a[5], "dh");
    ldd = of_h(dh, "dh");
    pd = dh.data_ptr();
  }
  Out dx;
  dx.ld = sh.cols;
  if (given(a[6])) {
    dx.t = tensor(a[6], "dx");
    dx.ld = of_h(dx.t, "dx");
  } else {
    dx.t = empty({sh.rows, sh.cols}, h.scalar_type(), h);
  }
  at::Tensor dw, ws;
  int32_t wdt = MXFP4_DTYPE_F32;
  size_t need = 0;
  if (given(a[3])) {
    const at::Tensor& w = tensor(a[3], "weight");
    vector(w, "weight", sh.cols, sh.dev);
    wdt = dtype_code(w, "weight");
    pw = w.data_ptr();
    if (given(a[7])) {
      dw = tensor(a[7], "dw");
      dense(dw, "dw", sh.cols, w.scalar_type(), sh.dev);
    } else if (truth(a[8])) {
      dw = empty({sh.cols}, w.scalar_type(), h);
    }
  } else if (given(a[7])) {
    throw Raise(PyExc_ValueError, "dw needs a weight");
  }
  if (dw.defined()) {
    need = lib.norm_workspace(sh.rows, sh.cols);
    if (given(a[9])) {
      ws = tensor(a[9], "workspace");
      dense(ws, "workspace", (int64_t)need, at::kByte, sh.dev);
    } else {
      ws = empty({(int64_t)need}, at::kByte, h);
    }
  }
  const mxfp4_status st =
      call(lib.norm_backward, dy.data_ptr(), ydt, ldy, h.data_ptr(), hdt, ldh, pw, wdt,
           static_cast<const float*>(rstd.data_ptr()), pd, ldd, sh.rows, sh.cols, dx.ptr(), dx.ld,
           dw.defined() ? dw.data_ptr() : nullptr, ws.defined() ? ws.data_ptr() : nullptr, need, stream_of(sh.dev));
  if (st) return PyLong_FromLong(st);
  return tuple({&dx.t, &dw});
}

// (table, gate, up, row, y_dtype, y, q, s) -> (q, s, y)
PyObject* swiglu(PyObject* const* a) {
  const Table& lib = table(a[0]);
  const at::Tensor& g = tensor(a[1], "gate");
  const Shape sh = shape_of(g, "gate");
  const OnDevice current(static_cast<c10::DeviceIndex>(sh.dev));
  const int64_t ldg = rows_ld(g, "gate", sh.rows, sh.cols, sh.dev);
  const int32_t dt = dtype_code(g, "gate");
  const at::Tensor& u = tensor(a[2], "up");
  if (u.scalar_type() != g.scalar_type())
    throw Raise(PyExc_TypeError, "up must have gate's type (got %s)", c10::toString(u.scalar_type()));
  const int64_t ldu = rows_ld(u, "up", sh.rows, sh.cols, sh.dev);
  Out y;
  y.ld = sh.cols;
  if (given(a[5])) {
    y.t = tensor(a[5], "y");
    y.ld = rows_ld(y.t, "y", sh.rows, sh.cols, sh.dev);
  } else if (given(a[4])) {
    const at::ScalarType t = scalar_type(a[4], "y_dtype");
    dtype_code(t, "y");
    y.t = empty({sh.rows, sh.cols}, t, g);
  }
  const int32_t ydt = y.t.defined() ? dtype_code(y.t, "y") : MXFP4_DTYPE_F32;
  Quantized z = quantized(a[3], a[6], a[7], sh, g);
  const mxfp4_status st = call(lib.swiglu, g.data_ptr(), ldg, u.data_ptr(), ldu, dt, sh.rows, sh.cols, y.ptr(), ydt,
                               y.ld, z.params(), z.codes(), z.scales(), stream_of(sh.dev));
  if (st) return PyLong_FromLong(st);
  return tuple({&z.q, &z.s, &y.t});
}

// (table, dy, gate, up, dgate, dup) -> (dgate, dup)
PyObject* swiglu_backward(PyObject* const* a) {
  const Table& lib = table(a[0]);
  const at::Tensor& g = tensor(a[2], "gate");
  const Shape sh = shape_of(g, "gate");
  const OnDevice current(static_cast<c10::DeviceIndex>(sh.dev));
  const int64_t ldg = rows_ld(g, "gate", sh.rows, sh.cols, sh.dev);
  const int32_t dt = dtype_code(g, "gate");
  const at::Tensor& dy = tensor(a[1], "dy");
  const int64_t ldy = rows_ld(dy, "dy", sh.rows, sh.cols, sh.dev);
  const int32_t ydt = dtype_code(dy, "dy");
  auto of_gate = [&](const at::Tensor& t, const char* name) {
    if (t.scalar_type() != g.scalar_type())
      throw Raise(PyExc_TypeError, "%s must have gate's type (got %s)", name, c10::toString(t.scalar_type()));
    return rows_ld(t, name, sh.rows, sh.cols, sh.dev);
  };
  const at::Tensor& u = tensor(a[3], "up");
  const int64_t ldu = of_gate(u, "up");
  const at::Tensor dg = given(a[4]) ? tensor(a[4], "dgate") : empty({sh.rows, sh.cols}, g.scalar_type(), g);
  const at::Tensor du = given(a[5]) ? tensor(a[5], "dup") : empty({sh.rows, sh.cols}, g.scalar_type(), g);
  const int64_t lddg = of_gate(dg, "dgate"), lddu = of_gate(du, "dup");
  const mxfp4_status st =
      call(lib.swiglu_backward, dy.data_ptr(), ydt, ldy, g.data_ptr(), ldg, u.data_ptr(), ldu, dt, sh.rows, sh.cols,
           dg.data_ptr(), lddg, du.data_ptr(), lddu, stream_of(sh.dev));
  if (st) return PyLong_FromLong(st);
  return tuple({&dg, &du});
}

// Weights from which a workspace gains (times without / with, row-major scales,
// bf16 x; tiled scales and MXFP8 x cross at the same sizes):
//  up to 8 rows   4 rows: 8192 x 8192 14.6 / 16.0 us, 28672 x 4096 21.0 / 18.7
//  9 to 16 rows   12 rows: 4096 x 4096 10.7 / 11.0, 8192 x 4096 15.5 / 14.6
//  17 to 32 rows  24 rows (one more tile of digits): 8192 x 4096 16.4 / 17.8,
//                 4096 x 8192 16.6 / 19.3, 11264 x 4096 21.1 / 18.5
//  more           64 rows: 4096 x 4096 16.7 / 18.5, 8192 x 4096 26.5 / 20.5
//  NVFP4 above 8  24 rows: 2048 x 4096 10.5 / 9.6 (less than the second launch
//                 costs the host), 4096 x 4096 11.8 / 10.9
int64_t workspace_from(int64_t rows, bool nv) {
  if (rows <= 8) return (int64_t)3 << 25;
  if (nv) return (int64_t)1 << 24;
  return rows > 16 && rows <= 32 ? (int64_t)5 << 23 : (int64_t)1 << 25;
}

// (table, x, qw, sw, N, K, w, sx, x_format, out_dtype, y, workspace) -> (y,)
PyObject* gemv(PyObject* const* a) {
  const Table& lib = table(a[0]);
  const at::Tensor& x = tensor(a[1], "x");
  const Shape sh = shape_of(x, "x");
  const OnDevice current(static_cast<c10::DeviceIndex>(sh.dev));
  const int64_t M = sh.rows, N = integer(a[4]), K = integer(a[5]);
  const int64_t ldx = rows_ld(x, "x", M, K, sh.dev);
  int32_t block = MXFP4_BLOCK_1X32, layout = MXFP4_LAYOUT_ROWMAJOR, exponent = 0;
  if (given(a[6])) {
    const mxfp4_quant_params w = params(a[6]);
    if (w.elem_format != MXFP4_FORMAT_E2M1) throw Raise(PyExc_ValueError, "the weights must be 4-bit (E2M1) codes");
    block = w.block;
    layout = w.scale_layout;
    exponent = w.tensor_exp;
  }
  int32_t kind = MXFP4_GEMV_X_BF16;
  const uint8_t* psx = nullptr;
  if (x.scalar_type() == at::kBFloat16) {
    if (given(a[7])) throw Raise(PyExc_ValueError, "sx goes with one-byte codes; x is bfloat16");
  } else if (x.scalar_type() == at::kByte) {
    if (!given(a[7])) throw Raise(PyExc_ValueError, "one-byte codes need their scales sx");
    const int64_t f = integer(a[8]);
    if (f != MXFP4_FORMAT_E4M3 && f != MXFP4_FORMAT_E5M2)
      throw Raise(PyExc_ValueError, "x_format %lld is not E4M3 or E5M2", (long long)f);
    kind = f == MXFP4_FORMAT_E4M3 ? MXFP4_GEMV_X_E4M3 : MXFP4_GEMV_X_E5M2;
    const at::Tensor& sx = tensor(a[7], "sx");
    dense(sx, "sx", M * (K / 32), at::kByte, sh.dev);
    psx = static_cast<const uint8_t*>(sx.data_ptr());
  } else {
    throw Raise(PyExc_TypeError, "x must be bfloat16 or uint8 codes (got %s)", c10::toString(x.scalar_type()));
  }
  int64_t weights;
  if (N < 0 || __builtin_mul_overflow(N, K, &weights)) throw Raise(PyExc_ValueError, "N %lld is out of range", (long long)N);
  const at::Tensor &qw = tensor(a[2], "qw"), &sw = tensor(a[3], "sw");
  dense(qw, "qw", N * (K / 2), at::kByte, sh.dev);
  dense(sw, "sw", N * scale_cols(block, K), at::kByte, sh.dev);
  Out y;
  y.ld = N;
  if (given(a[10])) {
    y.t = tensor(a[10], "y");
    y.ld = rows_ld(y.t, "y", M, N, sh.dev);
  } else {
    const at::ScalarType t = scalar_type(a[9], "out_dtype");
    dtype_code(t, "y");
    y.t = empty({M, N}, t, x);
  }
  const int32_t ydt = dtype_code(y.t, "y");
  at::Tensor ws;
  size_t bytes = 0;
  if (!given(a[11])) {
    if (weights >= workspace_from(M, block == MXFP4_BLOCK_1X16)) {
      bytes = lib.gemv_workspace(kind, block, M, N, K);
      if (bytes) ws = empty({(int64_t)bytes}, at::kByte, x);
    }
  } else if (a[11] != Py_False) {
    ws = tensor(a[11], "workspace");
    dense(ws, "workspace", 0, at::kByte, sh.dev);
    bytes = (size_t)ws.numel();
  }
  const mxfp4_status st =
      call(lib.gemv, x.data_ptr(), kind, ldx, psx, static_cast<const uint8_t*>(qw.data_ptr()),
           static_cast<const uint8_t*>(sw.data_ptr()), block, layout, exponent, M, N, K, y.ptr(), ydt, y.ld,
           ws.defined() ? ws.data_ptr() : nullptr, bytes, stream_of(sh.dev));
  if (st) return PyLong_FromLong(st);
  return tuple({&y.t});
}

PyMethodDef methods[] = {
    {"make_table", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&make_table<kFunctions>)), METH_FASTCALL, nullptr},
    method<norm, 13>("rmsnorm_quantize"),
    method<norm_backward, 10>("rmsnorm_backward"),
    method<swiglu, 8>("swiglu_quantize"),
    method<swiglu_backward, 6>("swiglu_backward"),
    method<gemv, 12>("gemv"),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  for (int i = 0; i < kFields; ++i)
    if (!(fields[i] = PyUnicode_InternFromString(field_names[i]))) return nullptr;
  return PyModule_Create(&module);
}
