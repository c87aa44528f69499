// cache_binding.cpp -- the calls on the 8-bit cache of keys and values from
// Python, as binding.cpp has the norm, activation and few-row calls.
#include "binding_util.h"

namespace {

// The library's functions.
struct Table {
  decltype(&mxfp8_cache_append) append;
  decltype(&mxfp8_cache_read) read;
  decltype(&mxfp8_cache_attention) attention;
  decltype(&mxfp8_cache_attention_workspace_size) workspace;
};
constexpr int kFunctions = sizeof(Table) / sizeof(void*);
const Table& table(PyObject* o) { return table_at<Table>(o); }

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}

void whole(const at::Tensor& t, const char* name) {
  if (t.scalar_type() != at::kInt) throw Raise(PyExc_TypeError, "%s must be int32 (got %s)", name, c10::toString(t.scalar_type()));
}

// codes [pages, 2, heads, page_tokens, head_dim] and scales [pages, 2, heads].
mxfp8_cache cache(PyObject* codes, PyObject* scales, int* dev) {
  const at::Tensor& q = tensor(codes, "codes");
  if (!q.is_cuda()) throw Raise(PyExc_ValueError, "codes must be a CUDA tensor");
  if (q.dim() != 5 || q.size(1) != 2) throw Raise(PyExc_ValueError, "codes must be [pages, 2, heads, page_tokens, head_dim]");
  *dev = q.get_device();
  dense(q, "codes", 0, at::kByte, *dev);
  const at::Tensor& s = tensor(scales, "scales");
  dense(s, "scales", 0, at::kByte, *dev);
  if (s.dim() != 3 || s.size(0) != q.size(0) || s.size(1) != 2 || s.size(2) != q.size(2))
    throw Raise(PyExc_ValueError, "scales must be [%lld, 2, %lld]", (long long)q.size(0), (long long)q.size(2));
  for (int i = 2; i < 5; ++i)
    if (q.size(i) > (1 << 20)) throw Raise(PyExc_ValueError, "codes are too large in dimension %d", i);
  return mxfp8_cache{static_cast<uint8_t*>(q.data_ptr()), static_cast<uint8_t*>(s.data_ptr()), q.size(0),
                     (int32_t)q.size(2), (int32_t)q.size(3), (int32_t)q.size(4)};
}

// page_table [sequences, max_pages], lens [sequences] and starts [sequences + 1] (each None: absent).
mxfp8_cache_batch batch(PyObject* page_table, PyObject* lens, PyObject* starts, int64_t tokens, int dev) {
  const at::Tensor& t = tensor(page_table, "page_table");
  whole(t, "page_table");
  if (t.dim() != 2) throw Raise(PyExc_ValueError, "page_table must be 2-D (got %d dimensions)", (int)t.dim());
  mxfp8_cache_batch b{};
  b.sequences = t.size(0);
  b.max_pages = t.size(1);
  b.ld_table = rows_ld(t, "page_table", b.sequences, b.max_pages, dev);
  b.page_table = static_cast<const int32_t*>(t.data_ptr());
  b.tokens = tokens;
  if (given(lens)) {
    const at::Tensor& l = tensor(lens, "lens");
    whole(l, "lens");
    vector(l, "lens", b.sequences, dev);
    b.lens = static_cast<const int32_t*>(l.data_ptr());
  }
  if (given(starts)) {
    const at::Tensor& s = tensor(starts, "starts");
    whole(s, "starts");
    vector(s, "starts", b.sequences + 1, dev);
    b.starts = static_cast<const int32_t*>(s.data_ptr());
  }
  return b;
}

// A [tokens, heads, head_dim] tensor. Strides of a single row or head are not used.
mxfp8_heads heads_of(const at::Tensor& t, const char* name, int64_t tokens, int64_t heads, int64_t dim, int dev) {
  on_device(t, name, dev);
  if (t.dim() != 3 || t.size(0) != tokens || t.size(1) != heads || t.size(2) != dim)
    throw Raise(PyExc_ValueError, "%s must be [%lld, %lld, %lld]", name, (long long)tokens, (long long)heads, (long long)dim);
  if (t.stride(2) != 1 && tokens) throw Raise(PyExc_ValueError, "%s must have a unit stride in its last dimension", name);
  return mxfp8_heads{t.data_ptr(), dtype_code(t, name), tokens > 1 ? t.stride(0) : heads * dim, heads > 1 ? t.stride(1) : dim};
}

int64_t rows_in(const at::Tensor& t, const char* name) {
  if (t.dim() != 3) throw Raise(PyExc_ValueError, "%s must be 3-D (got %d dimensions)", name, (int)t.dim());
  return t.size(0);
}

// (table, k, v, codes, scales, page_table, lens, starts)
PyObject* append(PyObject* const* a) {
  const Table& lib = table(a[0]);
  int dev = 0;
  const mxfp8_cache c = cache(a[3], a[4], &dev);
  const OnDevice current(static_cast<c10::DeviceIndex>(dev));
  const at::Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
  const int64_t rows = rows_in(k, "k");
  const mxfp8_cache_batch b = batch(a[5], a[6], a[7], rows, dev);
  const mxfp8_heads hk = heads_of(k, "k", rows, c.heads, c.head_dim, dev), hv = heads_of(v, "v", rows, c.heads, c.head_dim, dev);
  if (k.scalar_type() != v.scalar_type())
    throw Raise(PyExc_TypeError, "v must have k's type (got %s)", c10::toString(v.scalar_type()));
  const mxfp4_status st = call(lib.append, &c, &b, &hk, &hv, stream_of(dev));
  if (st) return PyLong_FromLong(st);
  Py_RETURN_NONE;
}

// (table, codes, scales, page_table, starts, rows, out_dtype, k, v) -> (k, v)
PyObject* read(PyObject* const* a) {
  const Table& lib = table(a[0]);
  int dev = 0;
  const mxfp8_cache c = cache(a[1], a[2], &dev);
  const OnDevice current(static_cast<c10::DeviceIndex>(dev));
  const int64_t rows = integer(a[5]);
  if (rows < 0 || rows >= (1 << 24)) throw Raise(PyExc_ValueError, "rows %lld is out of range", (long long)rows);
  const mxfp8_cache_batch b = batch(a[3], Py_None, a[4], rows, dev);
  const at::ScalarType type = scalar_type(a[6], "out_dtype");
  dtype_code(type, "out_dtype");
  const at::Tensor& like = tensor(a[1], "codes");
  const at::Tensor k = given(a[7]) ? tensor(a[7], "k") : empty({rows, c.heads, c.head_dim}, type, like);
  const at::Tensor v = given(a[8]) ? tensor(a[8], "v") : empty({rows, c.heads, c.head_dim}, k.scalar_type(), like);
  const mxfp8_heads hk = heads_of(k, "k", rows, c.heads, c.head_dim, dev), hv = heads_of(v, "v", rows, c.heads, c.head_dim, dev);
  if (k.scalar_type() != v.scalar_type())
    throw Raise(PyExc_TypeError, "v must have k's type (got %s)", c10::toString(v.scalar_type()));
  const mxfp4_status st = call(lib.read, &c, &b, &hk, &hv, stream_of(dev));
  if (st) return PyLong_FromLong(st);
  return tuple({&k, &v});
}

// (table, q, codes, scales, page_table, lens, starts, scale, window, softcap, slopes, out_dtype, with_lse, out, lse,
// workspace) -> (out, lse)
PyObject* attention(PyObject* const* a) {
  const Table& lib = table(a[0]);
  int dev = 0;
  const mxfp8_cache c = cache(a[2], a[3], &dev);
  const OnDevice current(static_cast<c10::DeviceIndex>(dev));
  const at::Tensor& q = tensor(a[1], "q");
  const int64_t rows = rows_in(q, "q"), heads = q.size(1);
  if (heads > 65535) throw Raise(PyExc_ValueError, "q has %lld heads; at most 65535 are supported", (long long)heads);
  if (q.scalar_type() != at::kBFloat16) throw Raise(PyExc_TypeError, "q must be bfloat16 (got %s)", c10::toString(q.scalar_type()));
  if (!given(a[5])) throw Raise(PyExc_TypeError, "lens must be a tensor");
  const mxfp8_cache_batch b = batch(a[4], a[5], a[6], rows, dev);
  const mxfp8_heads hq = heads_of(q, "q", rows, heads, c.head_dim, dev);
  mxfp8_attention_params p{};
  p.scale = (float)number(a[7]);
  const int64_t window = integer(a[8]);
  if (window < 0 || window > INT32_MAX) throw Raise(PyExc_ValueError, "window %lld is out of range", (long long)window);
  p.window = (int32_t)window;
  p.softcap = (float)number(a[9]);
  if (given(a[10])) {
    const at::Tensor& s = tensor(a[10], "slopes");
    if (s.scalar_type() != at::kFloat) throw Raise(PyExc_TypeError, "slopes must be float32 (got %s)", c10::toString(s.scalar_type()));
    vector(s, "slopes", heads, dev);
    p.slopes = static_cast<const float*>(s.data_ptr());
  }
  at::Tensor out, lse, ws;
  if (given(a[13])) {
    out = tensor(a[13], "out");
  } else {
    const at::ScalarType type = scalar_type(a[11], "out_dtype");
    dtype_code(type, "out_dtype");
    out = empty({rows, heads, c.head_dim}, type, q);
  }
  const mxfp8_heads ho = heads_of(out, "out", rows, heads, c.head_dim, dev);
  if (given(a[14])) {
    lse = tensor(a[14], "lse");
    dense(lse, "lse", rows * heads, at::kFloat, dev);
  } else if (truth(a[12])) {
    lse = empty({rows, heads}, at::kFloat, q);
  }
  const size_t need = lib.workspace(&c, &b, (int32_t)heads);
  if (given(a[15])) {
    ws = tensor(a[15], "workspace");
    dense(ws, "workspace", (int64_t)need, at::kByte, dev);
  } else if (need) {
    ws = empty({(int64_t)need}, at::kByte, q);
  }
  const mxfp4_status st =
      call(lib.attention, &c, &b, &hq, (int32_t)heads, &p, &ho, lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr,
           ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? (size_t)ws.numel() : 0, stream_of(dev));
  if (st) return PyLong_FromLong(st);
  return tuple({&out, &lse});
}

PyMethodDef methods[] = {
    {"make_table", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&make_table<kFunctions>)), METH_FASTCALL, nullptr},
    method<append, 8>("append"),
    method<read, 9>("read"),
    method<attention, 16>("attention"),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_cache_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__cache_binding() { return PyModule_Create(&module); }
