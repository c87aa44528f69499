// binding_util.h -- what the Python extensions share: checks of tensors,
// allocation, the call of the library, and the way out of an error. Header of
// host C++; everything is in the including file's anonymous namespace.
#pragma once
#define PY_SSIZE_T_CLEAN
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdio>
#include <initializer_list>

#include "../../include/mxfp4.h"

namespace {

// A Python exception on its way out.
struct Raise {
  PyObject* type;
  char text[256];
  Raise(PyObject* t, const char* fmt, ...) __attribute__((format(printf, 3, 4))) : type(t) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(text, sizeof(text), fmt, ap);
    va_end(ap);
  }
};
struct Raised {};  // the interpreter has the exception already

template <typename T>
const T& table_at(PyObject* o) {
  const T* t = static_cast<const T*>(PyLong_AsVoidPtr(o));
  if (!t) {
    if (PyErr_Occurred()) throw Raised{};
    throw Raise(PyExc_ValueError, "no library");
  }
  return *t;
}

bool given(PyObject* o) { return o != Py_None; }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Raise(PyExc_TypeError, "%s must be a tensor (got %s)", name, Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v;
}

at::ScalarType scalar_type(PyObject* o, const char* name) {
  if (!THPDtype_Check(o)) throw Raise(PyExc_TypeError, "%s must be a torch dtype (got %s)", name, Py_TYPE(o)->tp_name);
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

int32_t dtype_code(at::ScalarType t, const char* name) {
  if (t == at::kBFloat16) return MXFP4_DTYPE_BF16;
  if (t == at::kFloat) return MXFP4_DTYPE_F32;
  throw Raise(PyExc_TypeError, "%s must be bfloat16 or float32 (got %s)", name, c10::toString(t));
}
int32_t dtype_code(const at::Tensor& t, const char* name) { return dtype_code(t.scalar_type(), name); }

// The CUDA device and sizes of a matrix.
struct Shape {
  int64_t rows, cols;
  int dev;
};
Shape shape_of(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) throw Raise(PyExc_ValueError, "%s must be a CUDA tensor", name);
  if (t.dim() != 2) throw Raise(PyExc_ValueError, "%s must be 2-D (got %d dimensions)", name, (int)t.dim());
  return Shape{t.size(0), t.size(1), t.get_device()};
}

void on_device(const at::Tensor& t, const char* name, int dev) {
  if (!t.is_cuda() || t.get_device() != dev)
    throw Raise(PyExc_ValueError, "%s must be a CUDA tensor on device %d (got %s)", name, dev, t.device().str().c_str());
}

// Leading dimension of a matrix [rows, cols] with unit column stride. The
// stride of a single row (or of an empty matrix) is never used.
int64_t rows_ld(const at::Tensor& t, const char* name, int64_t rows, int64_t cols, int dev) {
  on_device(t, name, dev);
  if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
    throw Raise(PyExc_ValueError, "%s must be [%lld, %lld]", name, (long long)rows, (long long)cols);
  if (t.stride(1) != 1 && cols > 1 && rows) throw Raise(PyExc_ValueError, "%s must have unit column stride", name);
  return rows > 1 && cols ? t.stride(0) : cols;
}

void vector(const at::Tensor& t, const char* name, int64_t n, int dev) {
  on_device(t, name, dev);
  if (t.dim() != 1 || t.size(0) != n || (n > 1 && t.stride(0) != 1))
    throw Raise(PyExc_ValueError, "%s must be a contiguous vector of %lld elements", name, (long long)n);
}

// A buffer that holds at least n dense elements of one type.
void dense(const at::Tensor& t, const char* name, int64_t n, at::ScalarType type, int dev) {
  on_device(t, name, dev);
  if (t.scalar_type() != type)
    throw Raise(PyExc_TypeError, "%s must be %s (got %s)", name, c10::toString(type), c10::toString(t.scalar_type()));
  if (!t.is_contiguous()) throw Raise(PyExc_ValueError, "%s must be contiguous", name);
  if (t.numel() < n)
    throw Raise(PyExc_ValueError, "%s holds %lld elements; %lld are needed", name, (long long)t.numel(), (long long)n);
}

// Other Python threads run while an allocation or a launch waits.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// (without the dispatcher's way to the same allocation)
at::Tensor empty(at::IntArrayRef sizes, at::ScalarType type, const at::Tensor& like) {
  Unlocked u;
  return at::detail::empty_cuda(sizes, type, like.device(), std::nullopt);
}

// A call of the library.
template <class F, class... A>
mxfp4_status call(F f, A... a) {
  Unlocked u;
  return f(a...);
}

// The tensors' device is the thread's current one while the library runs: it
// launches there, and the default stream's handle names no device.
using OnDevice = c10::cuda::CUDAGuard;

void* stream_of(int dev) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream(); }

PyObject* wrap(const at::Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
PyObject* tuple(std::initializer_list<const at::Tensor*> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (!r) throw Raised{};
  Py_ssize_t i = 0;
  for (const at::Tensor* t : ts) {
    PyObject* o = wrap(*t);
    if (!o) {
      Py_DECREF(r);
      throw Raised{};
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// No C++ exception passes into the interpreter.
template <PyObject* (*F)(PyObject* const*), int kArgs>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != kArgs) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", kArgs, n);
    return nullptr;
  }
  try {
    return F(a);
  } catch (const Raise& e) {
    PyErr_SetString(e.type, e.text);
  } catch (const Raised&) {
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (type) PyErr_SetString(type, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// The addresses of the library's functions, in the order of a table of kFunctions pointers, to a table that
// lives as long as the process.
template <int kFunctions>
PyObject* make_table(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != kFunctions) {
    PyErr_Format(PyExc_TypeError, "%d addresses expected, got %zd", kFunctions, n);
    return nullptr;
  }
  void** t = static_cast<void**>(PyMem_RawMalloc(kFunctions * sizeof(void*)));
  if (!t) return PyErr_NoMemory();
  for (int i = 0; i < kFunctions; ++i) {
    t[i] = PyLong_AsVoidPtr(a[i]);
    if (!t[i]) {
      PyMem_RawFree(t);
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an address is NULL");
      return nullptr;
    }
  }
  return PyLong_FromVoidPtr(t);
}

template <PyObject* (*F)(PyObject* const*), int kArgs>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<F, kArgs>)), METH_FASTCALL, nullptr};
}
}  // namespace
