// Python entry of the calls on 4-bit matrices and of appending to a cache.
//
// The smallest of these calls take the GPU two to four microseconds, and what the host does with their arguments (types,
// devices, strides, addresses, the stream) takes as long when Python does it.  The functions here ask the tensors
// themselves and call the library through the addresses that use() was given; they raise ValueError for tensors that do
// not fit and return the call's pe_status.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "pe.h"

namespace {

struct Calls {
  decltype(&pe_quantize_mx) quantize;
  decltype(&pe_dequantize_mx) dequantize;
  decltype(&pe_matmul_mx) matmul;
  decltype(&pe_linear_mx) linear;
  decltype(&pe_append_kv) append;
  decltype(&pe_append_kv_packed) append_packed;
} calls;

struct Refused {};  // a Python exception is set

[[noreturn]] void refuse(const char* what, const std::string& expected) {
  PyErr_Format(PyExc_ValueError, "%s: expected %s", what, expected.c_str());
  throw Refused();
}
[[noreturn]] void refuse(const char* what, const std::string& expected, const at::Tensor& t) {
  std::string got = std::string(c10::toString(t.scalar_type())) + " (";
  for (int64_t s : t.sizes()) got += std::to_string(s) + ",";
  got += ") with strides (";
  for (int64_t s : t.strides()) got += std::to_string(s) + ",";
  refuse(what, expected + ", got " + got + ") on " + t.device().str());
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_ValueError, "%s: expected a tensor", what);
    throw Refused();
  }
  return THPVariable_Unpack(o);
}
std::string on(int dev) { return " on cuda:" + std::to_string(dev); }

// The device of a call's tensors, which has to be the current one (its stream is used).
int current(const at::Tensor& t) {
  const int dev = t.is_cuda() ? (int)t.get_device() : -1;
  if (dev < 0 || dev != (int)c10::cuda::current_device()) {
    PyErr_Format(PyExc_ValueError, "expected tensors on the current CUDA device, got %s", t.device().str().c_str());
    throw Refused();
  }
  return dev;
}
bool is_on(const at::Tensor& t, int dev) { return t.is_cuda() && (int)t.get_device() == dev; }

struct Rows {
  pe_dtype dtype;
  void* p;
  int64_t stride;
};
// n rows of `width` fp32 or bf16 elements, each row contiguous.
Rows any_rows(PyObject* o, const char* what, int dev, int64_t n, int64_t width) {
  const at::Tensor& t = tensor(o, what);
  const auto type = t.scalar_type();
  if ((type != at::kBFloat16 && type != at::kFloat) || !is_on(t, dev) || t.dim() != 2 || t.size(0) != n ||
      t.size(1) != width || (width > 1 && n > 0 && t.stride(1) != 1))
    refuse(what, std::to_string(n) + " rows of " + std::to_string(width) + " contiguous fp32 or bf16 elements" + on(dev), t);
  return Rows{type == at::kBFloat16 ? PE_BF16 : PE_F32, t.data_ptr(), n > 1 ? t.stride(0) : width};
}
// n rows of `width` elements of a type ([n][width] or [n][heads][head_dim], each row contiguous).
Rows typed_rows(PyObject* o, const char* what, int dev, at::ScalarType type, int64_t n, int64_t width) {
  const at::Tensor& t = tensor(o, what);
  bool fits = t.scalar_type() == type && is_on(t, dev) && t.dim() >= 2 && t.size(0) == n;
  int64_t inner = 1;
  for (int64_t d = t.dim() - 1; fits && d > 0; --d) {
    fits = t.size(d) == 1 || t.stride(d) == inner;
    inner *= t.size(d);
  }
  if (!fits || inner != width)
    refuse(what, std::to_string(n) + " rows of " + std::to_string(width) + " contiguous elements of " + c10::toString(type) +
                     on(dev), t);
  return Rows{PE_F32, t.data_ptr(), n > 1 ? t.stride(0) : width};
}
// A contiguous tensor of a type.
const at::Tensor& whole(PyObject* o, const char* what, int dev, at::ScalarType type) {
  const at::Tensor& t = tensor(o, what);
  if (t.scalar_type() != type || !is_on(t, dev) || !t.is_contiguous())
    refuse(what, std::string("a contiguous tensor of ") + c10::toString(type) + on(dev), t);
  return t;
}
int32_t* error_word(PyObject* o, int dev) {
  const at::Tensor& t = whole(o, "err", dev, at::kInt);
  if (t.numel() < 1) refuse("err", "an element", t);
  return static_cast<int32_t*>(t.data_ptr());
}

int64_t number(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}
int32_t small_number(PyObject* o) {
  const int64_t v = number(o);
  if (v < INT32_MIN || v > INT32_MAX) {
    PyErr_SetString(PyExc_OverflowError, "sizes: expected 32-bit numbers");
    throw Refused();
  }
  return (int32_t)v;
}
pe_stream_t stream(PyObject* o, int dev) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
  PyObject* raw = PyObject_GetAttrString(o, "cuda_stream");
  if (raw == nullptr) throw Refused();
  void* s = PyLong_AsVoidPtr(raw);
  Py_DECREF(raw);
  if (s == nullptr && PyErr_Occurred()) throw Refused();
  return static_cast<pe_stream_t>(s);
}

// A 4-bit matrix: (n_rows, width, data), data as large as its maker saw to.
struct Mx {
  int32_t n, width;
  void* p;
};
Mx matrix(PyObject* o, const char* what, int dev) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 3) {
    PyErr_Format(PyExc_ValueError, "%s: expected a matrix", what);
    throw Refused();
  }
  const at::Tensor& data = tensor(PyTuple_GET_ITEM(o, 2), what);
  if (!is_on(data, dev)) refuse(what, "a matrix" + on(dev) + ", got one on " + data.device().str());
  return Mx{small_number(PyTuple_GET_ITEM(o, 0)), small_number(PyTuple_GET_ITEM(o, 1)), data.data_ptr()};
}

// A call of the library, during which other Python threads run (a launch may wait for room in its queue).
template <typename F>
pe_status released(F f) {
  PyThreadState* s = PyEval_SaveThread();
  const pe_status st = f();
  PyEval_RestoreThread(s);
  return st;
}

void count(Py_ssize_t n, Py_ssize_t expected) {
  if (n != expected) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", expected, n);
    throw Refused();
  }
}
template <typename F>
PyObject* status(F f) {
  try {
    return PyLong_FromLong((long)f());
  } catch (const Refused&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// quantize_mx(x, m, err, stream)
PyObject* quantize_mx(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return status([&] {
    count(n, 4);
    const int dev = current(tensor(a[0], "x"));
    const Mx m = matrix(a[1], "m", dev);
    const Rows x = any_rows(a[0], "x", dev, m.n, m.width);
    int32_t* err = error_word(a[2], dev);
    pe_stream_t s = stream(a[3], dev);
    if (m.n == 0) return PE_OK;
    return released([&] { return calls.quantize(x.dtype, x.p, x.stride, m.n, m.width, m.p, err, s); });
  });
}
// dequantize_mx(m, x, stream)
PyObject* dequantize_mx(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return status([&] {
    count(n, 3);
    const int dev = current(tensor(a[1], "x"));
    const Mx m = matrix(a[0], "m", dev);
    const Rows x = any_rows(a[1], "x", dev, m.n, m.width);
    pe_stream_t s = stream(a[2], dev);
    if (m.n == 0) return PE_OK;
    return released([&] { return calls.dequantize(x.dtype, m.p, m.n, m.width, x.p, x.stride, s); });
  });
}

// y and what is added to it.
struct Out {
  Rows y;
  void* add = nullptr;
  int64_t add_stride = 0;
};
Out output(PyObject* y, PyObject* add, int dev, int64_t n, int64_t n_out) {
  Out o{any_rows(y, "y", dev, n, n_out)};
  if (add != Py_None) {
    const Rows r = any_rows(add, "add", dev, n, n_out);
    if (r.dtype != o.y.dtype) refuse("add", "y's type");
    o.add = r.p;
    o.add_stride = r.stride;
  }
  return o;
}
// matmul_mx(x, w, y, err, add, stream)
PyObject* matmul_mx(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return status([&] {
    count(n, 6);
    const int dev = current(tensor(a[2], "y"));
    const Mx x = matrix(a[0], "x", dev), w = matrix(a[1], "w", dev);
    if (x.width != w.width) {
      PyErr_Format(PyExc_ValueError, "x and w: widths %d and %d differ", x.width, w.width);
      throw Refused();
    }
    const Out o = output(a[2], a[4], dev, x.n, w.n);
    int32_t* err = error_word(a[3], dev);
    pe_stream_t s = stream(a[5], dev);
    if (x.n == 0) return PE_OK;
    return released([&] {
      return calls.matmul(x.p, x.n, w.p, w.n, w.width, o.add, o.add_stride, o.y.dtype, o.y.p, o.y.stride, err, s);
    });
  });
}
// linear_mx(x, w, y, workspace, err, add, stream)
PyObject* linear_mx(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return status([&] {
    count(n, 7);
    const int dev = current(tensor(a[2], "y"));
    const Mx w = matrix(a[1], "w", dev);
    const at::Tensor& xt = tensor(a[0], "x");
    if (xt.dim() != 2 || xt.size(0) > INT32_MAX) refuse("x", "rows of " + std::to_string(w.width) + " elements", xt);
    const int32_t rows = (int32_t)xt.size(0);
    const Rows x = any_rows(a[0], "x", dev, rows, w.width);
    const Out o = output(a[2], a[5], dev, rows, w.n);
    int32_t* err = error_word(a[4], dev);
    const at::Tensor& ws = whole(a[3], "workspace", dev, at::kByte);
    pe_stream_t s = stream(a[6], dev);
    if (rows == 0) return PE_OK;
    return released([&] {
      return calls.linear(x.dtype, x.p, x.stride, rows, w.p, w.n, w.width, o.add, o.add_stride, o.y.dtype, o.y.p, o.y.stride,
                          ws.data_ptr(), (size_t)ws.numel(), err, s);
    });
  });
}

struct Ref {  // a reference of this call's own
  PyObject* o;
  explicit Ref(PyObject* p) : o(p) {
    if (p == nullptr) throw Refused();
  }
  Ref(const Ref&) = delete;
  ~Ref() { Py_DECREF(o); }
};

// append_kv(cfg, q, k, v, positions, slots, cache, q_out, err, axes, stream)
struct ConfigView {  // the pe_config that a ctypes structure holds
  Py_buffer b;
  explicit ConfigView(PyObject* o) {
    if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) throw Refused();
    if (b.len != (Py_ssize_t)sizeof(pe_config)) {
      PyBuffer_Release(&b);
      refuse("cfg", "a Config");
    }
  }
  ~ConfigView() { PyBuffer_Release(&b); }
  const pe_config& operator*() const { return *static_cast<const pe_config*>(b.buf); }
};
PyObject* append_kv(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return status([&] {
    count(nargs, 11);
    const ConfigView view(a[0]);
    const pe_config& c = *view;
    const int dev = current(tensor(a[5], "slots"));
    const at::Tensor& slots = whole(a[5], "slots", dev, at::kLong);
    if (slots.dim() != 1 || slots.numel() > INT32_MAX) refuse("slots", "one dimension", slots);
    const int32_t n = (int32_t)slots.numel();
    const at::Tensor& pos = whole(a[4], "positions", dev, at::kInt);
    if (pos.dim() < 1 || pos.dim() > 2 || pos.size(-1) != n || (pos.dim() == 2 && pos.size(0) > INT32_MAX))
      refuse("positions", "[" + std::to_string(n) + "] or [axes][" + std::to_string(n) + "]", pos);
    const int32_t n_axes = pos.dim() == 2 ? (int32_t)pos.size(0) : 1;
    const uint8_t* axes = nullptr;
    if (a[9] != Py_None) {
      if (!PyBytes_Check(a[9]) || PyBytes_GET_SIZE(a[9]) != c.head_dim / 2)
        refuse("axes", std::to_string(c.head_dim / 2) + " bytes, one per pair");
      axes = reinterpret_cast<const uint8_t*>(PyBytes_AS_STRING(a[9]));
    }
    const at::ScalarType type = c.dtype == PE_BF16 ? at::kBFloat16 : at::kFloat;
    const int64_t kv_row = (int64_t)c.n_kv * c.head_dim, q_row = (int64_t)c.n_q * c.head_dim;
    const Rows k = typed_rows(a[2], "k", dev, type, n, kv_row), v = typed_rows(a[3], "v", dev, type, n, kv_row);
    Rows q{}, out{};
    if (a[1] != Py_None || a[7] != Py_None) {
      q = typed_rows(a[1], "q", dev, type, n, q_row);
      out = typed_rows(a[7], "q_out", dev, type, n, q_row);
    }
    int32_t* err = error_word(a[8], dev);
    pe_stream_t s = stream(a[10], dev);
    const auto* positions = static_cast<const int32_t*>(pos.data_ptr());
    const auto* slot = static_cast<const int64_t*>(slots.data_ptr());
    if (THPVariable_Check(a[6])) {
      const at::Tensor& pool = whole(a[6], "pool", dev, at::kByte);
      if (pool.dim() != 3 || pool.size(1) != c.n_kv || pool.size(2) != 18 * (int64_t)c.head_dim || pool.size(0) > INT32_MAX)
        refuse("pool", "[pages][" + std::to_string(c.n_kv) + "][" + std::to_string(18 * c.head_dim) + "]", pool);
      if (n == 0) return PE_OK;
      return released([&] {
        return calls.append_packed(&c, q.p, k.p, v.p, q.stride, k.stride, v.stride, positions, n_axes, axes, slot, n, out.p,
                                   out.stride, pool.data_ptr(), (int32_t)pool.size(0), err, s);
      });
    }
    if (!PySequence_Check(a[6]) || PySequence_Size(a[6]) != 2) refuse("cache", "a pool, or keys and values");
    // (a sequence may make its items when it is asked for them, and keep none)
    const Ref items[2] = {Ref(PySequence_GetItem(a[6], 0)), Ref(PySequence_GetItem(a[6], 1))};
    void* at_[2];
    int32_t pages = 0;
    for (int i = 0; i < 2; ++i) {
      const char* what = i == 0 ? "k_cache" : "v_cache";
      const at::Tensor& t = whole(items[i].o, what, dev, type);
      if (t.dim() != 4 || t.size(1) != 16 || t.size(2) != c.n_kv || t.size(3) != c.head_dim || t.size(0) > INT32_MAX ||
          (i == 1 && t.size(0) != pages))
        refuse(what, "[pages][16][" + std::to_string(c.n_kv) + "][" + std::to_string(c.head_dim) + "]", t);
      pages = (int32_t)t.size(0);
      at_[i] = t.data_ptr();
    }
    if (n == 0) return PE_OK;
    return released([&] {
      return calls.append(&c, q.p, k.p, v.p, q.stride, k.stride, v.stride, positions, n_axes, axes, slot, n, out.p, out.stride,
                          at_[0], at_[1], pages, err, s);
    });
  });
}

// use(addresses of quantize, dequantize, matmul, linear, append, append_packed)
PyObject* use(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return status([&] {
    count(n, 6);
    void* p[6];
    for (int i = 0; i < 6; ++i)
      if ((p[i] = PyLong_AsVoidPtr(a[i])) == nullptr) refuse("use", "addresses");
    calls = Calls{reinterpret_cast<decltype(calls.quantize)>(p[0]), reinterpret_cast<decltype(calls.dequantize)>(p[1]),
                  reinterpret_cast<decltype(calls.matmul)>(p[2]),   reinterpret_cast<decltype(calls.linear)>(p[3]),
                  reinterpret_cast<decltype(calls.append)>(p[4]),   reinterpret_cast<decltype(calls.append_packed)>(p[5])};
    return PE_OK;
  });
}

#define PE_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {PE_METHOD(use),       PE_METHOD(quantize_mx), PE_METHOD(dequantize_mx), PE_METHOD(matmul_mx),
                         PE_METHOD(linear_mx), PE_METHOD(append_kv),   {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "pe_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_pe_bind() { return PyModule_Create(&module); }
