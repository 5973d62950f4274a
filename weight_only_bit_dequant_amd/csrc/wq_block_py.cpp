// CPython entry points of block.py: check the tensors' types, shapes, strides
// and devices, and call the C ABI (include/wq_block.h) on torch's current
// stream.  A decode step's operators take a few microseconds on the GPU; the
// same checks in Python over ctypes cost the host 3 us a call (6.5 against 3.4
// us for a norm of one row), more than the kernels.
//
// The module holds no state but the C functions' addresses, which bind() takes
// from the library that wq.lib() loaded.
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <sstream>
#include <stdexcept>

#include "wq_block.h"

namespace {

decltype(&wq_block_quantize_act) p_quantize_act;
decltype(&wq_block_silu_mul_quantize) p_silu_mul_quantize;
decltype(&wq_block_add_rmsnorm_quantize) p_add_rmsnorm_quantize;
decltype(&wq_block_linear) p_linear;
decltype(&wq_block_grouped_linear) p_grouped_linear;

// What Python raises as ValueError.
struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Refused(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

[[noreturn]] void refuse(const at::Tensor& t, const char* name, const std::string& want) {
  std::ostringstream s;
  s << name << " must be " << want << " (got " << t.scalar_type() << " " << t.sizes() << ", strides " << t.strides()
    << ", on " << t.device() << ")";
  throw Refused(s.str());
}

// A contiguous tensor of this type, shape and device: its data.
void* data(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, c10::Device dev) {
  if (t.scalar_type() != type || t.sizes() != shape || t.device() != dev || !t.is_contiguous()) {
    std::ostringstream s;
    s << "a contiguous " << type << " tensor of shape " << shape << " on " << dev;
    refuse(t, name, s.str());
  }
  return t.data_ptr();
}

void* data(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, c10::Device dev) {
  return data(tensor(o, name), name, type, shape, dev);
}

void* data_or_null(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, c10::Device dev) {
  return o == Py_None ? nullptr : data(o, name, type, shape, dev);
}

// A bf16 matrix on the GPU whose rows are contiguous.
struct Rows {
  const void* p;
  int64_t M, K, ld;
  c10::Device dev;
};
Rows rows(PyObject* o, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != at::kBFloat16 || t.dim() != 2 || !t.is_cuda() || (t.size(1) > 1 && t.stride(1) != 1))
    refuse(t, name, "a bf16 matrix with contiguous rows on the GPU");
  // a single row's stride says nothing
  return {t.data_ptr(), t.size(0), t.size(1), t.size(0) > 1 ? t.stride(0) : t.size(1), t.device()};
}

constexpr int64_t kb(int64_t n) { return (n + WQ_BLOCK - 1) / WQ_BLOCK; }

// Runs `call(stream)` on the device's current stream with the device current.
template <typename F>
wq_status on(c10::Device dev, F&& call) {
  const c10::DeviceIndex was = c10::hip::current_device();
  if (was != dev.index()) c10::hip::set_device(dev.index());
  const wq_status st = call((void*)c10::hip::getCurrentHIPStream(dev.index()).stream());
  if (was != dev.index()) c10::hip::set_device(was);
  return st;
}

// Entry: `n` arguments, C++ exceptions turned into Python's.
template <typename F>
PyObject* entry(Py_ssize_t given, Py_ssize_t n, F&& body) {
  try {
    if (given != n) throw std::invalid_argument("wrong number of arguments");
    if (!p_linear) throw std::logic_error("bind() has not been called");
    return PyLong_FromLong(body());
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

template <typename Fn>
PyObject* quant(Fn fn, int halves, PyObject* const* a, Py_ssize_t n) {  // (X, codes, scales)
  return entry(n, 3, [&] {
    const Rows x = rows(a[0], halves == 2 ? "GU" : "X");
    if (x.K % halves) throw Refused("GU must have an even number of columns (gate and up)");
    const int64_t K = x.K / halves;
    void* xq = data(a[1], "codes", at::kByte, {x.M, K}, x.dev);
    void* xs = data(a[2], "scales", at::kFloat, {x.M, kb(K)}, x.dev);
    return on(x.dev, [&](void* s) { return fn(x.p, x.ld, x.M, K, xq, (float*)xs, s); });
  });
}

PyObject* quantize_act(PyObject*, PyObject* const* a, Py_ssize_t n) { return quant(p_quantize_act, 1, a, n); }
PyObject* silu_mul_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) { return quant(p_silu_mul_quantize, 2, a, n); }

// (X, gain, eps, residual, codes, scales, residual_out, y_out)
PyObject* add_rmsnorm_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 8, [&] {
    const Rows x = rows(a[0], "X");
    const void* g = data(a[1], "gain", at::kBFloat16, {x.K}, x.dev);
    const double eps = PyFloat_AsDouble(a[2]);
    if (eps == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      throw Refused("eps must be a number");
    }
    const void* r = data_or_null(a[3], "residual", at::kBFloat16, {x.M, x.K}, x.dev);
    void* xq = data(a[4], "codes", at::kByte, {x.M, x.K}, x.dev);
    void* xs = data(a[5], "scales", at::kFloat, {x.M, kb(x.K)}, x.dev);
    void* ro = data_or_null(a[6], "residual_out", at::kBFloat16, {x.M, x.K}, x.dev);
    void* yo = data_or_null(a[7], "y_out", at::kBFloat16, {x.M, x.K}, x.dev);
    return on(x.dev, [&](void* s) {
      return p_add_rmsnorm_quantize(x.p, x.ld, r, g, (float)eps, x.M, x.K, xq, (float*)xs, ro, yo, s);
    });
  });
}

const at::Tensor& weight(PyObject* o, int64_t dim) {
  const at::Tensor& w = tensor(o, "weight codes");
  if (w.scalar_type() != at::kByte || w.dim() != dim || !w.is_cuda() || !w.is_contiguous())
    refuse(w, "weight codes", dim == 2 ? "contiguous uint8 codes [N, K] on the GPU" : "contiguous uint8 codes [E, N, K] on the GPU");
  return w;
}

// (Xq, Xs, codes, scales, bias, out)
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 6, [&] {
    const at::Tensor& w = weight(a[2], 2);
    const c10::Device dev = w.device();
    const int64_t N = w.size(0), K = w.size(1);
    const at::Tensor& x = tensor(a[0], "Xq");
    const int64_t M = x.dim() ? x.size(0) : 0;
    const void* xq = data(x, "Xq", at::kByte, {M, K}, dev);
    const void* xs = data(a[1], "Xs", at::kFloat, {M, kb(K)}, dev);
    const void* ws = data(a[3], "weight scales", at::kFloat, {kb(N), kb(K)}, dev);
    const void* b = data_or_null(a[4], "bias", at::kBFloat16, {N}, dev);
    void* y = data(a[5], "out", at::kBFloat16, {M, N}, dev);
    return on(dev, [&](void* s) {
      return p_linear(xq, (const float*)xs, M, K, w.data_ptr(), (const float*)ws, b, N, y, s);
    });
  });
}

// (Xq, Xs, codes, scales, offsets, rows, out)
PyObject* grouped_linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 7, [&] {
    const at::Tensor& w = weight(a[2], 3);
    const c10::Device dev = w.device();
    const int64_t E = w.size(0), N = w.size(1), K = w.size(2);
    const at::Tensor& x = tensor(a[0], "Xq");
    const int64_t M = x.dim() ? x.size(0) : 0;
    const void* xq = data(x, "Xq", at::kByte, {M, K}, dev);
    const void* xs = data(a[1], "Xs", at::kFloat, {M, kb(K)}, dev);
    const void* ws = data(a[3], "weight scales", at::kFloat, {E, kb(N), kb(K)}, dev);
    const void* off = data(a[4], "offsets", at::kInt, {E + 1}, dev);
    int64_t T = M;
    const void* r = nullptr;
    if (a[5] != Py_None) {
      const at::Tensor& t = tensor(a[5], "rows");
      T = t.numel();
      r = data(t, "rows", at::kInt, {T}, dev);
    }
    void* y = data(a[6], "out", at::kBFloat16, {T, N}, dev);
    return on(dev, [&](void* s) {
      return p_grouped_linear(xq, (const float*)xs, M, K, (const int32_t*)r, (const int32_t*)off, T, E, w.data_ptr(),
                              (const float*)ws, N, y, s);
    });
  });
}

// bind(quantize_act, silu_mul_quantize, add_rmsnorm_quantize, linear, grouped_linear): addresses of the C functions
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 5) {
    PyErr_SetString(PyExc_TypeError, "bind() takes five addresses");
    return nullptr;
  }
  void* p[5];
  for (int i = 0; i < 5; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
      return nullptr;
    }
  }
  p_quantize_act = (decltype(p_quantize_act))p[0];
  p_silu_mul_quantize = (decltype(p_silu_mul_quantize))p[1];
  p_add_rmsnorm_quantize = (decltype(p_add_rmsnorm_quantize))p[2];
  p_linear = (decltype(p_linear))p[3];
  p_grouped_linear = (decltype(p_grouped_linear))p[4];
  Py_RETURN_NONE;
}

#define WQ_METHOD(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {WQ_METHOD(bind),   WQ_METHOD(quantize_act),   WQ_METHOD(silu_mul_quantize), WQ_METHOD(add_rmsnorm_quantize),
                         WQ_METHOD(linear), WQ_METHOD(grouped_linear), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_block_call", "Calls of the block-scaled FP8 operators.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__block_call(void) { return PyModule_Create(&module); }
