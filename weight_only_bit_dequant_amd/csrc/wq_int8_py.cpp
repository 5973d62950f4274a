// CPython entry points of int8.py: check the tensors' types, shapes, strides and
// devices, and call the C ABI (include/wq_int8.h) on torch's current stream (why
// compiled: wq_block_py.cpp).
#include "wq_int8.h"
#include "wq_py.hpp"

namespace {

using namespace wq_py;

decltype(&wq_int8_quantize_act) p_quantize_act;
decltype(&wq_int8_silu_mul_quantize) p_silu_mul_quantize;
decltype(&wq_int8_linear) p_linear;
decltype(&wq_int8_grouped_linear) p_grouped_linear;

template <typename F>
PyObject* entry(Py_ssize_t given, Py_ssize_t n, F&& body) {
  return wq_py::entry(p_linear != nullptr, given, n, body);
}

template <typename Fn>
PyObject* quant(Fn fn, int halves, PyObject* const* a, Py_ssize_t n) {  // (X, codes, scales)
  return entry(n, 3, [&] {
    const Rows x = rows(a[0], halves == 2 ? "GU" : "X");
    if (x.K % halves) throw Refused("GU must have an even number of columns (gate and up)");
    const int64_t K = x.K / halves;
    if (K == 0 && x.M > 0) throw Refused(std::string(halves == 2 ? "GU" : "X") + " must have columns (rows of none would be left without scales)");
    void* xq = data(a[1], "codes", at::kChar, {x.M, K}, x.dev);
    void* xs = data(a[2], "scales", at::kFloat, {x.M}, x.dev);
    return on(x.dev, [&](void* s) { return fn(x.p, x.ld, x.M, K, xq, (float*)xs, s); });
  });
}

PyObject* quantize_act(PyObject*, PyObject* const* a, Py_ssize_t n) { return quant(p_quantize_act, 1, a, n); }
PyObject* silu_mul_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) { return quant(p_silu_mul_quantize, 2, a, n); }

const at::Tensor& weight(PyObject* o, int64_t dim) {
  const at::Tensor& w = tensor(o, "weight codes");
  if (w.scalar_type() != at::kChar || w.dim() != dim || !w.is_cuda() || !w.is_contiguous())
    refuse(w, "weight codes", dim == 2 ? "contiguous int8 codes [N, K] on the GPU" : "contiguous int8 codes [E, N, K] on the GPU");
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
    const void* xq = data(x, "Xq", at::kChar, {M, K}, dev);
    const void* xs = data(a[1], "Xs", at::kFloat, {M}, dev);
    const void* ws = data(a[3], "weight scales", at::kFloat, {N}, dev);
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
    const void* xq = data(x, "Xq", at::kChar, {M, K}, dev);
    const void* xs = data(a[1], "Xs", at::kFloat, {M}, dev);
    const void* ws = data(a[3], "weight scales", at::kFloat, {E, N}, dev);
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

// bind(quantize_act, silu_mul_quantize, linear, grouped_linear): addresses of the C functions
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return bind_all(a, n, {(void**)&p_quantize_act, (void**)&p_silu_mul_quantize, (void**)&p_linear, (void**)&p_grouped_linear});
}

PyMethodDef methods[] = {WQ_METHOD(bind),   WQ_METHOD(quantize_act),   WQ_METHOD(silu_mul_quantize),
                         WQ_METHOD(linear), WQ_METHOD(grouped_linear), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_int8_call", "Calls of the 8-bit integer operators.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__int8_call(void) { return PyModule_Create(&module); }
