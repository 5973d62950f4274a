// CPython entry points of experts.py: check the tensors' types, shapes, strides
// and devices, and call the C ABI (include/wq_experts.h) on torch's current
// stream (why compiled: wq_block_py.cpp).
#include "wq_experts.h"
#include "wq_py.hpp"

namespace {

using namespace wq_py;

decltype(&wq_experts_route) p_route;
decltype(&wq_experts_combine) p_combine;

template <typename F>
PyObject* entry(Py_ssize_t given, Py_ssize_t n, F&& body) {
  return wq_py::entry(p_route != nullptr, given, n, body);
}

int64_t whole(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Refused(std::string(name) + " must be a whole number");
  }
  return v;
}

bool truth(PyObject* o, const char* name) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    throw Refused(std::string(name) + " must be true or false");
  }
  return v != 0;
}

// (logits, top, score, bias, groups, keep, pairs, renormalize, scale, valid, ids, weights, offsets, rows, places, workspace)
PyObject* route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 16, [&] {
    const at::Tensor& l = tensor(a[0], "logits");
    const bool half = l.scalar_type() == at::kBFloat16;
    if ((!half && l.scalar_type() != at::kFloat) || l.dim() != 2 || !l.is_cuda() || (l.size(1) > 1 && l.stride(1) != 1))
      refuse(l, "logits", "an fp32 or bf16 matrix with contiguous rows on the GPU");
    const c10::Device dev = l.device();
    const int64_t M = l.size(0), E = l.size(1), ld = M > 1 ? l.stride(0) : E, top = whole(a[1], "top");
    if (top < 1 || top > E) throw Refused("top must be 1 to the number of experts");
    const double scale = PyFloat_AsDouble(a[8]);
    if (scale == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      throw Refused("scale must be a number");
    }
    const void* bias = data_or_null(a[3], "bias", at::kFloat, {E}, dev);
    const void* valid = data_or_null(a[9], "valid", at::kBool, {M}, dev);
    void* ids = data(a[10], "ids", at::kInt, {M, top}, dev);
    void* weights = data(a[11], "weights", at::kFloat, {M, top}, dev);
    void* offsets = data(a[12], "offsets", at::kInt, {E + 1}, dev);
    void* rows = data(a[13], "rows", at::kInt, {M * top}, dev);
    void* places = data(a[14], "places", at::kInt, {M, top}, dev);
    void* ws = nullptr;
    size_t bytes = 0;
    if (a[15] != Py_None) {
      const at::Tensor& w = tensor(a[15], "workspace");
      ws = data(w, "workspace", at::kByte, {w.numel()}, dev);
      bytes = (size_t)w.numel();
    }
    const int64_t score = whole(a[2], "score"), groups = whole(a[4], "groups"), keep = whole(a[5], "keep_groups");
    const int pairs = truth(a[6], "pairs"), renorm = truth(a[7], "renormalize");
    return on(dev, [&](void* s) {
      return p_route(l.data_ptr(), half ? 16 : 32, ld, M, E, top, (int)score, (const float*)bias, groups, keep, pairs,
                     renorm, (float)scale, valid, (int32_t*)ids, (float*)weights, (int32_t*)offsets, (int32_t*)rows,
                     (int32_t*)places, ws, bytes, s);
    });
  });
}

// (Y, places, weights, base, out)
PyObject* combine(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 5, [&] {
    const at::Tensor& y = tensor(a[0], "Y");
    if (y.scalar_type() != at::kBFloat16 || y.dim() != 2 || !y.is_cuda() || !y.is_contiguous())
      refuse(y, "Y", "a contiguous bf16 matrix on the GPU");
    const c10::Device dev = y.device();
    const at::Tensor& p = tensor(a[1], "places");
    if (p.dim() != 2) refuse(p, "places", "a matrix [M, top]");
    const int64_t M = p.size(0), top = p.size(1), N = y.size(1);
    const void* places = data(p, "places", at::kInt, {M, top}, dev);
    const void* w = data(a[2], "weights", at::kFloat, {M, top}, dev);
    const void* base = data_or_null(a[3], "base", at::kBFloat16, {M, N}, dev);
    void* out = data(a[4], "out", at::kBFloat16, {M, N}, dev);
    return on(dev, [&](void* s) {
      return p_combine(y.data_ptr(), y.size(0), N, (const int32_t*)places, (const float*)w, M, top, base, out, s);
    });
  });
}

// bind(route, combine): addresses of the C functions
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) { return bind_all(a, n, {(void**)&p_route, (void**)&p_combine}); }

PyMethodDef methods[] = {WQ_METHOD(bind), WQ_METHOD(route), WQ_METHOD(combine), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_experts_call", "Calls of the experts' routing.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__experts_call(void) { return PyModule_Create(&module); }
