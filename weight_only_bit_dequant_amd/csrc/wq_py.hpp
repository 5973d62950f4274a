// What the modules of CPython entry points share: checks of tensors, the call on
// torch's current stream, C++ exceptions turned into Python's.
#pragma once

#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <sstream>
#include <stdexcept>

#include "wq.h"

namespace wq_py {

// What Python raises as ValueError.
struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};

inline const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Refused(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

[[noreturn]] inline void refuse(const at::Tensor& t, const char* name, const std::string& want) {
  std::ostringstream s;
  s << name << " must be " << want << " (got " << t.scalar_type() << " " << t.sizes() << ", strides " << t.strides()
    << ", on " << t.device() << ")";
  throw Refused(s.str());
}

// A contiguous tensor of this type, shape and device: its data.
inline void* data(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, c10::Device dev) {
  if (t.scalar_type() != type || t.sizes() != shape || t.device() != dev || !t.is_contiguous()) {
    std::ostringstream s;
    s << "a contiguous " << type << " tensor of shape " << shape << " on " << dev;
    refuse(t, name, s.str());
  }
  return t.data_ptr();
}

inline void* data(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, c10::Device dev) {
  return data(tensor(o, name), name, type, shape, dev);
}

inline void* data_or_null(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, c10::Device dev) {
  return o == Py_None ? nullptr : data(o, name, type, shape, dev);
}

// A bf16 matrix on the GPU whose rows are contiguous.
struct Rows {
  const void* p;
  int64_t M, K, ld;
  c10::Device dev;
};
inline Rows rows(PyObject* o, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != at::kBFloat16 || t.dim() != 2 || !t.is_cuda() || (t.size(1) > 1 && t.stride(1) != 1))
    refuse(t, name, "a bf16 matrix with contiguous rows on the GPU");
  // a single row's stride says nothing
  return {t.data_ptr(), t.size(0), t.size(1), t.size(0) > 1 ? t.stride(0) : t.size(1), t.device()};
}

// Runs `call(stream)` on the device's current stream with the device current.
template <typename F>
wq_status on(c10::Device dev, F&& call) {
  const c10::DeviceIndex was = c10::hip::current_device();
  if (was != dev.index()) c10::hip::set_device(dev.index());
  const wq_status st = call((void*)c10::hip::getCurrentHIPStream(dev.index()).stream());
  if (was != dev.index()) c10::hip::set_device(was);
  return st;
}

// Entry: `n` arguments, C++ exceptions turned into Python's.  `bound`: the
// module has the C functions' addresses.
template <typename F>
PyObject* entry(bool bound, Py_ssize_t given, Py_ssize_t n, F&& body) {
  try {
    if (given != n) throw std::invalid_argument("wrong number of arguments");
    if (!bound) throw std::logic_error("bind() has not been called");
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

// Takes the addresses of C functions, in the order of `to`.
inline PyObject* bind_all(PyObject* const* a, Py_ssize_t n, std::initializer_list<void**> to) {
  if (n != (Py_ssize_t)to.size()) {
    PyErr_SetString(PyExc_TypeError, "bind() takes an address for each entry point");
    return nullptr;
  }
  Py_ssize_t i = 0;
  for (void** p : to) {
    void* v = PyLong_AsVoidPtr(a[i++]);
    if (!v) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
      return nullptr;
    }
    *p = v;
  }
  Py_RETURN_NONE;
}

#define WQ_METHOD(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}

}  // namespace wq_py
