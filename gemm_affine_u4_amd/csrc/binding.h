// What the Python sides of the calls (mix_binding.cpp, serve_binding.cpp) share: a call's device
// and stream, checks of tensors, and errors.
#pragma once
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "qmm.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Bad {
  std::string what;
};
[[noreturn]] void bad(const std::string& s) { throw Bad{s}; }

// A call's tensors must live on the current device: the stream and the launch are its.
struct Call {
  int device = -1;
  hipStream_t stream = nullptr;
  explicit Call(PyObject* s) {
    c10::hip::HIPStream cur = c10::hip::getCurrentHIPStream();
    device = cur.device_index();
    stream = s == Py_None ? cur.stream() : static_cast<hipStream_t>(PyLong_AsVoidPtr(s));
    if (PyErr_Occurred()) bad("stream must be a stream or its handle");
  }
  Call() {}
  const Tensor* opt(PyObject* o, const char* name) const {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) bad(std::string(name) + " must be a tensor");
    const Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) bad(std::string(name) + " must be a device tensor");
    if (!t.is_contiguous()) bad(std::string(name) + " must be contiguous");
    if (device >= 0 && t.get_device() != device)
      bad(std::string(name) + " is on device " + std::to_string(t.get_device()) + ", the current device is " +
          std::to_string(device));
    return &t;
  }
  const Tensor& get(PyObject* o, const char* name) const {
    const Tensor* t = opt(o, name);
    if (!t) bad(std::string(name) + " is missing");
    return *t;
  }
};

void need(bool ok, const char* what) {
  if (!ok) bad(what);
}
bool half_type(const Tensor& t) {
  const ScalarType s = t.scalar_type();
  return s == ScalarType::BFloat16 || s == ScalarType::Short || s == ScalarType::UInt16;
}
int out_type(const Tensor& t, const char* name) {
  if (t.scalar_type() == ScalarType::Float) return QMM_OUT_F32;
  if (!half_type(t)) bad(std::string(name) + " must be bf16 or fp32");
  return QMM_OUT_BF16;
}
bool shaped(const Tensor& t, std::initializer_list<int64_t> s) {
  return t.sizes() == c10::IntArrayRef(s.begin(), s.size());
}
bool words(const Tensor& t) { return t.element_size() == 4 && !t.is_floating_point(); }
void* ptr(const Tensor* t) { return t ? t->data_ptr() : nullptr; }

template <class F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const Bad& b) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, b.what.c_str());
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}

}  // namespace
