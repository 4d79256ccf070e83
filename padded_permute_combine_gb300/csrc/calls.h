// What the native calls from Python share: tensors from arguments, outputs, the
// stream, errors, and the interpreter's lock.
#pragma once

#include <Python.h>
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty_cuda_dispatch.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "moe_route.h"

namespace moe_calls {

using at::Tensor;

inline int dtype_of(const Tensor& t) {
  if (t.scalar_type() == at::kBFloat16) return MOE_BF16;
  return t.scalar_type() == at::kFloat ? MOE_F32 : -1;
}

// On a GPU, fp32 or bf16, [rows, H] with contiguous rows that do not overlap.
inline bool rows_ok(const Tensor& t, int64_t* stride) {
  if (!t.is_cuda() || t.dim() != 2 || dtype_of(t) < 0) return false;
  const int64_t M = t.size(0), H = t.size(1);
  *stride = t.is_contiguous() ? H : t.stride(0);
  return t.is_contiguous() || ((H <= 1 || t.stride(1) == 1) && (M <= 1 || t.stride(0) >= H));
}
inline bool plain(const Tensor& t, const Tensor& x, at::ScalarType type, at::IntArrayRef sizes) {
  return t.scalar_type() == type && t.device() == x.device() && t.is_contiguous() && t.sizes() == sizes;
}
// The C ABI works on the current device: its launches, SM counts and limits.
using c10::cuda::CUDAGuard;
inline Tensor make(const Tensor& x, at::ScalarType type, at::IntArrayRef sizes) {
  return at::cuda::empty(sizes, at::TensorOptions().dtype(type).device(x.device()));
}
inline moe_stream_t stream_of(const Tensor& x) {
  return reinterpret_cast<moe_stream_t>(c10::cuda::getCurrentCUDAStream(x.device().index()).stream());
}
inline const void* at_or_null(const Tensor& t) { return t.defined() ? t.const_data_ptr() : nullptr; }

// Tensors of a call, in order; the ones that may be None come out undefined.
inline bool tensors(PyObject* const* args, int n, Tensor* out, unsigned optional = 0) {
  for (int i = 0; i < n; ++i) {
    if ((optional >> i & 1) && args[i] == Py_None) continue;
    if (!THPVariable_Check(args[i])) return false;
    out[i] = THPVariable_Unpack(args[i]);
  }
  return true;
}
inline PyObject* wrapped(std::initializer_list<Tensor> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  Py_ssize_t i = 0;
  if (r != nullptr)
    for (const Tensor& t : ts) {
      if (t.defined()) {
        PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(t));
      } else {
        Py_INCREF(Py_None);
        PyTuple_SET_ITEM(r, i++, Py_None);
      }
    }
  return r;
}
// The call's result or, with errors of torch as exceptions of Python, none.
template <typename F> PyObject* guarded(F f) {
  try {
    PyObject* r = f();
    if (r == nullptr && !PyErr_Occurred()) Py_RETURN_NONE;
    return r;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// The C ABI's call without the interpreter's lock, as ctypes makes it: a full
// launch queue blocks it for as long as the queue is full, and other threads
// go on meanwhile. The lock is taken again also when torch throws (a tensor
// without memory, such as a fake one).
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};
template <typename F> int unlocked(F f) {
  const Unlocked now;
  return f();
}

// What follows a code other than MOE_OK. Refused arguments (nothing is enqueued
// then) answer none, and block.py words the error. After any other code work
// may be enqueued already, and a second call would do it twice (gradients
// clipped in place, say): MoeError.
inline PyObject* failed(const char* name, int rc) {
  if (rc == MOE_ERR_INVALID_ARG || rc == MOE_ERR_UNSUPPORTED) return nullptr;
  PyObject* lib = PyImport_ImportModule("padded_permute_combine_gb300._lib");
  PyObject* type = lib == nullptr ? nullptr : PyObject_GetAttrString(lib, "MoeError");
  PyObject* error = type == nullptr ? nullptr : PyObject_CallFunction(type, "sis", name, rc, moe_error_string(rc));
  if (error != nullptr) PyErr_SetObject(type, error);
  Py_XDECREF(error);
  Py_XDECREF(type);
  Py_XDECREF(lib);
  return nullptr;
}

// The calls of decode_calls.cpp, for the module.
PyMethodDef* decode_methods();

#define CALL(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}

}  // namespace moe_calls
