// What the CPython modules over the C ABI share: checks of tensors, their
// device and stream, and the results.  Host code only.
#pragma once

#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include "qlora_nf4.h"

namespace qlora_py {

using at::Tensor;

// ------------------------------------------------------------- arguments

// An optional tensor: NULL for None.
inline const Tensor* opt(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
  return &THPVariable_Unpack(o);
}
inline const Tensor& need(PyObject* o, const char* name) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
  return THPVariable_Unpack(o);
}
inline int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
inline double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}
inline bool flag(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}
inline void* ptr(const Tensor* t) { return t ? t->data_ptr() : nullptr; }
inline void* ptr(const Tensor& t) { return t.data_ptr(); }
template <typename T>
T* as(const Tensor* t) { return (T*)ptr(t); }

// The device of a call's tensors.  `current` is false when it is not the
// current one.
struct Device {
  int index = -1;
  bool current = false;
  explicit Device(std::initializer_list<const Tensor*> ts) {
    for (const Tensor* t : ts) {
      if (!t) continue;
      TORCH_CHECK_VALUE(t->is_cuda(), "qlora_nf4 tensors must live on a HIP device");
      const int i = t->get_device();
      TORCH_CHECK_VALUE(index < 0 || i == index, "all tensors of a call must be on one device");
      index = i;
    }
    current = index == c10::hip::current_device();
  }
  void* stream() const { return (void*)c10::hip::getCurrentHIPStream((c10::DeviceIndex)index).stream(); }
};

inline int dtype_code(at::ScalarType t, const char* name) {
  TORCH_CHECK_VALUE(t == at::kFloat || t == at::kBFloat16, name, " must be float32 or bfloat16");
  return t == at::kFloat ? QLORA_DTYPE_F32 : QLORA_DTYPE_BF16;
}
inline at::ScalarType scalar_of(int code) { return code == QLORA_DTYPE_F32 ? at::kFloat : at::kBFloat16; }

inline void dense(const Tensor* t, const char* name, at::IntArrayRef shape, at::ScalarType type) {
  if (!t) return;
  TORCH_CHECK_VALUE(t->scalar_type() == type && t->sizes() == shape && t->is_contiguous(), name,
                    " must be a contiguous ", type, " tensor of shape ", shape);
}

// [T, heads, d] with the heads of a token dense.
struct Heads {
  int64_t heads = 0, stride = 0;
};
inline Heads heads_of(const Tensor& t, const char* name, int64_t T, int64_t d, at::ScalarType type) {
  TORCH_CHECK_VALUE(t.dim() == 3 && t.size(0) == T && t.size(2) == d && t.scalar_type() == type, name, " must be a ",
                    type, " tensor [", T, ", heads, ", d, "]");
  const int64_t h = t.size(1);
  TORCH_CHECK_VALUE(h <= INT32_MAX && d <= INT32_MAX, name, " has too many heads");
  if (t.is_contiguous()) return {h, h * d};
  TORCH_CHECK_VALUE((d <= 1 || t.stride(2) == 1) && (h <= 1 || t.stride(1) == d), "the heads of a token of ", name,
                    " must be dense");
  return {h, T > 1 ? t.stride(0) : h * d};
}

inline Tensor new_like(const Tensor& t) {
  return t.is_contiguous() ? at::empty_like(t) : at::empty(t.sizes(), t.options());
}

// ---------------------------------------------------------------- results

inline PyObject* wrap(const Tensor* t) {
  if (!t || !t->defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(*t);
}
inline PyObject* results(std::initializer_list<const Tensor*> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (!r) throw python_error();
  Py_ssize_t i = 0;
  for (const Tensor* t : ts) {
    PyObject* o = wrap(t);
    if (!o) {
      Py_DECREF(r);
      throw python_error();
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}
inline void count(Py_ssize_t n, Py_ssize_t want) { TORCH_CHECK_TYPE(n == want, "expected ", want, " arguments, got ", n); }

// A tensor that is either the caller's or made here.
struct Out {
  const Tensor* given;
  Tensor made;
  explicit Out(const Tensor* t) : given(t) {}
  const Tensor* get() const { return given ? given : made.defined() ? &made : nullptr; }
};

// The call has written these tensors of the caller: a backward that saved one
// of them raises, as after a torch operation in place.
inline void wrote(std::initializer_list<const Tensor*> ts) {
  for (const Tensor* t : ts)
    if (t && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

// Queries or keys with their destination.
struct Turned {
  const Tensor* in;
  Out out;
  Heads from, to;
  Turned(const Tensor* t, const Tensor* o, const char* name, const char* out_name, int64_t T, int64_t d,
         at::ScalarType type)
      : in(t), out(t ? o : nullptr) {
    if (!in) return;
    from = heads_of(*in, name, T, d, type);
    to = {from.heads, from.heads * d};
    if (!out.given) return;
    to = heads_of(*out.given, out_name, T, d, type);
    TORCH_CHECK_VALUE(to.heads == from.heads, out_name, " must have the heads of ", name);
  }
  void make() {
    if (in && !out.given) out.made = new_like(*in);
  }
};

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, (PyCFunction)(void*)F, METH_FASTCALL, nullptr};
}

}  // namespace qlora_py
