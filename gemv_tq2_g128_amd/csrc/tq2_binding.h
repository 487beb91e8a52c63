// What the compiled Python modules share: torch tensors into the pointers and sizes of a C entry point's arguments, and the
// call on the tensors' device and its current stream.
//
// A decode step makes a handful of these calls on small tensors, whose kernels
// take 3 to 10 us: reading the tensors' types, shapes and strides from Python
// took 7 us of an append's 11, here it takes under one.  Argument marshalling
// only: every check that the C entry points make is left to them, and their
// status is returned where it is not TQ2_OK.
#ifndef TQ2_BINDING_H
#define TQ2_BINDING_H

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cmath>
#include <optional>
#include <string>

#include <ATen/ops/empty.h>
#include <c10/hip/HIPGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "tq2.h"
#include "tq2_attn.h"

namespace {

// A Python exception to be: caught at each entry.
struct Refusal {
  PyObject* type;
  std::string text;
};

[[noreturn]] inline void refuse(const std::string& text) { throw Refusal{PyExc_ValueError, text}; }

inline const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) throw Refusal{PyExc_TypeError, std::string(what) + " must be a torch.Tensor"};
  return THPVariable_Unpack(o);
}

inline const at::Tensor* maybe(PyObject* o, const char* what) { return o == Py_None ? nullptr : &tensor(o, what); }

inline int64_t integer(PyObject* o, const char* what) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Refusal{PyExc_TypeError, std::string(what) + " must be an integer"};
  }
  return v;
}

inline double real(PyObject* o, const char* what) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Refusal{PyExc_TypeError, std::string(what) + " must be a number"};
  }
  return v;
}

inline const char* name_of(at::ScalarType t) { return c10::toString(t); }

inline void typed(const at::Tensor& t, at::ScalarType type, const char* what) {
  if (t.scalar_type() != type)
    refuse(std::string(what) + " must have dtype " + name_of(type) + ", got " + name_of(t.scalar_type()));
}

// The device all tensors of a call share: a kernel reads and writes only memory
// of the device it runs on.
struct Device {
  int index;

  Device(const at::Tensor& t, const char* what) : index(-1) {
    if (!t.is_cuda()) refuse(std::string(what) + " must be a device tensor");
    index = t.get_device();
  }
  void holds(const at::Tensor& t, const char* what) const {
    if (!t.is_cuda()) refuse(std::string(what) + " must be a device tensor");
    if (t.get_device() != index)
      refuse(std::string(what) + " is on " + t.device().str() + ", the other tensors on cuda:" + std::to_string(index));
  }
  // The address of a contiguous tensor of this type and size; nullptr for None.
  template <class T>
  T* plain(const at::Tensor* t, at::ScalarType type, int64_t numel, const char* what) const {
    if (!t) return nullptr;
    holds(*t, what);
    typed(*t, type, what);
    if (t->numel() != numel || !t->is_contiguous())
      refuse(std::string(what) + " must be contiguous with " + std::to_string(numel) + " elements");
    return static_cast<T*>(t->data_ptr());
  }
  // A [tokens, heads, head_dim] tensor: its address, and its strides.
  void* rows(const at::Tensor& t, at::ScalarType type, int64_t tokens, int64_t heads, int64_t dim, const char* what,
             int64_t* token_stride, int64_t* head_stride) const {
    holds(t, what);
    typed(t, type, what);
    if (t.dim() != 3 || t.size(0) != tokens || t.size(1) != heads || t.size(2) != dim)
      refuse(std::string(what) + " must be [" + std::to_string(tokens) + ", " + std::to_string(heads) + ", " +
             std::to_string(dim) + "]");
    if (t.stride(2) != 1) refuse(std::string(what) + " must have contiguous components");
    *token_stride = t.stride(0);
    *head_stride = t.stride(1);
    return t.data_ptr();
  }
  // Run a call with this device current, on its current stream.
  template <class Call>
  int launch(Call call) const {
    const c10::hip::OptionalHIPGuard guard(c10::hip::current_device() == index
                                               ? std::optional<c10::DeviceIndex>()
                                               : std::optional<c10::DeviceIndex>(c10::DeviceIndex(index)));
    void* stream = c10::hip::getCurrentHIPStream(c10::DeviceIndex(index)).stream();
    return call(stream);
  }
};

// TQ2_TYPE_* of a dtype, or -1, which the entry points refuse.
inline int64_t type_of(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return TQ2_TYPE_F32;
    case at::kHalf: return TQ2_TYPE_F16;
    case at::kBFloat16: return TQ2_TYPE_BF16;
    case at::kFloat8_e4m3fn: return TQ2_TYPE_E4M3;
    default: return -1;
  }
}

inline PyObject* new_ref(PyObject* o) {
  Py_INCREF(o);
  return o;
}

// An entry with `count` positional arguments; no C++ exception leaves it.
template <PyObject* (*body)(PyObject* const*), int count>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != count) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", count, n);
    return nullptr;
  }
  try {
    return body(args);
  } catch (const Refusal& r) {
    PyErr_SetString(r.type, r.text.c_str());
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    PyErr_Clear();
    PyErr_SetString(type ? type : PyExc_MemoryError, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

}  // namespace

#endif  // TQ2_BINDING_H
