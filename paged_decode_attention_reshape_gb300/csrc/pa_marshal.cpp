// pa_marshal.cpp -- pa_tensor descriptors (include/pa.h) of torch tensors, all of a call's at once.
//
// A small call is on the host for longer than on the GPU, and most of that in reading each tensor's
// pointer, type, extents and strides through Python (0.6 us a tensor); here they are read from the tensor
// itself.  describe(kinds, *tensors) returns a tuple with each tensor's descriptor as bytes, None for
// None.  kinds: one character per tensor, 't' or 'c' (a cache: a rank-3 uint8 tensor holds a 4-bit cache's
// pages).
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>

#include "../../include/pa.h"

namespace {

int dtype_code(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return PA_F32;
    case at::kBFloat16: return PA_BF16;
    case at::kHalf: return PA_F16;
    case at::kByte: case at::kFloat8_e4m3fn: return PA_FP8_E4M3;
    case at::kInt: return PA_I32;
    case at::kLong: return PA_I64;
    default: return -1;
  }
}

PyObject *one(PyObject *x, char kind) {
  if (x == Py_None) Py_RETURN_NONE;
  if (!THPVariable_Check(x)) {
    PyErr_Format(PyExc_TypeError, "expected a torch.Tensor, got %s", Py_TYPE(x)->tp_name);
    return nullptr;
  }
  const at::Tensor &t = THPVariable_Unpack(x);
  const int64_t rank = t.dim();
  if (rank > 5) {
    PyErr_SetString(PyExc_ValueError, "rank > 5");
    return nullptr;
  }
  int code = dtype_code(t.scalar_type());
  if (code < 0) {
    PyObject *name = PyObject_GetAttrString(x, "dtype");
    if (name) PyErr_SetObject(PyExc_KeyError, name);
    Py_XDECREF(name);
    return nullptr;
  }
  if (kind == 'c' && rank == 3 && t.scalar_type() == at::kByte) code = PA_FP4_E2M1;
  pa_tensor d;
  std::memset(&d, 0, sizeof(d));
  d.data = t.numel() ? t.data_ptr() : nullptr;
  d.dtype = code;
  d.ndim = static_cast<int32_t>(rank);
  for (int64_t i = 0; i < rank; ++i) {
    d.shape[i] = t.size(i);
    d.stride[i] = t.stride(i);
  }
  return PyBytes_FromStringAndSize(reinterpret_cast<const char *>(&d), sizeof(d));
}

PyObject *describe(PyObject *, PyObject *const *args, Py_ssize_t n) {
  Py_ssize_t len = 0;
  char *kinds = nullptr;
  if (n < 1 || PyBytes_AsStringAndSize(args[0], &kinds, &len) < 0 || len != n - 1) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "describe(kinds, *tensors): a character per tensor");
    return nullptr;
  }
  PyObject *out = PyTuple_New(len);
  if (!out) return nullptr;
  for (Py_ssize_t i = 0; i < len; ++i) {
    PyObject *d = nullptr;
    try {
      d = one(args[i + 1], kinds[i]);
    } catch (const std::exception &e) {
      PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    if (!d) {
      Py_DECREF(out);
      return nullptr;
    }
    PyTuple_SET_ITEM(out, i, d);
  }
  return out;
}

PyMethodDef methods[] = {{"describe", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(describe)), METH_FASTCALL,
                          "describe(kinds, *tensors) -> tuple of pa_tensor bytes"},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit__marshal(void) {
  PyObject *m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch", PA_TORCH) < 0) {  // whose tensors it reads
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
