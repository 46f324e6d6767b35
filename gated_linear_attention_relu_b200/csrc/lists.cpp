// lists.cpp -- CPython helper that turns a list of torch tensors into the la_grad array of the C ABI.
//
// A gradient list has hundreds of tensors, and asking each for its address, size, type, device and
// layout from Python takes longer than the kernels do; here it is a few nanoseconds a tensor.  It only
// marshals: nothing is computed and nothing is kept.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <torch/csrc/autograd/python_variable.h>

#include "la.h"

namespace {

// The tensor at place i, checked: CUDA, contiguous, bf16 or fp32, on device `dev` (-1: any, and then
// set).  Null with a Python exception otherwise.
const at::Tensor* take(PyObject* item, const char* what, Py_ssize_t i, int* dev) {
  if (!THPVariable_Check(item)) {
    PyErr_Format(PyExc_ValueError, "%s %zd: not a tensor", what, i);
    return nullptr;
  }
  const at::Tensor& t = THPVariable_Unpack(item);
  if (t.scalar_type() != at::kBFloat16 && t.scalar_type() != at::kFloat) {
    PyErr_Format(PyExc_ValueError, "%s %zd: %s, expected torch.bfloat16 or torch.float32", what, i,
                 c10::toString(t.scalar_type()));
    return nullptr;
  }
  if (!t.is_cuda() || t.layout() != at::kStrided || (*dev >= 0 && t.get_device() != *dev)) {
    PyErr_Format(PyExc_ValueError, "%s %zd: on %s, expected one CUDA device for all", what, i, t.device().str().c_str());
    return nullptr;
  }
  *dev = static_cast<int>(t.get_device());
  if (!t.is_contiguous()) {
    PyErr_Format(PyExc_ValueError, "%s %zd: must be contiguous", what, i);
    return nullptr;
  }
  return &t;
}

// grad_list(tensors, outs or None) -> (bytes of the la_grad array, device index or -1 for no tensors)
PyObject* grad_list(PyObject*, PyObject* args) {
  PyObject *grads, *outs;
  if (!PyArg_ParseTuple(args, "O!O", &PyList_Type, &grads, &outs)) return nullptr;
  const Py_ssize_t n = PyList_GET_SIZE(grads);
  if (outs != Py_None && !PyList_Check(outs)) {
    PyErr_SetString(PyExc_ValueError, "out: a list of tensors is expected");
    return nullptr;
  }
  if (outs != Py_None && PyList_GET_SIZE(outs) != n)
    return PyErr_Format(PyExc_ValueError, "out: %zd tensors for %zd gradients", PyList_GET_SIZE(outs), n);
  PyObject* bytes = PyBytes_FromStringAndSize(nullptr, n * static_cast<Py_ssize_t>(sizeof(la_grad)));
  if (!bytes) return nullptr;
  la_grad* g = reinterpret_cast<la_grad*>(PyBytes_AS_STRING(bytes));
  int dev = -1;
  try {
    for (Py_ssize_t i = 0; i < n; ++i) {
      const at::Tensor* t = take(PyList_GET_ITEM(grads, i), "gradient", i, &dev);
      const at::Tensor* o = t && outs != Py_None ? take(PyList_GET_ITEM(outs, i), "out", i, &dev) : t;
      if (o && (o->numel() != t->numel() || o->scalar_type() != t->scalar_type())) {
        PyErr_Format(PyExc_ValueError, "out %zd: must have its gradient's size and type", i);
        o = nullptr;
      }
      if (!o) {
        Py_DECREF(bytes);
        return nullptr;
      }
      g[i].in = t->const_data_ptr();
      g[i].out = o->mutable_data_ptr();
      g[i].numel = t->numel();
      g[i].dtype = t->scalar_type() == at::kBFloat16 ? LA_BF16 : LA_F32;
      g[i].reserved = 0;
    }
  } catch (const std::exception& e) {  // (a tensor without storage, for one)
    Py_DECREF(bytes);
    PyErr_SetString(PyExc_ValueError, e.what());
    return nullptr;
  }
  return Py_BuildValue("Ni", bytes, dev);
}

PyMethodDef methods[] = {{"grad_list", grad_list, METH_VARARGS, "The la_grad array of a list of tensors."},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_lists", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__lists(void) { return PyModule_Create(&module); }
