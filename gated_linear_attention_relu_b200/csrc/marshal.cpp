// marshal.cpp -- CPython module between block.py and the C ABI (include/la.h): checks tensors, reads
// their addresses and strides, allocates what the caller leaves out, and makes the call.
//
// It only marshals; nothing is computed and nothing is kept.  It exists because the same in Python
// takes longer than a small call's kernels do (a list of 157 gradients: 130 us, here 20; a layer norm
// of a few rows: 15 us, here 7).  The library's entry points come by address (bind), so that they are
// those of the library that the package loaded.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstddef>
#include <cstring>
#include <string>
#include <vector>

#include "la.h"

namespace {

struct Failed {};  // a Python exception is set

struct Library {
  decltype(&la_cross_workspace_bytes_of) cross_workspace_bytes;
  decltype(&la_cross_forward) cross_forward;
  decltype(&la_cross_backward) cross_backward;
  decltype(&la_layernorm_workspace_bytes) layernorm_workspace_bytes;
  decltype(&la_layernorm_forward) layernorm_forward;
  decltype(&la_layernorm_backward) layernorm_backward;
  decltype(&la_clip_workspace_bytes) clip_workspace_bytes;
  decltype(&la_grad_norm) grad_norm;
  decltype(&la_clip_grad_norm) clip_grad_norm;
} lib;

using Shape = at::IntArrayRef;

template <typename... A>
[[noreturn]] void fail(const char* format, A... args) {
  PyErr_Format(PyExc_ValueError, format, args...);
  throw Failed{};
}

std::string text(Shape s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += std::to_string(s[i]) + (i + 1 < s.size() ? ", " : s.size() == 1 ? ",)" : ")");
  return t;
}

const at::Tensor* tensor(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) fail("%s: not a tensor", name);
  return &THPVariable_Unpack(o);
}

// A CUDA tensor of this type, shape and device; `dense`: contiguous, else contiguous rows.
void want(const at::Tensor& t, const char* name, Shape shape, at::ScalarType type, at::Device dev, bool dense) {
  if (t.layout() != at::kStrided || !t.is_cuda() || t.device() != dev)
    fail("%s: on %s, expected %s (a CUDA device)", name, t.device().str().c_str(), dev.str().c_str());
  if (t.scalar_type() != type)
    fail("%s: torch.%s, expected torch.%s", name, c10::toString(t.scalar_type()), c10::toString(type));
  if (t.sizes() != shape) fail("%s: shape %s, expected %s", name, text(t.sizes()).c_str(), text(shape).c_str());
  if (dense ? !t.is_contiguous() : t.numel() > 0 && shape.back() > 1 && t.stride(-1) != 1)
    fail(dense ? "%s: must be contiguous" : "%s: the elements of a row must be contiguous", name);
}

at::Device device_of(const at::Tensor* t, const char* name) {
  if (!t) fail("%s: a tensor is expected", name);
  if (!t->is_cuda()) fail("%s: on %s, expected a CUDA device", name, t->device().str().c_str());
  return t->device();
}

at::TensorOptions options(at::ScalarType type, at::Device dev) { return at::TensorOptions().dtype(type).device(dev); }

// The given tensor, checked, or a new one.
at::Tensor given_or_new(PyObject* o, const char* name, Shape shape, at::ScalarType type, at::Device dev, bool dense = true) {
  const at::Tensor* t = tensor(o, name);
  if (!t) return at::empty(shape, options(type, dev));
  want(*t, name, shape, type, dev, dense);
  return *t;
}

void* ptr(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }
template <typename T>
T* as(const at::Tensor* t) { return static_cast<T*>(ptr(t)); }

la_strides strides(const at::Tensor& t) { return {t.stride(0), t.stride(1), t.stride(2)}; }

struct Workspace {
  at::Tensor t;
  size_t bytes;
};
template <typename F>
Workspace workspace(PyObject* o, at::Device dev, F&& need) {
  if (const at::Tensor* t = tensor(o, "ws")) {
    if (t->device() != dev || t->scalar_type() != at::kByte || !t->is_contiguous())
      fail("ws: a contiguous uint8 tensor on %s is expected", dev.str().c_str());
    return {*t, size_t(t->numel())};
  }
  const size_t n = need();
  return {at::empty({int64_t(n > 16 ? n : 16)}, options(at::kByte, dev)), n};
}

PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }
PyObject* wrap(const at::Tensor* t) {
  if (t) return THPVariable_Wrap(*t);
  Py_RETURN_NONE;
}

template <typename P>
P problem(PyObject* bytes, size_t most) {
  P p = {};
  if (!PyBytes_Check(bytes) || size_t(PyBytes_GET_SIZE(bytes)) > most) fail("problem: bytes are expected");
  std::memcpy(&p, PyBytes_AS_STRING(bytes), size_t(PyBytes_GET_SIZE(bytes)));
  return p;
}

at::ScalarType type_of(int32_t dtype) { return dtype == LA_BF16 ? at::kBFloat16 : at::kFloat; }

// The status of a call that failed, as an int (the caller makes an LaError of it).
PyObject* status(int rc) { return PyLong_FromLong(rc); }

// Sets torch.OutOfMemoryError, as torch's own allocations do.
void out_of_memory(const char* what) {
  PyObject* torch = PyImport_ImportModule("torch");
  PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
  if (type) PyErr_SetString(type, what);
  Py_XDECREF(type);
  Py_XDECREF(torch);
}

// Runs f(args) with this thread's exceptions turned into Python's.
template <typename F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const Failed&) {
    return nullptr;
  } catch (const c10::OutOfMemoryError& e) {
    out_of_memory(e.what_without_backtrace());
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

bool count_is(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments, expected %zd", n, want);
  return false;
}

void want_masks(const at::Tensor* len, const at::Tensor* mask, const la_cross_problem& p, at::Device dev) {
  if (len) want(*len, "kv_len", {p.B}, at::kInt, dev, true);
  if (mask) {
    if (mask->scalar_type() != at::kBool && mask->scalar_type() != at::kByte)
      fail("key_mask: torch.%s, expected torch.bool or torch.uint8", c10::toString(mask->scalar_type()));
    want(*mask, "key_mask", {p.B, p.Nk}, mask->scalar_type(), dev, true);
  }
}

unsigned uses(unsigned call, const at::Tensor* len, const at::Tensor* mask) {
  return call | (len ? LA_CROSS_LENGTHS : 0) | (mask ? LA_CROSS_MASK : 0);
}

// cross_forward(head, Q, K, V, kv_len, key_mask, O, lse, return_lse, ws)
PyObject* cross_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 10)) return nullptr;
  return guarded([&]() -> PyObject* {
    la_cross_problem p = problem<la_cross_problem>(a[0], offsetof(la_cross_problem, q));
    const at::Tensor *Q = tensor(a[1], "Q"), *K = tensor(a[2], "K"), *V = tensor(a[3], "V"), *len = tensor(a[4], "kv_len"),
                     *mask = tensor(a[5], "key_mask");
    const at::Device dev = device_of(Q, "Q");
    const at::ScalarType type = type_of(p.dtype);
    const int64_t qs[4] = {p.B, p.H, p.Nq, p.d}, ks[4] = {p.B, p.Hkv, p.Nk, p.d};
    if (!K || !V) fail("K, V: tensors are expected");
    want(*Q, "Q", qs, type, dev, false);
    want(*K, "K", ks, type, dev, false);
    want(*V, "V", ks, type, dev, false);
    want_masks(len, mask, p, dev);
    const c10::cuda::CUDAGuard guard(dev);
    const at::Tensor O = a[6] == Py_None ? at::empty_like(*Q) : given_or_new(a[6], "O", qs, type, dev, false);
    const bool back = PyObject_IsTrue(a[8]) == 1, stats = back || a[7] != Py_None;
    at::Tensor lse;
    if (stats) lse = given_or_new(a[7], "lse", Shape(qs, 3), at::kFloat, dev);
    p.q = strides(*Q); p.k = strides(*K); p.v = strides(*V); p.o = strides(O);
    const Workspace ws = workspace(a[9], dev, [&] { return lib.cross_workspace_bytes(&p, uses(LA_CROSS_FORWARD, len, mask), 0); });
    const int rc = lib.cross_forward(&p, ptr(Q), ptr(K), ptr(V), as<int32_t>(len), as<uint8_t>(mask), O.data_ptr(),
                                     stats ? as<float>(&lse) : nullptr, ws.t.data_ptr(), ws.bytes,
                                     c10::cuda::getCurrentCUDAStream(dev.index()));
    if (rc) return status(rc);
    return back ? Py_BuildValue("NN", wrap(O), wrap(lse)) : wrap(O);
  });
}

// cross_backward(head, Q, K, V, O, lse, dO, kv_len, key_mask, dQ, dK, dV, ws)
PyObject* cross_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 13)) return nullptr;
  return guarded([&]() -> PyObject* {
    la_cross_problem p = problem<la_cross_problem>(a[0], offsetof(la_cross_problem, q));
    const char* names[6] = {"Q", "K", "V", "O", "lse", "dO"};
    const at::Tensor* t[6];
    for (int i = 0; i < 6; ++i) t[i] = tensor(a[1 + i], names[i]);
    const at::Device dev = device_of(t[0], "Q");
    const at::ScalarType type = type_of(p.dtype);
    const int64_t qs[4] = {p.B, p.H, p.Nq, p.d}, ks[4] = {p.B, p.Hkv, p.Nk, p.d};
    for (int i = 0; i < 6; ++i) {
      if (!t[i]) fail("%s: a tensor is expected", names[i]);
      if (i == 4)
        want(*t[i], names[i], Shape(qs, 3), at::kFloat, dev, true);
      else
        want(*t[i], names[i], i == 1 || i == 2 ? Shape(ks) : Shape(qs), type, dev, false);
    }
    const at::Tensor *len = tensor(a[7], "kv_len"), *mask = tensor(a[8], "key_mask");
    want_masks(len, mask, p, dev);
    const c10::cuda::CUDAGuard guard(dev);
    const char* gnames[3] = {"dQ", "dK", "dV"};
    at::Tensor g[3];
    for (int i = 0; i < 3; ++i)
      g[i] = a[9 + i] == Py_None ? at::empty_like(*t[i])
                                 : given_or_new(a[9 + i], gnames[i], i == 0 ? Shape(qs) : Shape(ks), type, dev, false);
    p.q = strides(*t[0]); p.k = strides(*t[1]); p.v = strides(*t[2]); p.o = strides(*t[3]); p.dout = strides(*t[5]);
    p.dq = strides(g[0]); p.dk = strides(g[1]); p.dv = strides(g[2]);
    const Workspace ws = workspace(a[12], dev, [&] { return lib.cross_workspace_bytes(&p, uses(LA_CROSS_BACKWARD, len, mask), 0); });
    const int rc = lib.cross_backward(&p, ptr(t[0]), ptr(t[1]), ptr(t[2]), as<int32_t>(len), as<uint8_t>(mask), ptr(t[3]),
                                      as<float>(t[4]), ptr(t[5]), g[0].data_ptr(), g[1].data_ptr(), g[2].data_ptr(),
                                      ws.t.data_ptr(), ws.bytes, c10::cuda::getCurrentCUDAStream(dev.index()));
    if (rc) return status(rc);
    return Py_BuildValue("NNN", wrap(g[0]), wrap(g[1]), wrap(g[2]));
  });
}

// A weight, bias or gradient of one: [groups, cols], or [cols] with one group.
void want_param(const at::Tensor* t, const char* name, const la_norm_problem& p, at::Device dev) {
  if (!t) return;
  const int64_t s[2] = {p.groups, p.cols};
  want(*t, name, t->dim() == 1 && p.groups == 1 ? Shape(s + 1, 1) : Shape(s, 2), at::kFloat, dev, true);
}

// layernorm_forward(problem, x, weight, bias, y, mean, rstd, return_stats)
PyObject* layernorm_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 8)) return nullptr;
  return guarded([&]() -> PyObject* {
    la_norm_problem p = problem<la_norm_problem>(a[0], sizeof(la_norm_problem));
    const at::Tensor *x = tensor(a[1], "x"), *w = tensor(a[2], "weight"), *b = tensor(a[3], "bias");
    const at::Device dev = device_of(x, "x");
    const at::ScalarType type = type_of(p.dtype);
    const int64_t shape[2] = {p.rows, p.cols};
    want(*x, "x", shape, type, dev, false);
    want_param(w, "weight", p, dev);
    want_param(b, "bias", p, dev);
    const c10::cuda::CUDAGuard guard(dev);
    const at::Tensor y = given_or_new(a[4], "y", shape, type, dev, false);
    const bool back = PyObject_IsTrue(a[7]) == 1, stats = back || a[5] != Py_None || a[6] != Py_None;
    at::Tensor mean, rstd;
    if (stats) {
      mean = given_or_new(a[5], "mean", Shape(shape, 1), at::kFloat, dev);
      rstd = given_or_new(a[6], "rstd", Shape(shape, 1), at::kFloat, dev);
    }
    p.sx = x->stride(0);
    p.sy = y.stride(0);
    const int rc = lib.layernorm_forward(&p, ptr(x), as<float>(w), as<float>(b), y.data_ptr(), stats ? as<float>(&mean) : nullptr,
                                         stats ? as<float>(&rstd) : nullptr, c10::cuda::getCurrentCUDAStream(dev.index()));
    if (rc) return status(rc);
    return back ? Py_BuildValue("NNN", wrap(y), wrap(mean), wrap(rstd)) : wrap(y);
  });
}

// layernorm_backward(problem, x, dy, mean, rstd, weight, dx, dweight, dbias, param_grads, ws)
PyObject* layernorm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 11)) return nullptr;
  return guarded([&]() -> PyObject* {
    la_norm_problem p = problem<la_norm_problem>(a[0], sizeof(la_norm_problem));
    const at::Tensor *x = tensor(a[1], "x"), *dy = tensor(a[2], "dy"), *mean = tensor(a[3], "mean"), *rstd = tensor(a[4], "rstd"),
                     *w = tensor(a[5], "weight");
    const at::Device dev = device_of(x, "x");
    const at::ScalarType type = type_of(p.dtype);
    const int64_t shape[2] = {p.rows, p.cols}, params[2] = {p.groups, p.cols};
    if (!dy || !mean || !rstd) fail("dy, mean, rstd: tensors are expected");
    want(*x, "x", shape, type, dev, false);
    want(*dy, "dy", shape, type, dev, false);
    want(*mean, "mean", Shape(shape, 1), at::kFloat, dev, true);
    want(*rstd, "rstd", Shape(shape, 1), at::kFloat, dev, true);
    want_param(w, "weight", p, dev);
    const c10::cuda::CUDAGuard guard(dev);
    const at::Tensor dx = given_or_new(a[6], "dx", shape, type, dev, false);
    const bool make = PyObject_IsTrue(a[9]) == 1;
    const char* names[2] = {"dweight", "dbias"};
    at::Tensor made[2];
    const at::Tensor* g[2];
    for (int i = 0; i < 2; ++i) {
      g[i] = tensor(a[7 + i], names[i]);
      want_param(g[i], names[i], p, dev);
      if (!g[i] && make) {
        made[i] = at::empty(params, options(at::kFloat, dev));
        g[i] = &made[i];
      }
    }
    p.sx = x->stride(0);
    p.sdy = dy->stride(0);
    p.sdx = dx.stride(0);
    const Workspace ws = workspace(a[10], dev, [&] {
      la_norm_problem q = p;
      q.sy = p.cols;
      return lib.layernorm_workspace_bytes(&q);
    });
    const int rc = lib.layernorm_backward(&p, ptr(x), ptr(dy), as<float>(w), as<float>(mean), as<float>(rstd), dx.data_ptr(),
                                          as<float>(g[0]), as<float>(g[1]), ws.t.data_ptr(), ws.bytes,
                                          c10::cuda::getCurrentCUDAStream(dev.index()));
    if (rc) return status(rc);
    return Py_BuildValue("NNN", wrap(dx), wrap(g[0]), wrap(g[1]));
  });
}

// A tensor of a gradient list: CUDA, contiguous, bf16 or fp32, on the list's device (-1: any, then set).
const at::Tensor& of_list(PyObject* list, const char* what, Py_ssize_t i, int* dev) {
  PyObject* item = PyList_GET_ITEM(list, i);
  if (!THPVariable_Check(item)) fail("%s %zd: not a tensor", what, i);
  const at::Tensor& t = THPVariable_Unpack(item);
  if (t.scalar_type() != at::kBFloat16 && t.scalar_type() != at::kFloat)
    fail("%s %zd: torch.%s, expected torch.bfloat16 or torch.float32", what, i, c10::toString(t.scalar_type()));
  if (!t.is_cuda() || t.layout() != at::kStrided || (*dev >= 0 && t.get_device() != *dev))
    fail("%s %zd: on %s, expected one CUDA device for all", what, i, t.device().str().c_str());
  *dev = static_cast<int>(t.get_device());
  if (!t.is_contiguous()) fail("%s %zd: must be contiguous", what, i);
  return t;
}

// clip(grads, outs, max_norm or None, norm, ws)
PyObject* clip(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 5)) return nullptr;
  return guarded([&]() -> PyObject* {
    if (!PyList_Check(a[0]) || (a[1] != Py_None && !PyList_Check(a[1]))) fail("gradients: lists of tensors are expected");
    const Py_ssize_t count = PyList_GET_SIZE(a[0]);
    if (a[1] != Py_None && PyList_GET_SIZE(a[1]) != count)
      fail("out: %zd tensors for %zd gradients", PyList_GET_SIZE(a[1]), count);
    std::vector<la_grad> g(static_cast<size_t>(count));
    int index = -1;
    for (Py_ssize_t i = 0; i < count; ++i) {
      const at::Tensor& t = of_list(a[0], "gradient", i, &index);
      const at::Tensor& o = a[1] == Py_None ? t : of_list(a[1], "out", i, &index);
      if (o.numel() != t.numel() || o.scalar_type() != t.scalar_type())
        fail("out %zd: must have its gradient's size and type", i);
      g[i] = {t.data_ptr(), o.data_ptr(), t.numel(), t.scalar_type() == at::kBFloat16 ? LA_BF16 : LA_F32, 0};
    }
    const at::Tensor* given = tensor(a[3], "norm");
    if (index < 0) index = given && given->is_cuda() ? static_cast<int>(given->get_device()) : c10::cuda::current_device();
    const at::Device dev(at::kCUDA, static_cast<c10::DeviceIndex>(index));
    if (given && (given->numel() != 1 || given->scalar_type() != at::kFloat || given->device() != dev))
      fail("norm: one fp32 element on %s is expected", dev.str().c_str());
    double max_norm = 0.0;
    if (a[2] != Py_None) {
      max_norm = PyFloat_AsDouble(a[2]);
      if (max_norm == -1.0 && PyErr_Occurred()) throw Failed{};
    }
    const c10::cuda::CUDAGuard guard(dev);
    const at::Tensor norm = given ? *given : at::empty({}, options(at::kFloat, dev));
    const Workspace ws = workspace(a[4], dev, [&] { return lib.clip_workspace_bytes(count); });
    const cudaStream_t st = c10::cuda::getCurrentCUDAStream(dev.index());
    float* out = static_cast<float*>(norm.data_ptr());
    const int rc = a[2] == Py_None ? lib.grad_norm(g.data(), count, out, ws.t.data_ptr(), ws.bytes, st)
                                   : lib.clip_grad_norm(g.data(), count, static_cast<float>(max_norm), out, ws.t.data_ptr(),
                                                        ws.bytes, st);
    return rc ? status(rc) : wrap(norm);
  });
}

// bind(addresses): the library's entry points, in the order of Library.
PyObject* bind(PyObject*, PyObject* args) {
  constexpr Py_ssize_t N = sizeof(Library) / sizeof(void*);
  void* p[N];
  if (!count_is(PyTuple_GET_SIZE(args), N)) return nullptr;
  for (Py_ssize_t i = 0; i < N; ++i) {
    p[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(args, i));
    if (!p[i]) return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "entry point %zd is null", i);
  }
  std::memcpy(&lib, p, sizeof lib);
  Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"bind", bind, METH_VARARGS, nullptr},
                         FAST(cross_forward),
                         FAST(cross_backward),
                         FAST(layernorm_forward),
                         FAST(layernorm_backward),
                         FAST(clip),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module); }
