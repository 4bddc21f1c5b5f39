// marshal.cpp -- the Python binding's argument marshalling in C++ (module
// _marshal): a call of a C entry point of include/ep.h from torch tensors.  It
// does what the ctypes wrappers do -- checks that a tensor is a contiguous one
// on the device the call runs on, describes it as an ep_tensor_t, passes the
// current stream -- without a Python object per argument: a call of eight
// tensors takes 8.2 us through ctypes, of which the library and the launch take
// 3.9.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>

#include "ep.h"

namespace {

constexpr int kMaxArgs = 9;   // of an entry point, the stream among them
constexpr int kMaxViews = 12;  // of a struct of views

// ep_dtype_t of a tensor, -1 if the library has none.
int32_t dtype_of(const at::Tensor &t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return EP_DTYPE_BF16;
    case at::kFloat: return EP_DTYPE_FP32;
    case at::kFloat8_e4m3fn: return EP_DTYPE_FP8_E4M3;
    case at::kInt: return EP_DTYPE_INT32;
    case at::kChar: return EP_DTYPE_INT8;
    default: return -1;
  }
}

// Describes `o` (a tensor) with `tag` in *v; false with a Python error set.
bool describe(PyObject *o, int32_t tag, int64_t dev, ep_tensor_t *v) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "expected a torch.Tensor, got %s", Py_TYPE(o)->tp_name);
    return false;
  }
  const at::Tensor &t = THPVariable_Unpack(o);
  if (!t.is_cuda()) {
    PyErr_SetString(PyExc_ValueError, "tensors passed to the library must be on the GPU");
    return false;
  }
  if (t.get_device() != dev) {
    PyErr_Format(PyExc_ValueError, "tensor on cuda:%d, the call runs on cuda:%d", (int)t.get_device(),
                 (int)dev);
    return false;
  }
  if (!t.is_contiguous()) {
    PyErr_SetString(PyExc_ValueError, "tensors passed to the library must be contiguous");
    return false;
  }
  const int32_t dt = dtype_of(t);
  if (dt < 0) {
    PyErr_Format(PyExc_TypeError, "unsupported dtype %s", c10::toString(t.scalar_type()));
    return false;
  }
  const int64_t nd = t.dim();
  if (nd < 1 || nd > 4) {
    PyErr_SetString(PyExc_ValueError, "tensors must have 1..4 dimensions");
    return false;
  }
  v->data = t.numel() > 0 ? t.data_ptr() : nullptr;
  v->dtype = dt;
  v->tag = tag;
  v->ndim = (int32_t)nd;
  v->reserved = 0;
  for (int i = 0; i < 4; ++i) v->sizes[i] = i < nd ? t.size(i) : 0;
  return true;
}

// The device and address of a call's stream argument: None for the current
// stream, or a torch.cuda.Stream's (device, address) as two ints in a tuple.
bool stream_of(PyObject *o, int64_t *dev, void **stream) {
  if (o == Py_None) {
    *dev = c10::hip::current_device();
    *stream = c10::hip::getCurrentHIPStream((c10::DeviceIndex)*dev).stream();
    return true;
  }
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 2) {
    PyErr_SetString(PyExc_TypeError, "stream: None or (device, address)");
    return false;
  }
  *dev = PyLong_AsLongLong(PyTuple_GET_ITEM(o, 0));
  *stream = PyLong_AsVoidPtr(PyTuple_GET_ITEM(o, 1));
  return !PyErr_Occurred();
}

// call(fn, tags, stream, args...) -> status.  fn: address of the entry point;
// tags: one byte per argument, a tensor's ep_tensor_tag_t or 0xFF for an
// address given as an int; None is NULL.  stream: as stream_of takes it; it is
// passed last.
PyObject *call(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n < 3 || !PyBytes_Check(args[1])) {
    PyErr_SetString(PyExc_TypeError, "call(fn, tags, stream, args...)");
    return nullptr;
  }
  void *fn = PyLong_AsVoidPtr(args[0]);
  const Py_ssize_t m = n - 3;
  if (PyErr_Occurred()) return nullptr;
  if (!fn || m != PyBytes_GET_SIZE(args[1]) || m + 1 > kMaxArgs) {
    PyErr_SetString(PyExc_TypeError, "one tag per argument");
    return nullptr;
  }
  const auto *tags = reinterpret_cast<const unsigned char *>(PyBytes_AS_STRING(args[1]));
  int64_t dev;
  void *p[kMaxArgs] = {};
  ep_tensor_t views[kMaxArgs];
  try {
    if (!stream_of(args[2], &dev, &p[m])) return nullptr;
    for (Py_ssize_t i = 0; i < m; ++i) {
      PyObject *o = args[3 + i];
      if (o == Py_None) continue;
      if (tags[i] == 0xFF) {
        p[i] = PyLong_AsVoidPtr(o);
        if (PyErr_Occurred()) return nullptr;
        continue;
      }
      if (!describe(o, tags[i], dev, &views[i])) return nullptr;
      p[i] = &views[i];
    }
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
  ep_status_t st = EP_ERR_INVALID_ARG;
  // every entry point called here takes pointers only, the stream last
  using P = void *;
  Py_BEGIN_ALLOW_THREADS
  switch (m + 1) {
    case 4: st = reinterpret_cast<ep_status_t (*)(P, P, P, P)>(fn)(p[0], p[1], p[2], p[3]); break;
    case 6:
      st = reinterpret_cast<ep_status_t (*)(P, P, P, P, P, P)>(fn)(p[0], p[1], p[2], p[3], p[4], p[5]);
      break;
    case 7:
      st = reinterpret_cast<ep_status_t (*)(P, P, P, P, P, P, P)>(fn)(p[0], p[1], p[2], p[3], p[4],
                                                                      p[5], p[6]);
      break;
    case 8:
      st = reinterpret_cast<ep_status_t (*)(P, P, P, P, P, P, P, P)>(fn)(p[0], p[1], p[2], p[3],
                                                                         p[4], p[5], p[6], p[7]);
      break;
    case 9:
      st = reinterpret_cast<ep_status_t (*)(P, P, P, P, P, P, P, P, P)>(fn)(
          p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], p[8]);
      break;
    default: break;   // no entry point of this length: EP_ERR_INVALID_ARG
  }
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

// call_views(fn, tags, stream, rule, tensors...) -> status, for entry points
// (rule, struct of views, stream): the tensors' views, or NULL for None, are the
// struct's members in order.
PyObject *call_views(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n < 4 || !PyBytes_Check(args[1]) || n - 4 != PyBytes_GET_SIZE(args[1]) || n - 4 > kMaxViews) {
    PyErr_SetString(PyExc_TypeError, "call_views(fn, tags, stream, rule, tensors...), one tag per tensor");
    return nullptr;
  }
  void *fn = PyLong_AsVoidPtr(args[0]), *rule = PyLong_AsVoidPtr(args[3]), *stream;
  if (PyErr_Occurred()) return nullptr;
  const auto *tags = reinterpret_cast<const unsigned char *>(PyBytes_AS_STRING(args[1]));
  int64_t dev;
  ep_tensor_t views[kMaxViews];
  ep_tensor_t *p[kMaxViews] = {};
  try {
    if (!stream_of(args[2], &dev, &stream)) return nullptr;
    for (Py_ssize_t i = 0; i < n - 4; ++i) {
      if (args[4 + i] == Py_None) continue;
      if (!describe(args[4 + i], tags[i], dev, &views[i])) return nullptr;
      p[i] = &views[i];
    }
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
  ep_status_t st;
  Py_BEGIN_ALLOW_THREADS
  st = reinterpret_cast<ep_status_t (*)(void *, void *, void *)>(fn)(rule, p, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

PyMethodDef methods[] = {
    {"call_views", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call_views)), METH_FASTCALL,
     "call_views(fn, tags, stream, rule, tensors...) -> status"},
    {"call", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call)), METH_FASTCALL,
     "call(fn, tags, stream, args...) -> status"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
