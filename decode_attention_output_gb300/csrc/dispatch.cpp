// dispatch.cpp -- calls a C entry point of libdecode_attn with torch tensors: a CPython module
// with two functions,
//   call(address, stream, n, tensor_1 .. tensor_n, float ...) -> status
//   call_ints(address, stream, n, tensor_1 .. tensor_n, float, int ...) -> status
// the second for entry points that take one float and then one or two int32_t before the stream;
// it fills a da_tensor_t for each tensor (None: a null pointer) from the tensor's own fields
// and calls the function at `address`, whose parameters are n descriptors, the floats and the
// stream. It reads a tensor in some 20 ns; asking for the same fields from Python takes 0.8 us a
// tensor on the GB300's host, 6 us of a 10 us call that writes one decode step's tokens.
#include <Python.h>
#include <c10/core/impl/DeviceGuardImplInterface.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <exception>
#include <string>
#include <utility>

#include "decode_attn.h"

namespace {

constexpr int kMaxTensors = 8, kMaxFloats = 3, kMostTensors = 15, kMaxInts = 2;

int dtype_code(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return DA_DTYPE_BF16;
    case at::kFloat: return DA_DTYPE_F32;
    case at::kInt: return DA_DTYPE_I32;
    case at::kFloat8_e4m3fn: return DA_DTYPE_E4M3;
    default: return 0;
  }
}

// The library launches on the current device and reads every tensor there, but sees addresses
// alone. A tensor on the host or on another GPU goes to it with a null address, which every entry
// point refuses (a wrong type of that tensor before it); the caller is then told where it lies.
struct Devices {
  int current = -1;              // asked for once a call
  const at::Tensor* off = nullptr;  // the first tensor that is not there
};
bool on_current_device(const at::Tensor& t, Devices* dev) {
  if (!t.is_cuda()) return false;
  if (dev->current < 0) dev->current = c10::impl::getDeviceGuardImpl(c10::DeviceType::CUDA)->getDevice().index();
  return t.device().index() == dev->current;
}

bool describe(PyObject* o, da_tensor_t* d, Devices* dev) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "expected a torch.Tensor, got %.100s", Py_TYPE(o)->tp_name);
    return false;
  }
  const at::Tensor& t = THPVariable_Unpack(o);
  d->dtype = dtype_code(t.scalar_type());
  if (!d->dtype) {
    PyErr_Format(PyExc_TypeError, "unsupported dtype %s", c10::toString(t.scalar_type()));
    return false;
  }
  const int64_t n = t.dim();
  if (n > 4) {
    PyErr_SetString(PyExc_ValueError, "at most 4 dimensions");
    return false;
  }
  d->ndim = (int32_t)n;
  d->data = nullptr;
  if (t.numel()) {
    if (on_current_device(t, dev)) d->data = t.data_ptr();
    else if (!dev->off) dev->off = &t;
  }
  const at::IntArrayRef shape = t.sizes(), stride = t.strides();
  for (int64_t i = 0; i < 4; ++i) {
    d->shape[i] = i < n ? shape[i] : 0;
    d->stride[i] = i < n ? stride[i] : 0;
  }
  return true;
}

template <size_t>
using Desc = const da_tensor_t*;
template <size_t>
using F32 = float;

template <size_t... T, size_t... F>
int invoke(void* fn, const da_tensor_t* const* d, const float* f, void* stream, std::index_sequence<T...>,
           std::index_sequence<F...>) {
  return reinterpret_cast<int (*)(Desc<T>..., F32<F>..., void*)>(fn)(d[T]..., f[F]..., stream);
}

template <size_t T>
int invoke_floats(void* fn, const da_tensor_t* const* d, const float* f, int floats, void* stream) {
  using Ts = std::make_index_sequence<T>;
  switch (floats) {
    case 0: return invoke(fn, d, f, stream, Ts(), std::make_index_sequence<0>());
    case 1: return invoke(fn, d, f, stream, Ts(), std::make_index_sequence<1>());
    default: return invoke(fn, d, f, stream, Ts(), std::make_index_sequence<3>());
  }
}

template <size_t>
using I32 = int32_t;

template <size_t... T, size_t... I>
int invoke_ints(void* fn, const da_tensor_t* const* d, float f, const int32_t* x, void* stream, std::index_sequence<T...>,
                std::index_sequence<I...>) {
  return reinterpret_cast<int (*)(Desc<T>..., float, I32<I>..., void*)>(fn)(d[T]..., f, x[I]..., stream);
}

// What both calls begin with: the address, the stream, the count of tensors and the tensors.
struct Begun {
  void* fn;
  void* stream;
  long n;
  da_tensor_t desc[kMostTensors];
  const da_tensor_t* d[kMostTensors];
  Devices dev;
};
bool begin(PyObject* const* args, Py_ssize_t nargs, const char* form, Begun* c) {
  if (nargs < 3) {
    PyErr_SetString(PyExc_TypeError, form);
    return false;
  }
  c->fn = PyLong_AsVoidPtr(args[0]);
  if (!c->fn && !PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null function");
  if (PyErr_Occurred()) return false;
  c->stream = args[1] == Py_None ? nullptr : PyLong_AsVoidPtr(args[1]);
  c->n = PyLong_AsLong(args[2]);
  return !PyErr_Occurred();
}
bool take_tensors(PyObject* const* args, Begun* c) {
  try {
    for (long i = 0; i < c->n; ++i) {
      c->d[i] = nullptr;
      if (args[3 + i] == Py_None) continue;
      if (!describe(args[3 + i], &c->desc[i], &c->dev)) return false;
      c->d[i] = &c->desc[i];
    }
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return false;
  }
  return true;
}
PyObject* end(const Begun& c, int status) {
  const Devices& dev = c.dev;
  if (dev.off && (status == DA_ERR_NULL || status == DA_OK)) {
    const std::string where = dev.off->device().str();
    if (dev.off->is_cuda())
      PyErr_Format(PyExc_ValueError, "expected a tensor on the current device cuda:%d, got one on %s", dev.current, where.c_str());
    else
      PyErr_Format(PyExc_ValueError, "expected a CUDA tensor, got one on %s", where.c_str());
    return nullptr;
  }
  return PyLong_FromLong(status);
}

PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  Begun c;
  if (!begin(args, nargs, "call(address, stream, n, tensors ..., floats ...)", &c)) return nullptr;
  const long n = c.n;
  const Py_ssize_t floats = nargs - 3 - n;
  if (n < 3 || n > kMaxTensors || !(floats == 0 || floats == 1 || floats == kMaxFloats)) {
    PyErr_SetString(PyExc_TypeError, "3 to 8 tensors and none, one or three floats");
    return nullptr;
  }
  if (!take_tensors(args, &c)) return nullptr;
  float f[kMaxFloats] = {};
  for (Py_ssize_t i = 0; i < floats; ++i) {
    f[i] = (float)PyFloat_AsDouble(args[3 + n + i]);
    if (PyErr_Occurred()) return nullptr;
  }
  int status = 0;
  Py_BEGIN_ALLOW_THREADS;
  switch (n) {
    case 3: status = invoke_floats<3>(c.fn, c.d, f, (int)floats, c.stream); break;
    case 4: status = invoke_floats<4>(c.fn, c.d, f, (int)floats, c.stream); break;
    case 5: status = invoke_floats<5>(c.fn, c.d, f, (int)floats, c.stream); break;
    case 6: status = invoke_floats<6>(c.fn, c.d, f, (int)floats, c.stream); break;
    case 7: status = invoke_floats<7>(c.fn, c.d, f, (int)floats, c.stream); break;
    default: status = invoke_floats<8>(c.fn, c.d, f, (int)floats, c.stream); break;
  }
  Py_END_ALLOW_THREADS;
  return end(c, status);
}

PyObject* call_ints(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  Begun c;
  if (!begin(args, nargs, "call_ints(address, stream, n, tensors ..., float, ints ...)", &c)) return nullptr;
  const long n = c.n;
  const Py_ssize_t ints = nargs - 4 - n;
  if (!((n == 6 && ints == 2) || (n == 8 && ints == 2) || (n == 9 && ints == 1) || (n == 15 && ints == 1))) {
    PyErr_SetString(PyExc_TypeError, "6 or 8 tensors, a float and two ints, or 9 or 15 tensors, a float and an int");
    return nullptr;
  }
  if (!take_tensors(args, &c)) return nullptr;
  const float f = (float)PyFloat_AsDouble(args[3 + n]);
  if (PyErr_Occurred()) return nullptr;
  int32_t x[kMaxInts] = {};
  for (Py_ssize_t i = 0; i < ints; ++i) {
    const long long v = PyLong_AsLongLong(args[4 + n + i]);
    if (PyErr_Occurred()) return nullptr;
    if (v != (int32_t)v) {
      PyErr_SetString(PyExc_ValueError, "a number that does not fit 32 bits");
      return nullptr;
    }
    x[i] = (int32_t)v;
  }
  int status = 0;
  using One = std::make_index_sequence<1>;
  using Two = std::make_index_sequence<2>;
  Py_BEGIN_ALLOW_THREADS;
  switch (n) {
    case 6: status = invoke_ints(c.fn, c.d, f, x, c.stream, std::make_index_sequence<6>(), Two()); break;
    case 8: status = invoke_ints(c.fn, c.d, f, x, c.stream, std::make_index_sequence<8>(), Two()); break;
    case 9: status = invoke_ints(c.fn, c.d, f, x, c.stream, std::make_index_sequence<9>(), One()); break;
    default: status = invoke_ints(c.fn, c.d, f, x, c.stream, std::make_index_sequence<15>(), One()); break;
  }
  Py_END_ALLOW_THREADS;
  return end(c, status);
}

PyMethodDef methods[] = {
    {"call", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call)), METH_FASTCALL,
     "call(address, stream, n, tensors ..., floats ...) -> status"},
    {"call_ints", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call_ints)), METH_FASTCALL,
     "call_ints(address, stream, n, tensors ..., float, ints ...) -> status"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_da_dispatch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__da_dispatch() { return PyModule_Create(&module); }
