// dispatch.cpp -- calls a C entry point of libdecode_attn with torch tensors: a CPython module
// with one function,
//   call(address, stream, n, tensor_1 .. tensor_n, float ...) -> status
// which fills a da_tensor_t for each tensor (None: a null pointer) from the tensor's own fields
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

constexpr int kMaxTensors = 8, kMaxFloats = 3;

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

PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs < 3) {
    PyErr_SetString(PyExc_TypeError, "call(address, stream, n, tensors ..., floats ...)");
    return nullptr;
  }
  void* fn = PyLong_AsVoidPtr(args[0]);
  if (!fn && !PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null function");
  if (PyErr_Occurred()) return nullptr;
  void* stream = args[1] == Py_None ? nullptr : PyLong_AsVoidPtr(args[1]);
  const long n = PyLong_AsLong(args[2]);
  if (PyErr_Occurred()) return nullptr;
  const Py_ssize_t floats = nargs - 3 - n;
  if (n < 3 || n > kMaxTensors || !(floats == 0 || floats == 1 || floats == kMaxFloats)) {
    PyErr_SetString(PyExc_TypeError, "3 to 8 tensors and none, one or three floats");
    return nullptr;
  }
  da_tensor_t desc[kMaxTensors];
  const da_tensor_t* d[kMaxTensors];
  float f[kMaxFloats] = {};
  Devices dev;
  try {
    for (long i = 0; i < n; ++i) {
      d[i] = nullptr;
      if (args[3 + i] == Py_None) continue;
      if (!describe(args[3 + i], &desc[i], &dev)) return nullptr;
      d[i] = &desc[i];
    }
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
  for (Py_ssize_t i = 0; i < floats; ++i) {
    f[i] = (float)PyFloat_AsDouble(args[3 + n + i]);
    if (PyErr_Occurred()) return nullptr;
  }
  int status = 0;
  Py_BEGIN_ALLOW_THREADS;
  switch (n) {
    case 3: status = invoke_floats<3>(fn, d, f, (int)floats, stream); break;
    case 4: status = invoke_floats<4>(fn, d, f, (int)floats, stream); break;
    case 5: status = invoke_floats<5>(fn, d, f, (int)floats, stream); break;
    case 6: status = invoke_floats<6>(fn, d, f, (int)floats, stream); break;
    case 7: status = invoke_floats<7>(fn, d, f, (int)floats, stream); break;
    default: status = invoke_floats<8>(fn, d, f, (int)floats, stream); break;
  }
  Py_END_ALLOW_THREADS;
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

PyMethodDef methods[] = {
    {"call", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call)), METH_FASTCALL,
     "call(address, stream, n, tensors ..., floats ...) -> status"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_da_dispatch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__da_dispatch() { return PyModule_Create(&module); }
