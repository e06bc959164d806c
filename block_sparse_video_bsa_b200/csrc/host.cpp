// What the Python wrappers of the operators around the attention do a call, in
// C++: a call on one token is 5 us on the GPU, and reading a dozen tensors'
// layouts, making two outputs and passing the pointers on took Python 9.
//
//   layout(*tensors) -> bytes     types, devices, sizes and strides (never
//                                 addresses); None may stand for a tensor
//   empty(sizes, strides, dtype of, device of) -> tensor
//   call(function, *arguments) -> int
//
// Checks stay in Python, once a layout.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/core/LegacyTypeDispatch.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/Dtype.h>

#include <cstring>
#include <string>

namespace {

void put(std::string* s, const void* p, size_t n) { s->append(static_cast<const char*>(p), n); }

PyObject* layout(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  std::string key;
  key.reserve(512);
  for (Py_ssize_t i = 0; i < n; ++i) {
    if (args[i] == Py_None) {
      key.push_back('\0');
      continue;
    }
    if (!THPVariable_Check(args[i])) {
      PyErr_SetString(PyExc_TypeError, "a tensor or None is expected");
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(args[i]);
    const int32_t head[4] = {1 + static_cast<int32_t>(t.dim()), static_cast<int32_t>(t.scalar_type()),
                             static_cast<int32_t>(t.device().type()), t.get_device()};
    put(&key, head, sizeof(head));
    put(&key, t.sizes().data(), t.sizes().size() * sizeof(int64_t));
    put(&key, t.strides().data(), t.strides().size() * sizeof(int64_t));
  }
  return PyBytes_FromStringAndSize(key.data(), static_cast<Py_ssize_t>(key.size()));
  END_HANDLE_TH_ERRORS
}

bool numbers(PyObject* o, int64_t* out, Py_ssize_t* n) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) > 8) {
    PyErr_SetString(PyExc_TypeError, "a tuple of 8 numbers at most is expected");
    return false;
  }
  *n = PyTuple_GET_SIZE(o);
  for (Py_ssize_t i = 0; i < *n; ++i) out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(o, i));
  return !PyErr_Occurred();
}

PyObject* empty(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  int64_t size[8], stride[8];
  Py_ssize_t dims, same;
  if (n != 4 || !THPDtype_Check(args[2]) || !THPVariable_Check(args[3])) {
    PyErr_SetString(PyExc_TypeError, "empty(sizes, strides, dtype, tensor)");
    return nullptr;
  }
  if (!numbers(args[0], size, &dims) || !numbers(args[1], stride, &same)) return nullptr;
  if (dims != same) {
    PyErr_SetString(PyExc_ValueError, "sizes and strides differ in number");
    return nullptr;
  }
  at::AutoDispatchBelowADInplaceOrView plain;
  return THPVariable_Wrap(at::empty_strided(
      at::IntArrayRef(size, dims), at::IntArrayRef(stride, dims),
      at::TensorOptions()
          .dtype(reinterpret_cast<THPDtype*>(args[2])->scalar_type)
          .device(THPVariable_Unpack(args[3]).device())));
  END_HANDLE_TH_ERRORS
}

// A tensor's data, an address or null.
bool address(PyObject* o, void** out) {
  if (o == Py_None) {
    *out = nullptr;
  } else if (THPVariable_Check(o)) {
    *out = THPVariable_Unpack(o).mutable_data_ptr();   // of its own, where a lazy clone shares memory
  } else {
    *out = PyLong_AsVoidPtr(o);
    return !PyErr_Occurred();
  }
  return true;
}

// function: the address of int (*)(pointers); arguments: tensors, addresses,
// None, or a tuple of these for a struct of pointers.
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  constexpr int kArgs = 12, kInner = 16;
  void* p[kArgs] = {};
  void* inner[kInner];
  int used = 0, held = 0;
  void* f = n > 0 ? PyLong_AsVoidPtr(args[0]) : nullptr;
  if (!f) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "call(function, *arguments)");
    return nullptr;
  }
  for (Py_ssize_t i = 1; i < n; ++i) {
    const bool nested = PyTuple_Check(args[i]);
    const int count = nested ? static_cast<int>(PyTuple_GET_SIZE(args[i])) : 0;
    if (used == kArgs || held + count > kInner) {
      PyErr_SetString(PyExc_TypeError, "too many arguments");
      return nullptr;
    }
    if (!nested) {
      if (!address(args[i], &p[used++])) return nullptr;
      continue;
    }
    p[used++] = inner + held;
    for (int j = 0; j < count; ++j)
      if (!address(PyTuple_GET_ITEM(args[i], j), &inner[held++])) return nullptr;
  }
  int rc;
  Py_BEGIN_ALLOW_THREADS
  using P = void*;
  switch (used) {
    case 5: rc = reinterpret_cast<int (*)(P, P, P, P, P)>(f)(p[0], p[1], p[2], p[3], p[4]); break;
    case 6:
      rc = reinterpret_cast<int (*)(P, P, P, P, P, P)>(f)(p[0], p[1], p[2], p[3], p[4], p[5]);
      break;
    case 8:
      rc = reinterpret_cast<int (*)(P, P, P, P, P, P, P, P)>(f)(p[0], p[1], p[2], p[3], p[4], p[5],
                                                                p[6], p[7]);
      break;
    case 12:
      rc = reinterpret_cast<int (*)(P, P, P, P, P, P, P, P, P, P, P, P)>(f)(
          p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], p[8], p[9], p[10], p[11]);
      break;
    default: rc = -1;
  }
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
  END_HANDLE_TH_ERRORS
}

PyMethodDef kMethods[] = {
    {"layout", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(layout)), METH_FASTCALL, nullptr},
    {"empty", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(empty)), METH_FASTCALL, nullptr},
    {"call", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(call)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_host", nullptr, -1, kMethods, nullptr, nullptr,
                       nullptr, nullptr};

}  // namespace

// BSA_BUILT_FOR: the torch and Python that the build compiled against.
PyMODINIT_FUNC PyInit__host(void) {
  PyObject* m = PyModule_Create(&kModule);
  if (m && PyModule_AddStringConstant(m, "built_for", BSA_BUILT_FOR) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
