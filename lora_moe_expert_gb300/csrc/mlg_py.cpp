// mlg_py.cpp -- the calls of mlg.h as functions of a Python module, for the
// binding's device calls: the same arguments in the same order, an int status
// back.  A pointer argument is None (NULL), an int (an address) or a torch
// tensor.  Where mlg.h names the pointer's element type, the tensor has to be
// of it and contiguous (the rows behind a void pointer have a type and a stride
// among the arguments, which the binding takes from the tensor).  ctypes takes
// 1 to 1.5 us to marshal such a call, as long as a small kernel runs; this takes
// about 0.3 us.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstdint>
#include <tuple>
#include <type_traits>
#include <utility>

#include "mlg.h"

namespace {

PyObject *g_data_ptr, *g_dtype, *g_is_contiguous;  // the names

// Each returns false with a Python error set when the argument does not convert.
bool as_int(PyObject *o, int64_t lo, int64_t hi, int64_t *out) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) return false;
  if (v < lo || v > hi) {
    PyErr_SetString(PyExc_OverflowError, "integer argument out of range");
    return false;
  }
  *out = v;
  return true;
}

template <typename E>
constexpr const char *kElement = nullptr;  // torch's name of an element type
template <>
constexpr const char *kElement<int32_t> = "int32";
template <>
constexpr const char *kElement<float> = "float32";
template <>
constexpr const char *kElement<mlg_bf16> = "bfloat16";
template <>
constexpr const char *kElement<uint8_t> = "uint8";

// A tensor of elements E, one after the other.
template <typename E>
bool holds(PyObject *tensor) {
  static PyObject *expected = nullptr;
  if (expected == nullptr) {
    PyObject *torch = PyImport_ImportModule("torch");
    if (torch != nullptr) expected = PyObject_GetAttrString(torch, kElement<E>);
    Py_XDECREF(torch);
    if (expected == nullptr) return false;
  }
  PyObject *dtype = PyObject_GetAttr(tensor, g_dtype);
  if (dtype == nullptr) return false;
  const bool same = dtype == expected;
  if (!same) PyErr_Format(PyExc_TypeError, "%S: %s expected", dtype, kElement<E>);
  Py_DECREF(dtype);
  if (!same) return false;
  PyObject *contiguous = PyObject_CallMethodNoArgs(tensor, g_is_contiguous);
  if (contiguous == nullptr) return false;
  const bool yes = contiguous == Py_True;
  Py_DECREF(contiguous);
  if (!yes) PyErr_Format(PyExc_ValueError, "a contiguous %s tensor expected", kElement<E>);
  return yes;
}

template <typename E>
bool as_address(PyObject *o, void **out) {
  if (o == Py_None) {
    *out = nullptr;
    return true;
  }
  PyObject *own = nullptr;
  if (!PyLong_Check(o)) {
    if constexpr (kElement<E> != nullptr)
      if (!holds<E>(o)) return false;
    own = PyObject_CallMethodNoArgs(o, g_data_ptr);
    if (own == nullptr) return false;
    o = own;
  }
  *out = PyLong_AsVoidPtr(o);
  Py_XDECREF(own);
  return !PyErr_Occurred();
}

template <typename T>
bool convert(PyObject *o, T *out) {
  if constexpr (std::is_pointer_v<T>) {
    void *p = nullptr;
    if (!as_address<std::remove_const_t<std::remove_pointer_t<T>>>(o, &p)) return false;
    *out = static_cast<T>(p);
    return true;
  } else {
    static_assert(std::is_same_v<T, int32_t> || std::is_same_v<T, int64_t>, "an argument of mlg.h");
    int64_t v = 0;
    if (!as_int(o, std::is_same_v<T, int32_t> ? INT32_MIN : INT64_MIN,
                std::is_same_v<T, int32_t> ? INT32_MAX : INT64_MAX, &v))
      return false;
    *out = static_cast<T>(v);
    return true;
  }
}

template <auto F, typename R, typename... A, size_t... I>
PyObject *call(R (*)(A...), PyObject *const *args, std::index_sequence<I...>) {
  std::tuple<A...> v;
  if (!(convert(args[I], &std::get<I>(v)) && ...)) return nullptr;
  R status;  // other threads run meanwhile: a launch waits where the stream's queue is full
  Py_BEGIN_ALLOW_THREADS;
  status = F(std::get<I>(v)...);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(status);
}

template <auto F, typename R, typename... A>
PyObject *checked(R (*f)(A...), PyObject *const *args, Py_ssize_t n) {
  if (n != static_cast<Py_ssize_t>(sizeof...(A))) {
    PyErr_Format(PyExc_TypeError, "%zd arguments expected", static_cast<Py_ssize_t>(sizeof...(A)));
    return nullptr;
  }
  return call<F>(f, args, std::index_sequence_for<A...>());
}

template <auto F>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return checked<F>(F, args, n);
}

#define MLG_METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&entry<name>)), METH_FASTCALL, nullptr}

PyMethodDef kMethods[] = {
    MLG_METHOD(mlg_route_topk), MLG_METHOD(mlg_route_topk_backward), MLG_METHOD(mlg_sort_slots),
    MLG_METHOD(mlg_dispatch),   MLG_METHOD(mlg_combine),             MLG_METHOD(mlg_combine_backward),
    MLG_METHOD(mlg_gather_q4),  {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_mlg_py", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mlg_py() {
  g_data_ptr = PyUnicode_InternFromString("data_ptr");
  g_dtype = PyUnicode_InternFromString("dtype");
  g_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  return g_data_ptr && g_dtype && g_is_contiguous ? PyModule_Create(&kModule) : nullptr;
}
