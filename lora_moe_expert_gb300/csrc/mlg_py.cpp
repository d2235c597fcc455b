// mlg_py.cpp -- the calls of mlg.h as functions of a Python module, for the
// binding's device calls: the same arguments in the same order, an int status
// back.  A pointer argument is None (NULL), an int (an address) or a torch
// tensor, and tensors are checked here, so that a call reads no other elements
// than it is given:
//  * where mlg.h names the pointer's element type, the tensor is of it and
//    contiguous;
//  * the rows and logits (void pointers) of a call are of one type, given as the
//    argument after the first of them, or None: taken from them;
//  * a row stride (the only 64-bit arguments) is given, or None: that of the
//    tensor before it; rows without a stride argument are contiguous.
// The last argument is the stream's address, or something to call for it, which
// is called after the checks.  ctypes takes 1 to 1.5 us to marshal such a call, as
// long as a small kernel runs; this takes 0.3 us, and 0.1 a tensor for the checks.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstdint>
#include <tuple>
#include <type_traits>
#include <utility>

#include "mlg.h"

namespace {

PyObject *g_data_ptr, *g_dtype, *g_is_contiguous, *g_shape, *g_stride;  // the names

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

// torch.`name`, looked up once; nullptr with an error set.
PyObject *torch_dtype(const char *name) {
  PyObject *torch = PyImport_ImportModule("torch");
  PyObject *dtype = torch ? PyObject_GetAttrString(torch, name) : nullptr;
  Py_XDECREF(torch);
  return dtype;
}

bool contiguous(PyObject *tensor) {
  PyObject *answer = PyObject_CallMethodNoArgs(tensor, g_is_contiguous);
  if (answer == nullptr) return false;
  const bool yes = answer == Py_True;
  Py_DECREF(answer);
  if (!yes) PyErr_SetString(PyExc_ValueError, "a contiguous tensor expected");
  return yes;
}

// A tensor of elements E, one after the other.
template <typename E>
bool holds(PyObject *tensor) {
  static PyObject *expected = torch_dtype(kElement<E>);
  PyObject *dtype = expected ? PyObject_GetAttr(tensor, g_dtype) : nullptr;
  if (dtype == nullptr) return false;
  const bool same = dtype == expected;  // torch keeps one object of each
  if (!same) PyErr_Format(PyExc_TypeError, "%S: %s expected", dtype, kElement<E>);
  Py_DECREF(dtype);
  return same && contiguous(tensor);
}

bool as_address(PyObject *o, void **out) {
  PyObject *own = nullptr;
  if (!PyLong_Check(o)) {
    own = PyObject_CallMethodNoArgs(o, g_data_ptr);
    if (own == nullptr) return false;
    o = own;
  }
  *out = PyLong_AsVoidPtr(o);
  Py_XDECREF(own);
  return !PyErr_Occurred();
}

// The row stride of a 2-D tensor.
bool row_stride(PyObject *tensor, int64_t *out) {
  PyObject *stride = PyObject_CallMethodNoArgs(tensor, g_stride);
  if (stride == nullptr) return false;
  bool ok = PyTuple_Check(stride) && PyTuple_GET_SIZE(stride) == 2;
  if (ok) {
    *out = PyLong_AsLongLong(PyTuple_GET_ITEM(stride, 0));
    if (PyLong_AsLongLong(PyTuple_GET_ITEM(stride, 1)) != 1) {  // fine where a row has one element
      PyObject *shape = PyObject_GetAttr(tensor, g_shape);
      ok = shape != nullptr && PyLong_AsLongLong(PyTuple_GET_ITEM(shape, 1)) <= 1;
      Py_XDECREF(shape);
    }
  }
  Py_DECREF(stride);
  if (!ok && !PyErr_Occurred())
    PyErr_SetString(PyExc_ValueError, "rows of adjacent elements expected");
  return ok;
}

// The arguments A... of a call, by place.
template <typename... A>
struct Call {
  static constexpr size_t kN = sizeof...(A);
  template <size_t I>
  using Arg = std::tuple_element_t<I, std::tuple<A...>>;
  template <size_t I>
  static constexpr bool is_void() {
    return std::is_pointer_v<Arg<I>> && std::is_void_v<std::remove_pointer_t<Arg<I>>>;
  }
  template <size_t I>
  static constexpr bool is_stride() {
    if constexpr (I < kN) return std::is_same_v<Arg<I>, int64_t>;
    return false;
  }
  static constexpr bool kTyped = is_void<0>();  // argument 0 is rows, argument 1 their type
  template <size_t I>
  static constexpr bool strided() {
    return is_stride<I + 1>() || (I == 0 && is_stride<2>());
  }

  PyObject *const *args;
  PyObject *rows_dtype = nullptr;  // owned
  std::tuple<A...> v = {};

  explicit Call(PyObject *const *a) : args(a) {}
  Call(const Call &) = delete;
  ~Call() { Py_XDECREF(rows_dtype); }

  bool rows(PyObject *tensor, bool any_stride) {
    PyObject *dtype = PyObject_GetAttr(tensor, g_dtype);
    if (dtype == nullptr) return false;
    const bool same = rows_dtype == nullptr || dtype == rows_dtype;
    if (!same)
      PyErr_Format(PyExc_TypeError, "rows of one type expected: %S and %S", rows_dtype, dtype);
    if (rows_dtype == nullptr)
      rows_dtype = dtype;
    else
      Py_DECREF(dtype);
    return same && (any_stride || contiguous(tensor));
  }

  template <size_t I>
  bool take() {
    using T = Arg<I>;
    PyObject *o = args[I];
    if constexpr (I == kN - 1 || (I == 1 && kTyped)) {
      return true;  // the stream, and the type: after the others
    } else if constexpr (std::is_pointer_v<T>) {
      using E = std::remove_const_t<std::remove_pointer_t<T>>;
      if (o == Py_None) return true;
      if (!PyLong_Check(o)) {
        if constexpr (is_void<I>()) {
          if (!rows(o, strided<I>())) return false;
        } else {
          if (!holds<E>(o)) return false;
        }
      }
      void *p = nullptr;
      if (!as_address(o, &p)) return false;
      std::get<I>(v) = static_cast<T>(p);
      return true;
    } else if constexpr (std::is_same_v<T, int64_t>) {
      if (o != Py_None) return as_int(o, INT64_MIN, INT64_MAX, &std::get<I>(v));
      PyObject *before = args[is_void<I - 1>() ? I - 1 : 0];
      if (before == Py_None) return true;
      if (PyLong_Check(before)) return stated();
      return row_stride(before, &std::get<I>(v));
    } else {
      static_assert(std::is_same_v<T, int32_t>, "an argument of mlg.h");
      int64_t n = 0;
      if (!as_int(o, INT32_MIN, INT32_MAX, &n)) return false;
      std::get<I>(v) = static_cast<T>(n);
      return true;
    }
  }

  static bool stated() {
    PyErr_SetString(PyExc_TypeError, "an address needs its type and row stride beside it");
    return false;
  }

  bool take_type() {
    if constexpr (kTyped) {
      int64_t type = 0;
      if (args[1] != Py_None) {
        if (!as_int(args[1], INT32_MIN, INT32_MAX, &type)) return false;
      } else {
        static PyObject *bf16 = torch_dtype("bfloat16"), *f32 = torch_dtype("float32");
        if (bf16 == nullptr || f32 == nullptr) return false;
        if (rows_dtype == nullptr) return stated();
        if (rows_dtype != bf16 && rows_dtype != f32) {
          PyErr_Format(PyExc_TypeError, "%S: bfloat16 or float32 expected", rows_dtype);
          return false;
        }
        type = rows_dtype == bf16 ? MLG_TYPE_BF16 : MLG_TYPE_F32;
      }
      std::get<1>(v) = static_cast<Arg<1>>(type);
    }
    return true;
  }

  bool take_stream() {
    PyObject *o = args[kN - 1];
    if (o == Py_None) return true;
    PyObject *own = PyLong_Check(o) ? nullptr : PyObject_CallNoArgs(o);
    if (own == nullptr && PyErr_Occurred()) return false;
    std::get<kN - 1>(v) = PyLong_AsVoidPtr(own ? own : o);
    Py_XDECREF(own);
    return !PyErr_Occurred();
  }
};

template <auto F, typename R, typename... A, size_t... I>
PyObject *call(R (*)(A...), PyObject *const *args, std::index_sequence<I...>) {
  Call<A...> c(args);
  if (!(c.template take<I>() && ...) || !c.take_type() || !c.take_stream()) return nullptr;
  R status;  // other threads run meanwhile: a launch waits where the stream's queue is full
  Py_BEGIN_ALLOW_THREADS;
  status = F(std::get<I>(c.v)...);
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
  g_shape = PyUnicode_InternFromString("shape");
  g_stride = PyUnicode_InternFromString("stride");
  const bool named = g_data_ptr && g_dtype && g_is_contiguous && g_shape && g_stride;
  return named ? PyModule_Create(&kModule) : nullptr;
}
