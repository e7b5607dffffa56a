// Checks and addresses of tensor arguments for the Python binding: a module
// (_marshal) of four functions that say, in one call each, what the binding
// needs to know of a tensor.  Asked of it attribute by attribute from Python,
// a decode step's small calls took longer to check than to run (4 to 7 us).
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

// as lowbit_type, and what else the calls take
enum Code { kNone = 0, kF32 = 1, kF16 = 2, kBF16 = 3, kI32 = 4, kU8 = 5 };

int code_of(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return kF32;
    case at::kHalf: return kF16;
    case at::kBFloat16: return kBF16;
    case at::kInt: return kI32;
    case at::kByte: return kU8;
    default: return kNone;
  }
}

const char* name_of(long code) {
  static const char* const names[] = {"?", "float32", "float16", "bfloat16", "int32", "uint8"};
  return names[code >= 1 && code <= 5 ? code : 0];
}

// the tensor of argument `o`, on a GPU, or NULL with the error set
const at::Tensor* tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a CUDA (HIP) tensor, not %s", name, Py_TYPE(o)->tp_name);
    return nullptr;
  }
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) {
    PyErr_Format(PyExc_TypeError, "%s must be a CUDA (HIP) tensor", name);
    return nullptr;
  }
  return &t;
}

bool on_device(const at::Tensor& t, long dev, const char* name) {
  if (t.get_device() == dev) return true;
  PyErr_Format(PyExc_ValueError, "%s is on cuda:%d, expected cuda:%ld", name, (int)t.get_device(), dev);
  return false;
}

// rows, columns and row stride of [m][k], or of [k] as one row; rows contiguous
bool as_rows(const at::Tensor& t, const char* name, long long* m, long long* k, long long* ld) {
  const auto size = t.sizes(), stride = t.strides();
  if (size.size() != 1 && size.size() != 2) {
    PyErr_Format(PyExc_ValueError, "%s must have one or two dimensions, not %zd", name, (Py_ssize_t)size.size());
    return false;
  }
  *k = size.back();
  *m = size.size() == 2 ? size[0] : 1;
  if (stride.back() != 1 && *k > 1) {
    PyErr_Format(PyExc_ValueError, "%s: the elements of a row must be contiguous", name);
    return false;
  }
  *ld = *m > 1 ? (long long)stride[0] : *k;
  return true;
}

// Runs f, which may throw as torch's accessors do on tensors without memory.
template <class F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

bool count_ok(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
  return false;
}

// shape(name, t) -> (rows, columns, device)
PyObject* shape(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_ok(n, 2)) return nullptr;
  return guarded([&]() -> PyObject* {
    const char* name = PyUnicode_AsUTF8(a[0]);
    if (!name) return nullptr;
    const at::Tensor* t = tensor(a[1], name);
    long long m, k, ld;
    if (!t || !as_rows(*t, name, &m, &k, &ld)) return nullptr;
    return Py_BuildValue("LLi", m, k, (int)t->get_device());
  });
}

// rows(name, t, m, k, device) -> (address, type code, row stride) of an FP32,
// FP16 or BF16 tensor [m][k]
PyObject* rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_ok(n, 5)) return nullptr;
  return guarded([&]() -> PyObject* {
    const char* name = PyUnicode_AsUTF8(a[0]);
    const long long want_m = PyLong_AsLongLong(a[2]), want_k = PyLong_AsLongLong(a[3]);
    const long dev = PyLong_AsLong(a[4]);
    if (PyErr_Occurred()) return nullptr;
    const at::Tensor* t = tensor(a[1], name);
    if (!t) return nullptr;
    const int code = code_of(*t);
    if (code < kF32 || code > kBF16) {
      PyErr_Format(PyExc_TypeError, "%s must be float32, float16 or bfloat16", name);
      return nullptr;
    }
    long long m, k, ld;
    if (!on_device(*t, dev, name) || !as_rows(*t, name, &m, &k, &ld)) return nullptr;
    if (m != want_m || k != want_k) {
      PyErr_Format(PyExc_ValueError, "%s has shape [%lld, %lld], expected [%lld, %lld]", name, m, k, want_m, want_k);
      return nullptr;
    }
    return Py_BuildValue("KiL", (unsigned long long)(uintptr_t)t->data_ptr(), code, ld);
  });
}

// vector(name, t, type code, count, device) -> address of a contiguous tensor
// of at least `count` elements, or None for None
PyObject* vector(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_ok(n, 5)) return nullptr;
  if (a[1] == Py_None) Py_RETURN_NONE;
  return guarded([&]() -> PyObject* {
    const char* name = PyUnicode_AsUTF8(a[0]);
    const long code = PyLong_AsLong(a[2]), dev = PyLong_AsLong(a[4]);
    const long long count = PyLong_AsLongLong(a[3]);
    if (PyErr_Occurred()) return nullptr;
    const at::Tensor* t = tensor(a[1], name);
    if (!t) return nullptr;
    if (code_of(*t) != code) {
      PyErr_Format(PyExc_TypeError, "%s must be %s", name, name_of(code));
      return nullptr;
    }
    if (!on_device(*t, dev, name)) return nullptr;
    if (!t->is_contiguous()) {
      PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
      return nullptr;
    }
    if (t->numel() < count) {
      PyErr_Format(PyExc_ValueError, "%s holds %lld elements, needs at least %lld", name, (long long)t->numel(), count);
      return nullptr;
    }
    return PyLong_FromVoidPtr(t->data_ptr());
  });
}

// lists(name, t, type code, rows or -1, device) -> (address, columns, row
// stride) of a tensor [rows][columns], or (None, 0, 0) for None
PyObject* lists(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_ok(n, 5)) return nullptr;
  if (a[1] == Py_None) return Py_BuildValue("Oii", Py_None, 0, 0);
  return guarded([&]() -> PyObject* {
    const char* name = PyUnicode_AsUTF8(a[0]);
    const long code = PyLong_AsLong(a[2]), dev = PyLong_AsLong(a[4]);
    const long long want = PyLong_AsLongLong(a[3]);
    if (PyErr_Occurred()) return nullptr;
    const at::Tensor* t = tensor(a[1], name);
    if (!t) return nullptr;
    if (code_of(*t) != code) {
      PyErr_Format(PyExc_TypeError, "%s must be %s", name, name_of(code));
      return nullptr;
    }
    long long m, k, ld;
    if (!on_device(*t, dev, name) || !as_rows(*t, name, &m, &k, &ld)) return nullptr;
    if (t->dim() != 2 || (want >= 0 && m != want)) {
      PyErr_Format(PyExc_ValueError, "%s must have two dimensions and %lld rows", name, want >= 0 ? want : m);
      return nullptr;
    }
    return Py_BuildValue("KLL", (unsigned long long)(uintptr_t)t->data_ptr(), k, ld);
  });
}

PyMethodDef methods[] = {
    {"shape", (PyCFunction)(void (*)())shape, METH_FASTCALL, "shape(name, t) -> (rows, columns, device)"},
    {"rows", (PyCFunction)(void (*)())rows, METH_FASTCALL, "rows(name, t, m, k, device) -> (address, type, stride)"},
    {"vector", (PyCFunction)(void (*)())vector, METH_FASTCALL, "vector(name, t, type, count, device) -> address"},
    {"lists", (PyCFunction)(void (*)())lists, METH_FASTCALL,
     "lists(name, t, type, rows, device) -> (address, columns, stride)"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
