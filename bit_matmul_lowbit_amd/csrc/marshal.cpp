// The Python side of the operators beside the products: a module (_marshal)
// that checks a call's tensors, makes those that were not given and calls the
// library.  A decode step makes many small calls with eight to fifteen tensors
// each; checked attribute by attribute in Python and passed through ctypes, a
// call took 5 to 8 us before its first kernel was launched, with the checks
// alone compiled still 2.7 to 3.3.
#include <Python.h>
#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/autograd/python_variable.h>

#include "lowbit.h"

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

// What bind() was given.
struct {
  decltype(&lowbit_norm_residual) norm;
  decltype(&lowbit_logits_workspace_bytes) logits_bytes;
  decltype(&lowbit_logits_process) logits;
  decltype(&lowbit_lora_workspace_bytes) lora_bytes;
  decltype(&lowbit_lora_accumulate) lora;
  PyObject* raw_stream;  // device -> address of its current stream
  PyObject* empty;       // (shape, type code or dtype, device of, stream) -> tensor
  PyObject* error;       // LowbitError
} bound;

// an owned reference
struct Ref {
  PyObject* o = nullptr;
  ~Ref() { Py_XDECREF(o); }
  Ref() = default;
  Ref(const Ref&) = delete;
  Ref& operator=(const Ref&) = delete;
};

struct Rows {
  void* p = nullptr;
  int type = 0;
  int64_t ld = 0;
};

// an FP32, FP16 or BF16 tensor [m][k]
bool get_rows(PyObject* o, const char* name, long long want_m, long long want_k, int dev, Rows* out) {
  const at::Tensor* t = tensor(o, name);
  if (!t) return false;
  const int code = code_of(*t);
  if (code < kF32 || code > kBF16) {
    PyErr_Format(PyExc_TypeError, "%s must be float32, float16 or bfloat16", name);
    return false;
  }
  long long m, k, ld;
  if (!on_device(*t, dev, name) || !as_rows(*t, name, &m, &k, &ld)) return false;
  if (m != want_m || k != want_k) {
    PyErr_Format(PyExc_ValueError, "%s has shape [%lld, %lld], expected [%lld, %lld]", name, m, k, want_m, want_k);
    return false;
  }
  *out = {t->data_ptr(), code, ld};
  return true;
}

// rows and columns of an argument, and the device of the call
bool get_shape(PyObject* o, const char* name, long long* m, long long* k, int* dev) {
  const at::Tensor* t = tensor(o, name);
  long long ld;
  if (!t || !as_rows(*t, name, m, k, &ld)) return false;
  *dev = t->get_device();
  return true;
}

// a contiguous tensor of at least `count` elements, or NULL for None
template <class T>
bool get_vector(PyObject* o, const char* name, int code, long long count, int dev, T** out) {
  *out = nullptr;
  if (o == Py_None) return true;
  const at::Tensor* t = tensor(o, name);
  if (!t) return false;
  if (code_of(*t) != code) {
    PyErr_Format(PyExc_TypeError, "%s must be %s", name, name_of(code));
    return false;
  }
  if (!on_device(*t, dev, name)) return false;
  if (!t->is_contiguous()) {
    PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
    return false;
  }
  if (t->numel() < count) {
    PyErr_Format(PyExc_ValueError, "%s holds %lld elements, needs at least %lld", name, (long long)t->numel(), count);
    return false;
  }
  *out = static_cast<T*>(t->data_ptr());
  return true;
}

template <class T>
struct Lists {
  T* p = nullptr;
  long long rows = 0, columns = 0, ld = 0;
};

// a tensor [rows][columns], with `want` rows unless that is negative, or none
template <class T>
bool get_lists(PyObject* o, const char* name, int code, long long want, int dev, Lists<T>* out) {
  if (o == Py_None) return true;
  const at::Tensor* t = tensor(o, name);
  if (!t) return false;
  if (code_of(*t) != code) {
    PyErr_Format(PyExc_TypeError, "%s must be %s", name, name_of(code));
    return false;
  }
  if (!on_device(*t, dev, name) || !as_rows(*t, name, &out->rows, &out->columns, &out->ld)) return false;
  if (t->dim() != 2 || (want >= 0 && out->rows != want)) {
    PyErr_Format(PyExc_ValueError, "%s must have two dimensions and %lld rows", name, want >= 0 ? want : out->rows);
    return false;
  }
  out->p = static_cast<T*>(t->data_ptr());
  return true;
}

// `stream` (None: the current one of device `dev`) as the library takes it
bool get_stream(PyObject* stream, int dev, hipStream_t* out) {
  Ref raw;
  if (stream == Py_None) {
    Ref d;
    if (!(d.o = PyLong_FromLong(dev))) return false;
    raw.o = PyObject_CallOneArg(bound.raw_stream, d.o);
  } else {
    Ref index;
    if (!(index.o = PyObject_GetAttrString(stream, "device_index"))) return false;
    const long of = PyLong_AsLong(index.o);
    if (PyErr_Occurred()) return false;
    if (of != dev) {
      PyErr_Format(PyExc_ValueError, "stream is one of cuda:%ld, expected cuda:%d", of, dev);
      return false;
    }
    raw.o = PyObject_GetAttrString(stream, "cuda_stream");
  }
  if (!raw.o) return false;
  *out = static_cast<hipStream_t>(PyLong_AsVoidPtr(raw.o));
  return !PyErr_Occurred();
}

// A tensor that the caller did not give.  One for another stream than the
// current is made by `empty`, from that stream's memory.
bool make(const at::Tensor& like, at::IntArrayRef shape, at::ScalarType type, int code, PyObject* stream, Ref* out) {
  if (stream == Py_None) {
    out->o = THPVariable_Wrap(at::empty(shape, like.options().dtype(type)));
  } else {
    Ref dims;
    dims.o = PyTuple_New((Py_ssize_t)shape.size());
    if (!dims.o) return false;
    for (size_t i = 0; i < shape.size(); ++i) {
      PyObject* n = PyLong_FromLongLong(shape[i]);
      if (!n) return false;
      PyTuple_SET_ITEM(dims.o, (Py_ssize_t)i, n);
    }
    out->o = PyObject_CallFunction(bound.empty, "OiiO", dims.o, code, (int)like.get_device(), stream);
  }
  return out->o != nullptr;
}

// Runs `call` with device `dev` current and without the interpreter's lock.
template <class F>
bool launch(int dev, const char* where, F call) {
  int status;
  {
    const c10::DeviceGuard guard(c10::Device(c10::kCUDA, (c10::DeviceIndex)dev));
    PyThreadState* state = PyEval_SaveThread();
    status = call();
    PyEval_RestoreThread(state);
  }
  if (status == LOWBIT_OK) return true;
  Ref e;
  e.o = PyObject_CallFunction(bound.error, "is", status, where);
  if (e.o) PyErr_SetObject(bound.error, e.o);
  return false;
}

bool count_ok(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
  return false;
}

template <class T>
bool address(PyObject* o, T* out) {
  *out = reinterpret_cast<T>(PyLong_AsVoidPtr(o));
  return !PyErr_Occurred();
}

// bind(norm, logits_bytes, logits, lora_bytes, lora, raw_stream, empty, error)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_ok(n, 8)) return nullptr;
  if (!address(a[0], &bound.norm) || !address(a[1], &bound.logits_bytes) || !address(a[2], &bound.logits) ||
      !address(a[3], &bound.lora_bytes) || !address(a[4], &bound.lora))
    return nullptr;
  PyObject** const keep[] = {&bound.raw_stream, &bound.empty, &bound.error};
  for (int i = 0; i < 3; ++i) {
    Py_INCREF(a[5 + i]);
    Py_XDECREF(*keep[i]);
    *keep[i] = a[5 + i];
  }
  Py_RETURN_NONE;
}

bool ready() {
  if (bound.error) return true;
  PyErr_SetString(PyExc_RuntimeError, "not bound to the library");
  return false;
}

// norm(y, r, post, post_w, post_b, gate, scale, pre or -1, pre_w, pre_b, eps,
// r_out, x_out, x_code, stream) -> (r_out, x_out)
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_ok(n, 15) || !ready()) return nullptr;
  return guarded([&]() -> PyObject* {
    PyObject *y = a[0], *r = a[1], *gate = a[5], *r_out = a[11], *x_out = a[12], *stream = a[14];
    const long post = PyLong_AsLong(a[2]), pre = PyLong_AsLong(a[7]), x_code = PyLong_AsLong(a[13]);
    const float scale = (float)PyFloat_AsDouble(a[6]), eps = (float)PyFloat_AsDouble(a[10]);
    if (PyErr_Occurred()) return nullptr;
    long long m, k;
    int dev;
    hipStream_t st;
    Rows ry, rr, rg, ro, rx;
    if (!get_shape(r, "r", &m, &k, &dev) || !get_stream(stream, dev, &st) || !get_rows(r, "r", m, k, dev, &rr))
      return nullptr;
    if (y != Py_None) {
      if (!get_rows(y, "y", m, k, dev, &ry)) return nullptr;
      if (gate != Py_None) {
        const at::Tensor* t = tensor(gate, "gate");
        if (!t || !get_rows(gate, "gate", t->dim() == 1 ? 1 : m, k, dev, &rg)) return nullptr;
        if (t->dim() == 1) rg.ld = 0;
      }
      if (r_out == Py_None) {
        r_out = r;
        ro = rr;
      } else {
        if (!get_rows(r_out, "r_out", m, k, dev, &ro)) return nullptr;
        if (ro.type != rr.type) {
          PyErr_SetString(PyExc_TypeError, "r_out must have the type of r");
          return nullptr;
        }
      }
    } else if (r_out != Py_None) {
      PyErr_SetString(PyExc_ValueError, "r_out needs y");
      return nullptr;
    }
    const float *post_w, *post_b, *pre_w, *pre_b;
    if (!get_vector(a[3], "post_w", kF32, k, dev, &post_w) || !get_vector(a[4], "post_b", kF32, k, dev, &post_b) ||
        !get_vector(a[8], "pre_w", kF32, k, dev, &pre_w) || !get_vector(a[9], "pre_b", kF32, k, dev, &pre_b))
      return nullptr;
    Ref made;
    if (pre >= 0) {
      if (x_out == Py_None) {
        const at::Tensor& t = THPVariable_Unpack(r);
        const at::ScalarType type = x_code == kF32 ? at::kFloat : x_code == kF16 ? at::kHalf : at::kBFloat16;
        if (!make(t, t.sizes(), type, (int)x_code, stream, &made)) return nullptr;
        x_out = made.o;
      }
      if (!get_rows(x_out, "x_out", m, k, dev, &rx)) return nullptr;
    } else if (x_out != Py_None) {
      PyErr_SetString(PyExc_ValueError, "x_out needs pre");
      return nullptr;
    }
    if (!launch(dev, "lowbit_norm_residual", [&] {
          return bound.norm(ry.p, ry.type, ry.ld, rr.p, rr.type, rr.ld, ro.p, ro.ld, rx.p, rx.type, rx.ld, m, k,
                            (int)post, post_w, post_b, rg.p, rg.type, rg.ld, scale, pre >= 0 ? (int)pre : 0, pre_w,
                            pre_b, eps, st);
        }))
      return nullptr;
    return PyTuple_Pack(2, y != Py_None ? r_out : r, x_out);
  });
}

// logits(y, tokens, prompt_len, total_len, repetition, frequency, presence,
// bias_ids, bias_vals, bias_len, mask, mask_row, out, top1, idx, val,
// workspace, stream) -> (out, idx, val)
PyObject* logits(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_ok(n, 18) || !ready()) return nullptr;
  return guarded([&]() -> PyObject* {
    PyObject *y = a[0], *out = a[12], *idx = a[14], *val = a[15], *workspace = a[16], *stream = a[17];
    const int top1 = PyObject_IsTrue(a[13]);
    if (top1 < 0) return nullptr;
    long long b, v;
    int dev;
    hipStream_t st;
    Rows ry, ro;
    if (!get_shape(y, "y", &b, &v, &dev) || !get_stream(stream, dev, &st) || !get_rows(y, "y", b, v, dev, &ry))
      return nullptr;
    Lists<const int32_t> tokens, bias_ids, mask;
    Lists<const float> bias_vals;
    if (!get_lists(a[1], "tokens", kI32, b, dev, &tokens) || !get_lists(a[7], "bias_ids", kI32, b, dev, &bias_ids) ||
        !get_lists(a[8], "bias_vals", kF32, b, dev, &bias_vals) ||
        !get_lists(a[10], "mask", kI32, a[11] == Py_None ? b : -1, dev, &mask))
      return nullptr;
    if ((a[7] == Py_None) != (a[8] == Py_None) || bias_ids.columns != bias_vals.columns ||
        bias_ids.ld != bias_vals.ld) {
      PyErr_SetString(PyExc_ValueError, "bias_ids and bias_vals go together, with one shape and row stride");
      return nullptr;
    }
    if (a[10] != Py_None && mask.columns < (v + 31) / 32) {
      PyErr_Format(PyExc_ValueError, "mask has %lld words a row, needs %lld", mask.columns, (v + 31) / 32);
      return nullptr;
    }
    if (out != Py_None) {
      if (!get_rows(out, "out", b, v, dev, &ro)) return nullptr;
      if (ro.type != kF32) {
        PyErr_SetString(PyExc_TypeError, "out must be float32");
        return nullptr;
      }
    }
    const int32_t *prompt_len, *total_len, *bias_len, *mask_row;
    const float *repetition, *frequency, *presence;
    if (!get_vector(a[2], "prompt_len", kI32, b, dev, &prompt_len) ||
        !get_vector(a[3], "total_len", kI32, b, dev, &total_len) ||
        !get_vector(a[4], "repetition", kF32, b, dev, &repetition) ||
        !get_vector(a[5], "frequency", kF32, b, dev, &frequency) ||
        !get_vector(a[6], "presence", kF32, b, dev, &presence) ||
        !get_vector(a[9], "bias_len", kI32, b, dev, &bias_len) ||
        !get_vector(a[11], "mask_row", kI32, b, dev, &mask_row))
      return nullptr;
    Ref made_idx, made_val, made_ws;
    int32_t* idx_p = nullptr;
    float* val_p = nullptr;
    uint8_t* ws = nullptr;
    int64_t ws_bytes = 0;
    if (top1) {
      const at::Tensor& t = THPVariable_Unpack(y);
      if (idx == Py_None) {
        if (!make(t, {b}, at::kInt, kI32, stream, &made_idx)) return nullptr;
        idx = made_idx.o;
      }
      if (val == Py_None) {
        if (!make(t, {b}, at::kFloat, kF32, stream, &made_val)) return nullptr;
        val = made_val.o;
      }
      if (workspace == Py_None) {
        const int64_t need = (int64_t)bound.logits_bytes(v, b);
        if (!make(t, {need > 16 ? need : 16}, at::kByte, kU8, stream, &made_ws)) return nullptr;
        workspace = made_ws.o;
      }
      if (!get_vector(idx, "idx", kI32, b, dev, &idx_p) || !get_vector(val, "val", kF32, b, dev, &val_p) ||
          !get_vector(workspace, "workspace", kU8, 0, dev, &ws))
        return nullptr;
      ws_bytes = THPVariable_Unpack(workspace).numel();
    } else if (idx != Py_None || val != Py_None) {
      PyErr_SetString(PyExc_ValueError, "idx and val need top1");
      return nullptr;
    }
    if (!launch(dev, "lowbit_logits_process", [&] {
          return bound.logits(ry.p, ry.type, ry.ld, v, b, tokens.p, tokens.columns, tokens.ld, prompt_len, total_len,
                              repetition, frequency, presence, bias_ids.p, bias_vals.p, bias_ids.columns, bias_ids.ld,
                              bias_len, mask.p, mask.rows, mask.ld, mask_row, static_cast<float*>(ro.p), ro.ld, idx_p,
                              val_p, ws, (size_t)ws_bytes, st);
        }))
      return nullptr;
    return PyTuple_Pack(3, out, idx, val);
  });
}

// lora(x, ids, a, b, y, ranks, scales, workspace, stream) -> y
PyObject* lora(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_ok(n, 9) || !ready()) return nullptr;
  return guarded([&]() -> PyObject* {
    PyObject *x = a[0], *y = a[4], *workspace = a[7], *stream = a[8];
    long long m, k;
    int dev;
    hipStream_t st;
    Rows rx, ry;
    if (!get_shape(x, "x", &m, &k, &dev) || !get_stream(stream, dev, &st) || !get_rows(x, "x", m, k, dev, &rx))
      return nullptr;
    const at::Tensor *ta = tensor(a[2], "a"), *tb = ta ? tensor(a[3], "b") : nullptr;
    if (!tb) return nullptr;
    if (ta->dim() != 3 || tb->dim() != 3) {
      PyErr_SetString(PyExc_ValueError, "a must be [slots][r][k] and b [slots][n][r]");
      return nullptr;
    }
    const int64_t slots = tb->size(0), out = tb->size(1), r = tb->size(2);
    if (ta->size(0) != slots || ta->size(1) != r || ta->size(2) != k) {
      PyErr_Format(PyExc_ValueError, "a [%lld][%lld][%lld] does not fit x [%lld][%lld] and b [%lld][%lld][%lld]",
                   (long long)ta->size(0), (long long)ta->size(1), (long long)ta->size(2), m, k, (long long)slots,
                   (long long)out, (long long)r);
      return nullptr;
    }
    if (!get_rows(y, "y", m, out, dev, &ry)) return nullptr;
    const int32_t *ids, *ranks;
    const float* scales;
    const void *pa, *pb;
    uint8_t* ws;
    if (!get_vector(a[1], "ids", kI32, m, dev, &ids) || !get_vector(a[2], "a", rx.type, 0, dev, &pa) ||
        !get_vector(a[3], "b", rx.type, 0, dev, &pb) || !get_vector(a[5], "ranks", kI32, slots, dev, &ranks) ||
        !get_vector(a[6], "scales", kF32, slots, dev, &scales))
      return nullptr;
    Ref made;
    if (workspace == Py_None) {
      const int64_t need = (int64_t)bound.lora_bytes(m, out, k, r, slots);
      if (!make(THPVariable_Unpack(x), {need > 16 ? need : 16}, at::kByte, kU8, stream, &made)) return nullptr;
      workspace = made.o;
    }
    if (!get_vector(workspace, "workspace", kU8, 0, dev, &ws)) return nullptr;
    const int64_t ws_bytes = THPVariable_Unpack(workspace).numel();
    if (!launch(dev, "lowbit_lora_accumulate", [&] {
          return bound.lora(rx.p, rx.type, rx.ld, ids, m, out, k, r, slots, pa, pb, ranks, scales, ry.p, ry.type,
                            ry.ld, ws, (size_t)ws_bytes, st);
        }))
      return nullptr;
    Py_INCREF(y);
    return y;
  });
}

PyMethodDef methods[] = {{"bind", (PyCFunction)(void (*)())bind, METH_FASTCALL, nullptr},
                         {"norm", (PyCFunction)(void (*)())norm, METH_FASTCALL, nullptr},
                         {"logits", (PyCFunction)(void (*)())logits, METH_FASTCALL, nullptr},
                         {"lora", (PyCFunction)(void (*)())lora, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
