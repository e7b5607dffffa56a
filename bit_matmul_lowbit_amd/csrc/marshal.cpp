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

#include <algorithm>
#include <cmath>

#include "lowbit.h"

namespace {

// as lowbit_type, and what else the calls take
enum Code { kNone = 0, kF32 = 1, kF16 = 2, kBF16 = 3, kI32 = 4, kU8 = 5, kI64 = 6 };

int code_of(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return kF32;
    case at::kHalf: return kF16;
    case at::kBFloat16: return kBF16;
    case at::kInt: return kI32;
    case at::kByte: return kU8;
    case at::kLong: return kI64;
    default: return kNone;
  }
}

const char* name_of(long code) {
  static const char* const names[] = {"?", "float32", "float16", "bfloat16", "int32", "uint8", "int64"};
  return names[code >= 1 && code <= 6 ? code : 0];
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
  decltype(&lowbit_rope) rope;
  decltype(&lowbit_kv_page_bytes) page_bytes;
  decltype(&lowbit_kv_store) kv_store;
  decltype(&lowbit_kv_load) kv_load;
  decltype(&lowbit_attention_workspace_bytes) attention_bytes;
  decltype(&lowbit_attention) attention;
  decltype(&lowbit_sample_workspace_bytes) sample_bytes;
  decltype(&lowbit_sample) sample;
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

// bind(norm, logits_bytes, logits, lora_bytes, lora, rope, page_bytes, kv_store,
// kv_load, attention_bytes, attention, sample_bytes, sample, raw_stream, empty,
// error)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_ok(n, 16)) return nullptr;
  if (!address(a[0], &bound.norm) || !address(a[1], &bound.logits_bytes) || !address(a[2], &bound.logits) ||
      !address(a[3], &bound.lora_bytes) || !address(a[4], &bound.lora) || !address(a[5], &bound.rope) ||
      !address(a[6], &bound.page_bytes) || !address(a[7], &bound.kv_store) || !address(a[8], &bound.kv_load) ||
      !address(a[9], &bound.attention_bytes) || !address(a[10], &bound.attention) ||
      !address(a[11], &bound.sample_bytes) || !address(a[12], &bound.sample))
    return nullptr;
  PyObject** const keep[] = {&bound.raw_stream, &bound.empty, &bound.error};
  for (int i = 0; i < 3; ++i) {
    Py_INCREF(a[13 + i]);
    Py_XDECREF(*keep[i]);
    *keep[i] = a[13 + i];
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

// a tensor [m][heads][d] whose heads are contiguous; -1: any size
struct Heads {
  void* p = nullptr;
  int type = 0;
  int64_t m = 0, heads = 0, d = 0, ld = 0, ldh = 0;
};
bool get_heads(PyObject* o, const char* name, int64_t m, int64_t heads, int64_t d, int dev, Heads* out) {
  const at::Tensor* t = tensor(o, name);
  if (!t) return false;
  const int code = code_of(*t);
  if (code < kF32 || code > kBF16) {
    PyErr_Format(PyExc_TypeError, "%s must be float32, float16 or bfloat16", name);
    return false;
  }
  if (dev >= 0 && !on_device(*t, dev, name)) return false;
  const auto size = t->sizes(), stride = t->strides();
  if (size.size() != 3) {
    PyErr_Format(PyExc_ValueError, "%s must have three dimensions [m][heads][d], not %zd", name,
                 (Py_ssize_t)size.size());
    return false;
  }
  if ((m >= 0 && size[0] != m) || (heads >= 0 && size[1] != heads) || (d >= 0 && size[2] != d)) {
    PyErr_Format(PyExc_ValueError, "%s has shape [%lld, %lld, %lld], expected [%lld, %lld, %lld]", name,
                 (long long)size[0], (long long)size[1], (long long)size[2], (long long)(m >= 0 ? m : size[0]),
                 (long long)(heads >= 0 ? heads : size[1]), (long long)(d >= 0 ? d : size[2]));
    return false;
  }
  if (size[2] > 1 && stride[2] != 1) {
    PyErr_Format(PyExc_ValueError, "%s: the elements of a head must be contiguous", name);
    return false;
  }
  // the stride of a dimension of one is not used; it may be anything
  const int64_t ldh = size[1] > 1 ? stride[1] : size[2];
  const int64_t ld = size[0] > 1 ? stride[0] : size[1] * size[2];
  *out = {t->data_ptr(), code, size[0], size[1], size[2], ld, ldh};
  return true;
}

bool device_of(PyObject* o, const char* name, int* dev) {
  const at::Tensor* t = tensor(o, name);
  if (t) *dev = t->get_device();
  return t != nullptr;
}

at::ScalarType scalar_of(int code) {
  return code == kF32 ? at::kFloat : code == kF16 ? at::kHalf : at::kBFloat16;
}

// the pages of a cache: uint8 [pages][page_bytes], contiguous
bool get_pages(PyObject* o, int dev, int64_t* n, int64_t* bytes, uint8_t** p) {
  if (o == Py_None) {
    PyErr_SetString(PyExc_TypeError, "pages must be a CUDA (HIP) tensor");
    return false;
  }
  if (!get_vector(o, "pages", kU8, 0, dev, p)) return false;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.dim() != 2) {
    PyErr_SetString(PyExc_ValueError, "pages must be [pages][bytes of a page]");
    return false;
  }
  *n = t.size(0);
  *bytes = t.size(1);
  return true;
}
bool fits_page(int64_t bytes, int64_t heads, int64_t d, int64_t page) {
  const int64_t want = (int64_t)bound.page_bytes(heads, d, page);
  if (want == 0 || bytes == want) return true;  // a bad shape is the library's to refuse
  PyErr_Format(PyExc_ValueError, "pages of %lld bytes do not hold %lld tokens of %lld heads of %lld (%lld bytes)",
               (long long)bytes, (long long)page, (long long)heads, (long long)d, (long long)want);
  return false;
}

template <class T>
bool need_vector(PyObject* o, const char* name, int code, long long count, int dev, T** out) {
  if (o == Py_None) {
    PyErr_Format(PyExc_TypeError, "%s must be a CUDA (HIP) tensor", name);
    return false;
  }
  return get_vector(o, name, code, count, dev, out);
}

// rope(x, positions, turns, out, out_code, interleaved, gain, stream) -> out
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_ok(n, 8) || !ready()) return nullptr;
  return guarded([&]() -> PyObject* {
    PyObject *x = a[0], *out = a[3], *stream = a[7];
    const long code = PyLong_AsLong(a[4]);
    const int inter = PyObject_IsTrue(a[5]);
    const double gain = PyFloat_AsDouble(a[6]);
    if (PyErr_Occurred()) return nullptr;
    int dev;
    hipStream_t st;
    Heads hx, ho;
    if (!device_of(x, "x", &dev) || !get_stream(stream, dev, &st) || !get_heads(x, "x", -1, -1, -1, dev, &hx))
      return nullptr;
    const int32_t* positions;
    const uint64_t* turns;
    if (!need_vector(a[1], "positions", kI32, hx.m, dev, &positions) ||
        !need_vector(a[2], "turns", kI64, 0, dev, &turns))
      return nullptr;
    const int64_t rot = 2 * THPVariable_Unpack(a[2]).numel();
    Ref made;
    if (out == Py_None) {
      const int type = code ? (int)code : hx.type;
      if (!make(THPVariable_Unpack(x), THPVariable_Unpack(x).sizes(), scalar_of(type), type, stream, &made))
        return nullptr;
      out = made.o;
    }
    if (!get_heads(out, "out", hx.m, hx.heads, hx.d, dev, &ho)) return nullptr;
    if (!launch(dev, "lowbit_rope", [&] {
          return bound.rope(hx.p, hx.type, hx.ld, hx.ldh, positions, turns, hx.m, hx.heads, hx.d, rot, inter, gain,
                            ho.p, ho.type, ho.ld, ho.ldh, st);
        }))
      return nullptr;
    Py_INCREF(out);
    return out;
  });
}

// kv_store(k, v, slots, pages, page, positions, turns, interleaved, gain, q,
// q_out, q_code, stream) -> q_out or None
PyObject* kv_store(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_ok(n, 13) || !ready()) return nullptr;
  return guarded([&]() -> PyObject* {
    PyObject *k = a[0], *v = a[1], *q = a[9], *q_out = a[10], *stream = a[12];
    const int64_t page = PyLong_AsLongLong(a[4]);
    const int inter = PyObject_IsTrue(a[7]);
    const double gain = PyFloat_AsDouble(a[8]);
    const long code = PyLong_AsLong(a[11]);
    if (PyErr_Occurred()) return nullptr;
    int dev;
    hipStream_t st;
    Heads hk, hv, hq, ho;
    if (!device_of(k, "k", &dev) || !get_stream(stream, dev, &st) || !get_heads(k, "k", -1, -1, -1, dev, &hk) ||
        !get_heads(v, "v", hk.m, hk.heads, hk.d, dev, &hv))
      return nullptr;
    if (hv.type != hk.type) {
      PyErr_SetString(PyExc_TypeError, "k, v and q must have one type");
      return nullptr;
    }
    const int32_t *slots, *positions;
    const uint64_t* turns;
    uint8_t* pages;
    int64_t n_pages, bytes, rot = 0;
    if (!need_vector(a[2], "slots", kI32, hk.m, dev, &slots) || !get_pages(a[3], dev, &n_pages, &bytes, &pages) ||
        !fits_page(bytes, hk.heads, hk.d, page) || !get_vector(a[5], "positions", kI32, hk.m, dev, &positions) ||
        !get_vector(a[6], "turns", kI64, 0, dev, &turns))
      return nullptr;
    if ((a[5] == Py_None) != (a[6] == Py_None)) {
      PyErr_SetString(PyExc_ValueError, "positions and turns go together");
      return nullptr;
    }
    if (a[6] != Py_None) rot = 2 * THPVariable_Unpack(a[6]).numel();
    Ref made;
    if (q != Py_None) {
      if (a[6] == Py_None) {
        PyErr_SetString(PyExc_ValueError, "q needs positions and turns");
        return nullptr;
      }
      if (!get_heads(q, "q", hk.m, -1, hk.d, dev, &hq)) return nullptr;
      if (hq.type != hk.type) {
        PyErr_SetString(PyExc_TypeError, "k, v and q must have one type");
        return nullptr;
      }
      if (q_out == Py_None) {
        const int type = code ? (int)code : hq.type == kF32 ? (int)kF16 : hq.type;
        if (!make(THPVariable_Unpack(q), THPVariable_Unpack(q).sizes(), scalar_of(type), type, stream, &made))
          return nullptr;
        q_out = made.o;
      }
      if (!get_heads(q_out, "q_out", hk.m, hq.heads, hk.d, dev, &ho)) return nullptr;
    } else if (q_out != Py_None) {
      PyErr_SetString(PyExc_ValueError, "q_out needs q");
      return nullptr;
    }
    if (!launch(dev, "lowbit_kv_store", [&] {
          return bound.kv_store(hk.p, hk.ld, hk.ldh, hv.p, hv.ld, hv.ldh, hk.type, slots, hk.m, hk.heads, hk.d, pages,
                                n_pages, page, positions, turns, rot, inter, gain, hq.p, hq.ld, hq.ldh, hq.heads,
                                ho.p, ho.type, ho.ld, ho.ldh, st);
        }))
      return nullptr;
    Py_INCREF(q_out);
    return q_out;
  });
}

// kv_load(pages, page, slots, heads, d, k_out, v_out, code, stream) -> (k, v)
PyObject* kv_load(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_ok(n, 9) || !ready()) return nullptr;
  return guarded([&]() -> PyObject* {
    PyObject *k = a[5], *v = a[6], *stream = a[8];
    const int64_t page = PyLong_AsLongLong(a[1]), heads = PyLong_AsLongLong(a[3]), d = PyLong_AsLongLong(a[4]);
    const long code = PyLong_AsLong(a[7]);
    if (PyErr_Occurred()) return nullptr;
    int dev;
    hipStream_t st;
    uint8_t* pages;
    int64_t n_pages, bytes;
    const int32_t* slots;
    if (!device_of(a[0], "pages", &dev) || !get_stream(stream, dev, &st) ||
        !get_pages(a[0], dev, &n_pages, &bytes, &pages) || !fits_page(bytes, heads, d, page) ||
        !need_vector(a[2], "slots", kI32, 0, dev, &slots))
      return nullptr;
    const int64_t m = THPVariable_Unpack(a[2]).numel();
    if (heads < 0 || d < 0) {
      PyErr_SetString(PyExc_ValueError, "heads and d must not be negative");
      return nullptr;
    }
    Ref made_k, made_v;
    const at::Tensor& like = THPVariable_Unpack(a[0]);
    const bool both = k == Py_None && v == Py_None;
    if (both) {
      if (!make(like, {m, heads, d}, scalar_of((int)code), (int)code, stream, &made_k) ||
          !make(like, {m, heads, d}, scalar_of((int)code), (int)code, stream, &made_v))
        return nullptr;
      k = made_k.o;
      v = made_v.o;
    }
    Heads hk, hv;
    if ((k != Py_None && !get_heads(k, "k_out", m, heads, d, dev, &hk)) ||
        (v != Py_None && !get_heads(v, "v_out", m, heads, d, dev, &hv)))
      return nullptr;
    if (k != Py_None && v != Py_None && hk.type != hv.type) {
      PyErr_SetString(PyExc_TypeError, "k_out and v_out must have one type");
      return nullptr;
    }
    if (!launch(dev, "lowbit_kv_load", [&] {
          return bound.kv_load(pages, n_pages, heads, d, page, slots, m, hk.p, hk.ld, hk.ldh, hv.p, hv.ld, hv.ldh,
                               k != Py_None ? hk.type : hv.type, st);
        }))
      return nullptr;
    return PyTuple_Pack(2, k, v);
  });
}

// attention(q, pages, page, table, lengths, q_start, max_q, scale or None, out,
// out_code, lse, workspace, stream) -> out
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_ok(n, 13) || !ready()) return nullptr;
  return guarded([&]() -> PyObject* {
    PyObject *q = a[0], *out = a[8], *workspace = a[11], *stream = a[12];
    const int64_t page = PyLong_AsLongLong(a[2]);
    const long code = PyLong_AsLong(a[9]);
    if (PyErr_Occurred()) return nullptr;
    int dev;
    hipStream_t st;
    Heads hq, ho;
    uint8_t* pages;
    int64_t n_pages, bytes;
    if (!device_of(q, "q", &dev) || !get_stream(stream, dev, &st) || !get_heads(q, "q", -1, -1, -1, dev, &hq) ||
        !get_pages(a[1], dev, &n_pages, &bytes, &pages))
      return nullptr;
    // as many KV heads as a page has room for
    const int64_t one = (int64_t)bound.page_bytes(1, hq.d, page);
    const int64_t heads = one ? bytes / one : 1;
    if (one && (heads < 1 || heads * one != bytes)) {
      PyErr_Format(PyExc_ValueError, "pages of %lld bytes do not hold %lld tokens of heads of %lld", (long long)bytes,
                   (long long)page, (long long)hq.d);
      return nullptr;
    }
    if (a[3] == Py_None) {
      PyErr_SetString(PyExc_TypeError, "table must be a CUDA (HIP) tensor");
      return nullptr;
    }
    Lists<const int32_t> table;
    const int32_t *lengths, *q_start;
    if (!get_lists(a[3], "table", kI32, -1, dev, &table) ||
        !need_vector(a[4], "lengths", kI32, table.rows, dev, &lengths) ||
        !get_vector(a[5], "q_start", kI32, table.rows + 1, dev, &q_start))
      return nullptr;
    int64_t max_q = 1;
    if (a[5] != Py_None) {
      max_q = a[6] == Py_None ? hq.m : PyLong_AsLongLong(a[6]);
      if (PyErr_Occurred()) return nullptr;
    } else if (a[6] != Py_None) {
      max_q = PyLong_AsLongLong(a[6]);
      if (PyErr_Occurred()) return nullptr;
    }
    const double scale = a[7] == Py_None ? 1.0 / std::sqrt((double)std::max<int64_t>(hq.d, 1)) : PyFloat_AsDouble(a[7]);
    if (PyErr_Occurred()) return nullptr;
    Ref made, made_ws;
    if (out == Py_None) {
      const int type = code ? (int)code : hq.type;
      if (!make(THPVariable_Unpack(q), THPVariable_Unpack(q).sizes(), scalar_of(type), type, stream, &made))
        return nullptr;
      out = made.o;
    }
    float* lse;
    uint8_t* ws;
    if (!get_heads(out, "out", hq.m, hq.heads, hq.d, dev, &ho) ||
        !get_vector(a[10], "lse", kF32, hq.m * hq.heads, dev, &lse))
      return nullptr;
    if (workspace == Py_None) {
      const int64_t need = (int64_t)bound.attention_bytes(hq.m, table.rows, hq.heads, heads, hq.d, max_q);
      if (!make(THPVariable_Unpack(q), {need > 16 ? need : 16}, at::kByte, kU8, stream, &made_ws)) return nullptr;
      workspace = made_ws.o;
    }
    if (!get_vector(workspace, "workspace", kU8, 0, dev, &ws)) return nullptr;
    const int64_t ws_bytes = THPVariable_Unpack(workspace).numel();
    if (!launch(dev, "lowbit_attention", [&] {
          return bound.attention(hq.p, hq.type, hq.ld, hq.ldh, hq.m, hq.heads, pages, n_pages, heads, hq.d, page,
                                 table.p, table.columns, table.ld, lengths, q_start, table.rows, max_q, (float)scale,
                                 ho.p, ho.type, ho.ld, ho.ldh, lse, ws, (size_t)ws_bytes, st);
        }))
      return nullptr;
    Py_INCREF(out);
    return out;
  });
}

// sample(y, u, temperature, top_k, top_p, min_p, idx, prob, workspace, stream)
// -> (idx, prob)
PyObject* sample(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_ok(n, 10) || !ready()) return nullptr;
  return guarded([&]() -> PyObject* {
    PyObject *y = a[0], *idx = a[6], *prob = a[7], *workspace = a[8], *stream = a[9];
    long long b, v;
    int dev;
    hipStream_t st;
    Rows ry;
    if (!get_shape(y, "y", &b, &v, &dev) || !get_stream(stream, dev, &st) || !get_rows(y, "y", b, v, dev, &ry))
      return nullptr;
    const float *u, *temperature, *top_p, *min_p;
    const int32_t* top_k;
    if (!need_vector(a[1], "u", kF32, b, dev, &u) || !get_vector(a[2], "temperature", kF32, b, dev, &temperature) ||
        !get_vector(a[3], "top_k", kI32, b, dev, &top_k) || !get_vector(a[4], "top_p", kF32, b, dev, &top_p) ||
        !get_vector(a[5], "min_p", kF32, b, dev, &min_p))
      return nullptr;
    const at::Tensor& t = THPVariable_Unpack(y);
    Ref made_idx, made_prob, made_ws;
    if (idx == Py_None) {
      if (!make(t, {b}, at::kInt, kI32, stream, &made_idx)) return nullptr;
      idx = made_idx.o;
    }
    if (prob == Py_None) {
      if (!make(t, {b}, at::kFloat, kF32, stream, &made_prob)) return nullptr;
      prob = made_prob.o;
    }
    if (workspace == Py_None) {
      const int64_t need = (int64_t)bound.sample_bytes(v, b);
      if (!make(t, {need > 16 ? need : 16}, at::kByte, kU8, stream, &made_ws)) return nullptr;
      workspace = made_ws.o;
    }
    int32_t* idx_p;
    float* prob_p;
    uint8_t* ws;
    if (!get_vector(idx, "idx", kI32, b, dev, &idx_p) || !get_vector(prob, "prob", kF32, b, dev, &prob_p) ||
        !get_vector(workspace, "workspace", kU8, 0, dev, &ws))
      return nullptr;
    const int64_t ws_bytes = THPVariable_Unpack(workspace).numel();
    if (!launch(dev, "lowbit_sample", [&] {
          return bound.sample(ry.p, ry.type, ry.ld, v, b, temperature, top_k, top_p, min_p, u, idx_p, prob_p, ws,
                              (size_t)ws_bytes, st);
        }))
      return nullptr;
    return PyTuple_Pack(2, idx, prob);
  });
}

PyMethodDef methods[] = {{"bind", (PyCFunction)(void (*)())bind, METH_FASTCALL, nullptr},
                         {"norm", (PyCFunction)(void (*)())norm, METH_FASTCALL, nullptr},
                         {"logits", (PyCFunction)(void (*)())logits, METH_FASTCALL, nullptr},
                         {"lora", (PyCFunction)(void (*)())lora, METH_FASTCALL, nullptr},
                         {"rope", (PyCFunction)(void (*)())rope, METH_FASTCALL, nullptr},
                         {"kv_store", (PyCFunction)(void (*)())kv_store, METH_FASTCALL, nullptr},
                         {"kv_load", (PyCFunction)(void (*)())kv_load, METH_FASTCALL, nullptr},
                         {"attention", (PyCFunction)(void (*)())attention, METH_FASTCALL, nullptr},
                         {"sample", (PyCFunction)(void (*)())sample, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
