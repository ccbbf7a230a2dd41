// CPython module behind serving.py's allocating calls.  At decode a product
// takes a few microseconds on the device; checking its tensors, allocating its
// result and marshalling the C ABI call from Python took 10 to 20, here 3 to
// 5.  Everything it launches goes through the C ABI of libgptq.so
// (include/gptq.h); the checks are serving.py's.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <string>

#include "gptq.h"

namespace {

PyObject* g_error = nullptr;        // GptqError(status, message)
PyObject* g_tokens_type = nullptr;  // Int8Tokens(q, scale, sum)

// A Python exception is set.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const std::string& message) {
  PyErr_SetString(type, message.c_str());
  throw Raised();
}

std::string name_of(at::ScalarType t) {
  switch (t) {
    case at::kHalf: return "torch.float16";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kChar: return "torch.int8";
    case at::kInt: return "torch.int32";
    default: return at::toString(t);
  }
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

gptq_dtype_t code(at::ScalarType t) {
  if (t == at::kHalf) return GPTQ_F16;
  if (t == at::kBFloat16) return GPTQ_BF16;
  if (t == at::kFloat) return GPTQ_F32;
  raise(PyExc_TypeError, "unsupported dtype " + name_of(t));
}

int64_t round16(int64_t n) { return (n + 15) & ~(int64_t)15; }

// The row stride of a matrix with contiguous rows; a single row's is of no
// account and is given as the shortest any call accepts.
int64_t row_stride(const at::Tensor& t, const char* name) {
  if (t.dim() != 2 || (t.stride(1) != 1 && t.size(1) > 1))
    raise(PyExc_ValueError, std::string(name) + " must be a 2-D tensor with contiguous rows");
  return t.size(0) > 1 ? t.stride(0) : round16(t.size(1));
}

void* vector(const at::Tensor& t, int64_t n, at::ScalarType type, const at::Device& device, const char* name) {
  if (t.scalar_type() != type || t.dim() != 1 || t.size(0) != n || t.device() != device || !t.is_contiguous())
    raise(PyExc_ValueError, std::string(name) + " must be a contiguous " + name_of(type) + " vector of " +
                                std::to_string(n) + " elements on " + device.str());
  return t.data_ptr();
}

void* vector(PyObject* o, int64_t n, at::ScalarType type, const at::Device& device, const char* name) {
  return o == Py_None ? nullptr : vector(tensor(o, name), n, type, device, name);
}

struct Matrix {
  void* p = nullptr;
  int64_t ld = 0;
};
Matrix matrix(const at::Tensor& t, int64_t rows, int64_t cols, at::ScalarType type, const at::Device& device,
              const char* name) {
  if (t.scalar_type() != type || t.dim() != 2 || t.size(0) != rows || t.size(1) != cols || t.device() != device)
    raise(PyExc_ValueError, std::string(name) + " must be a " + name_of(type) + " matrix of " + std::to_string(rows) +
                                " x " + std::to_string(cols) + " on " + device.str());
  return {t.data_ptr(), row_stride(t, name)};
}

// (weight, scale[, zero])
int64_t layer(PyObject* o, int64_t in, const at::Device& device, const char* name, gptq_int8_layer_t* out) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) < 2 || PyTuple_GET_SIZE(o) > 3)
    raise(PyExc_TypeError, std::string(name) + " must be an Int8Layer or a tuple (weight, scale[, zero])");
  const std::string n(name);
  const at::Tensor& w = tensor(PyTuple_GET_ITEM(o, 0), (n + ".weight").c_str());
  if (w.dim() != 2) raise(PyExc_ValueError, n + ": the weight must be a 2-D tensor");
  const int64_t channels = w.size(0);
  const Matrix m = matrix(w, channels, in, at::kChar, device, (n + ".weight").c_str());
  out->w = (const int8_t*)m.p;
  out->ldw = m.ld;
  out->scale = (const float*)vector(tensor(PyTuple_GET_ITEM(o, 1), "scale"), channels, at::kFloat, device,
                                    (n + ".scale").c_str());
  PyObject* zero = PyTuple_GET_SIZE(o) == 3 ? PyTuple_GET_ITEM(o, 2) : Py_None;
  out->zero = (const int32_t*)vector(zero, channels, at::kInt, device, (n + ".zero").c_str());
  return channels;
}

void check(gptq_status_t status) {
  if (status == GPTQ_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "is", (int)status, gptq_last_error());
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Raised();
}

// The device current, and its current stream, for one call.
struct On {
  c10::cuda::OptionalCUDAGuard guard;
  void* stream;
  explicit On(const at::Device& d) {
    if (!d.is_cuda()) raise(PyExc_ValueError, "the tensors must be on a CUDA device, not " + d.str());
    if (c10::cuda::current_device() != d.index()) guard.set_index(d.index());
    stream = c10::cuda::getCurrentCUDAStream(d.index()).stream();
  }
};

// The interpreter is free for other threads: a launch may wait for room in a
// full queue and an allocation for the device, and a host callback that the
// stream has yet to run may need the interpreter.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  Unlocked() = default;
  Unlocked(const Unlocked&) = delete;
  ~Unlocked() { PyEval_RestoreThread(state); }
};

at::Tensor empty(at::IntArrayRef size, at::ScalarType type, const at::Device& device) {
  return at::empty(size, at::TensorOptions().dtype(type).device(device));
}

// An Int8Tokens to write to, in tensors of their own.
struct NewTokens {
  at::Tensor q, scale, sum;
  int64_t ld;
  NewTokens(int64_t tokens, int64_t in, const at::Device& device) : ld(round16(in)) {
    q = empty({tokens, ld}, at::kChar, device);
    if (ld != in) q = q.narrow(1, 0, in);
    scale = empty({tokens}, at::kFloat, device);
    sum = empty({tokens}, at::kInt, device);
  }
  PyObject* wrap() const {
    return PyObject_CallFunction(g_tokens_type, "NNN", THPVariable_Wrap(q), THPVariable_Wrap(scale),
                                 THPVariable_Wrap(sum));
  }
};

// linear (up == nullptr) and gated.  x: a floating matrix, or an Int8Tokens.
at::Tensor product(PyObject* x, PyObject* w, PyObject* up, PyObject* bias, int act, PyObject* dtype) {
  const bool tokens8 = PyTuple_Check(x);
  if (tokens8 && PyTuple_GET_SIZE(x) != 3) raise(PyExc_TypeError, "x must be a tensor or an Int8Tokens");
  const at::Tensor& X = tensor(tokens8 ? PyTuple_GET_ITEM(x, 0) : x, tokens8 ? "x.q" : "x");
  const char* name = tokens8 ? "x.q" : "x";
  if (tokens8 && X.scalar_type() != at::kChar)
    raise(PyExc_ValueError, "x.q must be int8, got " + name_of(X.scalar_type()));
  const int64_t ldx = row_stride(X, name), T = X.size(0), in = X.size(1);
  const at::Device device = X.device();
  gptq_int8_tokens_t q{};
  gptq_dtype_t xt{};
  if (tokens8) {
    q = {(const int8_t*)X.data_ptr(), ldx,
         (const float*)vector(tensor(PyTuple_GET_ITEM(x, 1), "x.scale"), T, at::kFloat, device, "x.scale"),
         (const int32_t*)vector(tensor(PyTuple_GET_ITEM(x, 2), "x.sum"), T, at::kInt, device, "x.sum")};
  } else {
    xt = code(X.scalar_type());
  }
  gptq_int8_layer_t lw{}, lu{};
  const int64_t out = layer(w, in, device, up ? "gate" : "layer", &lw);
  if (up) {
    const int64_t out_up = layer(up, in, device, "up", &lu);
    if (out_up != out)
      raise(PyExc_ValueError, "gate and up differ in size: " + std::to_string(out) + " and " + std::to_string(out_up) +
                                  " channels");
  }
  const float* b = up ? nullptr : (const float*)vector(bias, out, at::kFloat, device, "bias");
  if (dtype != Py_None && !THPDtype_Check(dtype)) raise(PyExc_TypeError, "dtype must be a torch.dtype");
  const at::ScalarType type = dtype != Py_None ? reinterpret_cast<THPDtype*>(dtype)->scalar_type
                              : tokens8        ? at::kBFloat16
                                               : X.scalar_type();
  const gptq_dtype_t yt = code(type);
  On on(device);
  at::Tensor Y, ws;
  gptq_status_t status;
  {
    Unlocked unlocked;
    Y = empty({T, out}, type, device);
    void* const y = Y.data_ptr();
    if (tokens8) {
      status = up ? gptq_matmul_int8_gated(&q, T, in, &lw, &lu, out, (gptq_act_t)act, y, yt, out, on.stream)
                  : gptq_matmul_int8(&q, T, in, &lw, out, b, y, yt, out, on.stream);
    } else {
      const size_t n = gptq_linear_int8_ws_bytes(T, in);
      if (n) ws = empty({(int64_t)n}, at::kByte, device);
      void* const wsp = n ? ws.data_ptr() : nullptr;
      status = up ? gptq_linear_int8_gated(X.data_ptr(), xt, T, in, ldx, &lw, &lu, out, (gptq_act_t)act, y, yt, out, wsp,
                                           n, on.stream)
                  : gptq_linear_int8(X.data_ptr(), xt, T, in, ldx, &lw, out, b, y, yt, out, wsp, n, on.stream);
    }
  }
  check(status);
  return Y;
}

void need(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) raise(PyExc_TypeError, "expected " + std::to_string(want) + " arguments");
}

int integer(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  return (int)v;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return v;
}

template <typename F>
PyObject* guarded(F f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// linear(x, layer, bias, dtype)
PyObject* py_linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need(n, 4);
    return THPVariable_Wrap(product(a[0], a[1], nullptr, a[2], 0, a[3]));
  });
}

// gated(x, gate, up, act, dtype)
PyObject* py_gated(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need(n, 5);
    return THPVariable_Wrap(product(a[0], a[1], a[2], Py_None, integer(a[3]), a[4]));
  });
}

// quantize(X)
PyObject* py_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need(n, 1);
    const at::Tensor& X = tensor(a[0], "X");
    const int64_t ld = row_stride(X, "X");
    const gptq_dtype_t xt = code(X.scalar_type());
    On on(X.device());
    std::optional<NewTokens> x;
    gptq_status_t status;
    {
      Unlocked unlocked;
      x.emplace(X.size(0), X.size(1), X.device());
      status = gptq_quantize_tokens(X.data_ptr(), xt, X.size(0), X.size(1), ld, (int8_t*)x->q.data_ptr(), x->ld,
                                    (float*)x->scale.data_ptr(), (int32_t*)x->sum.data_ptr(), on.stream);
    }
    check(status);
    return x->wrap();
  });
}

// norm(h, y, weight, bias, post_weight, post_bias, gate, alpha, beta, kind, eps, quantize, inplace)
PyObject* py_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need(n, 13);
    gptq_norm_t p = {};
    const at::Tensor& h = tensor(a[0], "h");
    p.ldh = row_stride(h, "h");
    const int64_t T = h.size(0), d = h.size(1);
    const at::Device device = h.device();
    const at::ScalarType ht = h.scalar_type();
    const at::ScalarType yt = tensor(a[1] != Py_None ? a[1] : a[2], "weight").scalar_type();
    p.tokens = T;
    p.d = d;
    p.ht = code(ht);
    p.yt = code(yt);
    p.h = h.data_ptr();
    if (a[1] != Py_None) {
      const Matrix m = matrix(tensor(a[1], "y"), T, d, yt, device, "y");
      p.y = m.p;
      p.ldy = m.ld;
    }
    p.weight = vector(a[2], d, yt, device, "weight");
    p.bias = vector(a[3], d, yt, device, "bias");
    p.post_weight = vector(a[4], d, yt, device, "post_weight");
    p.post_bias = vector(a[5], d, yt, device, "post_bias");
    if (a[6] != Py_None) {
      const at::Tensor& g = tensor(a[6], "gate");
      if (g.dim() == 2) {
        const Matrix m = matrix(g, T, d, yt, device, "gate");
        p.gate = m.p;
        p.ldgate = m.ld;
      } else {
        p.gate = vector(g, d, yt, device, "gate");
      }
    }
    const double alpha = number(a[7]);
    p.alpha = (float)alpha;
    p.beta = (float)number(a[8]);
    p.kind = (gptq_norm_kind_t)integer(a[9]);
    p.eps = (float)number(a[10]);
    const bool quantize = PyObject_IsTrue(a[11]) == 1, inplace = PyObject_IsTrue(a[12]) == 1;
    On on(device);
    at::Tensor h_out, x;
    std::optional<NewTokens> tokens;
    gptq_status_t status;
    {
      Unlocked unlocked;
      if (inplace) {
        p.h_out = h.data_ptr();
        p.ldh_out = p.ldh;
      } else if (a[1] != Py_None || alpha != 1.0) {
        h_out = empty({T, d}, ht, device);
        p.h_out = h_out.data_ptr();
        p.ldh_out = d;
      }
      if (quantize) {
        tokens.emplace(T, d, device);
        p.q = (int8_t*)tokens->q.data_ptr();
        p.ldq = tokens->ld;
        p.scale = (float*)tokens->scale.data_ptr();
        p.sum = (int32_t*)tokens->sum.data_ptr();
      } else {
        x = empty({T, d}, yt, device);
        p.x = x.data_ptr();
        p.ldx = d;
      }
      status = gptq_norm_tokens(&p, on.stream);
    }
    check(status);
    PyObject* second = quantize ? tokens->wrap() : THPVariable_Wrap(x);
    if (!second) return nullptr;
    PyObject* first = h_out.defined() ? THPVariable_Wrap(h_out) : (Py_INCREF(a[0]), a[0]);
    return Py_BuildValue("NN", first, second);
  });
}

// init(GptqError, Int8Tokens)
PyObject* py_init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need(n, 2);
    Py_INCREF(a[0]);
    Py_INCREF(a[1]);
    g_error = a[0];
    g_tokens_type = a[1];
    Py_RETURN_NONE;
  });
}

#define FAST(f) (PyCFunction)(void (*)(void)) f, METH_FASTCALL, nullptr
PyMethodDef methods[] = {{"init", FAST(py_init)},         {"linear", FAST(py_linear)}, {"gated", FAST(py_gated)},
                         {"quantize", FAST(py_quantize)}, {"norm", FAST(py_norm)},     {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serving", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serving(void) { return PyModule_Create(&module); }
