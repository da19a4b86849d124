// Python calls of the layer operators, of those on the residual stream and of sampling, from
// torch tensors to the C ABI.
//
// A call of a few microseconds on the GPU should not wait for the interpreter: these
// functions check the tensors, allocate outputs and scratch through torch's
// allocator and call the library on the tensors' device and its current CUDA stream.
// block.py, residual.py and sampling.py document them and handle calls that name a stream.
#include <Python.h>

#include <algorithm>
#include <array>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <exception>
#include <initializer_list>
#include <utility>
#include <vector>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "flce.h"

namespace {

using at::Tensor;

constexpr int kMaxDev = 64;
PyObject* g_error_class = nullptr;  // FlceError(status, what)
PyObject* g_error_word = nullptr;   // device index -> its int32 error word (a tensor)
void* g_words[kMaxDev] = {};

// A refusal: the Python exception is set.
struct Refused : std::exception {};

[[noreturn]] void refuse(PyObject* type, const char* format, const char* name) {
  PyErr_Format(type, format, name);
  throw Refused();
}

void done(flce_status_t st, const char* what) {
  if (st == FLCE_OK) return;
  PyObject* e = PyObject_CallFunction(g_error_class, "is", static_cast<int>(st), what);
  if (e) {
    PyErr_SetObject(g_error_class, e);
    Py_DECREF(e);
  }
  throw Refused();
}

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "flce: %s must be a tensor", name);
  return THPVariable_Unpack(o);
}
const Tensor* optional(PyObject* o, const char* name) {
  return o == Py_None ? nullptr : &tensor(o, name);
}

void* error_word(int index) {
  if (index < 0 || index >= kMaxDev) refuse(PyExc_ValueError, "flce: %s", "device index");
  if (!g_words[index]) {
    PyObject* w = PyObject_CallFunction(g_error_word, "i", index);
    if (!w) throw Refused();
    g_words[index] = tensor(w, "error word").data_ptr();
    Py_DECREF(w);  // the callable keeps the tensor
  }
  return g_words[index];
}

const char* const kActivations[] = {"none", "relu", "gelu", "gelu_tanh", "silu", "sigmoid"};
int activation(PyObject* o) {
  const char* s = PyUnicode_Check(o) ? PyUnicode_AsUTF8(o) : nullptr;
  for (int i = 0; s && i < 6; ++i)
    if (std::strcmp(s, kActivations[i]) == 0) return i;
  PyErr_Clear();
  PyErr_Format(PyExc_ValueError,
               "flce: activation must be one of none, relu, gelu, gelu_tanh, silu, sigmoid, got %R",
               o);
  throw Refused();
}

// x of a call: two-dimensional, bf16 or fp16, on a CUDA device.
void check_x(const Tensor& x) {
  if (!x.is_cuda() || (x.scalar_type() != at::kBFloat16 && x.scalar_type() != at::kHalf))
    refuse(PyExc_TypeError, "flce: %s must be a bf16 or fp16 CUDA tensor", "x");
  if (x.dim() != 2) refuse(PyExc_ValueError, "flce: %s must be two-dimensional", "x");
}

// `t` has x's type and device.
void check_like(const Tensor& t, const Tensor& x, const char* name) {
  if (t.scalar_type() != x.scalar_type() || !t.is_cuda())
    refuse(PyExc_TypeError, "flce: %s must be a CUDA tensor of x's type", name);
  if (t.get_device() != x.get_device())
    refuse(PyExc_ValueError, "flce: %s must be on x's device", name);
}

// The row pitch of a [rows, cols] tensor like x whose rows are contiguous.
int64_t rows_of(const Tensor& t, int64_t rows, int64_t cols, const Tensor& x, const char* name) {
  check_like(t, x, name);
  if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
    refuse(PyExc_ValueError, "flce: %s has another shape than the call's sizes", name);
  if (cols > 1 && t.stride(1) != 1)
    refuse(PyExc_ValueError, "flce: the rows of %s must be contiguous", name);
  if (rows <= 1) return cols;
  if (t.stride(0) < cols)
    refuse(PyExc_ValueError, "flce: the rows of %s must not overlap", name);
  return t.stride(0);
}

void dense(const Tensor& t, at::IntArrayRef shape, const Tensor& x, const char* name) {
  check_like(t, x, name);
  if (t.sizes() != shape || !t.is_contiguous())
    refuse(PyExc_ValueError, "flce: %s must be contiguous and of the call's shape", name);
}

// The kept values: of x's type in the fixed form, int16 in the relative one.
int32_t kept(const Tensor& t, at::IntArrayRef shape, const Tensor& x) {
  if (t.scalar_type() != at::kShort) {
    dense(t, shape, x, "pre");
    return FLCE_KEEP_FIXED;
  }
  if (!t.is_cuda() || t.get_device() != x.get_device())
    refuse(PyExc_ValueError, "flce: %s must be on x's device", "pre");
  if (t.sizes() != shape || !t.is_contiguous())
    refuse(PyExc_ValueError, "flce: %s must be contiguous and of the call's shape", "pre");
  return FLCE_KEEP_RELATIVE;
}

void check_weight(const Tensor& W, const Tensor& x, const char* name) {
  if (W.dim() != 2 || W.size(1) != x.size(1))
    refuse(PyExc_ValueError, "flce: %s must have as many columns as x", name);
  dense(W, W.sizes(), x, name);
}

Tensor scratch(PyObject* given, size_t need, const Tensor& x) {
  if (need == 0) return Tensor();
  if (given != Py_None) {
    const Tensor& w = tensor(given, "workspace");
    if (w.scalar_type() != at::kByte || !w.is_cuda() || !w.is_contiguous())
      refuse(PyExc_TypeError, "flce: %s must be a contiguous uint8 CUDA tensor", "workspace");
    if (w.get_device() != x.get_device())
      refuse(PyExc_ValueError, "flce: %s must be on x's device", "workspace");
    if (static_cast<size_t>(w.numel()) >= need) return w;
  }
  return at::empty({static_cast<int64_t>(need)}, x.options().dtype(at::kByte));
}

void* data(const Tensor* t) { return t && t->defined() ? t->data_ptr() : nullptr; }
void* data(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
size_t bytes(const Tensor& t) { return t.defined() ? static_cast<size_t>(t.numel()) : 0; }

bool aligned16(const Tensor& t) { return reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 == 0; }

void* stream_of(const Tensor& x) { return c10::cuda::getCurrentCUDAStream(x.get_device()).stream(); }

// A call wrote into a tensor of the caller's: autograd refuses a backward that saved the
// values from before, as with torch's own in-place operations.
void written(const Tensor& t) {
  if (t.defined() && !t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

PyObject* wrap(const Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
PyObject* wrap2(const Tensor& a, const Tensor& b) {
  PyObject *pa = wrap(a), *pb = wrap(b);
  if (!pa || !pb) throw Refused();
  PyObject* r = PyTuple_Pack(2, pa, pb);
  Py_DECREF(pa);
  Py_DECREF(pb);
  return r;
}
PyObject* wrap3(const Tensor& a, const Tensor& b, const Tensor& c) {
  PyObject *pa = wrap(a), *pb = wrap(b), *pc = wrap(c);
  if (!pa || !pb || !pc) throw Refused();
  PyObject* r = PyTuple_Pack(3, pa, pb, pc);
  Py_DECREF(pa);
  Py_DECREF(pb);
  Py_DECREF(pc);
  return r;
}

// Runs f, turning C++ exceptions into Python ones: none leaves the module.
template <class Fn>
PyObject* guarded(Py_ssize_t given, Py_ssize_t wanted, Fn f) {
  if (given != wanted) {
    PyErr_SetString(PyExc_TypeError, "flce: wrong number of arguments");
    return nullptr;
  }
  try {
    return f();
  } catch (const Refused&) {
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "flce: unknown error");
  }
  return nullptr;
}

flce_linear_params_t linear_params(const Tensor& x, const Tensor& W, const Tensor* b, PyObject* act) {
  check_x(x);
  check_weight(W, x, "W");
  flce_linear_params_t p;
  std::memset(&p, 0, sizeof(p));
  p.M = x.size(0);
  p.K = x.size(1);
  p.N = W.size(0);
  if (b) dense(*b, {p.N}, x, "b");
  p.ld_x = rows_of(x, p.M, p.K, x, "x");
  p.activation = activation(act);
  p.has_bias = b ? 1 : 0;
  p.input_fp16 = x.scalar_type() == at::kHalf ? 1 : 0;
  return p;
}

// linear_forward(x, W, b, residual, activation, pre, out, workspace) -> y
PyObject* linear_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&] {
    const Tensor &x = tensor(a[0], "x"), &W = tensor(a[1], "W");
    const Tensor *b = optional(a[2], "b"), *res = optional(a[3], "residual"),
                 *pre = optional(a[5], "pre"), *out = optional(a[6], "out");
    flce_linear_params_t p = linear_params(x, W, b, a[4]);
    const c10::cuda::CUDAGuard guard(x.device());
    p.has_residual = res ? 1 : 0;
    if (res) p.ld_res = rows_of(*res, p.M, p.N, x, "residual");
    if (pre) p.keep = kept(*pre, {p.M, p.N}, x);
    if (out) p.ld_y = rows_of(*out, p.M, p.N, x, "out");
    const Tensor y = out ? *out : at::empty({p.M, p.N}, x.options());
    const Tensor ws = scratch(a[7], flce_linear_workspace_size(&p, 0), x);
    done(flce_linear_forward(&p, data(x), data(W), data(b), data(res), data(y), data(pre), data(ws),
                             bytes(ws), static_cast<int32_t*>(error_word(x.get_device())),
                             stream_of(x)),
         "flce_linear_forward");
    if (out) written(*out);
    if (pre) written(*pre);
    return wrap(y);
  });
}

at::ScalarType grad_type(bool fp32, const Tensor& x) { return fp32 ? at::kFloat : x.scalar_type(); }

// linear_backward(dy, x, W, b, activation, pre, dW_fp32, db_fp32, need_dx, need_dW, need_db,
//                 workspace) -> (dx, dW, db)
PyObject* linear_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&] {
    const Tensor &dy = tensor(a[0], "dy"), &x = tensor(a[1], "x"), &W = tensor(a[2], "W");
    const Tensor *b = optional(a[3], "b"), *pre = optional(a[5], "pre");
    flce_linear_params_t p = linear_params(x, W, b, a[4]);
    const c10::cuda::CUDAGuard guard(x.device());
    p.ld_y = rows_of(dy, p.M, p.N, x, "dy");
    p.dW_fp32 = a[6] == Py_True ? 1 : 0;
    p.db_fp32 = a[7] == Py_True ? 1 : 0;
    if (p.activation == FLCE_ACT_NONE) {
      pre = nullptr;
    } else {
      if (!pre)
        refuse(PyExc_ValueError, "flce: the backward of a layer with an activation needs %s", "pre=");
      p.keep = kept(*pre, {p.M, p.N}, x);
    }
    Tensor dx, dW, db;
    if (PyObject_IsTrue(a[8])) dx = at::empty({p.M, p.K}, x.options());
    if (PyObject_IsTrue(a[9])) dW = at::empty({p.N, p.K}, x.options().dtype(grad_type(p.dW_fp32, x)));
    if (b && PyObject_IsTrue(a[10])) db = at::empty({p.N}, x.options().dtype(grad_type(p.db_fp32, x)));
    const Tensor ws = scratch(a[11], flce_linear_workspace_size(&p, aligned16(dy) ? 2 : 1), x);
    done(flce_linear_backward(&p, data(dy), data(x), data(W), data(pre), data(dx), data(dW), data(db),
                              data(ws), bytes(ws),
                              static_cast<int32_t*>(error_word(x.get_device())), stream_of(x)),
         "flce_linear_backward");
    return wrap3(dx, dW, db);
  });
}

flce_gated_params_t gated_params(const Tensor& x, const Tensor& Wg, const Tensor& Wu, PyObject* act) {
  check_x(x);
  check_weight(Wg, x, "Wg");
  dense(Wu, Wg.sizes(), x, "Wu");
  flce_gated_params_t p;
  std::memset(&p, 0, sizeof(p));
  p.M = x.size(0);
  p.K = x.size(1);
  p.F = Wg.size(0);
  p.ld_x = rows_of(x, p.M, p.K, x, "x");
  p.activation = activation(act);
  p.input_fp16 = x.scalar_type() == at::kHalf ? 1 : 0;
  return p;
}

// gated_forward(x, Wg, Wu, activation, pre, out, workspace) -> h
PyObject* gated_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&] {
    const Tensor &x = tensor(a[0], "x"), &Wg = tensor(a[1], "Wg"), &Wu = tensor(a[2], "Wu");
    const Tensor *pre = optional(a[4], "pre"), *out = optional(a[5], "out");
    flce_gated_params_t p = gated_params(x, Wg, Wu, a[3]);
    const c10::cuda::CUDAGuard guard(x.device());
    if (pre) p.keep = kept(*pre, {2, p.M, p.F}, x);
    if (out) p.ld_h = rows_of(*out, p.M, p.F, x, "out");
    const Tensor h = out ? *out : at::empty({p.M, p.F}, x.options());
    const Tensor ws = scratch(a[6], flce_gated_workspace_size(&p, 0), x);
    done(flce_gated_forward(&p, data(x), data(Wg), data(Wu), data(h), data(pre), data(ws), bytes(ws),
                            static_cast<int32_t*>(error_word(x.get_device())), stream_of(x)),
         "flce_gated_forward");
    if (out) written(*out);
    if (pre) written(*pre);
    return wrap(h);
  });
}

// gated_backward(dh, x, Wg, Wu, pre, activation, dW_fp32, need_dx, need_dW, workspace)
//   -> (dx, dWg, dWu)
PyObject* gated_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&] {
    const Tensor &dh = tensor(a[0], "dh"), &x = tensor(a[1], "x"), &Wg = tensor(a[2], "Wg"),
                 &Wu = tensor(a[3], "Wu"), &pre = tensor(a[4], "pre");
    flce_gated_params_t p = gated_params(x, Wg, Wu, a[5]);
    const c10::cuda::CUDAGuard guard(x.device());
    p.ld_h = rows_of(dh, p.M, p.F, x, "dh");
    p.keep = kept(pre, {2, p.M, p.F}, x);
    p.dW_fp32 = a[6] == Py_True ? 1 : 0;
    Tensor dx, dWg, dWu;
    if (PyObject_IsTrue(a[7])) dx = at::empty({p.M, p.K}, x.options());
    if (PyObject_IsTrue(a[8])) {
      const auto options = x.options().dtype(grad_type(p.dW_fp32, x));
      dWg = at::empty({p.F, p.K}, options);
      dWu = at::empty({p.F, p.K}, options);
    }
    const Tensor ws = scratch(a[9], flce_gated_workspace_size(&p, 1), x);
    done(flce_gated_backward(&p, data(dh), data(x), data(Wg), data(Wu), data(pre), data(dx),
                             data(dWg), data(dWu), data(ws), bytes(ws),
                             static_cast<int32_t*>(error_word(x.get_device())), stream_of(x)),
         "flce_gated_backward");
    return wrap3(dx, dWg, dWu);
  });
}

// The tensors of a gradient list as the C ABI's HOST arrays.
struct GradList {
  std::vector<const void*> ptrs;
  std::vector<void*> out;
  std::vector<int64_t> numel;
  std::vector<int32_t> types;
};

int32_t grad_dtype(const Tensor& g) {
  switch (g.is_cuda() ? g.scalar_type() : at::kDouble) {
    case at::kBFloat16: return FLCE_DTYPE_BF16;
    case at::kHalf: return FLCE_DTYPE_FP16;
    case at::kFloat: return FLCE_DTYPE_FP32;
    default: refuse(PyExc_TypeError, "flce: %s must be bf16, fp16 or fp32 CUDA tensors", "gradients");
  }
}

// grads, out: lists (out may be None). Returns the first gradient.
const Tensor& read_grads(PyObject* grads, PyObject* out, GradList* l) {
  if (!PyList_Check(grads) || (out != Py_None && !PyList_Check(out)))
    refuse(PyExc_TypeError, "flce: %s must be lists", "gradients and out");
  const Py_ssize_t n = PyList_GET_SIZE(grads);
  if (n == 0) refuse(PyExc_ValueError, "flce: no %s given", "gradients");
  if (out != Py_None && PyList_GET_SIZE(out) != n)
    refuse(PyExc_ValueError, "flce: %s must hold as many tensors as there are gradients", "out");
  const Tensor& first = tensor(PyList_GET_ITEM(grads, 0), "a gradient");
  l->ptrs.resize(n);
  l->numel.resize(n);
  l->types.resize(n);
  if (out != Py_None) l->out.resize(n);
  for (Py_ssize_t i = 0; i < n; ++i) {
    const Tensor& g = tensor(PyList_GET_ITEM(grads, i), "a gradient");
    l->types[i] = grad_dtype(g);
    if (g.get_device() != first.get_device())
      refuse(PyExc_ValueError, "flce: %s must be on one device", "gradients");
    if (!g.is_contiguous() && !g.is_non_overlapping_and_dense())
      refuse(PyExc_ValueError, "flce: %s must be dense", "gradients");
    l->ptrs[i] = g.data_ptr();
    l->numel[i] = g.numel();
    if (out == Py_None) continue;
    const Tensor& o = tensor(PyList_GET_ITEM(out, i), "an output");
    if (o.scalar_type() != g.scalar_type() || !o.is_cuda() || o.get_device() != g.get_device())
      refuse(PyExc_TypeError, "flce: %s must match the gradients' types and device", "out");
    if (o.sizes() != g.sizes() ||
        (o.strides() != g.strides() && !(o.is_contiguous() && g.is_contiguous())))
      refuse(PyExc_ValueError, "flce: %s must match the gradients' shapes and strides", "out");
    l->out[i] = o.data_ptr();
  }
  return first;
}

// Clipped tensors are written by different blocks: none may share memory with another.
void check_apart(const GradList& l) {
  std::vector<std::pair<uintptr_t, uintptr_t>> spans;
  spans.reserve(l.ptrs.size());
  for (size_t i = 0; i < l.ptrs.size(); ++i) {
    const void* to = l.out.empty() ? l.ptrs[i] : l.out[i];
    const uintptr_t begin = reinterpret_cast<uintptr_t>(to);
    const uintptr_t bytes = static_cast<uintptr_t>(l.numel[i]) * (l.types[i] == FLCE_DTYPE_FP32 ? 4 : 2);
    if (bytes > 0) spans.emplace_back(begin, begin + bytes);
  }
  std::sort(spans.begin(), spans.end());
  for (size_t i = 1; i < spans.size(); ++i)
    if (spans[i].first < spans[i - 1].second)
      refuse(PyExc_ValueError, "flce: %s must not overlap: give each once", "clipped tensors");
}

// clip_grads(grads, out, max_norm, eps, workspace) -> norm; max_norm None: the norm alone.
PyObject* clip_grads(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, [&] {
    GradList l;
    const Tensor& first = read_grads(a[0], a[1], &l);
    const c10::cuda::CUDAGuard guard(first.device());
    const int64_t count = static_cast<int64_t>(l.ptrs.size());
    double max_norm = 0.0, eps = 0.0;
    if (a[2] != Py_None) {
      check_apart(l);
      max_norm = PyFloat_AsDouble(a[2]);
      eps = PyFloat_AsDouble(a[3]);
      if (PyErr_Occurred()) throw Refused();
    }
    const Tensor norm = at::empty({}, first.options().dtype(at::kFloat));
    const Tensor ws = scratch(a[4], flce_grad_norm_workspace_size(count), first);
    float* to = static_cast<float*>(norm.data_ptr());
    if (a[2] == Py_None) {
      done(flce_grad_norm(count, l.ptrs.data(), l.numel.data(), l.types.data(), to, data(ws),
                          bytes(ws), stream_of(first)),
           "flce_grad_norm");
    } else {
      done(flce_clip_grads(count, l.ptrs.data(), l.out.empty() ? nullptr : l.out.data(),
                           l.numel.data(), l.types.data(), static_cast<float>(max_norm),
                           static_cast<float>(eps), to, data(ws), bytes(ws), stream_of(first)),
           "flce_clip_grads");
      PyObject* list = a[1] == Py_None ? a[0] : a[1];
      for (int64_t i = 0; i < count; ++i) written(tensor(PyList_GET_ITEM(list, i), "an output"));
    }
    return wrap(norm);
  });
}

// ---- operators on the residual stream, and sampling

int32_t float_type(const Tensor& t, const char* name) {
  switch (t.is_cuda() ? t.scalar_type() : at::kDouble) {
    case at::kBFloat16: return FLCE_DTYPE_BF16;
    case at::kHalf: return FLCE_DTYPE_FP16;
    case at::kFloat: return FLCE_DTYPE_FP32;
    default: refuse(PyExc_TypeError, "flce: %s must be a bf16, fp16 or fp32 CUDA tensor", name);
  }
}

// Rows of a tensor: [rows, cols] with contiguous rows, or contiguous of any other dimensions.
struct Rows {
  int64_t rows, cols, ld;
};
Rows rows_of(const Tensor& t, const char* name) {
  const int64_t dims = t.dim();
  if (dims == 0) refuse(PyExc_ValueError, "flce: %s must have a dimension", name);
  Rows r;
  r.cols = t.size(dims - 1);
  r.rows = 1;
  for (int64_t i = 0; i + 1 < dims; ++i) r.rows *= t.size(i);
  r.ld = r.cols;
  if (r.rows == 0 || r.cols == 0 || t.is_contiguous()) return r;
  if (dims != 2) refuse(PyExc_ValueError, "flce: %s must be contiguous, or have two dimensions", name);
  if (r.cols > 1 && t.stride(1) != 1)
    refuse(PyExc_ValueError, "flce: the rows of %s must be contiguous", name);
  if (r.rows > 1) {
    if (t.stride(0) < r.cols) refuse(PyExc_ValueError, "flce: the rows of %s must not overlap", name);
    r.ld = t.stride(0);
  }
  return r;
}
// The pitch of a tensor of x's shape and device.
int64_t pitch_like(const Tensor& t, const Tensor& x, const char* name) {
  if (!t.is_cuda() || t.get_device() != x.get_device())
    refuse(PyExc_ValueError, "flce: %s must be on x's device", name);
  if (t.sizes() != x.sizes())
    refuse(PyExc_ValueError, "flce: %s has another shape than the call's sizes", name);
  return rows_of(t, name).ld;
}
// A tensor of the stream: x's type or fp32.
int32_t stream_type(const Tensor& t, int32_t of, const char* name) {
  const int32_t type = float_type(t, name);
  if (type != of && type != FLCE_DTYPE_FP32)
    refuse(PyExc_TypeError, "flce: %s must be of x's type or fp32", name);
  return type;
}
void flat(const Tensor& t, at::ScalarType type, at::IntArrayRef shape, const Tensor& x, const char* name) {
  if (!t.is_cuda() || t.scalar_type() != type)
    refuse(PyExc_TypeError, "flce: %s must be a CUDA tensor of the type that the call documents", name);
  if (t.get_device() != x.get_device())
    refuse(PyExc_ValueError, "flce: %s must be on x's device", name);
  if (t.sizes() != shape || !t.is_contiguous())
    refuse(PyExc_ValueError, "flce: %s must be contiguous and of the call's shape", name);
}

// An output shares no memory with another tensor of the call, unless `same` allows it to be that
// one: then a thread reads an element before it writes it.
void apart(const Tensor& out, const Tensor* in, bool same, const char* name) {
  if (!in || !in->defined() || !out.defined() || out.numel() == 0 || in->numel() == 0) return;
  const Rows a = rows_of(out, name), b = rows_of(*in, name);
  const uintptr_t pa = reinterpret_cast<uintptr_t>(out.data_ptr()), pb = reinterpret_cast<uintptr_t>(in->data_ptr());
  const uintptr_t ea = out.element_size(), eb = in->element_size();
  const uintptr_t wa = a.cols * ea, wb = b.cols * eb, la = a.ld * ea, lb = b.ld * eb;
  if (pa >= pb + (b.rows - 1) * lb + wb || pb >= pa + (a.rows - 1) * la + wa) return;
  if (same && pa == pb && ea == eb && a.cols == b.cols && (la == lb || a.rows == 1)) return;
  // Columns of one buffer next to each other.
  if (la == lb && a.rows > 1 && b.rows > 1) {
    const uintptr_t off = pb >= pa ? (pb - pa) % la : (la - (pa - pb) % la) % la;
    if (off >= wa && off + wb <= la) return;
  }
  refuse(PyExc_ValueError, "flce: %s must not overlap another tensor of the call", name);
}

void apart_from(const Tensor& out, std::initializer_list<const Tensor*> others, const char* name) {
  for (const Tensor* t : others) apart(out, t, false, name);
}

double number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(PyExc_TypeError, "flce: %s must be a number", name);
  }
  return v;
}

// seed: an int (its low 64 bits), or an int64 CUDA tensor of one element; only with dropout.
const int64_t* read_seed(PyObject* o, PyObject* offset, double p, const Tensor& x, int64_t* seed, int64_t* off) {
  *seed = *off = 0;
  if (!(p > 0.0)) return nullptr;
  if (!PyLong_Check(offset)) refuse(PyExc_TypeError, "flce: %s must be an int", "offset");
  *off = static_cast<int64_t>(PyLong_AsUnsignedLongLongMask(offset));
  if (THPVariable_Check(o)) {
    const Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.scalar_type() != at::kLong || t.numel() != 1 || t.get_device() != x.get_device())
      refuse(PyExc_ValueError, "flce: a %s tensor must be one int64 on x's device", "seed");
    return t.data_ptr<int64_t>();
  }
  if (!PyLong_Check(o)) refuse(PyExc_TypeError, "flce: dropout needs a %s: an int or an int64 tensor", "seed");
  *seed = static_cast<int64_t>(PyLong_AsUnsignedLongLongMask(o));
  return nullptr;
}

struct NormCall {
  flce_rms_norm_params_t p;
  const int64_t* seed;
  Tensor h;  // the sum that the call writes, or x's
  bool write_h;
};

// What the two forwards share. h: None (allocated where the sum is not x), False, or a tensor.
NormCall norm_call(const Tensor& x, const Tensor* w, const Tensor* r, PyObject* eps, PyObject* dropout,
                   PyObject* seed, PyObject* offset, PyObject* h) {
  NormCall c;
  std::memset(&c.p, 0, sizeof(c.p));
  c.p.dtype = float_type(x, "x");
  const Rows rows = rows_of(x, "x");
  c.p.M = rows.rows;
  c.p.H = rows.cols;
  c.p.ld_x = rows.ld;
  c.p.eps = static_cast<float>(number(eps, "eps"));
  c.p.dropout = number(dropout, "dropout");
  c.seed = read_seed(seed, offset, c.p.dropout, x, &c.p.seed, &c.p.offset);
  c.p.weight_dtype = c.p.stream_dtype = c.p.dtype;
  if (w) {
    c.p.weight_dtype = stream_type(*w, c.p.dtype, "weight");
    flat(*w, w->scalar_type(), {c.p.H}, x, "weight");
  }
  if (r) {
    c.p.stream_dtype = stream_type(*r, c.p.dtype, "residual");
    c.p.ld_res = pitch_like(*r, x, "residual");
  }
  const bool sum = r || c.p.dropout > 0.0;
  c.write_h = false;
  if (h == Py_None) {
    c.write_h = sum;
    c.h = sum ? at::empty(x.sizes(), r ? r->options() : x.options()) : x;
    if (sum) c.p.ld_h = c.p.H;
  } else if (h != Py_False) {
    c.h = tensor(h, "h");
    const int32_t type = stream_type(c.h, c.p.dtype, "h");
    if (r && type != c.p.stream_dtype) refuse(PyExc_TypeError, "flce: %s must be of the residual's type", "h");
    c.p.stream_dtype = type;
    c.p.ld_h = pitch_like(c.h, x, "h");
    c.write_h = true;
    apart(c.h, &x, true, "h");
    apart(c.h, r, true, "h");
    apart(c.h, w, false, "h");
  }
  return c;
}

// rms_norm_forward(x, weight, residual, eps, dropout, seed, offset, h, rstd, out) -> (y, h)
PyObject* rms_norm_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&] {
    const Tensor& x = tensor(a[0], "x");
    const Tensor *w = optional(a[1], "weight"), *r = optional(a[2], "residual"), *rstd = optional(a[8], "rstd"),
                 *out = optional(a[9], "out");
    NormCall c = norm_call(x, w, r, a[3], a[4], a[5], a[6], a[7]);
    const c10::cuda::CUDAGuard guard(x.device());
    if (rstd) flat(*rstd, at::kFloat, {c.p.M}, x, "rstd");
    if (out) {
      if (out->scalar_type() != x.scalar_type()) refuse(PyExc_TypeError, "flce: %s must be of x's type", "out");
      c.p.ld_y = pitch_like(*out, x, "out");
      apart(*out, &x, true, "out");
      apart(*out, r, true, "out");
      apart(*out, w, false, "out");
      if (c.write_h) apart(*out, &c.h, false, "out");
    }
    if (rstd) apart_from(*rstd, {&x, w, r, &c.h, out}, "rstd");
    const Tensor y = out ? *out : at::empty(x.sizes(), x.options());
    done(flce_rms_norm_forward(&c.p, data(x), data(w), data(r), c.seed, data(y),
                               c.write_h ? data(c.h) : nullptr, static_cast<float*>(data(rstd)), nullptr,
                               stream_of(x)),
         "flce_rms_norm_forward");
    if (out) written(*out);
    if (c.write_h) written(c.h);
    if (rstd) written(*rstd);
    return wrap2(y, c.h);
  });
}

// rms_norm_quantized(x, weight, residual, eps, dropout, seed, offset, h, blocks, out, scale) -> (y8, scale, h)
PyObject* rms_norm_quantized(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&] {
    const Tensor& x = tensor(a[0], "x");
    const Tensor *w = optional(a[1], "weight"), *r = optional(a[2], "residual"), *out = optional(a[9], "out"),
                 *given = optional(a[10], "scale");
    NormCall c = norm_call(x, w, r, a[3], a[4], a[5], a[6], a[7]);
    const c10::cuda::CUDAGuard guard(x.device());
    c.p.scales = a[8] == Py_True ? FLCE_SCALES_BLOCK : FLCE_SCALES_ROW;
    if (out) {
      if (out->scalar_type() != at::kFloat8_e4m3fn)
        refuse(PyExc_TypeError, "flce: %s must be of type float8_e4m3fn", "out");
      c.p.ld_y = pitch_like(*out, x, "out");
      apart(*out, &x, false, "out");
      apart(*out, r, false, "out");
      apart(*out, w, false, "out");
      if (c.write_h) apart(*out, &c.h, false, "out");
    }
    std::vector<int64_t> shape(x.sizes().begin(), x.sizes().end() - 1);
    if (c.p.scales == FLCE_SCALES_BLOCK) shape.push_back((c.p.H + 127) / 128);
    if (given) {
      flat(*given, at::kFloat, shape, x, "scale");
      apart_from(*given, {&x, w, r, &c.h, out}, "scale");
    }
    const Tensor y = out ? *out : at::empty(x.sizes(), x.options().dtype(at::kFloat8_e4m3fn));
    const Tensor scale = given ? *given : at::empty(shape, x.options().dtype(at::kFloat));
    done(flce_rms_norm_forward(&c.p, data(x), data(w), data(r), c.seed, data(y),
                               c.write_h ? data(c.h) : nullptr, nullptr, static_cast<float*>(data(scale)),
                               stream_of(x)),
         "flce_rms_norm_forward");
    if (out) written(*out);
    if (given) written(*given);
    if (c.write_h) written(c.h);
    return wrap3(y, scale, c.h);
  });
}

// rms_norm_backward(dy, h, weight, rstd, dh, dropout, seed, offset, dW_fp32, need_dx, need_dr, need_dW,
//                   workspace) -> (dx, dresidual, dW)
PyObject* rms_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&] {
    const Tensor &dy = tensor(a[0], "dy"), &h = tensor(a[1], "h"), &rstd = tensor(a[3], "rstd");
    const Tensor *w = optional(a[2], "weight"), *dh = optional(a[4], "dh");
    flce_rms_norm_params_t p;
    std::memset(&p, 0, sizeof(p));
    p.dtype = float_type(dy, "dy");
    const Rows rows = rows_of(dy, "dy");
    p.M = rows.rows;
    p.H = rows.cols;
    p.ld_y = rows.ld;
    const c10::cuda::CUDAGuard guard(dy.device());
    p.stream_dtype = stream_type(h, p.dtype, "h");
    p.ld_h = pitch_like(h, dy, "h");
    flat(rstd, at::kFloat, {p.M}, dy, "rstd");
    p.weight_dtype = p.dtype;
    if (w) {
      p.weight_dtype = stream_type(*w, p.dtype, "weight");
      flat(*w, w->scalar_type(), {p.H}, dy, "weight");
    }
    if (dh) {
      if (float_type(*dh, "dh") != p.stream_dtype) refuse(PyExc_TypeError, "flce: %s must be of h's type", "dh");
      p.ld_res = pitch_like(*dh, dy, "dh");
    }
    p.dropout = number(a[5], "dropout");
    const int64_t* seed = read_seed(a[6], a[7], p.dropout, dy, &p.seed, &p.offset);
    p.dW_fp32 = a[8] == Py_True ? 1 : 0;
    const bool need_dx = PyObject_IsTrue(a[9]), need_dr = PyObject_IsTrue(a[10]);
    const bool equal = p.dropout == 0.0 && p.dtype == p.stream_dtype;
    Tensor dx, dr, dW;
    if (need_dx || (need_dr && equal)) dx = at::empty(dy.sizes(), dy.options());
    if (need_dr) dr = equal ? dx : at::empty(dy.sizes(), h.options());
    if (w && PyObject_IsTrue(a[11])) dW = at::empty({p.H}, dy.options().dtype(grad_type(p.dW_fp32, dy)));
    const Tensor ws = scratch(a[12], dW.defined() ? flce_rms_norm_workspace_size(&p) : 0, dy);
    done(flce_rms_norm_backward(&p, data(dy), data(h), data(w), static_cast<const float*>(data(rstd)), data(dh),
                                seed, data(dx), data(dr), data(dW), data(ws), bytes(ws), stream_of(dy)),
         "flce_rms_norm_backward");
    if (!need_dx) dx = Tensor();
    return wrap3(dx, dr, dW);
  });
}

// dropout(x, p, seed, offset, residual, out, like) -> y; like: a tensor of the output's type, or None
PyObject* dropout(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&] {
    const Tensor& x = tensor(a[0], "x");
    const Tensor *r = optional(a[4], "residual"), *out = optional(a[5], "out"), *like = optional(a[6], "like");
    flce_dropout_params_t p;
    std::memset(&p, 0, sizeof(p));
    p.dtype = float_type(x, "x");
    const Rows rows = rows_of(x, "x");
    p.M = rows.rows;
    p.H = rows.cols;
    p.ld_x = rows.ld;
    p.dropout = number(a[1], "p");
    const int64_t* seed = read_seed(a[2], a[3], p.dropout, x, &p.seed, &p.offset);
    const c10::cuda::CUDAGuard guard(x.device());
    const Tensor& typed = out ? *out : r ? *r : like ? *like : x;
    p.out_dtype = float_type(typed, "the output");
    if (p.out_dtype != p.dtype && p.out_dtype != FLCE_DTYPE_FP32 && p.dtype != FLCE_DTYPE_FP32)
      refuse(PyExc_TypeError, "flce: %s must be of x's type, or one of them fp32", "the output");
    if (r) {
      if (r->scalar_type() != typed.scalar_type())
        refuse(PyExc_TypeError, "flce: %s must be of the output's type", "residual");
      p.ld_res = pitch_like(*r, x, "residual");
    }
    if (out) {
      p.ld_y = pitch_like(*out, x, "out");
      apart(*out, &x, true, "out");
      apart(*out, r, true, "out");
    }
    const Tensor y = out ? *out : at::empty(x.sizes(), x.options().dtype(typed.scalar_type()));
    done(flce_dropout(&p, data(x), data(r), seed, data(y), stream_of(x)), "flce_dropout");
    if (out) written(*out);
    return wrap(y);
  });
}

// A sampling setting: a number, or a tensor with a value for each row.
template <class T>
const T* setting(PyObject* o, at::ScalarType type, const Tensor& z, const char* name, double* value) {
  if (THPVariable_Check(o)) {
    const Tensor& t = THPVariable_Unpack(o);
    flat(t, type, {z.size(0)}, z, name);
    return t.data_ptr<T>();
  }
  *value = number(o, name);
  return nullptr;
}

// sample(logits, u, temperature, top_k, top_p, min_p, out) -> tokens
PyObject* sample(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&] {
    const Tensor &z = tensor(a[0], "logits"), &u = tensor(a[1], "u");
    const Tensor* out = optional(a[6], "out");
    flce_sample_params_t p;
    std::memset(&p, 0, sizeof(p));
    p.dtype = float_type(z, "logits");
    if (z.dim() != 2) refuse(PyExc_ValueError, "flce: %s must be two-dimensional", "logits");
    const Rows rows = rows_of(z, "logits");
    p.B = rows.rows;
    p.V = rows.cols;
    p.ld = rows.ld;
    flat(u, at::kFloat, {p.B}, z, "u");
    double temperature = 0.0, top_k = 0.0, top_p = 1.0, min_p = 0.0;
    const float* temperatures = setting<float>(a[2], at::kFloat, z, "temperature", &temperature);
    const int32_t* top_ks = setting<int32_t>(a[3], at::kInt, z, "top_k", &top_k);
    const float* top_ps = setting<float>(a[4], at::kFloat, z, "top_p", &top_p);
    const float* min_ps = setting<float>(a[5], at::kFloat, z, "min_p", &min_p);
    p.temperature = static_cast<float>(temperature);
    if (top_k != std::floor(top_k)) refuse(PyExc_ValueError, "flce: %s must be a whole number", "top_k");
    p.top_k = top_k < 0.0 ? -1 : top_k > 2147483647.0 ? 2147483647 : static_cast<int32_t>(top_k);
    p.top_p = static_cast<float>(top_p);
    p.min_p = static_cast<float>(min_p);
    const c10::cuda::CUDAGuard guard(z.device());
    if (out) {
      flat(*out, at::kLong, {p.B}, z, "out");
      apart_from(*out, {&z, &u}, "out");
      for (PyObject* o : {a[2], a[3], a[4], a[5]})
        if (THPVariable_Check(o)) apart(*out, &THPVariable_Unpack(o), false, "out");
    }
    const Tensor tokens = out ? *out : at::empty({p.B}, z.options().dtype(at::kLong));
    done(flce_sample(&p, data(z), static_cast<const float*>(data(u)), temperatures, top_ks, top_ps, min_ps,
                     static_cast<int64_t*>(data(tokens)), stream_of(z)),
         "flce_sample");
    if (out) written(*out);
    return wrap(tokens);
  });
}

// bind(FlceError, error_word): what the calls take from the package.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 2, [&]() -> PyObject* {
    Py_INCREF(a[0]);
    Py_INCREF(a[1]);
    g_error_class = a[0];
    g_error_word = a[1];
    Py_RETURN_NONE;
  });
}

#define FLCE_METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {FLCE_METHOD(linear_forward), FLCE_METHOD(linear_backward),
                          FLCE_METHOD(gated_forward),  FLCE_METHOD(gated_backward),
                          FLCE_METHOD(clip_grads),     FLCE_METHOD(bind),
                          FLCE_METHOD(rms_norm_forward), FLCE_METHOD(rms_norm_quantized),
                          FLCE_METHOD(rms_norm_backward), FLCE_METHOD(dropout),
                          FLCE_METHOD(sample),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_flce_torch", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__flce_torch() { return PyModule_Create(&kModule); }
