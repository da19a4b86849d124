// Python calls of the layer operators, from torch tensors to the C ABI.
//
// A call of a few microseconds on the GPU should not wait for the interpreter: these
// functions check the tensors, allocate outputs and scratch through torch's
// allocator and call the library on the tensors' device and its current CUDA stream.
// block.py documents them and handles calls that name a stream.
#include <Python.h>

#include <algorithm>
#include <array>
#include <cstdint>
#include <cstring>
#include <exception>
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
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_flce_torch", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__flce_torch() { return PyModule_Create(&kModule); }
