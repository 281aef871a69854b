// Argument marshalling of the layer operators and of the many-tensor AdamW step: torch
// tensors to the C ABI's views.
//
// These calls are made per layer and, decoding, per token, so the look at each
// tensor and the allocation of results happen here rather than in Python (a
// one-token linear call: 9 us of host time by ctypes). Nothing is computed:
// every function checks what the C ABI cannot see (devices, ranks, strides, the
// lengths of vectors), calls one entry point of libmao.so and returns its results.
// The Python functions around these resolve names and defaults and pass the
// stream; workspaces and the error class are theirs too (set by init).
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/GradMode.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <exception>
#include <memory>
#include <vector>

#include "../../include/mao.h"

namespace {

PyObject* g_workspace = nullptr;  // (bytes, device index, stream) -> uint8 tensor
PyObject* g_check = nullptr;      // (status, name): raises
PyObject* g_q8 = nullptr;         // the checkpoint class
PyObject *g_codes = nullptr, *g_scales = nullptr;  // its attribute names

// An exception is set on the Python side.
struct Raised {};

[[noreturn]] void fail(PyObject* type, const char* text) {
  PyErr_SetString(type, text);
  throw Raised{};
}

const at::Tensor& tensor(PyObject* o) {
  if (!THPVariable_Check(o)) fail(PyExc_TypeError, "expected a tensor");
  return THPVariable_Unpack(o);
}

void on_device(const at::Tensor& t, int64_t dev) {
  if (!t.is_cuda()) fail(PyExc_ValueError, "tensors must be on the GPU");
  if (t.get_device() != dev) fail(PyExc_ValueError, "tensors on different devices");
}

// The calls have their own backward calls and record no graph: a tensor whose gradient
// autograd is to find would lose it without a word.
void no_graph(const at::Tensor& t) {
  if (t.requires_grad() && c10::GradMode::is_enabled())
    fail(PyExc_RuntimeError,
         "the layer operators record no autograd graph, and a tensor requires a gradient: call "
         "them under torch.no_grad(), with their own backward calls, or detach the tensor");
}

int32_t dtype_code(const at::Tensor& t) {
  if (t.scalar_type() == at::kFloat) return MAO_F32;
  if (t.scalar_type() == at::kBFloat16) return MAO_BF16;
  fail(PyExc_TypeError, "unsupported dtype: float32 or bfloat16 is needed");
}

mao_mat view(const at::Tensor& t, int64_t dev) {
  if (t.dim() != 2 || (t.stride(1) != 1 && t.size(1) != 1))
    fail(PyExc_ValueError, "expected a 2-D row-major tensor (unit column stride)");
  on_device(t, dev);
  no_graph(t);
  const int64_t rows = t.size(0), cols = t.size(1);
  // the row stride of a single row means nothing
  return mao_mat{t.data_ptr(), rows, cols, rows == 1 ? (cols + 7) & ~int64_t(7) : t.stride(0),
                 dtype_code(t)};
}

// A checkpoint's two tensors are attributes that a program may have set itself: all that
// the class checks as it is made is checked here again.
mao_q8 checkpoint(const at::Tensor& codes, const at::Tensor& scales, int64_t dev) {
  if (codes.scalar_type() != at::kChar && codes.scalar_type() != at::kFloat8_e4m3fn)
    fail(PyExc_TypeError, "a checkpoint's codes must be int8 or float8_e4m3fn");
  if (scales.scalar_type() != at::kByte)
    fail(PyExc_TypeError, "a checkpoint's scales must be uint8");
  if (codes.dim() != 2 || scales.dim() != 2 || (codes.stride(1) != 1 && codes.size(1) != 1) ||
      (scales.stride(1) != 1 && scales.size(1) != 1))
    fail(PyExc_ValueError, "a checkpoint's codes and scales must be 2-D and row-major");
  if (scales.size(0) != codes.size(0) || scales.size(1) < (codes.size(1) + 31) / 32)
    fail(PyExc_ValueError, "a checkpoint's scales need one byte per row and 32 columns");
  on_device(codes, dev);
  on_device(scales, dev);
  return mao_q8{codes.data_ptr(), (uint8_t*)scales.data_ptr(), codes.size(0), codes.size(1),
                codes.stride(0), scales.stride(0),
                codes.scalar_type() == at::kChar ? MAO_Q8_INT8 : MAO_Q8_E4M3};
}

// A tensor, a checkpoint or None.
struct Kept {
  mao_mat m;
  mao_q8 q;
  const mao_mat* mat = nullptr;
  const mao_q8* q8 = nullptr;
  int64_t cols = 0;
  Kept(PyObject* o, int64_t dev) {
    if (o == Py_None) return;
    if (THPVariable_Check(o)) {
      m = view(THPVariable_Unpack(o), dev);
      mat = &m;
      cols = m.cols;
      return;
    }
    if (PyObject_IsInstance(o, g_q8) != 1) fail(PyExc_TypeError, "expected a tensor or a Q8");
    PyObject* c = PyObject_GetAttr(o, g_codes);
    PyObject* s = PyObject_GetAttr(o, g_scales);
    const bool ok = c && s && THPVariable_Check(c) && THPVariable_Check(s);
    if (ok) {
      // o keeps both alive
      const at::Tensor &tc = THPVariable_Unpack(c), &ts = THPVariable_Unpack(s);
      Py_DECREF(c);
      Py_DECREF(s);
      q = checkpoint(tc, ts, dev);
      q8 = &q;
      cols = q.cols;
      return;
    }
    Py_XDECREF(c);
    Py_XDECREF(s);
    PyErr_Clear();
    fail(PyExc_TypeError, "codes and scales must be tensors");
  }
};

// An optional matrix.
struct Opt {
  mao_mat m;
  const mao_mat* p = nullptr;
  Opt(PyObject* o, int64_t dev) {
    if (o == Py_None) return;
    m = view(tensor(o), dev);
    p = &m;
  }
};

// An optional contiguous vector of n values.
struct Vec {
  void* p = nullptr;
  int32_t dtype = MAO_F32;
  Vec(PyObject* o, int64_t n, int64_t dev, const char* name, bool floats) {
    if (o == Py_None) return;
    const at::Tensor& t = tensor(o);
    if (t.dim() != 1 || t.size(0) != n || !t.is_contiguous()) {
      PyErr_Format(PyExc_ValueError, "%s must be a contiguous vector of %lld values", name,
                   (long long)n);
      throw Raised{};
    }
    on_device(t, dev);
    no_graph(t);
    dtype = dtype_code(t);
    if (floats && dtype != MAO_F32) {
      PyErr_Format(PyExc_TypeError, "%s must be float32", name);
      throw Raised{};
    }
    p = t.data_ptr();
  }
};

// A result that was passed in, or a new one whose rows meet the layout rule.
at::Tensor result(PyObject* o, int64_t rows, int64_t cols, at::ScalarType type,
                  const at::Tensor& like) {
  if (o != Py_None) return tensor(o);
  const int64_t ld = (cols + 7) & ~int64_t(7);
  at::Tensor t = at::empty({rows, ld}, like.options().dtype(type));
  return ld == cols ? t : t.narrow(1, 0, cols);
}

PyObject* wrap(const at::Tensor& t, PyObject* given) {
  if (given != Py_None) {
    Py_INCREF(given);
    return given;
  }
  return THPVariable_Wrap(t);
}

// A vector gradient: passed in, new (None) or not wanted (False).
struct VecResult {
  PyObject* given;
  at::Tensor t;
  float* p = nullptr;
  VecResult(PyObject* o, int64_t n, int64_t dev, const char* name, const at::Tensor& like)
      : given(o) {
    if (o == Py_False) return;
    if (o == Py_None)
      t = at::empty({n}, like.options().dtype(at::kFloat));
    else
      t = (Vec(o, n, dev, name, true), tensor(o));
    p = (float*)t.data_ptr();
  }
  PyObject* object() const { return given == Py_False ? Py_NewRef(Py_None) : wrap(t, given); }
};

struct Workspace {
  PyObject* keep = nullptr;
  void* p = nullptr;
  size_t bytes = 0;
  Workspace(size_t need, int64_t dev, int64_t stream) {
    if (need == 0) return;
    keep = PyObject_CallFunction(g_workspace, "nLL", (Py_ssize_t)need, (long long)dev,
                                 (long long)stream);
    if (!keep) throw Raised{};
    const at::Tensor& t = THPVariable_Unpack(keep);
    p = t.data_ptr();
    bytes = (size_t)t.numel();
  }
  ~Workspace() { Py_XDECREF(keep); }
  Workspace(const Workspace&) = delete;
};

void check(mao_status s, const char* name) {
  if (s == MAO_OK) return;
  PyObject* r = PyObject_CallFunction(g_check, "is", (int)s, name);
  if (r) {  // did not raise
    Py_DECREF(r);
    PyErr_SetString(PyExc_RuntimeError, name);
  }
  throw Raised{};
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}

at::ScalarType type_of(int64_t code) { return code == MAO_BF16 ? at::kBFloat16 : at::kFloat; }

template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return nullptr;
  }
  try {
    return f();
  } catch (const Raised&) {
  } catch (...) {  // torch's own, out of memory among them, as torch raises them
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 3, [&]() -> PyObject* {
    g_workspace = Py_NewRef(a[0]);
    g_check = Py_NewRef(a[1]);
    g_q8 = Py_NewRef(a[2]);
    g_codes = PyUnicode_InternFromString("codes");
    g_scales = PyUnicode_InternFromString("scales");
    Py_RETURN_NONE;
  });
}

// (X, format, codes, scales, device, stream) -> (codes, scales); new ones where None
PyObject* q8_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject* {
    const int64_t dev = integer(a[4]);
    const at::Tensor& X = tensor(a[0]);
    const mao_mat x = view(X, dev);
    const int64_t blocks = (x.cols + 31) / 32;
    at::Tensor codes, scales;
    if (a[2] != Py_None) {
      codes = tensor(a[2]);
      scales = tensor(a[3]);
    } else {
      codes = at::empty({x.rows, blocks * 32},
                        X.options().dtype(integer(a[1]) == MAO_Q8_INT8 ? at::kChar
                                                                       : at::kFloat8_e4m3fn))
                  .narrow(1, 0, x.cols);
      scales = at::empty({x.rows, blocks}, X.options().dtype(at::kByte));
    }
    const mao_q8 q = checkpoint(codes, scales, dev);
    check(mao_q8_quantize(x, &q, (void*)integer(a[5])), "mao_q8_quantize");
    return Py_BuildValue("NN", wrap(codes, a[2]), wrap(scales, a[2] == Py_None ? Py_None : a[3]));
  });
}

// (Q8, act, result type, out, device, stream) -> tensor
PyObject* q8_dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject* {
    const int64_t dev = integer(a[4]);
    const Kept k(a[0], dev);
    if (!k.q8) fail(PyExc_TypeError, "expected a Q8");
    PyObject* c = PyObject_GetAttr(a[0], g_codes);
    if (!c) throw Raised{};
    const at::Tensor like = THPVariable_Unpack(c);
    Py_DECREF(c);
    const at::Tensor out = result(a[3], k.q8->rows, k.q8->cols, type_of(integer(a[2])), like);
    check(mao_q8_dequantize(k.q8, (int32_t)integer(a[1]), view(out, dev), (void*)integer(a[5])),
          "mao_q8_dequantize");
    return wrap(out, a[3]);
  });
}

// (X, gamma, beta, eps, out, stats, device, stream) -> (Y, mean, rstd)
PyObject* layer_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    const int64_t dev = integer(a[6]);
    const at::Tensor& X = tensor(a[0]);
    const mao_mat x = view(X, dev);
    const Vec g(a[1], x.cols, dev, "gamma", false), b(a[2], x.cols, dev, "beta", false);
    if (g.p && b.p && g.dtype != b.dtype) fail(PyExc_TypeError, "gamma and beta must share a dtype");
    const double eps = PyFloat_AsDouble(a[3]);
    if (eps == -1.0 && PyErr_Occurred()) throw Raised{};
    const at::Tensor out = result(a[4], x.rows, x.cols, X.scalar_type(), X);
    at::Tensor mean, rstd;
    const bool stats = a[5] == Py_True;
    if (stats) {
      mean = at::empty({x.rows}, X.options().dtype(at::kFloat));
      rstd = at::empty({x.rows}, X.options().dtype(at::kFloat));
    }
    check(mao_layer_norm(x, g.p, b.p, g.p ? g.dtype : b.dtype, (float)eps, view(out, dev),
                         stats ? (float*)mean.data_ptr() : nullptr,
                         stats ? (float*)rstd.data_ptr() : nullptr, (void*)integer(a[7])),
          "mao_layer_norm");
    return Py_BuildValue("NNN", wrap(out, a[4]), stats ? THPVariable_Wrap(mean) : Py_NewRef(Py_None),
                         stats ? THPVariable_Wrap(rstd) : Py_NewRef(Py_None));
  });
}

// (dY, X, gamma, mean, rstd, add, out, dgamma, dbeta, device, stream)
// -> (dX, dgamma, dbeta); dgamma or dbeta False: not computed, None
PyObject* layer_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    const int64_t dev = integer(a[9]), stream = integer(a[10]);
    const at::Tensor& DY = tensor(a[0]);
    const mao_mat dy = view(DY, dev);
    const Kept x(a[1], dev);
    const Vec g(a[2], dy.cols, dev, "gamma", false);
    const Vec mean(a[3], dy.rows, dev, "mean", true), rstd(a[4], dy.rows, dev, "rstd", true);
    if (!mean.p || !rstd.p) fail(PyExc_ValueError, "mean and rstd of the forward pass are needed");
    const Opt add(a[5], dev);
    const VecResult dgamma(a[7], dy.cols, dev, "dgamma", DY), dbeta(a[8], dy.cols, dev, "dbeta", DY);
    const at::Tensor out = result(a[6], dy.rows, dy.cols, DY.scalar_type(), DY);
    const Workspace ws(dgamma.p || dbeta.p
                           ? mao_layer_norm_backward_workspace_size(dy.rows, dy.cols)
                           : 0,
                       dev, stream);
    check(mao_layer_norm_backward(dy, x.mat, x.q8, g.p, g.dtype, (const float*)mean.p,
                                  (const float*)rstd.p, add.p, view(out, dev),
                                  dgamma.p, dbeta.p, ws.p, ws.bytes, (void*)stream),
          "mao_layer_norm_backward");
    return Py_BuildValue("NNN", wrap(out, a[6]), dgamma.object(), dbeta.object());
  });
}

// (X, W, bias, act, residual, out, preact, device, stream) -> Y
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const int64_t dev = integer(a[7]), stream = integer(a[8]);
    const at::Tensor& X = tensor(a[0]);
    const mao_mat x = view(X, dev), w = view(tensor(a[1]), dev);
    const Vec b(a[2], w.rows, dev, "bias", false);
    const Opt res(a[4], dev), z(a[6], dev);
    const at::Tensor out = result(a[5], x.rows, w.rows, X.scalar_type(), X);
    const Workspace ws(mao_linear_workspace_size(x.rows, x.cols, w.rows, x.dtype), dev, stream);
    check(mao_linear(x, w, b.p, b.dtype, (int32_t)integer(a[3]), res.p, view(out, dev), z.p, ws.p,
                     ws.bytes, (void*)stream),
          "mao_linear");
    return wrap(out, a[5]);
  });
}

// (dY, W, act, preact, add, out, device, stream) -> dX
PyObject* linear_backward_input(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    const int64_t dev = integer(a[6]), stream = integer(a[7]);
    const at::Tensor& DY = tensor(a[0]);
    const mao_mat dy = view(DY, dev), w = view(tensor(a[1]), dev);
    const Kept z(a[3], dev);
    const Opt add(a[4], dev);
    const at::Tensor out = result(a[5], dy.rows, w.cols, DY.scalar_type(), DY);
    const Workspace ws(mao_linear_backward_input_workspace_size(dy.rows, w.cols, w.rows, dy.dtype),
                       dev, stream);
    check(mao_linear_backward_input(dy, w, (int32_t)integer(a[2]), z.mat, z.q8, add.p,
                                    view(out, dev), ws.p, ws.bytes, (void*)stream),
          "mao_linear_backward_input");
    return wrap(out, a[5]);
  });
}

// (dY, X, x_act, result type, out, dbias, accumulate, device, stream) -> (dW, dbias); dbias
// False: not computed, None
PyObject* linear_backward_weight(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const int64_t dev = integer(a[7]), stream = integer(a[8]), act = integer(a[2]);
    const at::Tensor& DY = tensor(a[0]);
    const mao_mat dy = view(DY, dev);
    const Kept x(a[1], dev);
    const VecResult dbias(a[5], dy.cols, dev, "dbias", DY);
    const at::Tensor out = result(a[4], dy.cols, x.cols, type_of(integer(a[3])), DY);
    const Workspace ws(mao_linear_backward_weight_workspace_size(
                           dy.rows, x.cols, dy.cols, dy.dtype, x.q8 != nullptr || act != 0),
                       dev, stream);
    check(mao_linear_backward_weight(dy, x.mat, x.q8, (int32_t)act, view(out, dev), dbias.p,
                                     a[6] == Py_True, ws.p, ws.bytes, (void*)stream),
          "mao_linear_backward_weight");
    return Py_BuildValue("NN", wrap(out, a[4]), dbias.object());
  });
}

// A norm's kind and parameters.
struct RowNorm {
  mao_row_norm n;
  RowNorm(PyObject* kind, PyObject* gamma, PyObject* beta, double eps, int64_t cols, int64_t dev,
          const char* name) {
    const Vec g(gamma, cols, dev, name, false), b(beta, cols, dev, name, false);
    if (g.p && b.p && g.dtype != b.dtype) fail(PyExc_TypeError, "gamma and beta must share a dtype");
    n = mao_row_norm{(int32_t)integer(kind), g.p, b.p, g.p ? g.dtype : b.dtype, (float)eps};
  }
};

// The gate: a vector, a matrix or None.
struct Gate {
  void* vec = nullptr;
  int32_t dtype = MAO_F32;
  mao_mat m;
  const mao_mat* mat = nullptr;
  Gate(PyObject* o, int64_t cols, int64_t dev) {
    if (o == Py_None) return;
    if (tensor(o).dim() == 1) {
      const Vec v(o, cols, dev, "gate", false);
      vec = v.p;
      dtype = v.dtype;
    } else {
      m = view(tensor(o), dev);
      mat = &m;
    }
  }
};

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}

// (X, B, gate, x_scale, b_scale, post, post_gamma, post_beta, pre, pre_gamma, pre_beta, eps, out,
// h, stats, device, stream) -> (R, H, stats)
PyObject* residual_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 17, [&]() -> PyObject* {
    const int64_t dev = integer(a[15]);
    const at::Tensor &X = tensor(a[0]), &B = tensor(a[1]);
    const mao_mat x = view(X, dev), b = view(B, dev);
    const Gate gate(a[2], b.cols, dev);
    const double eps = number(a[11]);
    const RowNorm post(a[5], a[6], a[7], eps, b.cols, dev, "post_gamma or post_beta"),
        pre(a[8], a[9], a[10], eps, b.cols, dev, "pre_gamma or pre_beta");
    const at::Tensor r = result(a[12], x.rows, x.cols, X.scalar_type(), X);
    at::Tensor h, stats;
    mao_mat hv;
    const bool normed = pre.n.kind != MAO_ROW_NORM_NONE || a[13] != Py_None;
    if (normed) {
      h = result(a[13], b.rows, b.cols, B.scalar_type(), B);
      hv = view(h, dev);
    }
    if (a[14] == Py_True) stats = at::empty({b.rows, 4}, B.options().dtype(at::kFloat));
    check(mao_residual_norm(x, b, &post.n, gate.vec, gate.dtype, gate.mat, (float)number(a[3]),
                            (float)number(a[4]), &pre.n, view(r, dev), normed ? &hv : nullptr,
                            stats.defined() ? (float*)stats.data_ptr() : nullptr,
                            (void*)integer(a[16])),
          "mao_residual_norm");
    return Py_BuildValue("NNN", wrap(r, a[12]), normed ? wrap(h, a[13]) : Py_NewRef(Py_None),
                         stats.defined() ? THPVariable_Wrap(stats) : Py_NewRef(Py_None));
  });
}

// (B, dH, dR, R, stats, gate, x_scale, b_scale, post, post_gamma, post_beta, pre, pre_gamma, out,
// sums, device, stream) -> (dX, dB, dgate, dpost_gamma, dpost_beta, dpre_gamma, dpre_beta)
PyObject* residual_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 17, [&]() -> PyObject* {
    const int64_t dev = integer(a[15]), stream = integer(a[16]);
    const at::Tensor& B = tensor(a[0]);
    const mao_mat b = view(B, dev);
    const Opt dh(a[1], dev), dr(a[2], dev), r(a[3], dev);
    const at::Tensor& st = tensor(a[4]);
    if (st.scalar_type() != at::kFloat) fail(PyExc_TypeError, "stats must be float32");
    if (st.dim() != 2 || st.size(0) != b.rows || st.size(1) != 4 || !st.is_contiguous())
      fail(PyExc_ValueError, "stats must be the forward pass's (rows x 4)");
    on_device(st, dev);
    const Gate gate(a[5], b.cols, dev);
    // eps has gone into the statistics
    const RowNorm post(a[8], a[9], a[10], 1.0, b.cols, dev, "post_gamma or post_beta"),
        pre(a[11], a[12], Py_None, 1.0, b.cols, dev, "pre_gamma");
    if (!dr.p && !r.p) fail(PyExc_ValueError, "dH (with R) or dR is needed");
    const at::Tensor& stream_like = tensor(r.p ? a[3] : a[2]);
    const at::Tensor dx = result(a[13], b.rows, b.cols, stream_like.scalar_type(), B);
    const at::Tensor db = result(Py_None, b.rows, b.cols, B.scalar_type(), B);
    at::Tensor dgates, vecs[5];
    mao_mat dgv;
    if (gate.mat) {
      dgates = result(Py_None, b.rows, b.cols, B.scalar_type(), B);
      dgv = view(dgates, dev);
    }
    float* p[5] = {};
    if (a[14] == Py_True) {
      const bool want[5] = {post.n.kind != MAO_ROW_NORM_NONE, post.n.kind == MAO_ROW_NORM_LAYER,
                            pre.n.kind != MAO_ROW_NORM_NONE, pre.n.kind == MAO_ROW_NORM_LAYER,
                            gate.vec != nullptr};
      for (int k = 0; k < 5; ++k)
        if (want[k]) {
          vecs[k] = at::empty({b.cols}, B.options().dtype(at::kFloat));
          p[k] = (float*)vecs[k].data_ptr();
        }
    }
    const mao_residual_norm_sums sums{p[0], p[1], p[2], p[3], p[4]};
    const bool any = p[0] || p[1] || p[2] || p[3] || p[4];
    const Workspace ws(any ? mao_residual_norm_backward_workspace_size(b.rows, b.cols) : 0, dev,
                       stream);
    check(mao_residual_norm_backward(dh.p, dr.p, b, r.p, (const float*)st.data_ptr(), &post.n,
                                     gate.vec, gate.dtype, gate.mat, (float)number(a[6]),
                                     (float)number(a[7]), &pre.n, view(dx, dev), view(db, dev),
                                     gate.mat ? &dgv : nullptr, &sums, ws.p, ws.bytes,
                                     (void*)stream),
          "mao_residual_norm_backward");
    const auto out = [](const at::Tensor& t) {
      return t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None);
    };
    return Py_BuildValue("NNNNNNN", wrap(dx, a[13]), THPVariable_Wrap(db),
                         gate.mat ? THPVariable_Wrap(dgates) : out(vecs[4]), out(vecs[0]),
                         out(vecs[1]), out(vecs[2]), out(vecs[3]));
  });
}

// One token per row.
const int64_t* tokens_of(PyObject* o, int64_t rows, int64_t dev) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o);
  if (t.scalar_type() != at::kLong) fail(PyExc_TypeError, "targets must be int64");
  if (t.dim() != 1 || t.size(0) != rows || !t.is_contiguous())
    fail(PyExc_ValueError, "targets must be a contiguous vector with one token per row");
  on_device(t, dev);
  return (const int64_t*)t.data_ptr();
}

// (X, targets, entropy, top, device, stream)
// -> (logprob, entropy, stats, top_logprobs, top_ids), None for what is not asked for
PyObject* token_logprobs(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject* {
    const int64_t dev = integer(a[4]), stream = integer(a[5]), top = integer(a[3]);
    const at::Tensor& X = tensor(a[0]);
    const mao_mat x = view(X, dev);
    const int64_t* targets = tokens_of(a[1], x.rows, dev);
    if (top < 0 || top > INT32_MAX) fail(PyExc_ValueError, "top must not be negative");
    const auto f = X.options().dtype(at::kFloat);
    at::Tensor lp, ent, top_lp, ids;
    if (targets) lp = at::empty({x.rows}, f);
    if (a[2] == Py_True) ent = at::empty({x.rows}, f);
    const at::Tensor stats = at::empty({x.rows, 2}, f);
    // a top that the call refuses allocates nothing
    const int64_t k = top <= x.cols && top <= 32 ? top : 0;
    if (k) {
      top_lp = at::empty({x.rows, k}, f);
      ids = at::empty({x.rows, k}, X.options().dtype(at::kLong));
    }
    check(mao_token_logprobs(x, targets, targets ? (float*)lp.data_ptr() : nullptr,
                             ent.defined() ? (float*)ent.data_ptr() : nullptr,
                             (float*)stats.data_ptr(), (int32_t)top,
                             k ? (float*)top_lp.data_ptr() : nullptr,
                             k ? (int64_t*)ids.data_ptr() : nullptr, (void*)stream),
          "mao_token_logprobs");
    const auto out = [](const at::Tensor& t) {
      return t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None);
    };
    return Py_BuildValue("NNNNN", out(lp), out(ent), out(stats), out(top_lp), out(ids));
  });
}

// (X, targets, stats, entropy, dlogprob, dentropy, dlse, out, device, stream) -> dX
PyObject* token_logprobs_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const int64_t dev = integer(a[8]), stream = integer(a[9]);
    const at::Tensor& X = tensor(a[0]);
    const mao_mat x = view(X, dev);
    const int64_t* targets = tokens_of(a[1], x.rows, dev);
    const at::Tensor& st = tensor(a[2]);
    if (st.scalar_type() != at::kFloat) fail(PyExc_TypeError, "stats must be float32");
    if (st.dim() != 2 || st.size(0) != x.rows || st.size(1) != 2 || !st.is_contiguous())
      fail(PyExc_ValueError, "stats must be the forward pass's (rows x 2)");
    on_device(st, dev);
    const Vec ent(a[3], x.rows, dev, "entropy", true), dlp(a[4], x.rows, dev, "dlogprob", true),
        de(a[5], x.rows, dev, "dentropy", true), dl(a[6], x.rows, dev, "dlse", true);
    const at::Tensor out = result(a[7], x.rows, x.cols, X.scalar_type(), X);
    check(mao_token_logprobs_backward(x, targets, (const float*)st.data_ptr(), (const float*)ent.p,
                                      (const float*)dlp.p, (const float*)de.p, (const float*)dl.p,
                                      view(out, dev), (void*)stream),
          "mao_token_logprobs_backward");
    return wrap(out, a[7]);
  });
}

// (X, targets, weight, out, device, stream) -> (logprob, dX)
PyObject* token_loss(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject* {
    const int64_t dev = integer(a[4]), stream = integer(a[5]);
    const at::Tensor& X = tensor(a[0]);
    const mao_mat x = view(X, dev);
    const int64_t* targets = tokens_of(a[1], x.rows, dev);
    const Vec w(a[2], x.rows, dev, "weight", true);
    const at::Tensor lp = at::empty({x.rows}, X.options().dtype(at::kFloat));
    const at::Tensor out = result(a[3], x.rows, x.cols, X.scalar_type(), X);
    check(mao_token_loss(x, targets, (const float*)w.p, (float*)lp.data_ptr(), view(out, dev),
                         (void*)stream),
          "mao_token_loss");
    return Py_BuildValue("NN", THPVariable_Wrap(lp), wrap(out, a[3]));
  });
}

// The elements of a tensor that an optimizer step reads or writes in place (autograd looks on
// at none of it, as with the other steps).
struct Flat {
  void* p = nullptr;
  int64_t n = 0;
  at::ScalarType type;
  Flat(PyObject* o, int64_t dev) {
    const at::Tensor& t = tensor(o);
    if (!t.is_contiguous()) fail(PyExc_ValueError, "adamw_step_many needs contiguous tensors");
    on_device(t, dev);
    p = t.data_ptr();
    n = t.numel();
    type = t.scalar_type();
  }
  void want(at::ScalarType ty, int64_t size, const char* name) const {
    if (type != ty) {
      PyErr_Format(PyExc_TypeError, "%s must be %s", name,
                   ty == at::kFloat ? "float32" : ty == at::kByte ? "uint8" : "bfloat16");
      throw Raised{};
    }
    if (n != size) {
      PyErr_Format(PyExc_ValueError, "%s needs %lld elements, not %lld", name, (long long)size,
                   (long long)n);
      throw Raised{};
    }
  }
  int32_t code() const {
    if (type == at::kFloat) return MAO_F32;
    if (type == at::kBFloat16) return MAO_BF16;
    fail(PyExc_TypeError, "unsupported dtype: float32 or bfloat16 is needed");
  }
};

// A list or tuple, held for the call.
struct Sequence {
  PyObject* s;
  explicit Sequence(PyObject* o, const char* what) : s(PySequence_Fast(o, what)) {
    if (!s) throw Raised{};
  }
  ~Sequence() { Py_DECREF(s); }
  Sequence(const Sequence&) = delete;
  int64_t size() const { return PySequence_Fast_GET_SIZE(s); }
  PyObject* operator[](int64_t i) const { return PySequence_Fast_GET_ITEM(s, i); }
};

// A number for all tensors, or one for each.
struct Numbers {
  float one = 0.f;
  std::vector<float> each;
  Numbers(PyObject* o, int64_t n, const char* name) {
    if (PyList_Check(o) || PyTuple_Check(o)) {
      const Sequence q(o, name);
      if (q.size() != n) {
        PyErr_Format(PyExc_ValueError, "%s: %lld values for %lld tensors", name,
                     (long long)q.size(), (long long)n);
        throw Raised{};
      }
      for (int64_t i = 0; i < n; ++i) each.push_back((float)number(q[i]));
    } else {
      one = (float)number(o);
    }
  }
  float operator[](int64_t i) const { return each.empty() ? one : each[(size_t)i]; }
};

constexpr int64_t kSpan = 256;  // elements per scale of an 8-bit state

// (first weight, items, t, lr, beta1, beta2, eps, weight_decay, grad_scale, device, stream):
// items of (w, g, m, v) or (w, g, m, m_scale, v, v_scale)
PyObject* adamw_step_many(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    const int64_t dev = integer(a[9]);
    const Sequence items(a[1], "expected a list of tensors' tuples");
    const int64_t count = items.size();
    const Numbers lr(a[3], count, "lr"), wd(a[7], count, "weight_decay");
    std::vector<mao_adamw_tensor> t((size_t)count);
    for (int64_t i = 0; i < count; ++i) {
      const Sequence q(items[i], "expected a tuple of tensors");
      if (q.size() != 4 && q.size() != 6)
        fail(PyExc_ValueError, "expected (w, g, m, v) or (w, g, m, m_scale, v, v_scale)");
      const bool q8 = q.size() == 6;
      const Flat w(q[0], dev), g(q[1], dev), m(q[2], dev), v(q[q8 ? 4 : 3], dev);
      if (g.n != w.n) fail(PyExc_ValueError, "w and g of different sizes");
      m.want(q8 ? at::kByte : at::kFloat, w.n, "m");
      v.want(q8 ? at::kByte : at::kFloat, w.n, "v");
      mao_adamw_tensor& x = t[(size_t)i];
      x = mao_adamw_tensor{w.p, g.p, m.p, v.p, nullptr, nullptr, w.n, w.code(), g.code(),
                           q8 ? MAO_ADAM_8BIT : MAO_ADAM_F32, lr[i], wd[i]};
      if (q8) {
        const Flat ms(q[3], dev), vs(q[5], dev);
        ms.want(at::kFloat, (w.n + kSpan - 1) / kSpan, "m_scale");
        vs.want(at::kFloat, (w.n + kSpan - 1) / kSpan, "v_scale");
        x.m_scale = (float*)ms.p;
        x.v_scale = (float*)vs.p;
      }
    }
    const float* gs = nullptr;
    if (a[8] != Py_None) {
      const Flat f(a[8], dev);
      f.want(at::kFloat, 1, "grad_scale");
      gs = (const float*)f.p;
    }
    check(adamw_step_many((int32_t)std::min<int64_t>(count, INT32_MAX), t.data(), integer(a[2]),
                          (float)number(a[4]), (float)number(a[5]), (float)number(a[6]), gs,
                          (void*)integer(a[10])),
          "adamw_step_many");
    Py_RETURN_NONE;
  });
}

// (first code tensor, states, type, out, device, stream): states of (m, m_scale, v, v_scale),
// out a list of (m, v) -> None, or None -> a list of (m, v)
PyObject* adamw8_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject* {
    const int64_t dev = integer(a[4]);
    const Sequence states(a[1], "expected a list of states");
    const int64_t count = states.size();
    std::vector<mao_adamw8_state> t((size_t)count);
    std::vector<at::Tensor> made;
    at::ScalarType type = type_of(integer(a[2]));
    const bool given = a[3] != Py_None;
    std::vector<std::unique_ptr<Sequence>> outs;
    if (given) {
      const Sequence o(a[3], "out must be a list of (m, v)");
      if (o.size() != count) fail(PyExc_ValueError, "out must hold one (m, v) for each state");
      for (int64_t i = 0; i < count; ++i) {
        outs.emplace_back(new Sequence(o[i], "out must be a list of (m, v)"));
        if (outs.back()->size() != 2) fail(PyExc_ValueError, "out must be a list of (m, v)");
      }
      if (count > 0) type = tensor((*outs[0])[0]).scalar_type();
    }
    if (type != at::kFloat && type != at::kBFloat16)
      fail(PyExc_TypeError, "unsupported dtype: float32 or bfloat16 is needed");
    for (int64_t i = 0; i < count; ++i) {
      const Sequence q(states[i], "expected a tuple (m, m_scale, v, v_scale)");
      if (q.size() != 4) fail(PyExc_ValueError, "expected a tuple (m, m_scale, v, v_scale)");
      const Flat m(q[0], dev), ms(q[1], dev), v(q[2], dev), vs(q[3], dev);
      m.want(at::kByte, m.n, "m");
      v.want(at::kByte, m.n, "v");
      ms.want(at::kFloat, (m.n + kSpan - 1) / kSpan, "m_scale");
      vs.want(at::kFloat, (m.n + kSpan - 1) / kSpan, "v_scale");
      void* to[2];
      for (int k = 0; k < 2; ++k) {
        if (given) {
          const Flat o((*outs[(size_t)i])[k], dev);
          o.want(type, m.n, "out");
          to[k] = o.p;
        } else {
          const at::Tensor& like = tensor(q[0]);
          made.push_back(at::empty(like.sizes(), like.options().dtype(type)));
          to[k] = made.back().data_ptr();
        }
      }
      t[(size_t)i] = mao_adamw8_state{m.p, v.p, (const float*)ms.p, (const float*)vs.p,
                                      to[0], to[1], m.n};
    }
    check(mao_adamw8_read((int32_t)std::min<int64_t>(count, INT32_MAX), t.data(),
                          type == at::kBFloat16 ? MAO_BF16 : MAO_F32, (void*)integer(a[5])),
          "mao_adamw8_read");
    if (given) return Py_NewRef(a[3]);
    PyObject* list = PyList_New(count);
    if (!list) throw Raised{};
    for (int64_t i = 0; i < count; ++i)
      PyList_SET_ITEM(list, i, Py_BuildValue("NN", THPVariable_Wrap(made[(size_t)(2 * i)]),
                                             THPVariable_Wrap(made[(size_t)(2 * i + 1)])));
    return list;
  });
}

#define MAO_METHOD(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {MAO_METHOD(init),
                           MAO_METHOD(q8_quantize),
                           MAO_METHOD(q8_dequantize),
                           MAO_METHOD(layer_norm),
                           MAO_METHOD(layer_norm_backward),
                           MAO_METHOD(linear),
                           MAO_METHOD(linear_backward_input),
                           MAO_METHOD(linear_backward_weight),
                           MAO_METHOD(residual_norm),
                           MAO_METHOD(residual_norm_backward),
                           MAO_METHOD(token_logprobs),
                           MAO_METHOD(token_logprobs_backward),
                           MAO_METHOD(token_loss),
                           MAO_METHOD(adamw_step_many),
                           MAO_METHOD(adamw8_read),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_layers", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layers(void) { return PyModule_Create(&g_module); }
