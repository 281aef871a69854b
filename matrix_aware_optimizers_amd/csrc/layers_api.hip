// C entry points of the layer operators: host-side validation, workspace
// carving, launches. Nothing here throws or allocates.
#include "layers.hpp"
#include "validate.hpp"

namespace mao {

namespace {

bool act_ok(int act) { return act >= MAO_ACT_NONE && act <= MAO_ACT_SILU; }

mao_status check_view(const char* name, const mao_mat& m) {
  return check_mat(name, m.data, m.rows, m.cols, m.ld, m.dtype, false);
}

mao_status check_shape(const char* name, const mao_mat& m, int64_t rows, int64_t cols) {
  MAO_TRY(check_view(name, m));
  if (m.rows != rows || m.cols != cols)
    MAO_FAIL(MAO_E_SHAPE, "%s: %lld x %lld, expected %lld x %lld", name, (long long)m.rows,
             (long long)m.cols, (long long)rows, (long long)cols);
  return MAO_OK;
}

mao_status check_q8(const char* name, const mao_q8& q, int64_t rows, int64_t cols) {
  if (!q.codes || !q.scales) MAO_FAIL(MAO_E_NULL, "%s: NULL codes or scales", name);
  if (q.rows != rows || q.cols != cols)
    MAO_FAIL(MAO_E_SHAPE, "%s: %lld x %lld, expected %lld x %lld", name, (long long)q.rows,
             (long long)q.cols, (long long)rows, (long long)cols);
  if (q.format != MAO_Q8_INT8 && q.format != MAO_Q8_E4M3)
    MAO_FAIL(MAO_E_DTYPE, "%s: format %d", name, q.format);
  if (q.ld < cols || q.ld % kQ8Block != 0)
    MAO_FAIL(MAO_E_LAYOUT, "%s: ld=%lld must be >= cols and a multiple of 32", name, (long long)q.ld);
  if (q.ld_scale < ceil_div(cols, kQ8Block))
    MAO_FAIL(MAO_E_LAYOUT, "%s: ld_scale=%lld below one byte per 32 columns", name, (long long)q.ld_scale);
  if ((uintptr_t)q.codes % 16 != 0) MAO_FAIL(MAO_E_LAYOUT, "%s: codes not 16-byte aligned", name);
  return MAO_OK;
}

mao_status check_vector(const char* name, const void* p, int dtype) {
  if (!p) return MAO_OK;
  if (!dtype_ok(dtype)) MAO_FAIL(MAO_E_DTYPE, "%s: unsupported dtype %d", name, dtype);
  if ((uintptr_t)p % 16 != 0) MAO_FAIL(MAO_E_LAYOUT, "%s: not 16-byte aligned", name);
  return MAO_OK;
}

mao_status check_floats(const char* name, const float* p) {
  if ((uintptr_t)p % 4 != 0) MAO_FAIL(MAO_E_LAYOUT, "%s: misaligned", name);
  return MAO_OK;
}

Range range_of(const mao_mat& m) {
  return mat_range(m.data, 1, m.rows, m.cols, m.ld, 0, dtype_size(m.dtype));
}
Range range_of(const void* p, int64_t bytes) {
  return Range{(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes};
}

bool same_view(const mao_mat& a, const mao_mat& b) {
  return a.data == b.data && a.ld == b.ld && a.dtype == b.dtype;
}

// The buffers of one call, outputs first: no output may share bytes with any
// other buffer.
struct Buffers {
  Range r[16];
  int n = 0, outs = 0;
  void out(Range x) {
    r[n++] = x;
    outs = n;
  }
  void in(Range x) { r[n++] = x; }
  void in(const mao_q8* q) {
    if (!q) return;
    in(mat_range(q->codes, 1, q->rows, q->cols, q->ld, 0, 1));
    in(mat_range(q->scales, 1, q->rows, ceil_div(q->cols, kQ8Block), q->ld_scale, 0, 1));
  }
  mao_status check() const {
    for (int i = 0; i < outs; ++i)
      for (int j = i + 1; j < n; ++j)
        if (overlap(r[i], r[j])) MAO_FAIL(MAO_E_ALIAS, "an output overlaps another buffer (%d, %d)", i, j);
    return MAO_OK;
  }
};

Q8View view_of(const mao_q8& q) { return {q.codes, q.scales, q.ld, q.ld_scale}; }
int kind_of(const mao_q8& q) { return q.format == MAO_Q8_INT8 ? kXInt8 : kXE4m3; }

bool sizes_ok(int64_t a, int64_t b, int64_t c) {
  const int64_t most = 1 << 20;
  return a >= 1 && b >= 1 && c >= 1 && a <= most && b <= most && c <= most;
}

// The weight gradient's workspace: the rebuilt input, the product's partial
// tiles, the bias gradient's partial rows.
struct WeightWs {
  char *x, *part;
  float* sums;
  int64_t ldx;
  size_t bytes, bare;  // bare: without a bias gradient
};
WeightWs carve_weight(void* base, int64_t rows, int64_t k, int64_t n, int dtype, bool rebuilt) {
  Carver c(base);
  WeightWs w = {};
  w.ldx = ws_ld(k);
  if (rebuilt) w.x = c.take<char>((size_t)rows * w.ldx * dtype_size(dtype));
  w.part = c.take<char>(lin_workspace(dtype, n, k, rows));
  w.bare = c.used;
  w.sums = c.take<float>((size_t)lin_sum_rows(dtype, n, k, rows) * n);
  w.bytes = c.used;
  return w;
}

}  // namespace
}  // namespace mao

using namespace mao;

extern "C" {

mao_status mao_q8_quantize(mao_mat X, const mao_q8* X8, void* stream) {
  MAO_TRY(check_view("X", X));
  if (!X8) MAO_FAIL(MAO_E_NULL, "X8 is NULL");
  MAO_TRY(check_q8("X8", *X8, X.rows, X.cols));
  Buffers b;
  b.out(mat_range(X8->codes, 1, X8->rows, X8->cols, X8->ld, 0, 1));
  b.out(mat_range(X8->scales, 1, X8->rows, ceil_div(X8->cols, kQ8Block), X8->ld_scale, 0, 1));
  b.in(range_of(X));
  MAO_TRY(b.check());
  return launch_q8_quantize(X.data, X.dtype, X.ld, (int)X.rows, (int)X.cols, view_of(*X8),
                            X8->format, (hipStream_t)stream);
}

mao_status mao_q8_dequantize(const mao_q8* X8, int32_t act, mao_mat Y, void* stream) {
  MAO_TRY(check_view("Y", Y));
  if (!X8) MAO_FAIL(MAO_E_NULL, "X8 is NULL");
  MAO_TRY(check_q8("X8", *X8, Y.rows, Y.cols));
  if (!act_ok(act)) MAO_FAIL(MAO_E_HPARAM, "act=%d", act);
  Buffers b;
  b.out(range_of(Y));
  b.in(X8);
  MAO_TRY(b.check());
  return launch_q8_dequantize(view_of(*X8), X8->format, (int)Y.rows, (int)Y.cols, act, false,
                              Y.data, Y.dtype, Y.ld, (hipStream_t)stream);
}

mao_status mao_layer_norm(mao_mat X, const void* gamma, const void* beta, int32_t param_dtype,
                          float eps, mao_mat Y, float* mean, float* rstd, void* stream) {
  MAO_TRY(check_view("X", X));
  MAO_TRY(check_shape("Y", Y, X.rows, X.cols));
  if (X.cols > kNormMaxCols) MAO_FAIL(MAO_E_UNSUPPORTED, "cols=%lld above %lld", (long long)X.cols, (long long)kNormMaxCols);
  MAO_TRY(check_vector("gamma", gamma, param_dtype));
  MAO_TRY(check_vector("beta", beta, param_dtype));
  MAO_TRY(check_floats("mean", mean));
  MAO_TRY(check_floats("rstd", rstd));
  if (!finite(eps) || eps <= 0.f) MAO_FAIL(MAO_E_HPARAM, "eps=%g must be > 0", (double)eps);
  const int64_t pb = X.cols * (int64_t)dtype_size(param_dtype);
  Buffers b;
  b.out(range_of(Y));
  if (mean) b.out(range_of(mean, X.rows * 4));
  if (rstd) b.out(range_of(rstd, X.rows * 4));
  b.in(range_of(X));
  if (gamma) b.in(range_of(gamma, pb));
  if (beta) b.in(range_of(beta, pb));
  MAO_TRY(b.check());
  NormFwdArgs a = {};
  a.x = X.data;
  a.gamma = gamma;
  a.beta = beta;
  a.y = Y.data;
  a.mean = mean;
  a.rstd = rstd;
  a.ldx = X.ld;
  a.ldy = Y.ld;
  a.rows = (int)X.rows;
  a.cols = (int)X.cols;
  a.p_dtype = param_dtype;
  a.y_dtype = Y.dtype;
  a.eps = eps;
  return launch_norm_fwd(a, X.dtype, (hipStream_t)stream);
}

size_t mao_layer_norm_backward_workspace_size(int64_t rows, int64_t cols) {
  if (!sizes_ok(rows, cols, 1) || cols > kNormMaxCols) return 0;
  return (size_t)norm_bwd_blocks(rows, cols) * 2 * cols * 4;
}

mao_status mao_layer_norm_backward(mao_mat dY, const mao_mat* X, const mao_q8* X8,
                                   const void* gamma, int32_t param_dtype, const float* mean,
                                   const float* rstd, const mao_mat* add, mao_mat dX,
                                   float* dgamma, float* dbeta, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  MAO_TRY(check_view("dY", dY));
  if ((X == nullptr) == (X8 == nullptr)) MAO_FAIL(MAO_E_NULL, "exactly one of X and X8 is needed");
  if (X) MAO_TRY(check_shape("X", *X, dY.rows, dY.cols));
  if (X8) MAO_TRY(check_q8("X8", *X8, dY.rows, dY.cols));
  MAO_TRY(check_shape("dX", dX, dY.rows, dY.cols));
  if (add) MAO_TRY(check_shape("add", *add, dY.rows, dY.cols));
  if (dY.cols > kNormMaxCols) MAO_FAIL(MAO_E_UNSUPPORTED, "cols=%lld above %lld", (long long)dY.cols, (long long)kNormMaxCols);
  MAO_TRY(check_vector("gamma", gamma, param_dtype));
  if (!mean || !rstd) MAO_FAIL(MAO_E_NULL, "mean or rstd is NULL");
  MAO_TRY(check_floats("mean", mean));
  MAO_TRY(check_floats("rstd", rstd));
  MAO_TRY(check_floats("dgamma", dgamma));
  MAO_TRY(check_floats("dbeta", dbeta));
  const bool sums = dgamma || dbeta;
  const size_t need = sums ? mao_layer_norm_backward_workspace_size(dY.rows, dY.cols) : 0;
  Buffers b;
  b.out(range_of(dX));
  if (dgamma) b.out(range_of(dgamma, dY.cols * 4));
  if (dbeta) b.out(range_of(dbeta, dY.cols * 4));
  if (sums) b.out(range_of(workspace, (int64_t)need));
  b.in(range_of(dY));
  if (X) b.in(range_of(*X));
  b.in(X8);
  if (gamma) b.in(range_of(gamma, dY.cols * (int64_t)dtype_size(param_dtype)));
  b.in(range_of(mean, dY.rows * 4));
  b.in(range_of(rstd, dY.rows * 4));
  if (add && !same_view(*add, dX)) b.in(range_of(*add));
  MAO_TRY(check_workspace(workspace, workspace_bytes, need));
  MAO_TRY(b.check());
  NormBwdArgs a = {};
  a.dy = dY.data;
  a.lddy = dY.ld;
  if (X) {
    a.x = X->data;
    a.ldx = X->ld;
  } else {
    a.x = X8->codes;
    a.ldx = X8->ld;
    a.scales = X8->scales;
    a.lds = X8->ld_scale;
  }
  a.gamma = gamma;
  a.p_dtype = param_dtype;
  a.mean = mean;
  a.rstd = rstd;
  if (add) {
    a.add = add->data;
    a.ldadd = add->ld;
    a.add_dtype = add->dtype;
  }
  a.dx = dX.data;
  a.lddx = dX.ld;
  a.dx_dtype = dX.dtype;
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  a.part = sums ? (float*)workspace : nullptr;
  a.rows = (int)dY.rows;
  a.cols = (int)dY.cols;
  return launch_norm_bwd(a, dY.dtype, X ? X->dtype : kind_of(*X8), (hipStream_t)stream);
}

size_t mao_linear_workspace_size(int64_t rows, int64_t k, int64_t n, int32_t dtype) {
  if (!sizes_ok(rows, k, n) || !dtype_ok(dtype) || rows <= kTokenRows) return 0;
  return lin_workspace(dtype, rows, n, k);
}

size_t mao_linear_backward_input_workspace_size(int64_t rows, int64_t k, int64_t n,
                                                int32_t dtype) {
  if (!sizes_ok(rows, k, n) || !dtype_ok(dtype)) return 0;
  return lin_workspace(dtype, rows, k, n);
}

size_t mao_linear_backward_weight_workspace_size(int64_t rows, int64_t k, int64_t n, int32_t dtype,
                                                 int32_t rebuilt) {
  if (!sizes_ok(rows, k, n) || !dtype_ok(dtype)) return 0;
  return carve_weight(nullptr, rows, k, n, dtype, rebuilt != 0).bytes;
}

mao_status mao_dbg_linear_cut(int32_t product, int64_t rows, int64_t k, int64_t n, int32_t dtype,
                              int32_t mixed, int32_t* tile_m, int32_t* tile_n, int32_t* split) {
  if (!tile_m || !tile_n || !split) MAO_FAIL(MAO_E_NULL, "NULL result");
  if (!sizes_ok(rows, k, n)) MAO_FAIL(MAO_E_SHAPE, "rows=%lld k=%lld n=%lld", (long long)rows, (long long)k, (long long)n);
  if (!dtype_ok(dtype)) MAO_FAIL(MAO_E_DTYPE, "dtype=%d", dtype);
  if (product < 0 || product > 2) MAO_FAIL(MAO_E_HPARAM, "product=%d", product);
  const LinCut c = product == 0 && rows <= kTokenRows ? LinCut{16, 16, 1}
                   : product == 0 ? lin_cut(dtype, mixed != 0, rows, n, k)
                   : product == 1 ? lin_cut(dtype, mixed != 0, rows, k, n)
                                  : lin_cut(dtype, false, n, k, rows);
  *tile_m = c.bm;
  *tile_n = c.bn;
  *split = c.split;
  return MAO_OK;
}

mao_status mao_linear(mao_mat X, mao_mat W, const void* bias, int32_t bias_dtype, int32_t act,
                      const mao_mat* residual, mao_mat Y, const mao_mat* preact, void* workspace,
                      size_t workspace_bytes, void* stream) {
  MAO_TRY(check_view("X", X));
  MAO_TRY(check_view("W", W));
  if (W.cols != X.cols) MAO_FAIL(MAO_E_SHAPE, "W has %lld columns, X %lld", (long long)W.cols, (long long)X.cols);
  if (W.dtype != X.dtype) MAO_FAIL(MAO_E_DTYPE, "X and W must share a dtype");
  MAO_TRY(check_shape("Y", Y, X.rows, W.rows));
  if (residual) MAO_TRY(check_shape("residual", *residual, X.rows, W.rows));
  if (preact) MAO_TRY(check_shape("preact", *preact, X.rows, W.rows));
  MAO_TRY(check_vector("bias", bias, bias_dtype));
  if (!act_ok(act)) MAO_FAIL(MAO_E_HPARAM, "act=%d", act);
  const size_t need = mao_linear_workspace_size(X.rows, X.cols, W.rows, X.dtype);
  MAO_TRY(check_workspace(workspace, workspace_bytes, need));
  Buffers b;
  b.out(range_of(Y));
  if (preact) b.out(range_of(*preact));
  if (need) b.out(range_of(workspace, (int64_t)need));
  b.in(range_of(X));
  b.in(range_of(W));
  if (bias) b.in(range_of(bias, W.rows * (int64_t)dtype_size(bias_dtype)));
  if (residual && !same_view(*residual, Y)) b.in(range_of(*residual));
  MAO_TRY(b.check());
  LinProblem p = {};
  p.A = X.data;
  p.lda = X.ld;
  p.B = W.data;
  p.ldb = W.ld;
  p.M = (int)X.rows;
  p.N = (int)W.rows;
  p.K = (int)X.cols;
  p.e.D = Y.data;
  p.e.ldd = Y.ld;
  p.e.d_dtype = Y.dtype;
  p.e.bias = bias;
  p.e.bias_dtype = bias_dtype;
  p.e.act = act;
  if (preact) {
    p.e.z_out = preact->data;
    p.e.ldzo = preact->ld;
    p.e.zo_dtype = preact->dtype;
  }
  if (residual) {
    p.e.add = residual->data;
    p.e.ldadd = residual->ld;
    p.e.add_dtype = residual->dtype;
  }
  if (X.rows <= kTokenRows) return launch_linear_token(X.dtype, p, (hipStream_t)stream);
  return launch_linear(X.dtype, p, workspace, nullptr, (hipStream_t)stream);
}

mao_status mao_linear_backward_input(mao_mat dY, mao_mat W, int32_t act, const mao_mat* Z,
                                     const mao_q8* Z8, const mao_mat* add, mao_mat dX,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  MAO_TRY(check_view("dY", dY));
  MAO_TRY(check_view("W", W));
  if (W.rows != dY.cols) MAO_FAIL(MAO_E_SHAPE, "W has %lld rows, dY %lld columns", (long long)W.rows, (long long)dY.cols);
  if (W.dtype != dY.dtype) MAO_FAIL(MAO_E_DTYPE, "dY and W must share a dtype");
  MAO_TRY(check_shape("dX", dX, dY.rows, W.cols));
  if (add) MAO_TRY(check_shape("add", *add, dY.rows, W.cols));
  if (!act_ok(act)) MAO_FAIL(MAO_E_HPARAM, "act=%d", act);
  if ((Z != nullptr) + (Z8 != nullptr) != (act == MAO_ACT_NONE ? 0 : 1))
    MAO_FAIL(MAO_E_NULL, "an activation needs exactly one of Z and Z8, no activation neither");
  if (Z) MAO_TRY(check_shape("Z", *Z, dY.rows, W.cols));
  if (Z8) MAO_TRY(check_q8("Z8", *Z8, dY.rows, W.cols));
  const size_t need = mao_linear_backward_input_workspace_size(dY.rows, W.cols, W.rows, dY.dtype);
  MAO_TRY(check_workspace(workspace, workspace_bytes, need));
  Buffers b;
  b.out(range_of(dX));
  if (need) b.out(range_of(workspace, (int64_t)need));
  b.in(range_of(dY));
  b.in(range_of(W));
  if (Z) b.in(range_of(*Z));
  b.in(Z8);
  if (add && !same_view(*add, dX)) b.in(range_of(*add));
  MAO_TRY(b.check());
  LinProblem p = {};
  p.A = dY.data;
  p.lda = dY.ld;
  p.B = W.data;
  p.ldb = W.ld;
  p.b_km = 1;
  p.M = (int)dY.rows;
  p.N = (int)W.cols;
  p.K = (int)W.rows;
  p.e.D = dX.data;
  p.e.ldd = dX.ld;
  p.e.d_dtype = dX.dtype;
  p.e.act = act;
  if (Z) {
    p.e.z_in = Z->data;
    p.e.ldzi = Z->ld;
    p.e.z_kind = Z->dtype;
  }
  if (Z8) {
    p.e.z_in = Z8->codes;
    p.e.ldzi = Z8->ld;
    p.e.z_scales = Z8->scales;
    p.e.ldzs = Z8->ld_scale;
    p.e.z_kind = kind_of(*Z8);
  }
  if (add) {
    p.e.add = add->data;
    p.e.ldadd = add->ld;
    p.e.add_dtype = add->dtype;
  }
  return launch_linear(dY.dtype, p, workspace, nullptr, (hipStream_t)stream);
}

mao_status mao_linear_backward_weight(mao_mat dY, const mao_mat* X, const mao_q8* X8,
                                      int32_t x_act, mao_mat dW, float* dbias, int32_t accumulate,
                                      void* workspace, size_t workspace_bytes, void* stream) {
  MAO_TRY(check_view("dY", dY));
  MAO_TRY(check_view("dW", dW));
  if ((X == nullptr) == (X8 == nullptr)) MAO_FAIL(MAO_E_NULL, "exactly one of X and X8 is needed");
  if (dW.rows != dY.cols) MAO_FAIL(MAO_E_SHAPE, "dW has %lld rows, dY %lld columns", (long long)dW.rows, (long long)dY.cols);
  if (X) {
    MAO_TRY(check_shape("X", *X, dY.rows, dW.cols));
    if (X->dtype != dY.dtype) MAO_FAIL(MAO_E_DTYPE, "dY and X must share a dtype");
  }
  if (X8) MAO_TRY(check_q8("X8", *X8, dY.rows, dW.cols));
  if (!act_ok(x_act)) MAO_FAIL(MAO_E_HPARAM, "x_act=%d", x_act);
  MAO_TRY(check_floats("dbias", dbias));
  const bool rebuilt = X8 != nullptr || x_act != MAO_ACT_NONE;
  const WeightWs w = carve_weight(workspace, dY.rows, dW.cols, dW.rows, dY.dtype, rebuilt);
  const size_t need = dbias ? w.bytes : w.bare;
  MAO_TRY(check_workspace(workspace, workspace_bytes, need));
  Buffers b;
  b.out(range_of(dW));
  if (dbias) b.out(range_of(dbias, dW.rows * 4));
  if (need) b.out(range_of(workspace, (int64_t)need));
  b.in(range_of(dY));
  if (X) b.in(range_of(*X));
  b.in(X8);
  MAO_TRY(b.check());
  hipStream_t s = (hipStream_t)stream;
  LinProblem p = {};
  p.A = dY.data;
  p.lda = dY.ld;
  p.a_km = p.b_km = 1;
  p.M = (int)dW.rows;
  p.N = (int)dW.cols;
  p.K = (int)dY.rows;
  // the input (or what its rounding to bf16 left) into the workspace
  auto rebuild = [&](bool rest) {
    return X8 ? launch_q8_dequantize(view_of(*X8), X8->format, (int)X8->rows, (int)X8->cols, x_act,
                                     rest, w.x, dY.dtype, w.ldx, s)
              : launch_act(X->data, X->dtype, X->ld, (int)X->rows, (int)X->cols, x_act, rest, w.x,
                           w.ldx, s);
  };
  if (rebuilt) {
    MAO_TRY(rebuild(false));
    p.B = w.x;
    p.ldb = w.ldx;
  } else {
    p.B = X->data;
    p.ldb = X->ld;
  }
  p.e.D = dW.data;
  p.e.ldd = dW.ld;
  p.e.d_dtype = dW.dtype;
  if (accumulate) {
    p.e.add = dW.data;
    p.e.ldadd = dW.ld;
    p.e.add_dtype = dW.dtype;
  }
  MAO_TRY(launch_linear(dY.dtype, p, w.part, dbias ? w.sums : nullptr, s));
  // bf16 matrix cores take a recomputed activation rounded to bf16. Into an fp32 dW
  // what that rounding left goes by a second product: two bf16 parts hold 16 bits of
  // it. (relu of a bf16 or 8-bit value needs one.) A bf16 dW takes the rounded value
  // alone, which is what a bf16 forward product read.
  // 8191 rows 14336 -> 4096, silu from e4m3, against the formula in 64 bits: fp32 dW
  // 1.5e-3 off with one product, 2.1e-6 with two (946 and 1921 us);
  // bf16 dW 2.25e-3 with one, and 1.66e-3 is its own rounding alone.
  if (x_act > MAO_ACT_RELU && dY.dtype == MAO_BF16 && dW.dtype == MAO_F32) {
    MAO_TRY(rebuild(true));
    p.e.add = dW.data;
    p.e.ldadd = dW.ld;
    p.e.add_dtype = dW.dtype;
    MAO_TRY(launch_linear(dY.dtype, p, w.part, nullptr, s));
  }
  if (dbias)
    MAO_TRY(launch_partial_sum(w.sums, p.M, lin_sum_rows(dY.dtype, p.M, p.N, p.K), p.M, dbias,
                               nullptr, 0, accumulate != 0, s));
  return MAO_OK;
}

}  // extern "C"
