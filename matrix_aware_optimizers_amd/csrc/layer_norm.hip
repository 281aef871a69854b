// Layer norm over the rows of a matrix, forward and backward.
//
//   mean = sum x / n,  rstd = (sum (x - mean)^2 / n + eps)^(-1/2)
//   y = (x - mean) rstd gamma + beta
//
//   xh = (x - mean) rstd,  g = dy gamma
//   dx = rstd (g - mean(g) - xh mean(g xh)) [+ add]
//   dgamma = sum over rows of dy xh,  dbeta = sum over rows of dy
//
// Bound: HBM. Each input is read once and each output written once: a row
// lives in the registers of its TPR threads (V runs of 8 columns each), so the
// variance is the two-pass one (deviations from the mean, no cancellation)
// without a second read. Grids are persistent: gamma and beta stay in
// registers, and the next row's loads are issued before the current row is
// reduced. One wavefront per row up to 2048 columns (reductions stay inside
// the wavefront: DPP adds and four lane reads, no LDS) in the forward pass, groups
// of 256 to 1024 threads above; in the backward pass groups of 128 to 1024 threads from
// 513 columns on.
//
// Measured (MI355X, bf16): forward 16384 x 1536 17.0 us, 101 MB, 5.9 TB/s (more than
// a large copy's 5.2: they fit the 256 MB cache behind the L2); one row 5.9 to 6.4 us on
// two cards, the kernel 3.4 of them. Backward with a joining gradient 16384 x 1536 44.3 us
// (34.4 and 4.2 for the partial rows; 201 MB, 5.9 TB/s over the first); 4093 x 4096
// from int8 codes 25.9 us (24.4 are the kernel, 84 MB, 3.5 TB/s: 16 rows per workgroup
// are too few to hide each row's reduction, both sums in one exchange). fp32, 16384 x
// 1536: forward 38.7 us, 201 MB, 5.2 TB/s, backward with a joining gradient 85 us, 403 MB,
// 4.7 TB/s. Rows above 8192 columns hold two or four runs per thread and spill a few
// registers in the backward pass (fp32 2000 x 8200 102 us, 262 MB, 2.6 TB/s).
//
// The column sums of the backward pass stay in registers over all rows a thread
// group handles, are joined inside the workgroup in a fixed order, and leave
// as one partial row per workgroup; a second kernel adds the partial rows in a
// fixed order. No atomics: results are bitwise repeatable. All sums are fp32.
#include "rows.hpp"

#include <algorithm>
#include <type_traits>

namespace mao {

namespace {

// CUT: a row's last run ends in its first 16-byte piece of fp32, so each run is loaded by
// its length. Kernels of their own: one branch a row in the backward kernel, whose code
// costs registers, took fp32 16384 x 1536 from 65 to 68 us and 2000 x 8200 from 102 to 116.
bool short_run(int cols) { return ((cols - 1) & 7) < 4; }

template <typename TIn, int TPR, int V, int BLK, bool CUT>
__global__ __launch_bounds__(BLK) void norm_fwd_kernel(NormFwdArgs a) {
  constexpr int RPB = BLK / TPR;
  __shared__ float red[2][BLK / 64];
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int nch = (a.cols + 7) >> 3;
  const bool ragged = (a.cols & 7) != 0;
  const float inv_n = 1.f / (float)a.cols;
  constexpr bool PRE = TPR < 1024 || V == 1;  // parameters stay in registers
  float gam[PRE ? V : 1][8], bet[PRE ? V : 1][8];
  if constexpr (PRE) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = t + v * TPR;
      load_param(a.gamma, a.p_dtype, 8 * c, a.cols - 8 * c, 1.f, gam[v]);
      load_param(a.beta, a.p_dtype, 8 * c, a.cols - 8 * c, 0.f, bet[v]);
    }
  }
  Raw8<TIn> raw[V];
  auto fetch = [&](int64_t row) __attribute__((always_inline)) {
    const TIn* x = (const TIn*)a.x + min(row, (int64_t)a.rows - 1) * a.ldx;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = t + v * TPR;
      if (c >= nch)
        raw[v].zero();
      else if constexpr (CUT)
        raw[v].load_cut(x + 8 * c, a.cols - 8 * c);
      else
        raw[v].load(x + 8 * c);
    }
  };
  const int step = gridDim.x * RPB;
  fetch((int64_t)blockIdx.x * RPB + sub);
  // every thread of the block runs the same number of rounds (barriers inside)
  for (int r0 = blockIdx.x * RPB; r0 < a.rows; r0 += step) {
    const int row = r0 + sub;
    float x[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      raw[v].get(x[v]);
      if (ragged) mask8(x[v], a.cols - 8 * (t + v * TPR));
    }
    if (r0 + step < a.rows) fetch((int64_t)row + step);
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) s += x[v][i];
    const float mean = group_total<TPR>(s, red[0]) * inv_n;
    float q = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int valid = a.cols - 8 * (t + v * TPR);
      if (valid <= 0) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[v][i] -= mean;
      if (ragged) mask8(x[v], valid);
#pragma unroll
      for (int i = 0; i < 8; ++i) q += x[v][i] * x[v][i];
    }
    const float rstd = 1.f / sqrtf(group_total<TPR>(q, red[1]) * inv_n + a.eps);
    if (row < a.rows) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = t + v * TPR;
        if (c >= nch) continue;
        float gl[8], bl[8];
        if constexpr (!PRE) {
          load_param(a.gamma, a.p_dtype, 8 * c, a.cols - 8 * c, 1.f, gl);
          load_param(a.beta, a.p_dtype, 8 * c, a.cols - 8 * c, 0.f, bl);
        }
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          y[i] = x[v][i] * rstd * (PRE ? gam[PRE ? v : 0][i] : gl[i]) +
                 (PRE ? bet[PRE ? v : 0][i] : bl[i]);
        store8n_any(a.y, a.y_dtype, (int64_t)row * a.ldy + 8 * c, y, a.cols - 8 * c);
      }
      if (t == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
      }
    }
  }
}

// Eight elements of the saved input: a tensor's, or decoded codes.
template <int XK> struct SavedRaw;
template <> struct SavedRaw<MAO_F32> {
  Raw8<float> r;
  template <bool CUT>
  __device__ __forceinline__ void load(const NormBwdArgs& a, int64_t row, int c) {
    const float* p = (const float*)a.x + row * a.ldx + 8 * c;
    if constexpr (CUT)
      r.load_cut(p, a.cols - 8 * c);
    else
      r.load(p);
  }
  __device__ __forceinline__ void zero() { r.zero(); }
  __device__ __forceinline__ void opaque() { r.opaque(); }
  __device__ __forceinline__ void get(float (&v)[8]) const { r.get(v); }
};
template <> struct SavedRaw<MAO_BF16> {
  Raw8<bf16_t> r;
  template <bool>
  __device__ __forceinline__ void load(const NormBwdArgs& a, int64_t row, int c) {
    r.load((const bf16_t*)a.x + row * a.ldx + 8 * c);
  }
  __device__ __forceinline__ void zero() { r.zero(); }
  __device__ __forceinline__ void opaque() { r.opaque(); }
  __device__ __forceinline__ void get(float (&v)[8]) const { r.get(v); }
};
template <int FMT> struct SavedCodes {
  uint2 q;
  int s;
  template <bool>
  __device__ __forceinline__ void load(const NormBwdArgs& a, int64_t row, int c) {
    q = *(const uint2*)((const uint8_t*)a.x + row * a.ldx + 8 * c);
    s = a.scales[row * a.lds + (c >> 2)];
  }
  __device__ __forceinline__ void zero() {
    q = make_uint2(0, 0);
    s = 0;
  }
  __device__ __forceinline__ void opaque() { asm volatile("" : "+v"(q.x), "+v"(q.y)); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const float sc = q8_scale_value(s);
    q8_decode4<FMT>(q.x, sc, v);
    q8_decode4<FMT>(q.y, sc, v + 4);
  }
};
template <> struct SavedRaw<kXInt8> : SavedCodes<MAO_Q8_INT8> {};
template <> struct SavedRaw<kXE4m3> : SavedCodes<MAO_Q8_E4M3> {};

template <typename TDy, int XK, int TPR, int V, int BLK, bool CUT>
__global__ __launch_bounds__(BLK) void norm_bwd_kernel(NormBwdArgs a) {
  constexpr int RPB = BLK / TPR;
  constexpr int kJoin = RPB > 1 ? 8 * V * TPR : 1;
  __shared__ float2 red[2][BLK / 64];
  __shared__ float join[kJoin];
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int nch = (a.cols + 7) >> 3;
  const float inv_n = 1.f / (float)a.cols;
  constexpr bool PRE = TPR < 1024 || V == 1;  // parameters stay in registers
  float gam[PRE ? V : 1][8];
  if constexpr (PRE) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = t + v * TPR;
      load_param(a.gamma, a.p_dtype, 8 * c, a.cols - 8 * c, 1.f, gam[v]);
    }
  }
  float dg[V][8], db[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) dg[v][i] = db[v][i] = 0.f;
  // the joining gradient comes with its row where it has dY's type (the usual
  // case), otherwise as it is needed
  using TOther = std::conditional_t<sizeof(TDy) == 2, float, bf16_t>;
  const bool add_early = a.add != nullptr && a.add_dtype == (sizeof(TDy) == 2 ? MAO_BF16 : MAO_F32);
  struct Row {
    Raw8<TDy> dy[V], add[V];
    SavedRaw<XK> x[V];
    float mean, rstd;
  };
  auto fetch = [&](Row& q, int64_t row) __attribute__((always_inline)) {
    row = min(row, (int64_t)a.rows - 1);
    q.mean = a.mean[row];
    q.rstd = a.rstd[row];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = t + v * TPR;
      if (c < nch) {
        const TDy* pd = (const TDy*)a.dy + row * a.lddy + 8 * c;
        const TDy* pa = (const TDy*)a.add + row * a.ldadd + 8 * c;
        if constexpr (CUT) {
          q.dy[v].load_cut(pd, a.cols - 8 * c);
          q.x[v].template load<true>(a, row, c);
          if (add_early) q.add[v].load_cut(pa, a.cols - 8 * c);
        } else {
          q.dy[v].load(pd);
          q.x[v].template load<false>(a, row, c);
          if (add_early) q.add[v].load(pa);
        }
      } else {
        q.dy[v].zero();
        q.x[v].zero();
      }
    }
  };
  const int step = gridDim.x * RPB;
  // The row stays in its stored form between the two passes over it (half the
  // registers of fp32 for bf16), values are rebuilt in the second.
  auto values = [&](const Row& q, int v, int lim, float (&dy)[8], float (&xh)[8], float (&g)[8])
                    __attribute__((always_inline)) {
    const int c = t + v * TPR, valid = lim - 8 * c;
    q.dy[v].get(dy);
    q.x[v].get(xh);
#pragma unroll
    for (int i = 0; i < 8; ++i) xh[i] = (xh[i] - q.mean) * q.rstd;
    if (valid < 8) {
      mask8(dy, valid);
      mask8(xh, valid);
    }
    float gl[8];
    if constexpr (!PRE) load_param(a.gamma, a.p_dtype, 8 * c, a.cols - 8 * c, 1.f, gl);
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = dy[i] * (PRE ? gam[PRE ? v : 0][i] : gl[i]);
  };
  auto handle = [&](Row& q, int row, float2* buf) __attribute__((always_inline)) {
    const bool live = row < a.rows;
    const int lim = live ? a.cols : 0;
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float dy[8], xh[8], g[8];
      values(q, v, lim, dy, xh, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dg[v][i] += dy[i] * xh[i];
        db[v][i] += dy[i];
        s0 += g[i];
        s1 += g[i] * xh[i];
      }
    }
    group_total2<TPR>(s0, s1, buf);
    const float c0 = s0 * inv_n, c1 = s1 * inv_n;
    if (!live) return;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = t + v * TPR;
      if (c >= nch) continue;
      q.dy[v].opaque();
      q.x[v].opaque();
      float dy[8], xh[8], g[8], o[8];
      values(q, v, lim, dy, xh, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = q.rstd * (g[i] - c0 - xh[i] * c1);
      if (a.add) {
        float w[8];
        if (add_early) {
          q.add[v].get(w);
        } else {
          Raw8<TOther> r;
          const TOther* p = (const TOther*)a.add + (int64_t)row * a.ldadd + 8 * c;
          if constexpr (CUT)
            r.load_cut(p, a.cols - 8 * c);
          else
            r.load(p);
          r.get(w);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] += w[i];
      }
      store8n_any(a.dx, a.dx_dtype, (int64_t)row * a.lddx + 8 * c, o, a.cols - 8 * c);
    }
  };
  int r0 = blockIdx.x * RPB;
  // every thread of the block runs the same number of rounds (barriers inside)
  if constexpr (TPR == 1024 && V > 1) {  // no registers for a second row
    Row q;
    for (int k = 0; r0 < a.rows; r0 += step, k ^= 1) {
      fetch(q, (int64_t)r0 + sub);
      handle(q, r0 + sub, red[k]);
    }
  } else {
    // two rows in turn: the next one is on its way while one is handled (a third
    // row in flight gained nothing)
    Row q0, q1;
    fetch(q0, (int64_t)r0 + sub);
    while (true) {
      if (r0 + step < a.rows) fetch(q1, (int64_t)r0 + step + sub);
      handle(q0, r0 + sub, red[0]);
      r0 += step;
      if (r0 >= a.rows) break;
      if (r0 + step < a.rows) fetch(q0, (int64_t)r0 + step + sub);
      handle(q1, r0 + sub, red[1]);
      r0 += step;
      if (r0 >= a.rows) break;
    }
  }
  if (a.part == nullptr) return;
  // partial row of the workgroup: its row groups' sums in order 0, 1, ...
  float* out = a.part + (int64_t)blockIdx.x * 2 * a.cols;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if constexpr (RPB > 1) {
      for (int k = 0; k < RPB - 1; ++k) {
        __syncthreads();
        if (sub == k) {
#pragma unroll
          for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float* p = &join[(v * 8 + i) * TPR + t];
              const float w = which ? db[v][i] : dg[v][i];
              *p = k == 0 ? w : *p + w;
            }
        }
      }
      __syncthreads();
    }
    if (sub == RPB - 1) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = t + v * TPR;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float w = (which ? db[v][i] : dg[v][i]) +
                          (RPB > 1 ? join[RPB > 1 ? (v * 8 + i) * TPR + t : 0] : 0.f);
          if (8 * c + i < a.cols) out[(int64_t)which * a.cols + 8 * c + i] = w;
        }
      }
    }
  }
}

// Threads per workgroup; the backward pass takes more, for fewer partial rows.
constexpr int fwd_block(int tpr) { return tpr > 256 ? tpr : 256; }
constexpr int bwd_block(int tpr) { return 1024 / tpr * tpr; }

template <typename TIn, int TPR, int V>
mao_status fwd_launch(const NormFwdArgs& a, hipStream_t s) {
  constexpr int BLK = fwd_block(TPR), RPB = BLK / TPR;
  const int grid = (int)std::min<int64_t>(ceil_div(a.rows, RPB), 256 * (2048 / BLK));
  constexpr bool F32 = sizeof(TIn) == 4;
  if (F32 && short_run(a.cols))
    hipLaunchKernelGGL((norm_fwd_kernel<TIn, TPR, V, BLK, F32>), dim3(grid), dim3(BLK), 0, s, a);
  else
    hipLaunchKernelGGL((norm_fwd_kernel<TIn, TPR, V, BLK, false>), dim3(grid), dim3(BLK), 0, s, a);
  MAO_LAUNCH_CHECK();
  return MAO_OK;
}

template <typename TIn>
mao_status fwd_pick(const NormFwdArgs& a, hipStream_t s) {
  if (a.cols <= 512) return fwd_launch<TIn, 64, 1>(a, s);
  if (a.cols <= 1024) return fwd_launch<TIn, 64, 2>(a, s);
  if (a.cols <= 1536) return fwd_launch<TIn, 64, 3>(a, s);
  if (a.cols <= 2048) return fwd_launch<TIn, 64, 4>(a, s);
  if (a.cols <= 4096) return fwd_launch<TIn, 256, 2>(a, s);
  if (a.cols <= 8192) return fwd_launch<TIn, 256, 4>(a, s);
  if (a.cols <= 16384) return fwd_launch<TIn, 512, 4>(a, s);
  return fwd_launch<TIn, 1024, 4>(a, s);
}

// Threads per row and runs of 8 columns per thread.
struct BwdShape {
  int tpr, v;
};
BwdShape bwd_shape(int64_t cols) {
  // One run per thread: column sums, gamma and two or three rows in flight fit
  // 128 registers, so that 16 wavefronts share a CU. (16384 x 1536 bf16: three runs
  // per lane of one wavefront, 8 wavefronts per CU, 50.8 us.)
  if (cols <= 512) return {64, 1};
  if (cols <= 1024) return {128, 1};
  if (cols <= 1536) return {192, 1};
  if (cols <= 2048) return {256, 1};
  if (cols <= 4096) return {512, 1};
  return {1024, cols <= 8192 ? 1 : cols <= 16384 ? 2 : 4};
}

template <typename TDy, int XK, int TPR, int V>
mao_status bwd_launch(const NormBwdArgs& a, hipStream_t s) {
  constexpr int BLK = bwd_block(TPR);
  const dim3 grid(norm_bwd_blocks(a.rows, a.cols));
  const bool f32 = sizeof(TDy) == 4 || XK == MAO_F32 || (a.add && a.add_dtype == MAO_F32);
  if (f32 && short_run(a.cols))
    hipLaunchKernelGGL((norm_bwd_kernel<TDy, XK, TPR, V, BLK, true>), grid, dim3(BLK), 0, s, a);
  else
    hipLaunchKernelGGL((norm_bwd_kernel<TDy, XK, TPR, V, BLK, false>), grid, dim3(BLK), 0, s, a);
  MAO_LAUNCH_CHECK();
  return MAO_OK;
}

template <typename TDy, int XK>
mao_status bwd_pick(const NormBwdArgs& a, hipStream_t s) {
  const BwdShape b = bwd_shape(a.cols);
  switch (b.tpr) {
    case 64: return bwd_launch<TDy, XK, 64, 1>(a, s);
    case 128: return bwd_launch<TDy, XK, 128, 1>(a, s);
    case 192: return bwd_launch<TDy, XK, 192, 1>(a, s);
    case 256: return bwd_launch<TDy, XK, 256, 1>(a, s);
    case 512: return bwd_launch<TDy, XK, 512, 1>(a, s);
    default:
      if (b.v == 1) return bwd_launch<TDy, XK, 1024, 1>(a, s);
      if (b.v == 2) return bwd_launch<TDy, XK, 1024, 2>(a, s);
      return bwd_launch<TDy, XK, 1024, 4>(a, s);
  }
}

template <typename TDy>
mao_status bwd_kind(const NormBwdArgs& a, int x_kind, hipStream_t s) {
  switch (x_kind) {
    case MAO_F32: return bwd_pick<TDy, MAO_F32>(a, s);
    case MAO_BF16: return bwd_pick<TDy, MAO_BF16>(a, s);
    case kXInt8: return bwd_pick<TDy, kXInt8>(a, s);
    default: return bwd_pick<TDy, kXE4m3>(a, s);
  }
}

}  // namespace

int norm_bwd_blocks(int64_t rows, int64_t cols) {
  const BwdShape b = bwd_shape(cols);
  return (int)std::min<int64_t>(ceil_div(rows, bwd_block(b.tpr) / b.tpr), 256);
}

mao_status launch_norm_fwd(const NormFwdArgs& a, int x_dtype, hipStream_t s) {
  return x_dtype == MAO_BF16 ? fwd_pick<bf16_t>(a, s) : fwd_pick<float>(a, s);
}

mao_status launch_norm_bwd(const NormBwdArgs& a, int dy_dtype, int x_kind, hipStream_t s) {
  MAO_TRY(dy_dtype == MAO_BF16 ? bwd_kind<bf16_t>(a, x_kind, s) : bwd_kind<float>(a, x_kind, s));
  if (a.part == nullptr) return MAO_OK;
  return launch_partial_sum(a.part, 2 * (int64_t)a.cols, norm_bwd_blocks(a.rows, a.cols), a.cols,
                            a.dgamma, a.dbeta, a.cols, 0, s);
}

}  // namespace mao
