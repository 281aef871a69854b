// What joins a block to the residual stream and begins the next one: the norm of the block's
// output, its gate and scale, the sum with the stream, and the next block's norm.
//
//   N(z) = xh gamma + beta,  xh = (z - mean) rstd,  rstd = (sum (z - mean)^2 / n + eps)^(-1/2)
//          (mean = 0 for the root-mean-square norm; without a norm N(z) = z)
//   u = N1(b);  r = xs x + bs gate . u;  h = N2(r)
//
// Backward, from dh (of h) and d (of r, from what follows):
//   q = dh gamma2;  dr = d + rstd2 (q - mean(q) - xh2 mean(q xh2))
//   dx = xs dr;  du = bs gate . dr;  p = du gamma1
//   db = rstd1 (p - mean(p) - xh1 mean(p xh1))          (no mean(q), mean(p) without a mean)
//   dgate = bs dr . u;  dgamma1 = sum du xh1, dbeta1 = sum du, dgamma2 = sum dh xh2,
//   dbeta2 = sum dh over the rows
//
// Bound: HBM, each matrix once. A row lives in the registers of its threads (one run of 4
// columns each up to 4096 columns), so that a deviation is one from the row's own mean; the
// next row's loads are issued before the current one is reduced. h is made from r as it is
// in fp32, before it is rounded to be stored.
//
// With a gate per channel (or none) its gradient and those of N1's parameters need two column
// sums: A = sum dr xh1 and D = sum dr give dgamma1 = bs gate A, dbeta1 = bs gate D and
// dgate = bs (gamma1 A + beta1 D). With a gate per element A and D are sums of gate . dr.
// Sums stay in registers over the rows of a workgroup, are joined in it in order, and
// leave as one partial row; a second kernel adds those in order. No atomics, fp32.
#include "rows.hpp"

#include <algorithm>

namespace mao {

namespace {

template <typename TX, typename TB, int TPR, int V>
__global__ __launch_bounds__(TPR) void join_fwd_kernel(JoinArgs a) {
  __shared__ float red[2][4][TPR / 64];
  int t = threadIdx.x;
  const float inv_n = 1.f / (float)a.cols;
  constexpr bool PRE = V == 1;  // parameters stay in registers
  constexpr int P = PRE ? V : 1;
  float g1[P][4], b1[P][4], g2[P][4], b2[P][4], gate[P][4];
  auto params = [&](int v, int i) __attribute__((always_inline)) {
    const int col = 4 * (t + v * TPR), valid = a.cols - col;
    load_param4(a.post.gamma, a.post.p_dtype, col, valid, 1.f, g1[i]);
    load_param4(a.post.beta, a.post.p_dtype, col, valid, 0.f, b1[i]);
    load_param4(a.pre.gamma, a.pre.p_dtype, col, valid, 1.f, g2[i]);
    load_param4(a.pre.beta, a.pre.p_dtype, col, valid, 0.f, b2[i]);
    load_param4(a.gate_vec, a.gate_dtype, col, valid, 1.f, gate[i]);
  };
  if constexpr (PRE) params(0, 0);
  Run4<TX> rx[V];
  Run4<TB> rb[V], rg[V];
  const int xbytes = run4_bytes<TX>(a.cols), bbytes = run4_bytes<TB>(a.cols);
  auto fetch = [&](int row) __attribute__((always_inline)) {
    const auto x = row_buffer(a.x, a.ldx * (int64_t)sizeof(TX), row, xbytes);
    const auto b = row_buffer(a.b, a.ldb * (int64_t)sizeof(TB), row, bbytes);
    const auto g = row_buffer(a.gate, a.ldgate * (int64_t)sizeof(TB), row, a.gate ? bbytes : 0);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      rx[v].load(x, t + v * TPR);
      rb[v].load(b, t + v * TPR);
      if (a.gate) rg[v].load(g, t + v * TPR);
    }
  };
  int row = blockIdx.x, turn = 0;
  fetch(row);
  for (; row < a.rows; row += gridDim.x, turn ^= 1) {
    // columns and parameters of several runs anew for each row: kept over the rows they spill
    if (V > 1) asm volatile("" : "+v"(t));
    float x[V][4], u[V][4], g[V][4];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int valid = a.cols - 4 * (t + v * TPR);
      rx[v].get(x[v]);
      rb[v].get(u[v]);
      if (a.gate) rg[v].get(g[v]);
      // past the row: storage, or 0 past its last run
      mask4(x[v], valid);
      mask4(u[v], valid);
    }
    if (row + (int)gridDim.x < a.rows) fetch(row + (int)gridDim.x);
    // z <- its deviations from the mean; (mean, rstd). Only the two sums depend on the kind.
    auto moments = [&](float (&z)[V][4], const JoinNorm& k, float* buf0, float* buf1, float& mean,
                       float& rstd) __attribute__((always_inline)) {
      mean = 0.f;
      rstd = 1.f;
      if (k.kind == MAO_ROW_NORM_LAYER) {
        float s = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int i = 0; i < 4; ++i) s += z[v][i];
        mean = group_total<TPR>(s, buf0) * inv_n;
      }
      float q = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int valid = a.cols - 4 * (t + v * TPR);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          z[v][i] = i < valid ? z[v][i] - mean : 0.f;
          q += z[v][i] * z[v][i];
        }
      }
      if (k.kind != MAO_ROW_NORM_NONE)
        rstd = 1.f / sqrtf(group_total<TPR>(q, buf1) * inv_n + k.eps);
    };
    float m1, r1, m2, r2;
    moments(u, a.post, red[turn][0], red[turn][1], m1, r1);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = t + v * TPR, valid = a.cols - 4 * c, i0 = PRE ? v : 0;
      if constexpr (!PRE) params(v, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float w = u[v][i] * r1 * g1[i0][i] + b1[i0][i];
        w *= a.gate ? g[v][i] : gate[i0][i];
        x[v][i] = a.xs * x[v][i] + a.bs * w;
      }
      mask4(x[v], valid);
      store_run4<TX>(a.r, a.ldr, row, a.cols, c, x[v]);
    }
    moments(x, a.pre, red[turn][2], red[turn][3], m2, r2);
    if (a.h) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = t + v * TPR, i0 = PRE ? v : 0;
        if constexpr (!PRE) params(v, 0);
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = x[v][i] * r2 * g2[i0][i] + b2[i0][i];
        store_run4<TB>(a.h, a.ldh, row, a.cols, c, y);
      }
    }
    if (t == 0 && a.stats) *(float4*)(a.stats + 4 * (int64_t)row) = make_float4(m1, r1, m2, r2);
  }
}

template <typename TX, typename TB, int TPR, int V, int BLK>
__global__ __launch_bounds__(BLK) void join_bwd_kernel(JoinBackArgs a) {
  constexpr int RPB = BLK / TPR;
  constexpr int kJoin = RPB > 1 ? 4 * V * TPR : 1;
  __shared__ float2 red[2][2][BLK / 64];
  __shared__ float join[kJoin];
  // a wavefront has one row
  int t = threadIdx.x % TPR;
  const int sub = __builtin_amdgcn_readfirstlane(threadIdx.x / TPR);
  const float inv_n = 1.f / (float)a.cols;
  constexpr bool PRE = V == 1;  // parameters stay in registers
  constexpr int P = PRE ? V : 1;
  // the last one: the gate of each channel, or with gates of their own beta1
  float g1[P][4], g2[P][4], last[P][4];
  auto params = [&](int v, int i) __attribute__((always_inline)) {
    const int col = 4 * (t + v * TPR), valid = a.cols - col;
    load_param4(a.post.gamma, a.post.p_dtype, col, valid, 1.f, g1[i]);
    load_param4(a.pre.gamma, a.pre.p_dtype, col, valid, 1.f, g2[i]);
    if (a.gate)
      load_param4(a.post.beta, a.post.p_dtype, col, valid, 0.f, last[i]);
    else
      load_param4(a.gate_vec, a.gate_dtype, col, valid, 1.f, last[i]);
  };
  if constexpr (PRE) params(0, 0);
  float sums[4][V][4];  // A, D, dgamma2, dbeta2
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i) sums[k][v][i] = 0.f;
  const bool pre = a.pre.kind != MAO_ROW_NORM_NONE, post = a.post.kind != MAO_ROW_NORM_NONE;
  const float pre_mean = a.pre.kind == MAO_ROW_NORM_LAYER ? inv_n : 0.f;
  const float post_mean = a.post.kind == MAO_ROW_NORM_LAYER ? inv_n : 0.f;
  struct Row {
    Run4<TX> d[V], r[V];
    Run4<TB> dh[V], b[V], g[V];
    float4 st;
  };
  const int xbytes = run4_bytes<TX>(a.cols), bbytes = run4_bytes<TB>(a.cols);
  auto fetch = [&](Row& q, int row) __attribute__((always_inline)) {
    row = min(row, a.rows - 1);
    q.st = *(const float4*)(a.stats + 4 * (int64_t)row);
    const auto d = row_buffer(a.dr, a.lddr * (int64_t)sizeof(TX), row, a.dr ? xbytes : 0);
    const auto r = row_buffer(a.r, a.ldr * (int64_t)sizeof(TX), row, pre ? xbytes : 0);
    const auto dh = row_buffer(a.dh, a.lddh * (int64_t)sizeof(TB), row, pre ? bbytes : 0);
    const auto b = row_buffer(a.b, a.ldb * (int64_t)sizeof(TB), row, bbytes);
    const auto g = row_buffer(a.gate, a.ldgate * (int64_t)sizeof(TB), row, a.gate ? bbytes : 0);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = t + v * TPR;
      q.dh[v].load(dh, c);
      q.r[v].load(r, c);
      q.d[v].load(d, c);
      q.b[v].load(b, c);
      if (a.gate) q.g[v].load(g, c);
    }
  };
  auto handle = [&](Row& q, int row, float2 (*buf)[BLK / 64]) __attribute__((always_inline)) {
    const bool live = row < a.rows;
    const int lim = live ? a.cols : 0;
    float d[V][4];  // dr
    float s0 = 0.f, s1 = 0.f;
    // dh and xh2 of a run; zero past the row
    auto values = [&](int v, float (&dh)[4], float (&xh)[4]) __attribute__((always_inline)) {
      const int valid = lim - 4 * (t + v * TPR);
      q.dh[v].get(dh);
      q.r[v].get(xh);
#pragma unroll
      for (int i = 0; i < 4; ++i) xh[i] = (xh[i] - q.st.z) * q.st.w;
      mask4(dh, valid);
      mask4(xh, valid);
    };
    // without a norm after the sum dh, r and all that is made of them are 0
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float dh[4], xh[4];
      values(v, dh, xh);
      if constexpr (!PRE) params(v, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sums[2][v][i] += dh[i] * xh[i];
        sums[3][v][i] += dh[i];
        const float w = dh[i] * g2[PRE ? v : 0][i];
        s0 += w;
        s1 += w * xh[i];
      }
    }
    if (pre) group_total2<TPR>(s0, s1, buf[0]);
    s0 *= pre_mean;
    s1 *= inv_n;
    float p0 = 0.f, p1 = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = t + v * TPR, valid = lim - 4 * c, i0 = PRE ? v : 0;
      q.d[v].get(d[v]);  // 0 if there is none
      if constexpr (!PRE) params(v, 0);
      {
        float dh[4], xh[4];
        q.dh[v].opaque();
        q.r[v].opaque();
        values(v, dh, xh);
#pragma unroll
        for (int i = 0; i < 4; ++i) d[v][i] += q.st.w * (dh[i] * g2[i0][i] - s0 - xh[i] * s1);
      }
      mask4(d[v], valid);
      if (live) {
        float o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = a.xs * d[v][i];
        store_run4<TX>(a.dx, a.lddx, row, a.cols, c, o);
      }
      float xh[4], g[4];
      q.b[v].get(xh);
#pragma unroll
      for (int i = 0; i < 4; ++i) xh[i] = (xh[i] - q.st.x) * q.st.y;
      mask4(xh, valid);
      if (a.gate) {
        q.g[v].get(g);
        mask4(g, valid);
        if (live && a.dgate) {
          float o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = a.bs * d[v][i] * (xh[i] * g1[i0][i] + last[i0][i]);
          store_run4<TB>(a.dgate, a.lddgate, row, a.cols, c, o);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) d[v][i] *= g[i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sums[0][v][i] += d[v][i] * xh[i];
        sums[1][v][i] += d[v][i];
        if (!a.gate) d[v][i] *= last[i0][i];
        d[v][i] *= a.bs * g1[i0][i];  // p (du without a norm: gamma1 is 1 then)
        p0 += d[v][i];
        p1 += d[v][i] * xh[i];
      }
    }
    // without a norm of the block's output its gradient is p itself (mean 0, rstd 1)
    if (post) group_total2<TPR>(p0, p1, buf[1]);
    p0 *= post_mean;
    p1 *= post ? inv_n : 0.f;
    if (!live) return;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float o[4], xh[4];
      q.b[v].opaque();
      q.b[v].get(xh);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        o[i] = q.st.y * (d[v][i] - p0 - (post ? (xh[i] - q.st.x) * q.st.y * p1 : 0.f));
      store_run4<TB>(a.db, a.lddb, row, a.cols, t + v * TPR, o);
    }
  };
  const int step = gridDim.x * RPB;
  int r0 = blockIdx.x * RPB;
  // every thread of the block runs the same number of rounds (barriers inside)
  if constexpr (V > 1) {  // no registers for a second row
    Row q;
    for (int k = 0; r0 < a.rows; r0 += step, k ^= 1) {
      // columns and parameters anew for each row: kept over the rows they spill
      asm volatile("" : "+v"(t));
      fetch(q, r0 + sub);
      handle(q, r0 + sub, red[k]);
    }
  } else {
    Row q0, q1;
    fetch(q0, r0 + sub);
    while (true) {
      if (r0 + step < a.rows) fetch(q1, r0 + step + sub);
      handle(q0, r0 + sub, red[0]);
      r0 += step;
      if (r0 >= a.rows) break;
      if (r0 + step < a.rows) fetch(q0, r0 + step + sub);
      handle(q1, r0 + sub, red[1]);
      r0 += step;
      if (r0 >= a.rows) break;
    }
  }
  if (a.part == nullptr) return;
  // partial row of the workgroup: its row groups' sums in order 0, 1, ...
  float* out = a.part + (int64_t)blockIdx.x * 4 * a.cols;
#pragma unroll
  for (int which = 0; which < 4; ++which) {
    if constexpr (RPB > 1) {
      for (int k = 0; k < RPB - 1; ++k) {
        __syncthreads();
        if (sub == k) {
#pragma unroll
          for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float* p = &join[(v * 4 + i) * TPR + t];
              *p = k == 0 ? sums[which][v][i] : *p + sums[which][v][i];
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
        for (int i = 0; i < 4; ++i) {
          const float w = sums[which][v][i] + (RPB > 1 ? join[RPB > 1 ? (v * 4 + i) * TPR + t : 0] : 0.f);
          if (4 * c + i < a.cols) out[(int64_t)which * a.cols + 4 * c + i] = w;
        }
      }
    }
  }
}

// The join of the partial rows: 64 columns per workgroup, 16 wavefronts that each add every 16th
// row, joined in order. y = 0: A and D, y = 1: N2's parameters.
__global__ __launch_bounds__(1024) void join_sums_kernel(JoinBackArgs a, int blocks) {
  __shared__ float2 join[16][64];
  const bool second = blockIdx.y != 0;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = blockIdx.x * 64 + lane;
  float2 s = make_float2(0.f, 0.f);
  if (col < a.cols) {
    const float* p = a.part + (second ? 2 * (int64_t)a.cols : 0) + col;
    int b = wave;
    for (; b + 3 * 16 < blocks; b += 4 * 16) {
      float2 w[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float* q = p + (int64_t)(b + 16 * u) * 4 * a.cols;
        w[u] = make_float2(q[0], q[a.cols]);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        s.x += w[u].x;
        s.y += w[u].y;
      }
    }
    for (; b < blocks; b += 16) {
      const float* q = p + (int64_t)b * 4 * a.cols;
      s.x += q[0];
      s.y += q[a.cols];
    }
  }
  join[wave][lane] = s;
  __syncthreads();
  if (wave != 0 || col >= a.cols) return;
  s = make_float2(0.f, 0.f);
#pragma unroll
  for (int w = 0; w < 16; ++w) {
    s.x += join[w][lane].x;
    s.y += join[w][lane].y;
  }
  if (second) {
    if (a.dpre_gamma) a.dpre_gamma[col] = s.x;
    if (a.dpre_beta) a.dpre_beta[col] = s.y;
    return;
  }
  const float g = a.gate_vec ? load1_any(a.gate_vec, a.gate_dtype, col) : 1.f;
  if (a.dpost_gamma) a.dpost_gamma[col] = a.bs * g * s.x;
  if (a.dpost_beta) a.dpost_beta[col] = a.bs * g * s.y;
  if (a.dgate_vec) {
    const float gam = a.post.gamma ? load1_any(a.post.gamma, a.post.p_dtype, col) : 1.f;
    const float bet = a.post.beta ? load1_any(a.post.beta, a.post.p_dtype, col) : 0.f;
    a.dgate_vec[col] = a.bs * (gam * s.x + bet * s.y);
  }
}

// Threads per row and runs of 4 columns a thread.
struct JoinShape {
  int tpr, v;
};
JoinShape join_shape(int64_t cols) {
  if (cols <= 256) return {64, 1};
  if (cols <= 512) return {128, 1};
  if (cols <= 1024) return {256, 1};
  if (cols <= 2048) return {512, 1};
  return {1024, cols <= 4096 ? 1 : cols <= 8192 ? 2 : 4};
}
constexpr int bwd_block(int tpr) { return 1024 / tpr * tpr; }

template <typename TX, typename TB, int TPR, int V>
mao_status fwd_launch(const JoinArgs& a, hipStream_t s) {
  const int grid = std::min(a.rows, 256 * (2048 / TPR));
  hipLaunchKernelGGL((join_fwd_kernel<TX, TB, TPR, V>), dim3(grid), dim3(TPR), 0, s, a);
  MAO_LAUNCH_CHECK();
  return MAO_OK;
}

template <typename TX, typename TB, int TPR, int V>
mao_status bwd_launch(const JoinBackArgs& a, hipStream_t s) {
  constexpr int BLK = bwd_block(TPR);
  hipLaunchKernelGGL((join_bwd_kernel<TX, TB, TPR, V, BLK>), dim3(join_blocks(a.rows, a.cols)),
                     dim3(BLK), 0, s, a);
  MAO_LAUNCH_CHECK();
  return MAO_OK;
}

#define MAO_JOIN_PICK(NAME, GO, ARGS)                  \
  template <typename TX, typename TB>                  \
  mao_status NAME(const ARGS& a, hipStream_t s) {      \
    const JoinShape k = join_shape(a.cols);            \
    switch (k.tpr) {                                   \
      case 64: return GO<TX, TB, 64, 1>(a, s);         \
      case 128: return GO<TX, TB, 128, 1>(a, s);       \
      case 256: return GO<TX, TB, 256, 1>(a, s);       \
      case 512: return GO<TX, TB, 512, 1>(a, s);       \
      default: break;                                  \
    }                                                  \
    if (k.v == 1) return GO<TX, TB, 1024, 1>(a, s);    \
    if (k.v == 2) return GO<TX, TB, 1024, 2>(a, s);    \
    return GO<TX, TB, 1024, 4>(a, s);                  \
  }
MAO_JOIN_PICK(fwd_pick, fwd_launch, JoinArgs)
MAO_JOIN_PICK(bwd_pick, bwd_launch, JoinBackArgs)
#undef MAO_JOIN_PICK

}  // namespace

int join_blocks(int64_t rows, int64_t cols) {
  const int tpr = join_shape(cols).tpr;
  return (int)std::min<int64_t>(ceil_div(rows, bwd_block(tpr) / tpr), 256);
}

mao_status launch_join(const JoinArgs& a, int stream_type, int block_type, hipStream_t s) {
  if (stream_type == MAO_BF16)
    return block_type == MAO_BF16 ? fwd_pick<bf16_t, bf16_t>(a, s) : fwd_pick<bf16_t, float>(a, s);
  return block_type == MAO_BF16 ? fwd_pick<float, bf16_t>(a, s) : fwd_pick<float, float>(a, s);
}

mao_status launch_join_backward(const JoinBackArgs& a, int stream_type, int block_type,
                                hipStream_t s) {
  if (stream_type == MAO_BF16)
    MAO_TRY((block_type == MAO_BF16 ? bwd_pick<bf16_t, bf16_t>(a, s) : bwd_pick<bf16_t, float>(a, s)));
  else
    MAO_TRY((block_type == MAO_BF16 ? bwd_pick<float, bf16_t>(a, s) : bwd_pick<float, float>(a, s)));
  if (a.part == nullptr) return MAO_OK;
  hipLaunchKernelGGL(join_sums_kernel, dim3((int)ceil_div(a.cols, 64), 2), dim3(1024), 0, s, a,
                     join_blocks(a.rows, a.cols));
  MAO_LAUNCH_CHECK();
  return MAO_OK;
}

}  // namespace mao
