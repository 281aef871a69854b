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
// Bound: HBM, each matrix once; with few rows the launch, backward two of them. A row lives in
// the registers of its threads (one to four runs of 4 columns each), so that a deviation is one
// from the row's own mean; the next row's loads are issued before the current one is reduced.
// h is made from r as it is in fp32, before it is rounded to be stored.
//
// With a gate per channel (or none) its gradient and those of N1's parameters need two column
// sums: A = sum dr xh1 and D = sum dr give dgamma1 = bs gate A, dbeta1 = bs gate D and
// dgate = bs (gamma1 A + beta1 D). With a gate per element A and D are sums of gate . dr.
// Sums stay in registers over the rows of a workgroup, are joined in it in order, and
// leave as one partial row; a second kernel adds those in order. No atomics, fp32.
//
// Measured (bf16, both norms; a copy of 1 GiB reaches 5.2 TB/s): forward 16384 x 1536 40 us on
// resident inputs (5.0 TB/s), 8192 x 4096 57 (4.7), 2048 x 16384 69 (3.9), one row of 1536 7 (host
// time; the kernel is 4.2 to 4.4 under the profiler). Backward 16384 x 1536 68 us (4.5 TB/s, 4 of
// them the second kernel), 8192 x 4096 86 (4.7), 4093 x 4096 with an fp32 stream and gates 76 (4.9),
// 4096 x 8192 with gates 116 (4.6), 2048 x 16384 172 (2.3: 128 registers a thread are full,
// parameters come from the L2 for each row; loads of a row held from its first pass to its
// second spilt more). One row of 1536 13 (kernels 7.4 and 2.6, the rest host time).
// Forms of 1024 threads that spill, of their 128 registers (stream, block): backward above 8192
// columns 4 to 11 in all types, 6145 to 8192 10 (bf16, fp32) and 20 (both fp32); forward above 8192
// 4 and 11 of the same two. Two rms norms, forward and backward, bf16 / fp32 stream / fp32 block /
// both fp32: 4096 x 8192 59 and 93 us / 81 and 126 / 81 and 128 / 98 and 171 (4.6 to 5.5 TB/s, 4.3 to
// 4.8); 2048 x 12288 59 and 133 / 73 and 158 / 79 and 172 / 108 and 198 (3.4 to 4.1, 2.3 to 3.1);
// 2048 x 16384 65 and 171 / 90 and 194 / 99 and 209 / 127 and 240 (4.0 to 4.5, 2.3 to 3.4).
#include "rows.hpp"

#include <algorithm>

namespace mao {

namespace {

// Large results go past the caches. Measured on both sides, us, through them / past them, two rms
// norms forward (with a reading of h right after): bf16 2048 x 1536 8.3 / 6.9 (12.6 / 11.5), 5461 x
// 1536, the limit, 17.4 / 15.6 (23.6 / 23.7), 16384 x 1536 41.3 / 35.7 (56.6 / 59.9), 8192 x 4096
// 63.4 / 55.3 (85.4 / 90.6); fp32 5461 x 1536 20.9 / 20.9 (31.2 / 34.0), 16384 x 1536 76.1 / 73.4
// (109.7 / 117.3). Backward 16384 x 1536 bf16 67.4 / 60.4 (with a reading of dB 84.5 / 86.2), 2048 x
// 4096, the limit, 28.9 / 29.4 (34.8 / 36.9). So the call gains up to 14%, and a next reader pays that
// back and up to 9% of the two on top. The limit is the size at which two bf16 results fill the
// L2s (32 MB); no size divides gain from loss.
__device__ __forceinline__ bool past_l2(int rows, int cols) {
  return (int64_t)rows * cols >= (int64_t)1 << 23;
}

// Parameter vectors of a workgroup in LDS, as fp32 (LDS: up to 6144 columns forward, 8192
// backward; rows of a CU read them from there instead of holding 5 values a column in
// registers), in registers, or read where they are.
struct Vector {
  const void* p;  // or nullptr: dflt
  int dtype;
  float dflt;
};
template <int N, int COLS, int BLK>
__device__ __forceinline__ void stage(const Vector (&from)[N], int cols, float (*to)[COLS]) {
  constexpr int K = (COLS + BLK - 1) / BLK;
  uint32_t raw[N][K];
  // all loads first, conversions after
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (int)threadIdx.x + k * BLK;
      raw[n][k] = 0;
      if (from[n].p && c < cols)
        raw[n][k] = from[n].dtype == MAO_BF16 ? ((const bf16_t*)from[n].p)[c]
                                              : ((const uint32_t*)from[n].p)[c];
    }
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (int)threadIdx.x + k * BLK;
      const uint32_t u = from[n].dtype == MAO_BF16 ? raw[n][k] << 16 : raw[n][k];
      if (c < COLS) to[n][c] = from[n].p ? __uint_as_float(u) : from[n].dflt;
    }
}
// Where a kernel has its vectors: a thread with one run of columns keeps their values, and one with
// two where LDS has no room for them (forward 4096 x 8192 bf16 80 us, read for each row 90;
// 6106 x 8187 from fp32 113 for 157).
enum { kInRegisters, kInLds, kInMemory };
constexpr int vectors_at(int v, bool lds) {
  return v == 1 ? kInRegisters : lds ? kInLds : v == 2 ? kInRegisters : kInMemory;
}

template <bool LDS>
__device__ __forceinline__ void vector4(const Vector& from, const float* staged, int run, int cols,
                                        float (&v)[4]) {
  if constexpr (LDS) {
    const float4 k = *(const float4*)(staged + 4 * run);
    v[0] = k.x;
    v[1] = k.y;
    v[2] = k.z;
    v[3] = k.w;
  } else {
    load_param4(from.p, from.dtype, 4 * run, cols - 4 * run, from.dflt, v);
  }
}

template <typename TX, typename TB, int TPR, int V, int BLK, bool LDS>
__global__ __launch_bounds__(BLK) void join_fwd_kernel(JoinArgs a) {
  constexpr int RPB = BLK / TPR, COLS = 4 * TPR * V;
  __shared__ float red[2][4][BLK / 64];
  constexpr bool STAGED = vectors_at(V, LDS) == kInLds;
  __shared__ float vecs[STAGED ? 5 : 1][STAGED ? COLS : 1];
  // a wavefront has one row
  const int sub = __builtin_amdgcn_readfirstlane(threadIdx.x / TPR);
  int t = threadIdx.x % TPR;
  const float inv_n = 1.f / (float)a.cols;
  const bool past = past_l2(a.rows, a.cols);
  const Vector from[5] = {{a.post.gamma, a.post.p_dtype, 1.f}, {a.post.beta, a.post.p_dtype, 0.f},
                          {a.gate_vec, a.gate_dtype, 1.f}, {a.pre.gamma, a.pre.p_dtype, 1.f},
                          {a.pre.beta, a.pre.p_dtype, 0.f}};
  constexpr int AT = vectors_at(V, LDS);
  float held[AT == kInRegisters ? 5 : 1][AT == kInRegisters ? V : 1][4];
  auto vec = [&](int n, int v, float (&w)[4]) __attribute__((always_inline)) {
    if constexpr (AT == kInRegisters) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = held[AT == kInRegisters ? n : 0][AT == kInRegisters ? v : 0][i];
    } else {
      vector4<AT == kInLds>(from[n], vecs[AT == kInLds ? n : 0], t + v * TPR, a.cols, w);
    }
  };
  Run4<TX> rx[V];
  Run4<TB> rb[V], rg[V];
  const int xbytes = run4_bytes<TX>(a.cols), bbytes = run4_bytes<TB>(a.cols);
  auto fetch = [&](int row) __attribute__((always_inline)) {
    const bool live = row < a.rows;
    const auto x = row_buffer(a.x, a.ldx * (int64_t)sizeof(TX), row, live ? xbytes : 0);
    const auto b = row_buffer(a.b, a.ldb * (int64_t)sizeof(TB), row, live ? bbytes : 0);
    const auto g = row_buffer(a.gate, a.ldgate * (int64_t)sizeof(TB), row, live && a.gate ? bbytes : 0);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      rx[v].load(x, t + v * TPR);
      rb[v].load(b, t + v * TPR);
      if (a.gate) rg[v].load(g, t + v * TPR);
    }
  };
  const int step = gridDim.x * RPB;
  int r0 = blockIdx.x * RPB, turn = 0;
  fetch(r0 + sub);
  if constexpr (AT == kInLds) {
    stage<5, COLS, BLK>(from, a.cols, vecs);
    __syncthreads();
  }
  if constexpr (AT == kInRegisters) {
#pragma unroll
    for (int n = 0; n < 5; ++n)
#pragma unroll
      for (int v = 0; v < V; ++v) vector4<false>(from[n], nullptr, t + v * TPR, a.cols, held[n][v]);
  }
  // every thread of the block runs the same number of rounds (barriers inside)
  for (; r0 < a.rows; r0 += step, turn ^= 1) {
    // columns anew for each row: kept over the rows they spill
    if (V > 1) asm volatile("" : "+v"(t));
    const int row = r0 + sub;
    const bool live = row < a.rows;
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
    if (r0 + step < a.rows) fetch(row + step);
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
      const int c = t + v * TPR, valid = a.cols - 4 * c;
      float g1[4], b1[4], gate[4];
      vec(0, v, g1);
      vec(1, v, b1);
      vec(2, v, gate);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float w = (u[v][i] * r1 * g1[i] + b1[i]) * (a.gate ? g[v][i] : gate[i]);
        x[v][i] = a.xs * x[v][i] + a.bs * w;
      }
      mask4(x[v], valid);
      if (live) store_run4<TX>(a.r, a.ldr, row, a.cols, c, x[v], past);
    }
    moments(x, a.pre, red[turn][2], red[turn][3], m2, r2);
    if (!live) continue;
    if (a.h) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float g2[4], b2[4], y[4];
        vec(3, v, g2);
        vec(4, v, b2);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = x[v][i] * r2 * g2[i] + b2[i];
        store_run4<TB>(a.h, a.ldh, row, a.cols, t + v * TPR, y, past);
      }
    }
    if (t == 0 && a.stats) *(float4*)(a.stats + 4 * (int64_t)row) = make_float4(m1, r1, m2, r2);
  }
}

template <typename TX, typename TB, int TPR, int V, int BLK, bool LDS>
__global__ __launch_bounds__(BLK) void join_bwd_kernel(JoinBackArgs a) {
  constexpr int RPB = BLK / TPR, COLS = 4 * TPR * V;
  __shared__ float2 red[2][2][BLK / 64];
  // parameters (the last one: the gate of each channel, or with gates of their own beta1)
  constexpr int AT = vectors_at(V, LDS);
  __shared__ float vecs[AT == kInLds ? 3 : 1][AT == kInLds ? COLS : 1];
  // a wavefront has one row
  int t = threadIdx.x % TPR;
  const int sub = __builtin_amdgcn_readfirstlane(threadIdx.x / TPR);
  const float inv_n = 1.f / (float)a.cols;
  const bool past = past_l2(a.rows, a.cols);
  const Vector from[3] = {{a.post.gamma, a.post.p_dtype, 1.f}, {a.pre.gamma, a.pre.p_dtype, 1.f},
                          {a.gate ? a.post.beta : a.gate_vec, a.gate ? a.post.p_dtype : a.gate_dtype,
                           a.gate ? 0.f : 1.f}};
  float held[AT == kInRegisters ? 3 : 1][AT == kInRegisters ? V : 1][4];
  auto vec = [&](int n, int v, float (&w)[4]) __attribute__((always_inline)) {
    if constexpr (AT == kInRegisters) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = held[AT == kInRegisters ? n : 0][AT == kInRegisters ? v : 0][i];
    } else {
      vector4<AT == kInLds>(from[n], vecs[AT == kInLds ? n : 0], t + v * TPR, a.cols, w);
    }
  };
  // A, D, dgamma2, dbeta2. With four runs a thread the last two are in LDS, each thread's its
  // own (2048 x 16384 bf16 180 us; in registers, which spilt, 341).
  constexpr bool HALF = V > 2;
  constexpr int S = HALF ? 2 : 4;
  __shared__ float rest[HALF ? 2 : 1][HALF ? COLS : 1];
  float sums[S][V][4];
  if constexpr (HALF) {
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int k = 0; k < 2; ++k)
        *(float4*)&rest[k][4 * (t + v * TPR)] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
#pragma unroll
  for (int k = 0; k < S; ++k)
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i) sums[k][v][i] = 0.f;
  const bool pre = a.pre.kind != MAO_ROW_NORM_NONE, post = a.post.kind != MAO_ROW_NORM_NONE;
  const bool pre_mean = a.pre.kind == MAO_ROW_NORM_LAYER;
  const bool post_mean = a.post.kind == MAO_ROW_NORM_LAYER;
  // One row in its stored form; a run of the next row is on its way as soon as this row's has
  // been used for the last time. (KEEP; else no registers are left for it, and each run is
  // loaded, from the cache after the first time, where it is used.)
  constexpr bool KEEP = V <= 2;
  constexpr int Q = KEEP ? V : 1;
  Run4<TX> qd[Q], qr[Q];
  Run4<TB> qh[Q], qb[Q], qg[Q];
  float4 st, next_st;
  const int xbytes = run4_bytes<TX>(a.cols), bbytes = run4_bytes<TB>(a.cols);
  struct Bufs {
    __amdgpu_buffer_rsrc_t d, r, dh, b, g;
  };
  auto buffers = [&](int row) __attribute__((always_inline)) {
    return Bufs{row_buffer(a.dr, a.lddr * (int64_t)sizeof(TX), row, a.dr ? xbytes : 0),
                row_buffer(a.r, a.ldr * (int64_t)sizeof(TX), row, pre ? xbytes : 0),
                row_buffer(a.dh, a.lddh * (int64_t)sizeof(TB), row, pre ? bbytes : 0),
                row_buffer(a.b, a.ldb * (int64_t)sizeof(TB), row, bbytes),
                row_buffer(a.gate, a.ldgate * (int64_t)sizeof(TB), row, a.gate ? bbytes : 0)};
  };
  auto fetch = [&](int row) __attribute__((always_inline)) {  // all but b
    row = min(row, a.rows - 1);
    next_st = *(const float4*)(a.stats + 4 * (int64_t)row);
    if constexpr (KEEP) {
      const Bufs f = buffers(row);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        qh[v].load(f.dh, t + v * TPR);
        qr[v].load(f.r, t + v * TPR);
        qd[v].load(f.d, t + v * TPR);
        if (a.gate) qg[v].load(f.g, t + v * TPR);
      }
    }
  };
  auto fetch_b = [&](int row) __attribute__((always_inline)) {
    if constexpr (KEEP) {
      const Bufs f = buffers(min(row, a.rows - 1));
#pragma unroll
      for (int v = 0; v < V; ++v) qb[v].load(f.b, t + v * TPR);
    }
  };
  auto handle = [&](int row, int next, float2 (*buf)[BLK / 64]) __attribute__((always_inline)) {
    if (V > 1) asm volatile("" : "+v"(t));
    const bool live = row < a.rows;
    st = next_st;
    const Bufs now = buffers(min(row, a.rows - 1));
    const int lim = live ? a.cols : 0;
    float d[V][4];  // dr
    float s0 = 0.f, s1 = 0.f;
    // dh and xh2 of a run; zero past the row
    auto values = [&](int v, float (&dh)[4], float (&xh)[4]) __attribute__((always_inline)) {
      const int valid = lim - 4 * (t + v * TPR), i0 = KEEP ? v : 0;
      if constexpr (!KEEP) {
        __builtin_amdgcn_sched_barrier(0);  // one run's registers at a time
        qh[0].load(now.dh, t + v * TPR);
        qr[0].load(now.r, t + v * TPR);
      }
      qh[i0].get(dh);
      qr[i0].get(xh);
#pragma unroll
      for (int i = 0; i < 4; ++i) xh[i] = (xh[i] - st.z) * st.w;
      mask4(dh, valid);
      mask4(xh, valid);
    };
    // without a norm after the sum dh, r and all that is made of them are 0
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float dh[4], xh[4], g2[4];
      values(v, dh, xh);
      vec(1, v, g2);
      if constexpr (HALF) {
        float4* p0 = (float4*)&rest[0][4 * (t + v * TPR)];
        float4* p1 = (float4*)&rest[HALF ? 1 : 0][4 * (t + v * TPR)];
        float4 k0 = *p0, k1 = *p1;
        k0.x += dh[0] * xh[0];
        k0.y += dh[1] * xh[1];
        k0.z += dh[2] * xh[2];
        k0.w += dh[3] * xh[3];
        k1.x += dh[0];
        k1.y += dh[1];
        k1.z += dh[2];
        k1.w += dh[3];
        *p0 = k0;
        *p1 = k1;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sums[S - 2][v][i] += dh[i] * xh[i];
          sums[S - 1][v][i] += dh[i];
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float w = dh[i] * g2[i];
        s0 += w;
        s1 += w * xh[i];
      }
    }
    if (pre) group_total2<TPR>(s0, s1, buf[0]);
    s0 = pre_mean ? s0 * inv_n : 0.f;  // chosen, not times 0: the sum may be infinite
    s1 *= inv_n;
    float p0 = 0.f, p1 = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = t + v * TPR, valid = lim - 4 * c;
      float g1[4], last[4];
      const int i0 = KEEP ? v : 0;
      if constexpr (!KEEP) {
        qd[0].load(now.d, c);
        qb[0].load(now.b, c);
        if (a.gate) qg[0].load(now.g, c);
      }
      qd[i0].get(d[v]);  // 0 if there is none
      {
        float dh[4], xh[4], g2[4];
        qh[i0].opaque();
        qr[i0].opaque();
        values(v, dh, xh);
        vec(1, v, g2);
#pragma unroll
        for (int i = 0; i < 4; ++i) d[v][i] += st.w * (dh[i] * g2[i] - s0 - xh[i] * s1);
      }
      mask4(d[v], valid);
      if (live) {
        float o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = a.xs * d[v][i];
        store_run4<TX>(a.dx, a.lddx, row, a.cols, c, o, past);
      }
      vec(0, v, g1);
      vec(2, v, last);
      float xh[4], g[4];
      qb[i0].get(xh);
#pragma unroll
      for (int i = 0; i < 4; ++i) xh[i] = (xh[i] - st.x) * st.y;
      mask4(xh, valid);
      if (a.gate) {
        qg[i0].get(g);
        mask4(g, valid);
        if (live && a.dgate) {
          float o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = a.bs * d[v][i] * (xh[i] * g1[i] + last[i]);
          store_run4<TB>(a.dgate, a.lddgate, row, a.cols, c, o, past);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) d[v][i] *= g[i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sums[0][v][i] += d[v][i] * xh[i];
        sums[1][v][i] += d[v][i];
        if (!a.gate) d[v][i] *= last[i];
        d[v][i] *= a.bs * g1[i];  // p (du without a norm: gamma1 is 1 then)
        p0 += d[v][i];
        p1 += d[v][i] * xh[i];
      }
    }
    fetch(next);
    // without a norm of the block's output its gradient is p itself (mean 0, rstd 1)
    if (post) group_total2<TPR>(p0, p1, buf[1]);
    p0 = post_mean ? p0 * inv_n : 0.f;
    p1 *= inv_n;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i0 = KEEP ? v : 0;
      float o[4], xh[4];
      if constexpr (!KEEP) {
        __builtin_amdgcn_sched_barrier(0);
        qb[0].load(now.b, t + v * TPR);
      }
      qb[i0].opaque();
      qb[i0].get(xh);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        o[i] = st.y * (d[v][i] - p0 - (post ? (xh[i] - st.x) * st.y * p1 : 0.f));
      if (live) store_run4<TB>(a.db, a.lddb, row, a.cols, t + v * TPR, o, past);
    }
    fetch_b(next);
  };
  const int step = gridDim.x * RPB;
  int r0 = blockIdx.x * RPB;
  fetch(r0 + sub);
  fetch_b(r0 + sub);
  if constexpr (AT == kInLds) {
    stage<3, COLS, BLK>(from, a.cols, vecs);
    __syncthreads();
  }
  if constexpr (AT == kInRegisters) {
#pragma unroll
    for (int n = 0; n < 3; ++n)
#pragma unroll
      for (int v = 0; v < V; ++v) vector4<false>(from[n], nullptr, t + v * TPR, a.cols, held[n][v]);
  }
  // every thread of the block runs the same number of rounds (barriers inside)
  for (int k = 0; r0 < a.rows; r0 += step, k ^= 1) handle(r0 + sub, r0 + step + sub, red[k]);
  if (a.part == nullptr) return;
  // partial row of the workgroup: its row groups' sums in order 0, 1, ...
  float* out = a.part + (int64_t)blockIdx.x * 4 * a.cols;
#pragma unroll
  for (int which = 0; which < 4; ++which) {
    if constexpr (RPB > 1) {
      __shared__ float join[RPB][COLS];
      if (which > 0) __syncthreads();
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float(&w)[4] = sums[which < S ? which : 0][v];
        *(float4*)&join[sub][4 * (t + v * TPR)] = make_float4(w[0], w[1], w[2], w[3]);
      }
      __syncthreads();
      for (int c = threadIdx.x; c < a.cols; c += BLK) {
        float w = join[0][c];
#pragma unroll
        for (int k = 1; k < RPB; ++k) w += join[k][c];
        out[(int64_t)which * a.cols + c] = w;
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = t + v * TPR;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float w = HALF && which >= 2 ? rest[HALF ? which - 2 : 0][HALF ? 4 * c + i : 0]
                                             : sums[which < S ? which : 0][v][i];
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
    float w = gam * s.x;
    if (a.post.beta) w += load1_any(a.post.beta, a.post.p_dtype, col) * s.y;  // s.y may be infinite
    a.dgate_vec[col] = a.bs * w;
  }
}

// Threads of a row. bf16: several runs of 8 bytes a thread, so that the reductions of a row
// cost fewer instructions a column; fp32 (a stream or block in it): one run of 16 bytes.
// Forward, us (runs x threads, in workgroups of): 16384 x 1536 bf16 3 x 128 in 512 39.2, in 256 43,
// in 1024 50, 6 x 64 42, 2 x 192 52, 1 x 384 45; with an fp32 stream and one norm 1 x 384 in 768 47,
// 3 x 128 50; 8192 x 4096 bf16 2 x 512 in 1024 59, 4 x 256 63, 1 x 1024 69; 8192 x 6144 bf16 3 x 512
// in 1024 102, 2 x 768 122, 2 x 1024 143; 4096 x 5120 fp32 2 x 768 80, 2 x 1024 82; 8192 x 2560 bf16
// 2 x 320 in 640 43, in 960 44, 2 x 512 59; 16384 x 768 bf16 3 x 64 21, 1 x 192 25, 2 x 128 26.
// Backward: 16384 x 1536 bf16 2 x 192 68, 1 x 384 82, 3 x 128 185 (spills); fp32 1 x 384 112, 2 x 192
// 138. 4093 x 4096 with an fp32 stream and gates 1 x 1024 76, 2 x 512 94. 8192 x 6144 bf16 2 x 768
// 139, 2 x 1024 155; 4096 x 5120 fp32 104 and 130; 8192 x 2560 bf16 2 x 320 61, 2 x 512 76, fp32
// 1 x 640 99, 1 x 1024 103; 16384 x 768 bf16 1 x 192 36, 2 x 128 43, fp32 1 x 192 62, 1 x 256 61.
template <typename TX, typename TB> constexpr bool kAllBf16 = sizeof(TX) + sizeof(TB) == 4;

constexpr int fwd_block(int tpr) {
  return tpr % 192 == 0 ? 768 : tpr == 320 ? 640 : tpr >= 512 ? 1024 : 512;
}
constexpr int bwd_block(int tpr) { return 1024 / tpr * tpr; }  // few partial rows

template <typename TX, typename TB, int TPR, int V, bool LDS>
mao_status fwd_launch(const JoinArgs& a, hipStream_t s) {
  constexpr int BLK = fwd_block(TPR);
  const int grid = (int)std::min<int64_t>(ceil_div(a.rows, BLK / TPR), 256 * (2048 / BLK));
  hipLaunchKernelGGL((join_fwd_kernel<TX, TB, TPR, V, BLK, LDS>), dim3(grid), dim3(BLK), 0, s, a);
  MAO_LAUNCH_CHECK();
  return MAO_OK;
}

template <typename TX, typename TB>
mao_status fwd_pick(const JoinArgs& a, hipStream_t s) {
  if constexpr (kAllBf16<TX, TB>) {
    if (a.cols <= 256) return fwd_launch<TX, TB, 64, 1, true>(a, s);
    if (a.cols <= 512) return fwd_launch<TX, TB, 64, 2, true>(a, s);
    if (a.cols <= 768) return fwd_launch<TX, TB, 64, 3, true>(a, s);
    if (a.cols <= 1024) return fwd_launch<TX, TB, 128, 2, true>(a, s);
    if (a.cols <= 1536) return fwd_launch<TX, TB, 128, 3, true>(a, s);
    if (a.cols <= 2048) return fwd_launch<TX, TB, 256, 2, true>(a, s);
    if (a.cols <= 2560) return fwd_launch<TX, TB, 320, 2, true>(a, s);
    if (a.cols <= 4096) return fwd_launch<TX, TB, 512, 2, true>(a, s);
    if (a.cols <= 6144) return fwd_launch<TX, TB, 512, 3, true>(a, s);
  } else {
    if (a.cols <= 256) return fwd_launch<TX, TB, 64, 1, true>(a, s);
    if (a.cols <= 512) return fwd_launch<TX, TB, 128, 1, true>(a, s);
    if (a.cols <= 768) return fwd_launch<TX, TB, 192, 1, true>(a, s);
    if (a.cols <= 1024) return fwd_launch<TX, TB, 256, 1, true>(a, s);
    if (a.cols <= 1536) return fwd_launch<TX, TB, 384, 1, true>(a, s);
    if (a.cols <= 2048) return fwd_launch<TX, TB, 512, 1, true>(a, s);
    if (a.cols <= 4096) return fwd_launch<TX, TB, 1024, 1, true>(a, s);
    if (a.cols <= 6144) return fwd_launch<TX, TB, 768, 2, false>(a, s);
  }
  if (a.cols <= 8192) return fwd_launch<TX, TB, 1024, 2, false>(a, s);
  return fwd_launch<TX, TB, 1024, 4, false>(a, s);
}

int bwd_threads(bool all_bf16, int64_t cols) {
  if (cols <= 256) return 64;
  if (cols > 512 && cols <= 768) return 192;
  if (cols > 4096) return cols <= 6144 ? 768 : 1024;
  const int t = cols <= 512    ? 64
                : cols <= 1024 ? 128
                : cols <= 1536 ? 192
                : cols <= 2048 ? 256
                : cols <= 2560 ? 320
                               : 512;
  return all_bf16 ? t : 2 * t;
}

template <typename TX, typename TB, int TPR, int V, bool LDS>
mao_status bwd_launch(const JoinBackArgs& a, hipStream_t s) {
  constexpr int BLK = bwd_block(TPR);
  const int grid = join_blocks(kAllBf16<TX, TB>, a.rows, a.cols);
  hipLaunchKernelGGL((join_bwd_kernel<TX, TB, TPR, V, BLK, LDS>), dim3(grid), dim3(BLK), 0, s, a);
  MAO_LAUNCH_CHECK();
  return MAO_OK;
}

template <typename TX, typename TB>
mao_status bwd_pick(const JoinBackArgs& a, hipStream_t s) {
  constexpr bool H = kAllBf16<TX, TB>;
  constexpr int V = H ? 2 : 1, M = H ? 1 : 2;
  if (a.cols <= 256) return bwd_launch<TX, TB, 64, 1, true>(a, s);
  if (a.cols <= 512) return bwd_launch<TX, TB, 64 * M, V, true>(a, s);
  if (a.cols <= 768) return bwd_launch<TX, TB, 192, 1, true>(a, s);
  if (a.cols <= 1024) return bwd_launch<TX, TB, 128 * M, V, true>(a, s);
  if (a.cols <= 1536) return bwd_launch<TX, TB, 192 * M, V, true>(a, s);
  if (a.cols <= 2048) return bwd_launch<TX, TB, 256 * M, V, true>(a, s);
  if (a.cols <= 2560) return bwd_launch<TX, TB, 320 * M, V, true>(a, s);
  if (a.cols <= 4096) return bwd_launch<TX, TB, 512 * M, V, true>(a, s);
  if (a.cols <= 6144) return bwd_launch<TX, TB, 768, 2, true>(a, s);
  if (a.cols <= 8192) return bwd_launch<TX, TB, 1024, 2, true>(a, s);
  return bwd_launch<TX, TB, 1024, 4, false>(a, s);
}

}  // namespace

int join_blocks(bool all_bf16, int64_t rows, int64_t cols) {
  const int tpr = bwd_threads(all_bf16, cols);
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
                     join_blocks(stream_type == MAO_BF16 && block_type == MAO_BF16, a.rows, a.cols));
  MAO_LAUNCH_CHECK();
  return MAO_OK;
}

}  // namespace mao
