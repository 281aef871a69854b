// Launchers of the layer operators: layer norm, the linear layer, 8-bit
// activation checkpoints. Arguments are validated by the C entry points.
#pragma once

#include "common.hpp"
#include "q8.hpp"

namespace mao {

// Eight consecutive elements (16-byte aligned) as fp32. load_cut reads, of a run with
// `valid` elements of a row, only the 16-byte pieces that hold one (the first one
// twice): storage may end with the row, and a piece never crosses a page.
template <typename T> struct Raw8;
template <> struct Raw8<bf16_t> {
  uint4 a;
  __device__ __forceinline__ void load(const bf16_t* p) { a = *(const uint4*)p; }
  __device__ __forceinline__ void load_cut(const bf16_t* p, int /*valid*/) { load(p); }
  __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
  // the compiler may not carry values derived from here on across this point
  __device__ __forceinline__ void opaque() {
    asm volatile("" : "+v"(a.x), "+v"(a.y), "+v"(a.z), "+v"(a.w));
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <> struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *(const float4*)p;
    b = *(const float4*)(p + 4);
  }
  __device__ __forceinline__ void load_cut(const float* p, int valid) {
    a = *(const float4*)p;
    b = *(const float4*)(p + (valid > 4 ? 4 : 0));
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void opaque() {
    asm volatile("" : "+v"(a.x), "+v"(a.y), "+v"(a.z), "+v"(a.w));
    asm volatile("" : "+v"(b.x), "+v"(b.y), "+v"(b.z), "+v"(b.w));
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};

__device__ __forceinline__ void load8_any(const void* p, int dtype, int64_t off, float (&v)[8],
                                          int valid) {
  if (dtype == MAO_BF16) {
    Raw8<bf16_t> r;
    r.load((const bf16_t*)p + off);
    r.get(v);
  } else {
    Raw8<float> r;
    r.load_cut((const float*)p + off, valid);
    r.get(v);
  }
}

__device__ __forceinline__ float load1_any(const void* p, int dtype, int64_t off) {
  return dtype == MAO_BF16 ? bf16_to_f32(((const bf16_t*)p)[off]) : ((const float*)p)[off];
}

// Stores the first n (1..8) of v at element off; a whole run of 8 in 16-byte
// pieces.
__device__ __forceinline__ void store8n_any(void* p, int dtype, int64_t off, const float (&v)[8],
                                            int n) {
  if (dtype == MAO_BF16) {
    bf16_t* d = (bf16_t*)p + off;
    if (n >= 8) {
      uint4 k;
      k.x = pack_bf16x2(v[0], v[1]);
      k.y = pack_bf16x2(v[2], v[3]);
      k.z = pack_bf16x2(v[4], v[5]);
      k.w = pack_bf16x2(v[6], v[7]);
      *(uint4*)d = k;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) d[i] = f32_to_bf16(v[i]);
    }
  } else {
    float* d = (float*)p + off;
    if (n >= 8) {
      *(float4*)d = make_float4(v[0], v[1], v[2], v[3]);
      *(float4*)(d + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) d[i] = v[i];
    }
  }
}

// ---- layer norm (layer_norm.hip) -----------------------------------------
constexpr int64_t kNormMaxCols = 32768;

struct NormFwdArgs {
  const void* x;
  const void* gamma;  // or nullptr (1)
  const void* beta;   // or nullptr (0)
  void* y;
  float *mean, *rstd;  // or nullptr
  int64_t ldx, ldy;
  int rows, cols, p_dtype, y_dtype;
  float eps;
};
mao_status launch_norm_fwd(const NormFwdArgs& a, int x_dtype, hipStream_t s);

struct NormBwdArgs {
  const void* dy;
  const void* x;  // tensor, or the codes of a checkpoint
  const uint8_t* scales;
  const void* gamma;
  const float *mean, *rstd;
  const void* add;  // or nullptr
  void* dx;
  float *dgamma, *dbeta;  // or nullptr
  float* part;            // [blocks][2][cols] (nullptr without dgamma and dbeta)
  int64_t lddy, ldx, lds, ldadd, lddx;
  int rows, cols, p_dtype, add_dtype, dx_dtype;
};
// x_kind: MAO_F32, MAO_BF16, or kXInt8 / kXE4m3 for a checkpoint
enum { kXInt8 = 2, kXE4m3 = 3 };
int norm_bwd_blocks(int64_t rows, int64_t cols);
mao_status launch_norm_bwd(const NormBwdArgs& a, int dy_dtype, int x_kind, hipStream_t s);

// ---- join of partial column sums (partial_sum.hip) ----------------------------------------
// out0[j] (+)= sum_b part[b * stride + j]; out1 the same from part + off1. Either
// may be nullptr.
mao_status launch_partial_sum(const float* part, int64_t stride, int blocks, int cols, float* out0,
                              float* out1, int64_t off1, int accumulate, hipStream_t s);

// ---- 8-bit checkpoints (q8.hip) --------------------------------------------
mao_status launch_q8_quantize(const void* x, int dtype, int64_t ldx, int rows, int cols, Q8View q,
                              int fmt, hipStream_t s);
// rest: what rounding to bf16 leaves of each value instead of the value (0 where that
// rounding is not finite), so that value and rest together carry 16 bits of it.
mao_status launch_q8_dequantize(Q8View q, int fmt, int rows, int cols, int act, bool rest, void* y,
                                int dtype, int64_t ldy, hipStream_t s);

// y = act(x) or its rest, one dtype
mao_status launch_act(const void* x, int dtype, int64_t ldx, int rows, int cols, int act, bool rest,
                      void* y, int64_t ldy, hipStream_t s);

// ---- linear layer (linear.hip, linear_token.hip) ---------------------------
// What happens to a result before it is stored:
//   t = acc + bias[j]; z_out = t
//   t = act(t), or with slope_of t = acc * act'(z_in) (a tensor or checkpoint)
//   D = t + add
struct LinEpilogue {
  void* D;
  const void* bias;
  void* z_out;
  const void* z_in;       // tensor, or codes
  const uint8_t* z_scales;
  const void* add;
  int64_t ldd, ldzo, ldzi, ldzs, ldadd;
  int d_dtype, bias_dtype, zo_dtype, add_dtype, act;
  int z_kind;  // of z_in: MAO_F32, MAO_BF16, kXInt8, kXE4m3
};

// D[i][j] = sum_k A(i, k) B(j, k), M x N. a_km / b_km: the operand is stored
// K x M (K x N) instead of M x K (N x K).
struct LinProblem {
  const void *A, *B;
  int64_t lda, ldb;
  int M, N, K;
  int a_km, b_km;
  LinEpilogue e;
};
struct LinCut {
  int bm, bn, split;
};
LinCut lin_cut(int dtype, bool mixed, int64_t M, int64_t N, int64_t K);
size_t lin_workspace(int dtype, int64_t M, int64_t N, int64_t K);
// sums (weight gradient, or nullptr): lin_sum_rows x M floats that receive
// partial column sums of A.
int lin_sum_rows(int dtype, int64_t M, int64_t N, int64_t K);
mao_status launch_linear(int dtype, const LinProblem& p, void* ws, float* sums, hipStream_t s);

// Up to kTokenRows rows of X against W (N x K), both K-contiguous.
constexpr int kTokenRows = 16;
mao_status launch_linear_token(int dtype, const LinProblem& p, hipStream_t s);

}  // namespace mao
