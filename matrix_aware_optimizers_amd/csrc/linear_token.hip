// The linear layer's forward product for up to 16 rows (decoded tokens): y = act(x W^T
// + b) + res.
//
// Bound: reading W once (one row, bf16, call after call on one stream: 1536 -> 6144 5.5 to
// 5.9 us, 3.6 of them the bytes at the copy rate and the rest the launch, 512 -> 512 takes
// 3.7; 4096 -> 14336 22.3 us, the copy rate; fp32 1536 -> 6144 10.7 us, 7.2 of them bytes.
// By itself, under the profiler, the first takes 6.5: neighbours in a stream overlap.) A
// workgroup takes 16 rows of W and all of K; its wavefronts take 256-byte blocks of those
// rows in turn, straight from memory into registers in the MFMA operand layout (16 x 16
// results: W rows x tokens, so a wavefront's load is 64 contiguous bytes of each of 16
// rows), the next block requested before the current one is multiplied. x is small and
// comes from L2. The wavefronts' sums are joined through LDS in a fixed order.
//
// 16 rows fill one MFMA result; the tile kernels take the rest. Timed against them
// (this kernel : tiles, us, bf16): 1536 -> 6144 1 row 5.9 : 11.4, 16 rows 7.5 : 11.4;
// 6144 -> 1536 8.9 : 10.7 and 12.7 : 11.5; 4096 -> 14336 22.3 : 39.2 and 33.3 : 39.5.
// Several results a wavefront, for up to 64 rows, read x again for every 16 rows of W:
// 32 rows 10.5 : 11.5, 18.5 : 11.3 and 52 : 40, 60 rows 17 : 12, 28 : 12 and 80 : 40.
// It won only between 17 and about 32 rows of the first of these shapes.
#include "act.hpp"
#include "layers.hpp"

#include <algorithm>

namespace mao {

namespace {

constexpr int kStep = 64;      // bytes of a row per MFMA step
constexpr int kSteps = 4;      // steps per block
constexpr int kBlockBytes = kStep * kSteps;

template <typename T>
__device__ __forceinline__ void mma16(const uint4& w, const uint4& x, f32x4_t& acc) {
  if constexpr (sizeof(T) == 2) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, w),
                                                  __builtin_bit_cast(bf16x8_t, x), acc, 0, 0, 0);
  } else {
    const uint32_t a[4] = {w.x, w.y, w.z, w.w}, b[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[e]), __uint_as_float(b[e]), acc,
                                                 0, 0, 0);
  }
}

// 16 bytes of a row from element k, zero from K on
template <typename T>
__device__ __forceinline__ uint4 load_masked(const T* row, int k, int K) {
  constexpr int EPC = 16 / (int)sizeof(T);
  union {
    uint4 v;
    T e[EPC];
  } u;
  u.v = make_uint4(0, 0, 0, 0);
  if (k + EPC <= K) {
    u.v = *(const uint4*)(row + k);
  } else {
#pragma unroll
    for (int i = 0; i < EPC; ++i)
      if (k + i < K) u.e[i] = row[k + i];
  }
  return u.v;
}

template <typename T, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void linear_token_kernel(LinProblem P) {
  constexpr int EPC = 16 / (int)sizeof(T), KSTEP = kStep / (int)sizeof(T);
  constexpr int KBLK = KSTEP * kSteps;
  __shared__ __attribute__((aligned(16))) float red[WAVES][256];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * 16;
  const T* wrow = (const T*)P.B + (int64_t)min(n0 + r, P.N - 1) * P.ldb;
  const T* xrow = (const T*)P.A + (int64_t)min(r, P.M - 1) * P.lda;
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};

  uint4 w[2][kSteps], x[2][kSteps];
  auto load = [&](int b, int s) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int k = b * KBLK + i * KSTEP + q * EPC;
      w[s][i] = *(const uint4*)(wrow + k);
      x[s][i] = *(const uint4*)(xrow + k);
    }
  };
  const int nb = P.K / KBLK;
  int b = wave;
  if (b < nb) load(b, 0);
  while (b < nb) {
    if (b + WAVES < nb) load(b + WAVES, 1);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) mma16<T>(w[0][i], x[0][i], acc);
    b += WAVES;
    if (b >= nb) break;
    if (b + WAVES < nb) load(b + WAVES, 0);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) mma16<T>(w[1][i], x[1][i], acc);
    b += WAVES;
  }
  // steps past the last whole block, one per wavefront in turn
  const int k1 = nb * KBLK;
  for (int t = wave; k1 + t * KSTEP < P.K; t += WAVES) {
    const int k = k1 + t * KSTEP + q * EPC;
    mma16<T>(load_masked(wrow, k, P.K), load_masked(xrow, k, P.K), acc);
  }
  *(float4*)&red[wave][lane * 4] = make_float4(acc[0], acc[1], acc[2], acc[3]);
  __syncthreads();
  // the first wavefront: lane l has columns n0 + 4 (l / 16) + 0..3 of row l % 16
  if (wave == 0) {
    const int row = r, col = n0 + 4 * q;
    if (row >= P.M || col >= P.N) return;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < WAVES; ++k) {
      const float4 t = *(const float4*)&red[k][lane * 4];
      v[0] += t.x;
      v[1] += t.y;
      v[2] += t.z;
      v[3] += t.w;
    }
    const LinEpilogue& e = P.e;
    const int n = min(4, P.N - col);
    auto put = [&](void* p, int dtype, int64_t off) {
      if (dtype == MAO_BF16) {
        bf16_t* d = (bf16_t*)p + off;
        if (n == 4) {
          *(uint2*)d = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i < n) d[i] = f32_to_bf16(v[i]);
        }
      } else {
        float* d = (float*)p + off;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < n) d[i] = v[i];
      }
    };
    if (e.bias) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) v[i] += load1_any(e.bias, e.bias_dtype, col + i);
    }
    if (e.z_out) put(e.z_out, e.zo_dtype, (int64_t)row * e.ldzo + col);
    act_apply(e.act, v);
    if (e.add) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) v[i] += load1_any(e.add, e.add_dtype, (int64_t)row * e.ldadd + col + i);
    }
    put(e.D, e.d_dtype, (int64_t)row * e.ldd + col);
  }
}

template <typename T>
mao_status go(const LinProblem& p, hipStream_t s) {
  const dim3 grid((int)ceil_div(p.N, 16));
  // from 32 blocks of K on, eight wavefronts (bf16, one row: 4096 -> 14336 25.0 -> 22.4
  // us); below, four (1536 -> 6144 6.3 against 6.4 us)
  if (p.K / (kBlockBytes / (int)sizeof(T)) >= 32)
    hipLaunchKernelGGL((linear_token_kernel<T, 8>), grid, dim3(512), 0, s, p);
  else
    hipLaunchKernelGGL((linear_token_kernel<T, 4>), grid, dim3(256), 0, s, p);
  MAO_LAUNCH_CHECK();
  return MAO_OK;
}

}  // namespace

mao_status launch_linear_token(int dtype, const LinProblem& p, hipStream_t s) {
  return dtype == MAO_BF16 ? go<bf16_t>(p, s) : go<float>(p, s);
}

}  // namespace mao
