// Column sums in two fixed-order stages (bias gradients, and the join of the
// partial rows that other kernels leave).
//
// Stage 1 reads the matrix once (HBM bound): a workgroup covers 512 columns
// (64 lanes x 8) of a band of rows, its four wavefronts take rows in turn and
// are joined in order. Stage 2 adds the bands' partial rows: 64 columns per
// workgroup, 16 wavefronts that each add every 16th partial row.
#include "layers.hpp"

#include <algorithm>

namespace mao {

namespace {

template <typename T>
__global__ __launch_bounds__(256) void column_partial_kernel(const T* x, int64_t ldx, int rows,
                                                             int cols, int band, float* part) {
  __shared__ float join[4][512];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;  // run of 8 columns
  const int r0 = blockIdx.y * band, r1 = min(rows, r0 + band);
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  if (8 * c < cols) {
    const T* p = x + 8 * c;
    int r = r0 + wave;
    for (; r + 12 < r1; r += 16) {
      Raw8<T> q[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) q[u].load(p + (int64_t)(r + 4 * u) * ldx);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        float v[8];
        q[u].get(v);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += v[i];
      }
    }
    for (; r < r1; r += 4) {
      Raw8<T> q;
      q.load(p + (int64_t)r * ldx);
      float v[8];
      q.get(v);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += v[i];
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) join[wave][i * 64 + lane] = acc[i];
  __syncthreads();
  for (int k = threadIdx.x; k < 512; k += 256) {
    const int col = blockIdx.x * 512 + k;
    const int j = (k & 7) * 64 + (k >> 3);
    if (col < cols)
      part[(int64_t)blockIdx.y * cols + col] = (join[0][j] + join[1][j]) + (join[2][j] + join[3][j]);
  }
}

__global__ __launch_bounds__(1024) void partial_sum_kernel(const float* part, int64_t stride,
                                                           int blocks, int cols, float* out0,
                                                           float* out1, int64_t off1,
                                                           int accumulate) {
  __shared__ float join[16][64];
  float* out = blockIdx.y ? out1 : out0;
  if (out == nullptr) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = blockIdx.x * 64 + lane;
  float t = 0.f;
  if (col < cols) {
    const float* p = part + (blockIdx.y ? off1 : 0) + col;
    int b = wave;
    for (; b + 7 * 16 < blocks; b += 8 * 16) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = p[(int64_t)(b + 16 * u) * stride];
#pragma unroll
      for (int u = 0; u < 8; ++u) t += v[u];
    }
    for (; b < blocks; b += 16) t += p[(int64_t)b * stride];
  }
  join[wave][lane] = t;
  __syncthreads();
  if (wave == 0 && col < cols) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 16; ++w) v += join[w][lane];
    out[col] = accumulate ? out[col] + v : v;
  }
}

}  // namespace

int column_sum_blocks(int64_t rows, int64_t cols) {
  // about four workgroups per CU, bands of at least 16 rows
  const int64_t strips = ceil_div(cols, 512);
  const int64_t want = std::max<int64_t>(1, 1024 / strips);
  const int64_t band = std::max<int64_t>(16, ceil_div(rows, want));
  return (int)ceil_div(rows, band);
}

mao_status launch_partial_sum(const float* part, int64_t stride, int blocks, int cols, float* out0,
                              float* out1, int64_t off1, int accumulate, hipStream_t s) {
  const dim3 grid((int)ceil_div(cols, 64), out1 ? 2 : 1);
  hipLaunchKernelGGL(partial_sum_kernel, grid, dim3(1024), 0, s, part, stride, blocks, cols, out0,
                     out1, off1, accumulate);
  MAO_LAUNCH_CHECK();
  return MAO_OK;
}

mao_status launch_column_sum(const void* x, int dtype, int64_t ldx, int rows, int cols,
                             float* part, float* out, int accumulate, hipStream_t s) {
  const int nb = column_sum_blocks(rows, cols);
  const int band = (int)ceil_div(rows, nb);
  const dim3 grid((int)ceil_div(cols, 512), nb);
  if (dtype == MAO_BF16)
    hipLaunchKernelGGL((column_partial_kernel<bf16_t>), grid, dim3(256), 0, s, (const bf16_t*)x,
                       ldx, rows, cols, band, part);
  else
    hipLaunchKernelGGL((column_partial_kernel<float>), grid, dim3(256), 0, s, (const float*)x, ldx,
                       rows, cols, band, part);
  MAO_LAUNCH_CHECK();
  return launch_partial_sum(part, cols, nb, cols, out, nullptr, 0, accumulate, s);
}

}  // namespace mao
