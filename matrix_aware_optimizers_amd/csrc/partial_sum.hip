// The join of partial column sums (bias and norm-parameter gradients): 64 columns
// per workgroup, 16 wavefronts that each add every 16th partial row, joined in
// order. Bound by the launch and the latency of a few dependent loads: 4.1 us for 256
// rows of 2 x 1536 or 2 x 4096 columns (3.1 MB and 8.4 MB), 4.8 for 6144.
#include "layers.hpp"

namespace mao {

namespace {

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

mao_status launch_partial_sum(const float* part, int64_t stride, int blocks, int cols, float* out0,
                              float* out1, int64_t off1, int accumulate, hipStream_t s) {
  const dim3 grid((int)ceil_div(cols, 64), out1 ? 2 : 1);
  hipLaunchKernelGGL(partial_sum_kernel, grid, dim3(1024), 0, s, part, stride, blocks, cols, out0,
                     out1, off1, accumulate);
  MAO_LAUNCH_CHECK();
  return MAO_OK;
}

}  // namespace mao
