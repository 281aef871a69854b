// Adds the fp32 partial results of a product whose K was split, in a fixed order,
// and finishes them as the tile kernels do: eight columns of a row per thread,
// one pass over the partial results, bound by reading them from the caches. 77 rows of
// 1536 columns in 16 parts take 5 us, most of it the launch; 6144 x 1536 in 3 parts
// 27 us (113 MB of them, and 38 MB of fp32 results: 5.6 TB/s).
#include "act.hpp"
#include "linear.hpp"

namespace mao {

namespace {

__global__ __launch_bounds__(256) void linear_join_kernel(LinProblem P, const float* part,
                                                          int64_t ldpart, int split, int slope,
                                                          int nch) {
  const int64_t w = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int row = (int)(w / nch), col = (int)(w - (int64_t)row * nch) * 8;
  if (row >= P.M) return;
  const LinEpilogue& e = P.e;
  const int valid = P.N - col;
  const float* p = part + (int64_t)row * ldpart + col;
  const int64_t step = (int64_t)P.M * ldpart;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = 0; s < split; ++s) {
    const float4 a = *(const float4*)(p + s * step), b = *(const float4*)(p + s * step + 4);
    v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
    v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
  }
  if (slope) {
    if (e.act != MAO_ACT_NONE) {
      float z[8];
      const int64_t off = (int64_t)row * e.ldzi + col;
      if (e.z_kind <= MAO_BF16) {
        load8_any(e.z_in, e.z_kind, off, z, valid);
      } else {
        const uint2 q = *(const uint2*)((const uint8_t*)e.z_in + off);
        const float sc = q8_scale_value(e.z_scales[(int64_t)row * e.ldzs + (col >> 5)]);
        const int fmt = e.z_kind == kXInt8 ? MAO_Q8_INT8 : MAO_Q8_E4M3;
        q8_decode4_any(fmt, q.x, sc, z);
        q8_decode4_any(fmt, q.y, sc, z + 4);
      }
      act_slope_apply(e.act, z, v);
    }
  } else {
    if (e.bias != nullptr) {
      float b[8];
      if (valid >= 8) {
        load8_any(e.bias, e.bias_dtype, col, b, 8);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) b[i] = i < valid ? load1_any(e.bias, e.bias_dtype, col + i) : 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += b[i];
    }
    if (e.z_out) store8n_any(e.z_out, e.zo_dtype, (int64_t)row * e.ldzo + col, v, valid);
    act_apply(e.act, v);
  }
  if (e.add != nullptr) {
    float a[8];
    load8_any(e.add, e.add_dtype, (int64_t)row * e.ldadd + col, a, valid);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += a[i];
  }
  store8n_any(e.D, e.d_dtype, (int64_t)row * e.ldd + col, v, valid);
}

}  // namespace

mao_status launch_linear_join(const LinProblem& p, const float* part, int64_t ldpart, int split,
                              bool slope, hipStream_t s) {
  const int nch = (int)ceil_div(p.N, 8);
  const int64_t grid = ceil_div((int64_t)p.M * nch, 256);
  hipLaunchKernelGGL(linear_join_kernel, dim3((uint32_t)grid), dim3(256), 0, s, p, part, ldpart,
                     split, slope ? 1 : 0, nch);
  MAO_LAUNCH_CHECK();
  return MAO_OK;
}

}  // namespace mao
