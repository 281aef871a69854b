// Rows held by groups of threads: sums over a group, runs of 8 columns, parameters.
#pragma once

#include "layers.hpp"

namespace mao {

// Sum over the 64 lanes, in every lane: quad and row adds by DPP, then the
// four 16-lane rows by lane reads.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float wave_total(float v) {
  v = dpp_add<0xB1>(v);   // quad_perm [1,0,3,2]
  v = dpp_add<0x4E>(v);   // quad_perm [2,3,0,1]
  v = dpp_add<0x141>(v);  // row_half_mirror
  v = dpp_add<0x140>(v);  // row_mirror
  const int b = __float_as_int(v);
  return (__int_as_float(__builtin_amdgcn_readlane(b, 0)) +
          __int_as_float(__builtin_amdgcn_readlane(b, 16))) +
         (__int_as_float(__builtin_amdgcn_readlane(b, 32)) +
          __int_as_float(__builtin_amdgcn_readlane(b, 48)));
}

// Largest of the 64 lanes, in every lane; NaN counts as nothing.
template <int CTRL>
__device__ __forceinline__ float dpp_fmax(float v) {
  return fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf,
                                                             true)));
}
__device__ __forceinline__ float wave_max(float v) {
  v = dpp_fmax<0xB1>(v);
  v = dpp_fmax<0x4E>(v);
  v = dpp_fmax<0x141>(v);
  v = dpp_fmax<0x140>(v);
  const int b = __float_as_int(v);
  return fmaxf(fmaxf(__int_as_float(__builtin_amdgcn_readlane(b, 0)),
                     __int_as_float(__builtin_amdgcn_readlane(b, 16))),
               fmaxf(__int_as_float(__builtin_amdgcn_readlane(b, 32)),
                     __int_as_float(__builtin_amdgcn_readlane(b, 48))));
}

// Sum over the TPR threads of a row group. buf: one float per wavefront of the
// block, one such array per call site so that a later reduction never
// overwrites one still being read (two barriers lie between reuses).
template <int TPR>
__device__ __forceinline__ float group_total(float v, float* buf) {
  v = wave_total(v);
  if constexpr (TPR == 64) return v;
  const int w = threadIdx.x >> 6, w0 = w / (TPR / 64) * (TPR / 64);
  if ((threadIdx.x & 63) == 0) buf[w] = v;
  __syncthreads();
  float t = 0.f;
#pragma unroll
  for (int i = 0; i < TPR / 64; ++i) t += buf[w0 + i];
  return t;
}

// Two sums behind one barrier; buf alternates between two arrays from one call
// to the next, so the barrier of the call between them separates its reads from
// the next writes.
template <int TPR>
__device__ __forceinline__ void group_total2(float& a, float& b, float2* buf) {
  a = wave_total(a);
  b = wave_total(b);
  if constexpr (TPR > 64) {
    constexpr int NW = TPR / 64;
    const int w = threadIdx.x >> 6, w0 = w / NW * NW;
    if ((threadIdx.x & 63) == 0) buf[w] = make_float2(a, b);
    __syncthreads();
    if constexpr (NW == 3) {
      const float2 t0 = buf[w0], t1 = buf[w0 + 1], t2 = buf[w0 + 2];
      a = (t0.x + t1.x) + t2.x;
      b = (t0.y + t1.y) + t2.y;
    } else {  // one partial sum per lane, joined across 2, 4, 8 or 16 lanes
      const float2 t = buf[w0 + (threadIdx.x & (NW - 1))];
      a = dpp_add<0xB1>(t.x);
      b = dpp_add<0xB1>(t.y);
      if constexpr (NW >= 4) a = dpp_add<0x4E>(a), b = dpp_add<0x4E>(b);
      if constexpr (NW >= 8) a = dpp_add<0x141>(a), b = dpp_add<0x141>(b);
      if constexpr (NW >= 16) a = dpp_add<0x140>(a), b = dpp_add<0x140>(b);
    }
  }
}

// Column runs past the row read as zero; so do the columns of a partial last
// run that lie past the row (its storage is read in whole 16-byte pieces).
__device__ __forceinline__ void mask8(float (&v)[8], int valid) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = i < valid ? v[i] : 0.f;
}

__device__ __forceinline__ void load_param(const void* p, int dtype, int col, int valid,
                                           float dflt, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = dflt;
  if (p == nullptr || valid <= 0) return;
  if (valid >= 8) {
    load8_any(p, dtype, col, v, 8);
    return;
  }
  // parameters are plain arrays: the last run may end with the allocation
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < valid) v[i] = load1_any(p, dtype, col + i);
}

}  // namespace mao
