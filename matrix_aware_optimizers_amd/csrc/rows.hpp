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
    } else if constexpr ((NW & (NW - 1)) != 0) {
      a = b = 0.f;
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        a += buf[w0 + i].x;
        b += buf[w0 + i].y;
      }
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

// A row (the same one for a whole wavefront) for buffer instructions: past its `bytes` they read 0
// and write nothing. One offset register serves every access of a thread, where 64-bit
// addresses of several matrices take as many registers as the data.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_buffer(const void* p, int64_t row_bytes,
                                                             int row, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((char*)p + row_bytes * row, 0, bytes, 0x00027000);
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Four elements of such a row, in their stored form: 8 bytes of bf16, 16 of fp32.
template <typename T> struct Run4;
template <> struct Run4<bf16_t> {
  u32x2 a;
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t row, int run) {
    a = __builtin_amdgcn_raw_buffer_load_b64(row, run * 8, 0, 0);
  }
  // the compiler may not carry values derived from here on across this point
  __device__ __forceinline__ void opaque() { asm volatile("" : "+v"(a[0]), "+v"(a[1])); }
  __device__ __forceinline__ void get(float (&v)[4]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[2 * i] = __uint_as_float(a[i] << 16);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
    }
  }
};
template <> struct Run4<float> {
  u32x4 a;
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t row, int run) {
    a = __builtin_amdgcn_raw_buffer_load_b128(row, run * 16, 0, 0);
  }
  __device__ __forceinline__ void opaque() {
    asm volatile("" : "+v"(a[0]), "+v"(a[1]), "+v"(a[2]), "+v"(a[3]));
  }
  __device__ __forceinline__ void get(float (&v)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(a[i]);
  }
};
// The bytes of whole runs that a row of `cols` columns is read in: of the storage past the row
// at most the rest of its last run.
template <typename T> __device__ __forceinline__ int run4_bytes(int cols) {
  return (cols + 3) / 4 * 4 * (int)sizeof(T);
}

// Writes run `run` of a row; past: past the L2.
template <typename T>
__device__ __forceinline__ void store_run4(void* p, int64_t ld, int row, int cols, int run,
                                           const float (&v)[4], bool past) {
  constexpr int NT = 2;
  const auto whole = row_buffer(p, ld * (int64_t)sizeof(T), row, cols / 4 * 4 * (int)sizeof(T));
  if constexpr (sizeof(T) == 2) {
    const u32x2 k = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    if (past)
      __builtin_amdgcn_raw_buffer_store_b64(k, whole, run * 8, 0, NT);
    else
      __builtin_amdgcn_raw_buffer_store_b64(k, whole, run * 8, 0, 0);
  } else {
    const u32x4 k = {__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                     __float_as_uint(v[3])};
    if (past)
      __builtin_amdgcn_raw_buffer_store_b128(k, whole, run * 16, 0, NT);
    else
      __builtin_amdgcn_raw_buffer_store_b128(k, whole, run * 16, 0, 0);
  }
  const int n = cols - 4 * run;
  if (n > 0 && n < 4) {
    T* d = (T*)p + ld * row + 4 * run;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) store_f32(d + i, v[i]);
  }
}

// Elements past the row count as zero.
__device__ __forceinline__ void mask4(float (&v)[4], int valid) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = i < valid ? v[i] : 0.f;
}

__device__ __forceinline__ void load_param4(const void* p, int dtype, int col, int valid,
                                            float dflt, float (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = dflt;
  if (p == nullptr || valid <= 0) return;
  if (valid >= 4) {
    if (dtype == MAO_BF16) {
      const uint2 k = *(const uint2*)((const bf16_t*)p + col);
      v[0] = __uint_as_float(k.x << 16);
      v[1] = __uint_as_float(k.x & 0xffff0000u);
      v[2] = __uint_as_float(k.y << 16);
      v[3] = __uint_as_float(k.y & 0xffff0000u);
    } else {
      const float4 k = *(const float4*)((const float*)p + col);
      v[0] = k.x;
      v[1] = k.y;
      v[2] = k.z;
      v[3] = k.w;
    }
    return;
  }
  // parameters are plain arrays: the last run may end with the allocation
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < valid) v[i] = load1_any(p, dtype, col + i);
}

}  // namespace mao
