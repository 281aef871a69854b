// 8-bit activation checkpoints: codes (int8 or OCP e4m3), and per row and 32
// columns one scale byte s that stands for 2^(s - 127).
//
// The scale is the smallest power of two that keeps every rounded code in
// range (|code| <= 127, or <= 448), so each stored value code * 2^(s - 127) has
// at most 8 significant bits and is exact in bf16: products over it on bf16
// matrix cores add no rounding. s = 0: a block of zeros. s = 255: a block that
// held a NaN or an infinity; its codes are 0 and it reads as NaN (0 * inf), so a
// diverged activation is not hidden.
#pragma once

#include "common.hpp"

namespace mao {

constexpr int kQ8Block = 32;

struct Q8View {
  void* codes;
  uint8_t* scales;
  int64_t ld, ld_scale;
};

// Scale byte for a block with largest magnitude amax (given as fp32 bits with
// the sign cleared; any NaN or infinity gives an exponent field of 255).
template <int FMT>
__device__ __forceinline__ int q8_scale(uint32_t amax_bits) {
  const int E = (int)(amax_bits >> 23), M = (int)(amax_bits & 0x7fffff);
  if (E == 255) return 255;
  if (amax_bits == 0) return 0;
  // amax = (1 + M 2^-23) 2^(E - 127). int8: 127 = 1.984 * 2^6, and values below
  // 127.5 steps round to 127 or less; e4m3: 448 = 1.75 * 2^8, and 464 rounds to
  // it (tie to even).
  const int s = FMT == MAO_Q8_INT8 ? E - 6 + (M >= 0x7f0000) : E - 8 + (M > 0x680000);
  // lowest scales: the smallest nonzero value, one step (2^-9 for e4m3), is then
  // at least 2^-133, the smallest bf16 number
  constexpr int kLowest = FMT == MAO_Q8_INT8 ? 1 : 3;
  return s < kLowest ? kLowest : s;
}

// Codes of four values, packed; inv = 2^(127 - s) (0 for s = 0 or 255).
template <int FMT>
__device__ __forceinline__ uint32_t q8_encode4(const float* x, float inv) {
  if constexpr (FMT == MAO_Q8_INT8) {
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) r |= ((uint32_t)(int)rintf(x[i] * inv) & 0xffu) << (8 * i);
    return r;
  } else {
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] * inv, x[1] * inv, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[2] * inv, x[3] * inv, r, true);
  }
}

__device__ __forceinline__ float q8_inv_scale(int s) {
  return (s == 0 || s == 255) ? 0.f : __uint_as_float((uint32_t)(254 - s) << 23);
}

__device__ __forceinline__ float q8_scale_value(int s) {
  return __uint_as_float((uint32_t)s << 23);
}

// Four values from packed codes.
template <int FMT>
__device__ __forceinline__ void q8_decode4(uint32_t c, float scale, float* v) {
  if constexpr (FMT == MAO_Q8_INT8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (float)(int)(int8_t)(c >> (8 * i)) * scale;
  } else {
    const f32x2_cvt_t lo = __builtin_amdgcn_cvt_pk_f32_fp8(c, false);
    const f32x2_cvt_t hi = __builtin_amdgcn_cvt_pk_f32_fp8(c, true);
    v[0] = lo.x * scale;
    v[1] = lo.y * scale;
    v[2] = hi.x * scale;
    v[3] = hi.y * scale;
  }
}

// Runtime-format forms (the format is the same for the whole launch).
__device__ __forceinline__ void q8_decode4_any(int fmt, uint32_t c, float scale, float* v) {
  if (fmt == MAO_Q8_INT8)
    q8_decode4<MAO_Q8_INT8>(c, scale, v);
  else
    q8_decode4<MAO_Q8_E4M3>(c, scale, v);
}

}  // namespace mao
