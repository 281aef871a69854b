// 8-bit optimizer states: codes, scales, and runs of elements of any alignment.
#pragma once

#include "common.hpp"

namespace mao {

constexpr int kAdamSpan = 256;  // elements per scale: 32 lanes of 8

// Runs of 8 elements: a tensor may begin at any element of a flat buffer. gfx950 reads and
// writes 16 bytes at any element's address in one instruction.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));

// The first `valid` elements; 0 for the others. FULL: all 8, known beforehand, so that the
// loads of a kernel's inputs go out together.
template <bool FULL>
__device__ __forceinline__ void load_run(const float* p, int valid, float (&v)[8]) {
  if (FULL || valid >= 8) {
    const u32x4_any a = *(const u32x4_any*)p, b = *(const u32x4_any*)(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __uint_as_float(a[i]);
      v[4 + i] = __uint_as_float(b[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < valid ? p[i] : 0.f;
  }
}
template <bool FULL>
__device__ __forceinline__ void load_run(const bf16_t* p, int valid, float (&v)[8]) {
  if (FULL || valid >= 8) {
    const u32x4_any a = *(const u32x4_any*)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(a[i] << 16);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < valid ? bf16_to_f32(p[i]) : 0.f;
  }
}
template <bool FULL>
__device__ __forceinline__ uint2 load_codes(const uint8_t* p, int valid) {
  if (FULL || valid >= 8) {
    const u32x2_any a = *(const u32x2_any*)p;
    return make_uint2(a[0], a[1]);
  }
  uint2 c = make_uint2(0, 0);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i < valid) c.x |= (uint32_t)p[i] << (8 * i);
    if (4 + i < valid) c.y |= (uint32_t)p[4 + i] << (8 * i);
  }
  return c;
}

template <bool FULL>
__device__ __forceinline__ void store_run(float* p, int valid, const float (&v)[8]) {
  if (FULL || valid >= 8) {
    u32x4_any a, b;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = __float_as_uint(v[i]);
      b[i] = __float_as_uint(v[4 + i]);
    }
    *(u32x4_any*)p = a;
    *(u32x4_any*)(p + 4) = b;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) p[i] = v[i];
  }
}
template <bool FULL>
__device__ __forceinline__ void store_run(bf16_t* p, int valid, const float (&v)[8]) {
  if (FULL || valid >= 8) {
    u32x4_any a;
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    *(u32x4_any*)p = a;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) p[i] = f32_to_bf16(v[i]);
  }
}
template <bool FULL>
__device__ __forceinline__ void store_codes(uint8_t* p, int valid, uint2 c) {
  if (FULL || valid >= 8) {
    u32x2_any a;
    a[0] = c.x;
    a[1] = c.y;
    *(u32x2_any*)p = a;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) p[i] = (uint8_t)((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
  }
}

// Code formats: SIGNED the first moment's (sign, 4-bit exponent, 3-bit mantissa), else the
// second's root (4-bit exponent, 4-bit mantissa). Shifted to the top of an fp32's mantissa, a
// code is that float times 2^-112, subnormals included.
template <bool SIGNED> struct Adam8 {
  static constexpr int kDrop = SIGNED ? 20 : 19;  // fp32 mantissa bits below the code's
  static constexpr uint32_t kTop = SIGNED ? 127 : 255;
  static constexpr float kMax = SIGNED ? 1.875f : 1.9375f;  // the largest code's float
  // dither of element i at step t: kElement i + kStep t
  static constexpr uint32_t kElement = SIGNED ? 0x9E3779B9u : 0xC13FA9A9u;
  static constexpr uint32_t kStep = SIGNED ? 0xC13FA9A9u : 0x9E3779B9u;
};

template <bool SIGNED>
__device__ __forceinline__ void adam8_decode(uint2 codes, float scale, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t c = ((i < 4 ? codes.x : codes.y) >> (8 * (i & 3))) & 0xffu;
    const uint32_t bits = SIGNED ? (c & 127) << 20 | (c & 128) << 24 : c << 19;
    v[i] = __uint_as_float(bits) * 0x1p112f * scale;
  }
}

template <int CTRL> __device__ __forceinline__ uint32_t dpp_max(uint32_t x) {
  return max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, true));
}

// Codes of 8 values (elements first, first + 1, ...) and the scale of the span that the 32
// lanes around this one hold. Quotients are rounded to nearest, not the hardware's reciprocal: a
// last bit decides a code where a border is near.
template <bool SIGNED>
__device__ __forceinline__ uint2 adam8_encode(const float (&v)[8], uint32_t first, uint32_t step,
                                              float& scale) {
  typedef Adam8<SIGNED> F;
  // magnitudes as integers: NaN and infinity above every number
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
  top = dpp_max<0xB1>(top);   // quad_perm [1,0,3,2]
  top = dpp_max<0x4E>(top);   // quad_perm [2,3,0,1]
  top = dpp_max<0x141>(top);  // row_half_mirror
  top = dpp_max<0x140>(top);  // row_mirror
  top = max(top, (uint32_t)__builtin_amdgcn_ds_swizzle((int)top, 0x401F));  // lane ^ 16
  const float largest = __uint_as_float(top);
  const bool bad = top >= 0x7f800000u;
  const bool live = largest >= 0x1p-100f && !bad;
  scale = bad ? __uint_as_float(0x7fc00000u) : live ? largest * (1.f / F::kMax) : 0.f;
  float inv = 0.f;
  if (live) {
    inv = __builtin_amdgcn_rcpf(largest);
    inv = __builtin_fmaf(__builtin_fmaf(-largest, inv, 1.f), inv, inv) * F::kMax;
    if (largest > 0x1p120f) inv = 1.f / largest * F::kMax;  // a reciprocal near the end of the range
  }
  uint32_t c[2] = {0, 0};
  const uint32_t d0 = first * F::kElement + step * F::kStep;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // y's places from the code's on down: its own bits, or among the subnormals (below 2^-14)
    // whole multiples of 2^-37
    const float y = fabsf(v[i]) * inv;
    const uint32_t places = y < 0x1p-14f ? (uint32_t)(y * 0x1p37f) : __float_as_uint(y) - (112u << 23);
    const uint32_t d = (d0 + (uint32_t)i * F::kElement) >> (32 - F::kDrop);
    uint32_t k = min((places + d) >> F::kDrop, F::kTop);
    if (SIGNED)
      k |= __float_as_uint(v[i]) >> 24 & 128u;
    else
      k = v[i] > 0.f && live ? max(k, 1u) : 0u;
    c[i >> 2] |= k << (8 * (i & 3));
  }
  if (bad) c[0] = c[1] = 0;
  return make_uint2(c[0], c[1]);
}

}  // namespace mao
