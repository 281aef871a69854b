// 8-bit activation checkpoints: quantise as they are kept, read back.
//
// Bound: HBM, one pass each way: 2 (bf16) or 4 (fp32) bytes in and 1 + 1/32
// out per element, and the reverse. A thread holds 16 consecutive columns (16
// bytes of codes per store), two neighbouring threads one scale block: the
// block's largest magnitude is one exchange between them (DPP). Magnitudes are
// compared as integers (fp32 bits without the sign), which orders NaN and
// infinity above every number.
//
// Measured (MI355X, 16384 x 6144 bf16, int8): 67 us to quantise and 68 to read back,
// 305 MB each, 4.5 TB/s, against 5.2 of a large copy; 125 us for the pair where the
// codes are read back from the cache behind the L2. fp32: 109 and 149 us, 507 MB each, 4.6
// and 3.4 TB/s.
#include "act.hpp"
#include "layers.hpp"

#include <algorithm>

namespace mao {

namespace {

// Work item (16 columns, 8 of launch_act) of a rows x nch grid of items.
struct Item {
  int row, c;
};
__device__ __forceinline__ Item item_of(int64_t base_row, int base_c, int nch) {
  // base + threadIdx.x, with base split once per workgroup
  const int off = base_c + (int)threadIdx.x;
  const int d = off / nch;
  return {(int)(base_row + d), off - d * nch};
}

template <typename T, int FMT>
__global__ __launch_bounds__(256) void q8_quantize_kernel(const T* x, int64_t ldx, int rows,
                                                          int cols, Q8View q, int nch) {
  const int64_t total = (int64_t)rows * nch;
  for (int64_t base = (int64_t)blockIdx.x * 256; base < total; base += (int64_t)gridDim.x * 256) {
    const int64_t br = base / nch;
    const Item it = item_of(br, (int)(base - br * nch), nch);
    // nch is even, so both threads of a block are in or out together
    if (it.row >= rows) continue;
    const int col = it.c * 16, valid = cols - col;
    float v[16];
    {
      float lo[8], hi[8];
      Raw8<T> r0, r1;
      const T* p = x + (int64_t)it.row * ldx + col;
      if (valid > 0) r0.load_cut(p, valid); else r0.zero();
      if (valid > 8) r1.load_cut(p + 8, valid - 8); else r1.zero();
      r0.get(lo);
      r1.get(hi);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = i < valid ? lo[i] : 0.f;
        v[8 + i] = 8 + i < valid ? hi[i] : 0.f;
      }
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xf, 0xf, true));
    const int s = q8_scale<FMT>(m);
    const float inv = q8_inv_scale(s);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // a block with a NaN or an infinity keeps zero codes
      float z[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) z[k] = s == 255 ? 0.f : v[4 * i + k];
      w[i] = q8_encode4<FMT>(z, inv);
    }
    uint8_t* d = (uint8_t*)q.codes + (int64_t)it.row * q.ld + col;
    if (valid >= 16) {
      *(uint4*)d = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < valid) d[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
    }
    if ((it.c & 1) == 0) q.scales[(int64_t)it.row * q.ld_scale + (it.c >> 1)] = (uint8_t)s;
  }
}

// v[i] <- v[i] - bf16(v[i]), exact in fp32; 0 where bf16(v[i]) is not finite
__device__ __forceinline__ void rest8(float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float h = bf16_to_f32(f32_to_bf16(v[i]));
    v[i] = fabsf(h) < INFINITY ? v[i] - h : 0.f;
  }
}

template <int FMT>
__global__ __launch_bounds__(256) void q8_dequantize_kernel(Q8View q, int rows, int cols, int act,
                                                            int rest, void* y, int dtype,
                                                            int64_t ldy, int nch) {
  const int64_t total = (int64_t)rows * nch;
  for (int64_t base = (int64_t)blockIdx.x * 256; base < total; base += (int64_t)gridDim.x * 256) {
    const int64_t br = base / nch;
    const Item it = item_of(br, (int)(base - br * nch), nch);
    if (it.row >= rows) continue;
    const int col = it.c * 16, valid = cols - col;
    const uint4 c = *(const uint4*)((const uint8_t*)q.codes + (int64_t)it.row * q.ld + col);
    const float sc = q8_scale_value(q.scales[(int64_t)it.row * q.ld_scale + (it.c >> 1)]);
    float lo[8], hi[8];
    q8_decode4<FMT>(c.x, sc, lo);
    q8_decode4<FMT>(c.y, sc, lo + 4);
    q8_decode4<FMT>(c.z, sc, hi);
    q8_decode4<FMT>(c.w, sc, hi + 4);
    act_apply(act, lo);
    act_apply(act, hi);
    if (rest) {
      rest8(lo);
      rest8(hi);
    }
    const int64_t off = (int64_t)it.row * ldy + col;
    store8n_any(y, dtype, off, lo, valid);
    if (valid > 8) store8n_any(y, dtype, off + 8, hi, valid - 8);
  }
}

// y = act(x), or its rest: 8 columns per thread
template <typename T>
__global__ __launch_bounds__(256) void act_kernel(const T* x, int64_t ldx, int rows, int cols,
                                                  int act, int rest, T* y, int64_t ldy, int nch) {
  const int64_t total = (int64_t)rows * nch;
  for (int64_t base = (int64_t)blockIdx.x * 256; base < total; base += (int64_t)gridDim.x * 256) {
    const int64_t br = base / nch;
    const Item it = item_of(br, (int)(base - br * nch), nch);
    if (it.row >= rows) continue;
    Raw8<T> r;
    r.load_cut(x + (int64_t)it.row * ldx + it.c * 8, cols - it.c * 8);
    float v[8];
    r.get(v);
    act_apply(act, v);
    if (rest) rest8(v);
    store8n_any(y, sizeof(T) == 2 ? MAO_BF16 : MAO_F32, (int64_t)it.row * ldy + it.c * 8, v,
                cols - it.c * 8);
  }
}

int q8_grid(int64_t total) { return (int)std::min<int64_t>(ceil_div(total, 256), 256 * 32); }

}  // namespace

mao_status launch_q8_quantize(const void* x, int dtype, int64_t ldx, int rows, int cols, Q8View q,
                              int fmt, hipStream_t s) {
  const int nch = (int)ceil_div(cols, kQ8Block) * 2;
  const dim3 grid(q8_grid((int64_t)rows * nch));
#define MAO_Q8_GO(T, F)                                                                       \
  hipLaunchKernelGGL((q8_quantize_kernel<T, F>), grid, dim3(256), 0, s, (const T*)x, ldx, rows, \
                     cols, q, nch)
  if (dtype == MAO_BF16) {
    if (fmt == MAO_Q8_INT8) MAO_Q8_GO(bf16_t, MAO_Q8_INT8);
    else MAO_Q8_GO(bf16_t, MAO_Q8_E4M3);
  } else {
    if (fmt == MAO_Q8_INT8) MAO_Q8_GO(float, MAO_Q8_INT8);
    else MAO_Q8_GO(float, MAO_Q8_E4M3);
  }
#undef MAO_Q8_GO
  MAO_LAUNCH_CHECK();
  return MAO_OK;
}

mao_status launch_act(const void* x, int dtype, int64_t ldx, int rows, int cols, int act, bool rest,
                      void* y, int64_t ldy, hipStream_t s) {
  const int nch = (int)ceil_div(cols, 8);
  const dim3 grid(q8_grid((int64_t)rows * nch));
  if (dtype == MAO_BF16)
    hipLaunchKernelGGL((act_kernel<bf16_t>), grid, dim3(256), 0, s, (const bf16_t*)x, ldx, rows,
                       cols, act, (int)rest, (bf16_t*)y, ldy, nch);
  else
    hipLaunchKernelGGL((act_kernel<float>), grid, dim3(256), 0, s, (const float*)x, ldx, rows, cols,
                       act, (int)rest, (float*)y, ldy, nch);
  MAO_LAUNCH_CHECK();
  return MAO_OK;
}

mao_status launch_q8_dequantize(Q8View q, int fmt, int rows, int cols, int act, bool rest, void* y,
                                int dtype, int64_t ldy, hipStream_t s) {
  const int nch = (int)ceil_div(cols, 16);
  const dim3 grid(q8_grid((int64_t)rows * nch));
  if (fmt == MAO_Q8_INT8)
    hipLaunchKernelGGL((q8_dequantize_kernel<MAO_Q8_INT8>), grid, dim3(256), 0, s, q, rows, cols,
                       act, (int)rest, y, dtype, ldy, nch);
  else
    hipLaunchKernelGGL((q8_dequantize_kernel<MAO_Q8_E4M3>), grid, dim3(256), 0, s, q, rows, cols,
                       act, (int)rest, y, dtype, ldy, nch);
  MAO_LAUNCH_CHECK();
  return MAO_OK;
}

}  // namespace mao
