// AdamW over many tensors in one call, with states in 32 or 8 bits.
//
//   m = b1 m + (1 - b1) s g;  v = b2 v + (1 - b2) (s g)^2       (s: *grad_scale or 1)
//   w -= lr (wd w + (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps))
//
// 8-bit states hold m and r = sqrt(v) in floats with a 4-bit exponent (bias 15, subnormals)
// and a mantissa of 3 bits (m, with a sign) or 4 bits (r, never negative), times one fp32
// scale per 256 elements that makes the largest of them the largest code. sqrt(v), not v:
// the denominator's relative error is what matters, and half the exponent range covers it. A
// nonzero r has a code of at least 1, so that no update is divided by eps alone.
//
// Rounding: an average of many steps moves by less than half a code's step at a time, and
// rounding to the nearest would hold it where it is. What is cut off is rounded up with
// its own fraction as probability instead: the code's places and the 20 (r: 19) bits
// below them, plus a dither of as many bits, cut off. The dither of element i at step t is
// the top of (a i + b t) mod 2^32, an additive recurrence (Kronecker's sequence; a and b
// are 2^32 times the golden ratio's fraction and times that of the next such ratio), equally
// spread over the steps of one element and over the elements of one step. No random
// state, the same results for the same inputs.
//
// A span of 256 whose m or r holds a NaN or an infinity gets a NaN scale: all of it reads as
// NaN. A span whose largest m is below 2^-100 counts as zeros.
#include "adam8.hpp"
#include "validate.hpp"

#include <algorithm>
#include <math.h>
#include <new>

namespace mao {

namespace {

struct AdamTensor {
  void* w;
  const void* g;
  void *m, *v;
  float *ms, *vs;
  int64_t n;
  float lr, wd;
};

constexpr int kTensors = 48;  // per launch: the table is a kernel argument of 3.6 KB
constexpr int kThreads = 256;
constexpr int kChunk = kThreads * 8;  // elements of one workgroup

struct AdamTable {
  AdamTensor t[kTensors];
  uint32_t first[kTensors];  // workgroup that begins with the tensor
  const float* grad_scale;
  float beta1, beta2, ob1, ob2, ib1, ib2, eps;
  uint32_t step;
  int count;
};

// The tensor of this workgroup: the last one that begins at or before it.
__device__ __forceinline__ int tensor_of_block(const uint32_t (&first)[kTensors], int count) {
  const int lane = threadIdx.x & 63;
  const bool begun = lane < count && first[min(lane, kTensors - 1)] <= blockIdx.x;
  return __popcll(__ballot(begun)) - 1;
}

// 8 elements of a tensor, from element base on; FULL: the whole workgroup lies inside it.
template <typename TW, typename TG, bool STATE8, bool FULL>
__device__ __forceinline__ void adamw_run(const AdamTable& a, const AdamTensor& t, int64_t base) {
  const int valid = FULL ? 8 : (int)min((int64_t)8, t.n - base);
  // with 8-bit states a lane past the end takes part in its span's reductions
  if (!STATE8 && valid <= 0) return;
  const float gs = a.grad_scale ? *a.grad_scale : 1.f;
  float w[8], g[8], m[8], v[8];
  if constexpr (STATE8) {
    const int64_t span = base >> 8;
    const float ms = valid > 0 ? t.ms[span] : 0.f, vs = valid > 0 ? t.vs[span] : 0.f;
    uint2 mc = load_codes<FULL>((const uint8_t*)t.m + base, valid);
    uint2 vc = load_codes<FULL>((const uint8_t*)t.v + base, valid);
    load_run<FULL>((const TW*)t.w + base, valid, w);
    load_run<FULL>((const TG*)t.g + base, valid, g);
    adam8_decode<true>(mc, ms, m);
    adam8_decode<false>(vc, vs, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (a.grad_scale) g[i] *= gs;
      m[i] = a.beta1 * m[i] + a.ob1 * g[i];
      const float vv = a.beta2 * (v[i] * v[i]) + a.ob2 * g[i] * g[i];
      v[i] = __builtin_amdgcn_sqrtf(vv);
      // sqrt(vv ib2) = sqrt(vv) sqrt(ib2); hardware square root and reciprocal, 1 ulp each
      const float u = (m[i] * a.ib1) * __builtin_amdgcn_rcpf(v[i] * a.ib2 + a.eps);
      w[i] = w[i] - t.lr * (t.wd * w[i] + u);
    }
    float mscale, vscale;
    mc = adam8_encode<true>(m, (uint32_t)base, a.step, mscale);
    vc = adam8_encode<false>(v, (uint32_t)base, a.step, vscale);
    if (valid <= 0) return;
    store_codes<FULL>((uint8_t*)t.m + base, valid, mc);
    store_codes<FULL>((uint8_t*)t.v + base, valid, vc);
    if ((threadIdx.x & 31) == 0) {
      t.ms[span] = mscale;
      t.vs[span] = vscale;
    }
  } else {
    load_run<FULL>((const TW*)t.w + base, valid, w);
    load_run<FULL>((const TG*)t.g + base, valid, g);
    load_run<FULL>((const float*)t.m + base, valid, m);
    load_run<FULL>((const float*)t.v + base, valid, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (a.grad_scale) g[i] *= gs;
      m[i] = a.beta1 * m[i] + a.ob1 * g[i];
      v[i] = a.beta2 * v[i] + a.ob2 * g[i] * g[i];
      const float u = (m[i] * a.ib1) / (sqrtf(v[i] * a.ib2) + a.eps);
      w[i] = w[i] - t.lr * (t.wd * w[i] + u);
    }
    store_run<FULL>((float*)t.m + base, valid, m);
    store_run<FULL>((float*)t.v + base, valid, v);
  }
  store_run<FULL>((TW*)t.w + base, valid, w);
}

template <typename TW, typename TG, bool STATE8>
__global__ __launch_bounds__(kThreads) void adamw_many_kernel(AdamTable a) {
  const int idx = tensor_of_block(a.first, a.count);
  const AdamTensor& t = a.t[idx];
  const int64_t begin = (int64_t)(blockIdx.x - a.first[idx]) * kChunk;
  const int64_t base = begin + threadIdx.x * 8;
  if (begin + kChunk <= t.n)
    adamw_run<TW, TG, STATE8, true>(a, t, base);
  else
    adamw_run<TW, TG, STATE8, false>(a, t, base);
}

struct ReadTensor {
  const void *m, *v;
  const float *ms, *vs;
  void *m_out, *v_out;
  int64_t n;
};
struct ReadTable {
  ReadTensor t[kTensors];
  uint32_t first[kTensors];
  int count;
};

template <typename T>
__global__ __launch_bounds__(kThreads) void adamw8_read_kernel(ReadTable a) {
  const int idx = tensor_of_block(a.first, a.count);
  const ReadTensor& t = a.t[idx];
  const int64_t base = (int64_t)(blockIdx.x - a.first[idx]) * kChunk + threadIdx.x * 8;
  const int valid = (int)min((int64_t)8, t.n - base);
  if (valid <= 0) return;
  float m[8], v[8];
  adam8_decode<true>(load_codes<false>((const uint8_t*)t.m + base, valid), t.ms[base >> 8], m);
  adam8_decode<false>(load_codes<false>((const uint8_t*)t.v + base, valid), t.vs[base >> 8], v);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= v[i];
  store_run<false>((T*)t.m_out + base, valid, m);
  store_run<false>((T*)t.v_out + base, valid, v);
}

// Byte ranges of one call, to be checked against each other: none that is written may
// share bytes with another. Sorted by their beginnings, one pass sees every pair that does.
struct Spans {
  struct Span {
    uintptr_t lo, hi;
    bool written;
  };
  Span few[256];
  Span* s = few;
  int64_t n = 0;
  bool room(int64_t most) {
    if (most > 256) s = new (std::nothrow) Span[most];
    return s != nullptr;
  }
  ~Spans() {
    if (s != few) delete[] s;
  }
  void add(const void* p, int64_t bytes, bool written) {
    if (p) s[n++] = Span{(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes, written};
  }
  mao_status check() {
    std::sort(s, s + n, [](const Span& x, const Span& y) { return x.lo < y.lo; });
    uintptr_t any = 0, written = 0;
    for (int64_t i = 0; i < n; ++i) {
      if (s[i].lo < (s[i].written ? any : written))
        MAO_FAIL(MAO_E_ALIAS, "a written buffer overlaps another one");
      any = std::max(any, s[i].hi);
      if (s[i].written) written = std::max(written, s[i].hi);
    }
    return MAO_OK;
  }
};

constexpr int kMostTensors = 4096;
constexpr int64_t kMostElements = (int64_t)1 << 34;

mao_status check_count(int32_t count, const void* items) {
  if (!items) MAO_FAIL(MAO_E_NULL, "tensors is NULL");
  if (count < 1 || count > kMostTensors) MAO_FAIL(MAO_E_SHAPE, "count=%d outside 1..4096", count);
  return MAO_OK;
}

mao_status check_element(const char* name, int i, const void* p, size_t es) {
  if (!p) MAO_FAIL(MAO_E_NULL, "tensor %d: %s is NULL", i, name);
  if ((uintptr_t)p % es != 0) MAO_FAIL(MAO_E_LAYOUT, "tensor %d: %s not aligned to its elements", i, name);
  return MAO_OK;
}

mao_status check_size(int i, int64_t n) {
  if (n < 0 || n > kMostElements) MAO_FAIL(MAO_E_SHAPE, "tensor %d: n=%lld", i, (long long)n);
  return MAO_OK;
}

template <typename TW, typename TG>
mao_status go(const AdamTable& a, bool state8, uint32_t blocks, hipStream_t s) {
  if (state8)
    hipLaunchKernelGGL((adamw_many_kernel<TW, TG, true>), dim3(blocks), dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((adamw_many_kernel<TW, TG, false>), dim3(blocks), dim3(kThreads), 0, s, a);
  MAO_LAUNCH_CHECK();
  return MAO_OK;
}

// One launch's table, sent off when it is full or its grid is (2^32 threads).
constexpr int64_t kMostBlocks = (1 << 24) - 1;

mao_status send(AdamTable& a, int kind, int64_t& blocks, hipStream_t s) {
  if (a.count == 0) return MAO_OK;
  const bool state8 = (kind & 4) != 0;
  const uint32_t nb = (uint32_t)blocks;
  blocks = 0;
  mao_status r;
  switch (kind & 3) {
    case 0: r = go<float, float>(a, state8, nb, s); break;
    case 1: r = go<float, bf16_t>(a, state8, nb, s); break;
    case 2: r = go<bf16_t, float>(a, state8, nb, s); break;
    default: r = go<bf16_t, bf16_t>(a, state8, nb, s); break;
  }
  a.count = 0;
  return r;
}

}  // namespace
}  // namespace mao

using namespace mao;

extern "C" {

mao_status adamw_step_many(int32_t count, const mao_adamw_tensor* tensors, int64_t t, float beta1,
                           float beta2, float eps, const float* grad_scale, void* stream) {
  MAO_TRY(check_count(count, tensors));
  if (t < 1) MAO_FAIL(MAO_E_HPARAM, "t=%lld must be >= 1", (long long)t);
  if (!(beta1 >= 0.f && beta1 < 1.f) || !(beta2 >= 0.f && beta2 < 1.f))
    MAO_FAIL(MAO_E_HPARAM, "beta1=%g beta2=%g must be in [0, 1)", (double)beta1, (double)beta2);
  if (!finite(eps) || eps <= 0.f) MAO_FAIL(MAO_E_HPARAM, "eps=%g must be > 0", (double)eps);
  if ((uintptr_t)grad_scale % 4 != 0) MAO_FAIL(MAO_E_LAYOUT, "grad_scale misaligned");
  Spans spans;
  if (!spans.room((int64_t)count * 6 + 1)) MAO_FAIL(MAO_E_UNSUPPORTED, "out of host memory");
  unsigned kinds = 0;
  for (int i = 0; i < count; ++i) {
    const mao_adamw_tensor& p = tensors[i];
    MAO_TRY(check_size(i, p.n));
    if (!dtype_ok(p.w_dtype) || !dtype_ok(p.g_dtype)) MAO_FAIL(MAO_E_DTYPE, "tensor %d: w or g dtype", i);
    if (p.state != MAO_ADAM_F32 && p.state != MAO_ADAM_8BIT) MAO_FAIL(MAO_E_DTYPE, "tensor %d: state=%d", i, p.state);
    if (!finite(p.lr) || p.lr < 0.f || !finite(p.weight_decay) || p.weight_decay < 0.f)
      MAO_FAIL(MAO_E_HPARAM, "tensor %d: lr=%g weight_decay=%g must be >= 0", i, (double)p.lr, (double)p.weight_decay);
    if (p.n == 0) continue;
    const bool q = p.state == MAO_ADAM_8BIT;
    const int64_t ss = q ? 1 : 4;
    MAO_TRY(check_element("w", i, p.w, dtype_size(p.w_dtype)));
    MAO_TRY(check_element("g", i, p.g, dtype_size(p.g_dtype)));
    MAO_TRY(check_element("m", i, p.m, (size_t)ss));
    MAO_TRY(check_element("v", i, p.v, (size_t)ss));
    spans.add(p.w, p.n * (int64_t)dtype_size(p.w_dtype), true);
    spans.add(p.g, p.n * (int64_t)dtype_size(p.g_dtype), false);
    spans.add(p.m, p.n * ss, true);
    spans.add(p.v, p.n * ss, true);
    if (q) {
      MAO_TRY(check_element("m_scale", i, p.m_scale, 4));
      MAO_TRY(check_element("v_scale", i, p.v_scale, 4));
      spans.add(p.m_scale, ceil_div(p.n, kAdamSpan) * 4, true);
      spans.add(p.v_scale, ceil_div(p.n, kAdamSpan) * 4, true);
    }
    kinds |= 1u << ((q ? 4 : 0) + (p.w_dtype == MAO_BF16 ? 2 : 0) + (p.g_dtype == MAO_BF16 ? 1 : 0));
  }
  spans.add(grad_scale, 4, false);
  MAO_TRY(spans.check());
  AdamTable a = {};
  a.grad_scale = grad_scale;
  a.beta1 = beta1;
  a.beta2 = beta2;
  a.ob1 = 1.f - beta1;
  a.ob2 = 1.f - beta2;
  a.eps = eps;
  a.step = (uint32_t)t;
  const float bc1 = (float)(1.0 - pow((double)beta1, (double)t));
  const float bc2 = (float)(1.0 - pow((double)beta2, (double)t));
  a.ib1 = 1.f / bc1;
  for (int kind = 0; kind < 8; ++kind) {
    if (!(kinds >> kind & 1)) continue;
    a.ib2 = kind & 4 ? (float)(1.0 / sqrt((double)bc2)) : 1.f / bc2;
    int64_t blocks = 0;
    for (int i = 0; i < count; ++i) {
      const mao_adamw_tensor& p = tensors[i];
      if (p.n == 0 || kind != (p.state == MAO_ADAM_8BIT ? 4 : 0) + (p.w_dtype == MAO_BF16 ? 2 : 0) + (p.g_dtype == MAO_BF16 ? 1 : 0))
        continue;
      const int64_t nb = ceil_div(p.n, kChunk);
      if (a.count == kTensors || blocks + nb > kMostBlocks)
        MAO_TRY(send(a, kind, blocks, (hipStream_t)stream));
      a.t[a.count] = AdamTensor{p.w, p.g, p.m, p.v, p.m_scale, p.v_scale, p.n, p.lr, p.weight_decay};
      a.first[a.count++] = (uint32_t)blocks;
      blocks += nb;
    }
    MAO_TRY(send(a, kind, blocks, (hipStream_t)stream));
  }
  return MAO_OK;
}

mao_status mao_adamw8_read(int32_t count, const mao_adamw8_state* states, int32_t dtype,
                           void* stream) {
  MAO_TRY(check_count(count, states));
  if (!dtype_ok(dtype)) MAO_FAIL(MAO_E_DTYPE, "dtype=%d", dtype);
  Spans spans;
  if (!spans.room((int64_t)count * 6)) MAO_FAIL(MAO_E_UNSUPPORTED, "out of host memory");
  for (int i = 0; i < count; ++i) {
    const mao_adamw8_state& p = states[i];
    MAO_TRY(check_size(i, p.n));
    if (p.n == 0) continue;
    const size_t es = dtype_size(dtype);
    MAO_TRY(check_element("m", i, p.m, 1));
    MAO_TRY(check_element("v", i, p.v, 1));
    MAO_TRY(check_element("m_scale", i, p.m_scale, 4));
    MAO_TRY(check_element("v_scale", i, p.v_scale, 4));
    MAO_TRY(check_element("m_out", i, p.m_out, es));
    MAO_TRY(check_element("v_out", i, p.v_out, es));
    spans.add(p.m, p.n, false);
    spans.add(p.v, p.n, false);
    spans.add(p.m_scale, ceil_div(p.n, kAdamSpan) * 4, false);
    spans.add(p.v_scale, ceil_div(p.n, kAdamSpan) * 4, false);
    spans.add(p.m_out, p.n * (int64_t)es, true);
    spans.add(p.v_out, p.n * (int64_t)es, true);
  }
  MAO_TRY(spans.check());
  ReadTable a = {};
  int64_t blocks = 0;
  auto send_read = [&]() -> mao_status {
    if (a.count == 0) return MAO_OK;
    if (dtype == MAO_BF16)
      hipLaunchKernelGGL((adamw8_read_kernel<bf16_t>), dim3((uint32_t)blocks), dim3(kThreads), 0, (hipStream_t)stream, a);
    else
      hipLaunchKernelGGL((adamw8_read_kernel<float>), dim3((uint32_t)blocks), dim3(kThreads), 0, (hipStream_t)stream, a);
    a.count = 0;
    blocks = 0;
    MAO_LAUNCH_CHECK();
    return MAO_OK;
  };
  for (int i = 0; i < count; ++i) {
    const mao_adamw8_state& p = states[i];
    if (p.n == 0) continue;
    const int64_t nb = ceil_div(p.n, kChunk);
    if (a.count == kTensors || blocks + nb > kMostBlocks) MAO_TRY(send_read());
    a.t[a.count] = ReadTensor{p.m, p.v, p.m_scale, p.v_scale, p.m_out, p.v_out, p.n};
    a.first[a.count++] = (uint32_t)blocks;
    blocks += nb;
  }
  return send_read();
}

}  // extern "C"
