// AdamW over many tensors in one call, with states in 32 or 8 bits.
//
//   m = b1 m + (1 - b1) s g;  v = b2 v + (1 - b2) (s g)^2       (s: *grad_scale or 1)
//   w -= lr (wd w + (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps))
//
// 8-bit states hold m and r = sqrt(v) in floats with a 4-bit exponent (bias 15, subnormals)
// and a mantissa of 3 bits (m, with a sign) or 4 bits (r, never negative), times one fp32
// scale per 256 elements that makes the largest of them the largest code. sqrt(v), not v:
// the denominator's relative error is what matters, and half the exponent range covers it. A
// nonzero r has a code of at least 1, so that no update is divided by eps alone; an r below that
// code, 2^-19 of its span's largest, gives smaller updates than its own.
//
// Rounding: an average of many steps moves by less than half a code's step at a time, and
// rounding to the nearest would hold it where it is. What is cut off is rounded up with
// its own fraction as probability instead: the code's places and the 20 (r: 19) bits
// below them, plus a dither of as many bits, cut off. The dither of element i at step t is
// the top of (a i + b t) mod 2^32, an additive recurrence (Kronecker's sequence; a and b
// are 2^32 times the golden ratio's fraction and times that of the next such ratio), equally
// spread over the steps of one element and over the elements of one step. No random
// state, the same results for the same inputs. It leaves r, not r^2, where it is on average: r^2
// gains each rounding's variance, up to 3% in all at beta2 = 0.999 (a rounding's variance is at
// most a code's step, r / 16, times what r moves in a step).
//
// A span of 256 whose m or r holds a NaN or an infinity gets a NaN scale: all of it reads as
// NaN. A span whose largest m is below 2^-100 counts as zeros.
//
// Bound: memory traffic where the tensors are large, the launch and the list's host time (about
// 3 us and 0.1 us a tensor) where they are small. 8 elements a thread make 16-byte loads of
// bf16 and 8-byte ones of codes; a span is the 32 lanes that hold it, so that its maximum takes
// five exchanges. The tensors' addresses are the kernel's argument, array by array, and each
// wavefront finds its own by a ballot over the first workgroups: nothing is copied to the card,
// and 68 (fp32 states: 96) tensors share a launch. As an array of structures of 64 bytes 48 did,
// and 61 tensors of 9 million elements with 8-bit states took 52 us for 41.
//
// Measured: 757 million bf16 parameters with fp32 states 2.86 to 3.05 ms (5.5 to 5.8 TB/s, where a
// copy of 1 GiB reaches 5.2); 218 million bf16 parameters with 8-bit states, and the reading of
// those states 608 us (5.8 TB/s of what the two kernels move, 10.06 and 6.03 bytes an element);
// four vectors of 1536 to 6144 elements 5 us.
#include "adam8.hpp"
#include "validate.hpp"

#include <algorithm>
#include <math.h>
#include <new>
#include <type_traits>

namespace mao {

namespace {

constexpr int kThreads = 256;
constexpr int kChunk = kThreads * 8;  // elements of one workgroup
constexpr int kRates = 8;
constexpr uint32_t kFirst = (1 << 24) - 1;

// The tensors of one launch, a kernel argument of at most 4 KB. Learning rates and weight decays
// repeat, so that a launch has few pairs of them.
template <bool STATE8> struct AdamTable {
  static constexpr int N = STATE8 ? 68 : 96;
  void* w[N];
  const void* g[N];
  void *m[N], *v[N];
  float *ms[STATE8 ? N : 1], *vs[STATE8 ? N : 1];
  const float* grad_scale;
  uint32_t n[N];      // elements, the lower 32 bits
  // Workgroup that begins with the tensor (24 bits), which rates it has (4), and the upper bits of
  // its elements (4).
  uint32_t first[N];
  float lr[kRates], wd[kRates];
  float beta1, beta2, ob1, ob2, ib1, ib2, eps;
  uint32_t step;
  int32_t count, rates;
};
static_assert(sizeof(AdamTable<true>) <= 4096 && sizeof(AdamTable<false>) <= 4096, "kernel argument");

// The tensor of this workgroup: the last one that begins at or before it.
template <int N>
__device__ __forceinline__ int tensor_of_block(const uint32_t (&first)[N], int count) {
  const int lane = threadIdx.x & 63;
  int begun = 0;
#pragma unroll
  for (int k = 0; k < N; k += 64)
    begun += __popcll(
        __ballot(lane + k < count && (first[min(lane + k, N - 1)] & kFirst) <= blockIdx.x));
  return begun - 1;
}

struct AdamTensor {
  void* w;
  const void* g;
  void *m, *v;
  float *ms, *vs;
  int64_t n;
  float lr, wd;
};

// m and r = sqrt(v) of 8-bit states, every operation rounded by itself, in the formula's order.
// Where a code's border is near their last bits decide the code, and with it all later steps:
// with fused operations and the hardware's square root one element in 300000 a step got another
// code than the formula's own. (Square root: one correction by its exact residual, off the nearest
// number in about one of a million, the reciprocal of a scale likewise: the step of 218 million
// bf16 parameters and the reading of its states took 603 us before, 608 so, and 632 with the
// compiler's own square root and division.)
template <bool STATE8>
__device__ __forceinline__ void moments8(const AdamTable<STATE8>& a, const float (&g)[8], float (&m)[8],
                                         float (&r)[8]) {
#pragma clang fp contract(off)
  float low = 1.f, high = 1.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m[i] = a.beta1 * m[i] + a.ob1 * g[i];
    r[i] = a.beta2 * (r[i] * r[i]) + a.ob2 * g[i] * g[i];
    low = fminf(low, r[i]);
    high = fmaxf(high, r[i]);
  }
  if (low >= 0x1p-90f && high <= 0x1p90f) {  // else zeros, infinities and residuals that underflow
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = __builtin_amdgcn_rsqf(r[i]), s = r[i] * q;
      r[i] = __builtin_fmaf(__builtin_fmaf(-s, s, r[i]), 0.5f * q, s);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = sqrtf(r[i]);
  }
}

// 8 elements of a tensor, from element base on; FULL: the whole workgroup lies inside it.
template <typename TW, typename TG, bool STATE8, bool FULL>
__device__ __forceinline__ void adamw_run(const AdamTable<STATE8>& a, const AdamTensor& t,
                                          int64_t base) {
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
    for (int i = 0; i < 8; ++i)
      if (a.grad_scale) g[i] *= gs;
    moments8(a, g, m, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // sqrt(v ib2) = r sqrt(ib2); the hardware's reciprocal, 1 ulp
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
__global__ __launch_bounds__(kThreads) void adamw_many_kernel(AdamTable<STATE8> a) {
  const int idx = tensor_of_block(a.first, a.count);
  const uint32_t first = a.first[idx], rates = first >> 24 & 15;
  const int q = STATE8 ? idx : 0;
  const AdamTensor t = {a.w[idx],
                        a.g[idx],
                        a.m[idx],
                        a.v[idx],
                        a.ms[q],
                        a.vs[q],
                        (int64_t)(first >> 28) << 32 | a.n[idx],
                        a.lr[rates],
                        a.wd[rates]};
  const int64_t begin = (int64_t)(blockIdx.x - (first & kFirst)) * kChunk;
  const int64_t base = begin + threadIdx.x * 8;
  if (begin + kChunk <= t.n)
    adamw_run<TW, TG, STATE8, true>(a, t, base);
  else
    adamw_run<TW, TG, STATE8, false>(a, t, base);
}

struct ReadTable {
  static constexpr int N = 68;
  const void *m[N], *v[N];
  const float *ms[N], *vs[N];
  void *m_out[N], *v_out[N];
  uint32_t n[N], first[N];  // as above, without rates
  int32_t count;
};
static_assert(sizeof(ReadTable) <= 4096, "kernel argument");

template <typename T>
__global__ __launch_bounds__(kThreads) void adamw8_read_kernel(ReadTable a) {
  const int idx = tensor_of_block(a.first, a.count);
  const uint32_t first = a.first[idx];
  const int64_t n = (int64_t)(first >> 28) << 32 | a.n[idx];
  const int64_t begin = (int64_t)(blockIdx.x - (first & kFirst)) * kChunk;
  const int64_t base = begin + threadIdx.x * 8, span = base >> 8;
  const uint8_t *mc = (const uint8_t*)a.m[idx] + base, *vc = (const uint8_t*)a.v[idx] + base;
  float m[8], v[8];
  auto run = [&](auto whole, int valid) __attribute__((always_inline)) {
    constexpr bool FULL = decltype(whole)::value;
    const uint2 km = load_codes<FULL>(mc, valid), kv = load_codes<FULL>(vc, valid);
    adam8_decode<true>(km, a.ms[idx][span], m);
    adam8_decode<false>(kv, a.vs[idx][span], v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= v[i];
    store_run<FULL>((T*)a.m_out[idx] + base, valid, m);
    store_run<FULL>((T*)a.v_out[idx] + base, valid, v);
  };
  if (begin + kChunk <= n)
    run(std::true_type(), 8);
  else if (base < n)
    run(std::false_type(), (int)min((int64_t)8, n - base));
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
constexpr int64_t kMostElements = (int64_t)1 << 34;  // its upper bits fit 4 bits of a table

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

// 2^32 threads to a launch.
constexpr int64_t kMostBlocks = kFirst;

template <bool STATE8>
mao_status send(const AdamTable<STATE8>& a, int kind, int64_t blocks, hipStream_t s) {
  const dim3 grid((uint32_t)blocks);
#define MAO_ADAM(W, G) hipLaunchKernelGGL((adamw_many_kernel<W, G, STATE8>), grid, dim3(kThreads), 0, s, a)
  switch (kind) {
    case 0: MAO_ADAM(float, float); break;
    case 1: MAO_ADAM(float, bf16_t); break;
    case 2: MAO_ADAM(bf16_t, float); break;
    default: MAO_ADAM(bf16_t, bf16_t); break;
  }
#undef MAO_ADAM
  MAO_LAUNCH_CHECK();
  return MAO_OK;
}

// What all launches of a step share.
struct AdamStep {
  float beta1, beta2, eps, bc1, bc2;
  const float* grad_scale;
  int64_t t;
};

int kind_of(const mao_adamw_tensor& p) {
  return (p.w_dtype == MAO_BF16 ? 2 : 0) + (p.g_dtype == MAO_BF16 ? 1 : 0);
}

// The tensors of one kind of state and types, in as few launches as they fit.
template <bool STATE8>
mao_status step_kind(int32_t count, const mao_adamw_tensor* tensors, int kind, const AdamStep& st,
                     hipStream_t s) {
  AdamTable<STATE8> a = {};
  a.grad_scale = st.grad_scale;
  a.beta1 = st.beta1;
  a.beta2 = st.beta2;
  a.ob1 = 1.f - st.beta1;
  a.ob2 = 1.f - st.beta2;
  a.ib1 = 1.f / st.bc1;
  a.ib2 = STATE8 ? (float)(1.0 / sqrt((double)st.bc2)) : 1.f / st.bc2;
  a.eps = st.eps;
  a.step = (uint32_t)st.t;
  int64_t blocks = 0;
  for (int i = 0; i < count; ++i) {
    const mao_adamw_tensor& p = tensors[i];
    if (p.n == 0 || (p.state == MAO_ADAM_8BIT) != STATE8 || kind_of(p) != kind) continue;
    int r = 0;
    while (r < a.rates && !(a.lr[r] == p.lr && a.wd[r] == p.weight_decay)) ++r;
    const int64_t nb = ceil_div(p.n, kChunk);
    if (a.count == AdamTable<STATE8>::N || r == kRates || blocks + nb > kMostBlocks) {
      MAO_TRY(send<STATE8>(a, kind, blocks, s));
      a.count = a.rates = r = 0;
      blocks = 0;
    }
    if (r == a.rates) {
      a.lr[r] = p.lr;
      a.wd[r] = p.weight_decay;
      ++a.rates;
    }
    const int k = a.count++;
    a.w[k] = p.w;
    a.g[k] = p.g;
    a.m[k] = p.m;
    a.v[k] = p.v;
    if (STATE8) {
      a.ms[STATE8 ? k : 0] = p.m_scale;
      a.vs[STATE8 ? k : 0] = p.v_scale;
    }
    a.n[k] = (uint32_t)p.n;
    a.first[k] = (uint32_t)(blocks | r << 24 | p.n >> 32 << 28);
    blocks += nb;
  }
  return a.count ? send<STATE8>(a, kind, blocks, s) : MAO_OK;
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
    kinds |= 1u << ((q ? 4 : 0) + kind_of(p));
  }
  spans.add(grad_scale, 4, false);
  MAO_TRY(spans.check());
  AdamStep st = {};
  st.beta1 = beta1;
  st.beta2 = beta2;
  st.eps = eps;
  st.bc1 = (float)(1.0 - pow((double)beta1, (double)t));
  st.bc2 = (float)(1.0 - pow((double)beta2, (double)t));
  st.grad_scale = grad_scale;
  st.t = t;
  for (int kind = 0; kind < 4; ++kind) {
    if (kinds >> kind & 1)
      MAO_TRY(step_kind<false>(count, tensors, kind, st, (hipStream_t)stream));
    if (kinds >> kind & 16)
      MAO_TRY(step_kind<true>(count, tensors, kind, st, (hipStream_t)stream));
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
    const dim3 grid((uint32_t)blocks);
    if (dtype == MAO_BF16)
      hipLaunchKernelGGL((adamw8_read_kernel<bf16_t>), grid, dim3(kThreads), 0, (hipStream_t)stream, a);
    else
      hipLaunchKernelGGL((adamw8_read_kernel<float>), grid, dim3(kThreads), 0, (hipStream_t)stream, a);
    a.count = 0;
    blocks = 0;
    MAO_LAUNCH_CHECK();
    return MAO_OK;
  };
  for (int i = 0; i < count; ++i) {
    const mao_adamw8_state& p = states[i];
    if (p.n == 0) continue;
    const int64_t nb = ceil_div(p.n, kChunk);
    if (a.count == ReadTable::N || blocks + nb > kMostBlocks) MAO_TRY(send_read());
    const int k = a.count++;
    a.m[k] = p.m;
    a.v[k] = p.v;
    a.ms[k] = p.m_scale;
    a.vs[k] = p.v_scale;
    a.m_out[k] = p.m_out;
    a.v_out[k] = p.v_out;
    a.n[k] = (uint32_t)p.n;
    a.first[k] = (uint32_t)(blocks | p.n >> 32 << 28);
    blocks += nb;
  }
  return a.count ? send_read() : MAO_OK;
}

}  // extern "C"
