// Log probabilities of tokens: of given ones, with the entropy and the most likely
// alternatives of each row of logits; the gradient of those; and a loss's gradient in the
// same pass as its log probabilities.
//
//   M = max x, S = sum e^(x - M), T = sum (x - M) e^(x - M)
//   logprob = (x_t - M) - log S,  entropy = log S - T / S
//   dx_j = dlp (d_jt - p_j) + dlse p_j - dent p_j (log p_j + entropy)
//   loss: dx_j = w (p_j - d_jt)
//
// M and log S are kept apart (their sum, the log of the sum of exponentials, would round away
// log S where logits are large: a row of the type's lowest values still is uniform).
//
// Bound: HBM. Forward: one pass, each thread with a running maximum and the two sums, joined
// at the end; a masked logit (-inf) adds nothing, a row of them has entropy 0 and log
// probabilities of -inf; a NaN or +inf makes all results of its row NaN.
#include "rows.hpp"

#include <algorithm>

namespace mao {

namespace {

constexpr float kLog2E = 1.4426950408889634f;
constexpr float kNone = -3.4028234663852886e38f;  // below every logit but -inf
__device__ __forceinline__ float exp_hw(float x) { return __builtin_amdgcn_exp2f(x * kLog2E); }

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}

// Running softmax sums of a part of a row.
struct Sums {
  float m, s, t;
  __device__ __forceinline__ void init() {
    m = kNone;
    s = t = 0.f;
  }
  // to the maximum to >= m. Beyond e^-1e4 nothing is left, and the product stays finite.
  __device__ __forceinline__ void raise(float to) {
    const float d = fminf(to - m, 1e4f), f = exp_hw(-d);
    t = f * (t - d * s);
    s *= f;
    m = to;
  }
};

// Elements valid.. of a run are past the row.
__device__ __forceinline__ void cut_run(float (&v)[8], int valid) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = i < valid ? v[i] : -INFINITY;
}

template <typename T>
__device__ __forceinline__ void load_logits(const T* x, int run, int vocab, float (&v)[8]) {
  Raw8<T> r;
  const int valid = vocab - 8 * run;
  r.load_cut(x + 8 * (int64_t)run, valid);
  r.get(v);
  if (valid < 8) cut_run(v, valid);
}

template <bool ENT, int R>
__device__ __forceinline__ void add_runs(Sums& q, const float (&v)[R][8]) {
  float c = max3(v[0][0], v[0][1], v[0][2]);
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = r == 0 ? 3 : 0; i + 1 < 8; i += 2) c = max3(c, v[r][i], v[r][i + 1]);
  c = max3(c, v[0][7], v[R - 1][7]);
  if (c > q.m) q.raise(c);
  float s[4] = {0.f, 0.f, 0.f, 0.f}, t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float y = v[r][i] - q.m, e = exp_hw(y);
      s[i & 3] += e;
      if (ENT) t[i & 3] += e * fmaxf(y, -200.f);  // 0 times -inf is none
    }
  q.s += (s[0] + s[1]) + (s[2] + s[3]);
  if (ENT) q.t += (t[0] + t[1]) + (t[2] + t[3]);
}

// Sums over the block's threads, in every thread. buf: 3 floats per wavefront, used once.
template <int THREADS>
__device__ __forceinline__ Sums block_sums(Sums q, float (*buf)[3]) {
  const float m = wave_max(q.m);
  q.raise(m);
  q.s = wave_total(q.s);
  q.t = wave_total(q.t);
  if constexpr (THREADS > 64) {
    constexpr int NW = THREADS / 64;
    const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
    if (lane == 0) {
      buf[w][0] = q.m;
      buf[w][1] = q.s;
      buf[w][2] = q.t;
    }
    __syncthreads();
    q.init();
    if (lane < NW) {
      q.m = buf[lane][0];
      q.s = buf[lane][1];
      q.t = buf[lane][2];
    }
    const float all = wave_max(q.m);
    q.raise(all);
    q.s = wave_total(q.s);
    q.t = wave_total(q.t);
  }
  return q;
}

// ---- the most likely alternatives ------------------------------------------
//
// Order: larger logits first, of equal ones (-0 and 0 among them) the lower token. A key
// holds both: the logit's bits in an order of unsigned integers, and the token's complement.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint64_t key_of(float x, int token) {
  return (uint64_t)ordered(x) << 32 | (uint32_t)~token;
}

constexpr int kList = 1024;  // candidates that fit

struct TopShared {
  uint64_t list[kList];
  uint32_t group[64];
  uint32_t hist[256];
  uint32_t count, limit, need;
};

// The `top` largest keys of the runs [lo, hi) of a row, each handed to emit with its place
// in the order; places past the part's elements get key 0. m: the largest logit of this
// thread's runs, which `kept` holds if KEEP (one block of R a thread).
//
// The threads form 64 groups; the top-th largest of the groups' maxima (its upper 16 bits)
// is a limit that at least `top` logits reach and, of logits in no order, few more do. Threads
// whose own maximum reaches it look through their runs. Where too many reach it (ties; a
// mask that leaves a few neighbours), the exact limit is found by four histograms of 8
// bits each, and of the logits equal to it the lowest tokens are taken.
template <int THREADS>
__device__ __forceinline__ void group_maxima(float m, bool any, TopShared& sh) {
  constexpr int GROUP = THREADS / 64;
  uint32_t g = any ? ordered(m) : 0;
#pragma unroll
  for (int off = 1; off < GROUP; off <<= 1) g = max(g, (uint32_t)__shfl_xor((int)g, off, 64));
  if ((threadIdx.x & (GROUP - 1)) == 0) sh.group[threadIdx.x / GROUP] = g;
  if (threadIdx.x == 0) sh.count = 0;
}

// After group_maxima and a barrier.
template <typename T, int THREADS, bool KEEP, int R, typename Emit>
__device__ __forceinline__ void select_top(const T* x, int vocab, int lo, int hi, int top, float m,
                                           const float (&kept)[R][8], TopShared& sh, Emit emit) {
  const int tid = threadIdx.x;
  uint32_t limit = 0;
  {
    const uint32_t g = sh.group[tid & 63];
#pragma unroll
    for (int bit = 31; bit >= 16; --bit) {
      const uint32_t higher = limit | 1u << bit;
      if (__popcll(__ballot(g >= higher)) >= top) limit = higher;
    }
  }
  auto offer = [&](const float (&v)[8], int run) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (8 * run + i < vocab && ordered(v[i]) >= limit) {
        const uint32_t at = atomicAdd(&sh.count, 1u);
        if (at < kList) sh.list[at] = key_of(v[i], 8 * run + i);
      }
    }
  };
  if (lo + tid < hi && ordered(m) >= limit) {
    if constexpr (KEEP) {
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (lo + tid + r * THREADS < hi) offer(kept[r], lo + tid + r * THREADS);
    } else {
      for (int run = lo + tid; run < hi; run += THREADS) {
        float v[8];
        load_logits(x, run, vocab, v);
        offer(v, run);
      }
    }
  }
  __syncthreads();
  if (sh.count > kList) {
    // the top-th largest logit, 8 bits at a time
    uint32_t prefix = 0;
    if (tid == 0) sh.need = (uint32_t)top;
    for (int shift = 24; shift >= 0; shift -= 8) {
      __syncthreads();
      for (int b = tid; b < 256; b += THREADS) sh.hist[b] = 0;
      __syncthreads();
      for (int run = lo + tid; run < hi; run += THREADS) {
        float v[8];
        load_logits(x, run, vocab, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t k = ordered(v[i]);
          if (8 * run + i < vocab && (shift == 24 || (k ^ prefix) >> (shift + 8) == 0))
            atomicAdd(&sh.hist[k >> shift & 255], 1u);
        }
      }
      __syncthreads();
      if (tid == 0) {
        uint32_t left = sh.need;
        int b = 255;
        while (sh.hist[b] < left) left -= sh.hist[b--];
        sh.need = left;  // of that bin
        sh.limit = (uint32_t)b;
      }
      __syncthreads();
      prefix |= sh.limit << shift;
    }
    // larger ones, fewer than top, in any order; then the lowest tokens of the equal ones
    const uint32_t need = sh.need;
    __syncthreads();
    if (tid == 0) sh.count = 0;
    __syncthreads();
    for (int run = lo + tid; run < hi; run += THREADS) {
      float v[8];
      load_logits(x, run, vocab, v);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (8 * run + i < vocab && ordered(v[i]) > prefix)
          sh.list[atomicAdd(&sh.count, 1u)] = key_of(v[i], 8 * run + i);
    }
    __syncthreads();
    const uint32_t above = (uint32_t)top - need;
    uint32_t found = 0;
    for (int base = lo; found < need && base < hi; base += THREADS) {
      const int run = base + tid;
      uint32_t mine = 0;
      if (run < hi) {
        float v[8];
        load_logits(x, run, vocab, v);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (8 * run + i < vocab && ordered(v[i]) == prefix) mine |= 1u << i;
      }
      // how many lie in the runs before this one
      uint32_t before = (uint32_t)__popc(mine);
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const uint32_t o = (uint32_t)__shfl_up((int)before, off, 64);
        if ((tid & 63) >= off) before += o;
      }
      __syncthreads();
      if ((tid & 63) == 63) sh.group[tid >> 6] = before;
      __syncthreads();
      before -= (uint32_t)__popc(mine);
      uint32_t all = 0;
      for (int w = 0; w < THREADS / 64; ++w) {
        if (w < tid >> 6) before += sh.group[w];
        all += sh.group[w];
      }
      before += found;
      for (int i = 0; i < 8; ++i)
        if (mine >> i & 1) {
          if (before < need) sh.list[above + before] = key_of(unordered(prefix), 8 * run + i);
          ++before;
        }
      found += all;
    }
    __syncthreads();
    if (tid == 0) sh.count = (uint32_t)top;
    __syncthreads();
  }
  // in order by counting the larger ones: keys are distinct, and at least min(top, elements)
  const int n = (int)sh.count;
  for (int c = tid; c < n; c += THREADS) {
    const uint64_t mine = sh.list[c];
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) rank += sh.list[j] > mine;
    if (rank < top) emit(rank, mine);
  }
  for (int k = n + tid; k < top; k += THREADS) emit(k, 0);
}

// What a row's sums give.
__device__ __forceinline__ float log_prob(float x, const Sums& q, float log_s) {
  // no finite logit: all probabilities are 0. (x - m is NaN for an infinity on both sides.)
  return x == -INFINITY && q.s == q.s ? -INFINITY : (x - q.m) - log_s;
}

// The row's results but the alternatives, by one thread.
template <typename T>
__device__ __forceinline__ void write_row(const TokenArgs& a, int64_t row, const Sums& q) {
  const float log_s = q.s == 0.f ? 0.f : logf(q.s);
  if (a.stats) {
    a.stats[2 * row] = q.s == 0.f ? -INFINITY : q.m;
    a.stats[2 * row + 1] = log_s;
  }
  if (a.entropy) a.entropy[row] = q.s == 0.f ? 0.f : log_s - q.t / q.s;
  if (a.logprob) {
    const int64_t t = a.targets[row];
    float lp = 0.f;
    if (t >= a.vocab)
      lp = NAN;
    else if (t >= 0)
      lp = log_prob(load_f32((const T*)a.x + row * a.ldx + t), q, log_s);
    a.logprob[row] = lp;
  }
}
__device__ __forceinline__ void write_top(const TokenArgs& a, int64_t row, const Sums& q, int k,
                                          uint64_t key) {
  const bool bad = q.s != q.s;
  const float log_s = q.s == 0.f ? 0.f : logf(q.s);
  const int64_t at = row * a.top + k;
  if (a.top_logprobs) a.top_logprobs[at] = bad ? NAN : log_prob(unordered((uint32_t)(key >> 32)), q, log_s);
  if (a.top_ids) a.top_ids[at] = bad ? -1 : (int64_t)(uint32_t)~(uint32_t)key;
}

// One workgroup per part of a row; parts == 1: the row's results, else the part's sums
// (a.part_sums) and alternatives (a.part_keys). KEEP: the part is one block of R runs a thread.
template <typename T, int THREADS, bool ENT, bool TOP, bool KEEP>
__global__ __launch_bounds__(THREADS) void token_kernel(TokenArgs a) {
  constexpr int R = 4;
  __shared__ float buf[THREADS / 64][3];
  const uint32_t line = blockIdx.x / (uint32_t)a.parts;
  const int64_t row = line;
  const int part = (int)(blockIdx.x - line * (uint32_t)a.parts);
  const T* x = (const T*)a.x + row * a.ldx;
  const int runs = (a.vocab + 7) >> 3;
  const int lo = part * a.part_runs, hi = min(runs, lo + a.part_runs);
  Sums q;
  q.init();
  float v[R][8];
  int base = lo + (int)threadIdx.x;
  do {
    Raw8<T> raw[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int run = base + r * THREADS;
      // past the end: the part's first run once more, replaced below
      raw[r].load_cut(x + 8 * (int64_t)(run < hi ? run : lo), run < hi ? a.vocab - 8 * run : 8);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int run = base + r * THREADS;
      raw[r].get(v[r]);
      const int valid = run < hi ? a.vocab - 8 * run : 0;
      if (valid < 8) cut_run(v[r], valid);
    }
    add_runs<ENT, R>(q, v);
    base += R * THREADS;
  } while (!KEEP && base < hi);
  if constexpr (TOP) {
    __shared__ TopShared sh;
    // kNone: masked logits alone, or none that is larger than the lowest number
    const float mine = q.m == kNone ? -INFINITY : q.m;
    group_maxima<THREADS>(mine, lo + (int)threadIdx.x < hi, sh);
    if constexpr (THREADS == 64) __syncthreads();
    q = block_sums<THREADS>(q, buf);
    if (a.parts == 1) {
      auto out = [&](int k, uint64_t key) { write_top(a, row, q, k, key); };
      if (q.s == q.s)
        select_top<T, THREADS, KEEP, R>(x, a.vocab, lo, hi, a.top, mine, v, sh, out);
      else
        for (int k = threadIdx.x; k < a.top; k += THREADS) out(k, 0);
    } else {
      uint64_t* keys = a.part_keys + (int64_t)blockIdx.x * a.top;
      auto out = [&](int k, uint64_t key) { keys[k] = key; };
      if (q.s == q.s)
        select_top<T, THREADS, KEEP, R>(x, a.vocab, lo, hi, a.top, mine, v, sh, out);
      else
        for (int k = threadIdx.x; k < a.top; k += THREADS) out(k, 0);
    }
  } else {
    q = block_sums<THREADS>(q, buf);
  }
  if (threadIdx.x != 0) return;
  if (a.parts == 1) {
    write_row<T>(a, row, q);
  } else {
    float* p = a.part_sums + 4 * (int64_t)blockIdx.x;
    p[0] = q.m;
    p[1] = q.s;
    p[2] = q.t;
  }
}

// The join of a row's parts: one workgroup per row, of one wavefront without alternatives.
template <typename T, bool TOP>
__global__ __launch_bounds__(TOP ? 256 : 64) void token_join_kernel(TokenArgs a) {
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63;
  Sums q;
  q.init();
  if (lane < a.parts) {
    const float* p = a.part_sums + 4 * (row * a.parts + lane);
    q.m = p[0];
    q.s = p[1];
    q.t = p[2];
  }
  if constexpr (TOP) {
    constexpr int kMost = kTokenParts * kTokenTop;
    __shared__ uint64_t keys[kMost];
    const int n = a.parts * a.top;
    for (int k = tid; k < n; k += 256) keys[k] = a.part_keys[row * n + k];
    q.raise(wave_max(q.m));
    q.s = wave_total(q.s);
    q.t = wave_total(q.t);
    __syncthreads();
    for (int k = tid; k < n; k += 256) {
      const uint64_t mine = keys[k];
      if (mine == 0 && q.s == q.s) continue;  // no element
      int rank = 0;
      // equal ones only in a row with a NaN, whose parts have none
#pragma unroll 8
      for (int j = 0; j < n; ++j) rank += keys[j] > mine || (keys[j] == mine && j < k);
      if (rank < a.top) write_top(a, row, q, rank, mine);
    }
  } else {
    q.raise(wave_max(q.m));
    q.s = wave_total(q.s);
    q.t = wave_total(q.t);
  }
  if (tid == 0) write_row<T>(a, row, q);
}

// The gradient, a segment of a row per workgroup. ENT: the entropy's too.
template <typename T, typename TO, int THREADS, bool ENT>
__global__ __launch_bounds__(THREADS) void token_backward_kernel(TokenBackArgs a) {
  const uint32_t line = blockIdx.x / (uint32_t)a.parts;
  const int64_t row = line;
  const int part = (int)(blockIdx.x - line * (uint32_t)a.parts);
  const int runs = (a.vocab + 7) >> 3;
  const int lo = part * a.part_runs, hi = min(runs, lo + a.part_runs);
  const T* x = (const T*)a.x + row * a.ldx;
  constexpr int R = 4;  // a segment is one block of runs
  Raw8<T> raw[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int run = lo + (int)threadIdx.x + r * THREADS;
    if (run < hi) raw[r].load_cut(x + 8 * (int64_t)run, a.vocab - 8 * run);
  }
  const int64_t target = a.targets ? a.targets[row] : -1;
  const float m = a.stats[2 * row], log_s = a.stats[2 * row + 1];
  float dlp = a.dlogprob && target >= 0 ? a.dlogprob[row] : 0.f;
  if (target >= a.vocab) dlp = NAN;
  const float dl = (a.dlse ? a.dlse[row] : 0.f) - dlp;
  const float de = ENT ? a.dentropy[row] : 0.f, h = ENT ? a.entropy[row] : 0.f;
  const bool empty = m == -INFINITY;
  if (empty) dlp = 0.f;
  const bool nothing = empty || (dl == 0.f && de == 0.f);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int run = lo + (int)threadIdx.x + r * THREADS;
    if (run >= hi) break;
    float v[8], o[8];
    raw[r].get(v);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float y = (v[i] - m) - log_s, p = exp_hw(y);
      o[i] = p * (ENT ? dl - de * (fmaxf(y, -1e4f) + h) : dl);
    }
    if (nothing) {  // whatever the row holds
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = 0.f;
    }
    const int64_t at = target - 8 * (int64_t)run;
    if (at >= 0 && at < 8) {
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] += i == (int)at ? dlp : 0.f;
    }
    store8n_any(a.dx, sizeof(TO) == 2 ? MAO_BF16 : MAO_F32, row * a.lddx + 8 * (int64_t)run, o,
                a.vocab - 8 * run);
  }
}

// Log probability and the gradient of -w logprob, a row per workgroup. KEEP: the row stays in
// registers (R runs of 8 a thread), else it is read twice.
template <typename T, int THREADS, int R, bool KEEP>
__global__ __launch_bounds__(THREADS) void token_loss_kernel(TokenBackArgs a) {
  __shared__ float buf[THREADS / 64][3];
  const int64_t row = blockIdx.x;
  const int runs = (a.vocab + 7) >> 3, tid = threadIdx.x;
  const T* x = (const T*)a.x + row * a.ldx;
  const int64_t target = a.targets[row];
  const int out_type = a.dx_dtype;
  if (target < 0) {  // nothing of the row matters
    const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int run = tid; run < runs; run += THREADS)
      store8n_any(a.dx, out_type, row * a.lddx + 8 * (int64_t)run, zero, a.vocab - 8 * run);
    if (tid == 0 && a.logprob) a.logprob[row] = 0.f;
    return;
  }
  float w = a.weight ? a.weight[row] : 1.f;
  if (target >= a.vocab) {
    w = NAN;
    if (tid == 0 && a.logprob) a.logprob[row] = NAN;
  }
  Raw8<T> raw[R];
  Sums q;
  q.init();
  if constexpr (KEEP) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int run = tid + r * THREADS;
      if (run < runs) raw[r].load_cut(x + 8 * (int64_t)run, a.vocab - 8 * run);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int run = tid + r * THREADS;
      if (run < runs) {
        float v[1][8];
        raw[r].get(v[0]);
        if (a.vocab - 8 * run < 8) cut_run(v[0], a.vocab - 8 * run);
        add_runs<false, 1>(q, v);
      }
    }
  } else {
    for (int base = tid; base < runs; base += THREADS * R) {
      float v[R][8];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int run = base + r * THREADS;
        raw[r].load_cut(x + 8 * (int64_t)(run < runs ? run : 0), run < runs ? a.vocab - 8 * run : 8);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int run = base + r * THREADS;
        raw[r].get(v[r]);
        const int valid = run < runs ? a.vocab - 8 * run : 0;
        if (valid < 8) cut_run(v[r], valid);
      }
      add_runs<false, R>(q, v);
    }
  }
  // dx may be x: a thread writes what it alone has read
  q = block_sums<THREADS>(q, buf);
  if (q.s == 0.f) w = 0.f;  // no finite logit
  const float scale = q.s == 0.f ? 0.f : w / q.s;
  auto finish = [&](int run, float (&v)[8]) __attribute__((always_inline)) {
    const int64_t at = target - 8 * (int64_t)run;
    float xt = 0.f;
    if (at >= 0 && at < 8) {
#pragma unroll
      for (int i = 0; i < 8; ++i) xt = i == (int)at ? v[i] : xt;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = exp_hw(v[i] - q.m) * scale;
    if (at >= 0 && at < 8 && target < a.vocab) {
      if (a.logprob) a.logprob[row] = log_prob(xt, q, q.s == 0.f ? 0.f : logf(q.s));
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] -= i == (int)at ? w : 0.f;
    }
    store8n_any(a.dx, out_type, row * a.lddx + 8 * (int64_t)run, v, a.vocab - 8 * run);
  };
  if constexpr (KEEP) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int run = tid + r * THREADS;
      if (run < runs) {
        float v[8];
        raw[r].opaque();
        raw[r].get(v);
        finish(run, v);
      }
    }
  } else {
    for (int run = tid; run < runs; run += THREADS) {
      float v[8];
      raw[0].load_cut(x + 8 * (int64_t)run, a.vocab - 8 * run);
      raw[0].get(v);
      finish(run, v);
    }
  }
}

template <typename T, int THREADS, bool KEEP>
mao_status forward_go(const TokenArgs& a, hipStream_t s) {
  const dim3 grid((uint32_t)((int64_t)a.rows * a.parts));
  const bool ent = a.entropy != nullptr, top = a.top != 0;
#define MAO_TOKEN(E, P) \
  hipLaunchKernelGGL((token_kernel<T, THREADS, E, P, KEEP>), grid, dim3(THREADS), 0, s, a)
  if (ent && top) MAO_TOKEN(true, true);
  else if (ent) MAO_TOKEN(true, false);
  else if (top) MAO_TOKEN(false, true);
  else MAO_TOKEN(false, false);
#undef MAO_TOKEN
  MAO_LAUNCH_CHECK();
  if (a.parts == 1) return MAO_OK;
  if (top)
    hipLaunchKernelGGL((token_join_kernel<T, true>), dim3(a.rows), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((token_join_kernel<T, false>), dim3(a.rows), dim3(64), 0, s, a);
  MAO_LAUNCH_CHECK();
  return MAO_OK;
}

template <typename T>
mao_status forward_pick(const TokenArgs& a, hipStream_t s) {
  if (a.part_runs <= 64 * 4) return forward_go<T, 64, true>(a, s);
  if (a.part_runs <= 256 * 4) return forward_go<T, 256, true>(a, s);
  return forward_go<T, 256, false>(a, s);
}

template <typename T, typename TO, int THREADS>
mao_status backward_go(TokenBackArgs a, hipStream_t s) {
  const int64_t runs = ceil_div(a.vocab, 8);
  a.parts = (int)ceil_div(runs, 4 * THREADS);
  a.part_runs = (int)ceil_div(runs, a.parts);
  const dim3 grid((uint32_t)((int64_t)a.rows * a.parts));
  if (a.dentropy)
    hipLaunchKernelGGL((token_backward_kernel<T, TO, THREADS, true>), grid, dim3(THREADS), 0, s, a);
  else
    hipLaunchKernelGGL((token_backward_kernel<T, TO, THREADS, false>), grid, dim3(THREADS), 0, s, a);
  MAO_LAUNCH_CHECK();
  return MAO_OK;
}

template <typename T, typename TO>
mao_status backward_pick(const TokenBackArgs& a, hipStream_t s) {
  return a.vocab <= 64 * 4 * 8 ? backward_go<T, TO, 64>(a, s) : backward_go<T, TO, 256>(a, s);
}

template <typename T, int THREADS, int R, bool KEEP>
mao_status loss_go(const TokenBackArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((token_loss_kernel<T, THREADS, R, KEEP>), dim3(a.rows), dim3(THREADS), 0, s, a);
  MAO_LAUNCH_CHECK();
  return MAO_OK;
}

template <typename T>
mao_status loss_pick(const TokenBackArgs& a, hipStream_t s) {
  const int64_t runs = ceil_div(a.vocab, 8);
  if (runs <= 64 * 2) return loss_go<T, 64, 2, true>(a, s);
  if (runs <= 256 * 4) return loss_go<T, 256, 4, true>(a, s);
  if (runs <= 1024 * 4) return loss_go<T, 1024, 4, true>(a, s);
  if (runs <= 1024 * 8) return loss_go<T, 1024, 8, true>(a, s);
  if (sizeof(T) == 2 && runs <= 1024 * 16) return loss_go<T, 1024, sizeof(T) == 2 ? 16 : 8, true>(a, s);
  return loss_go<T, 1024, 4, false>(a, s);
}

}  // namespace

TokenCut token_cut(int64_t rows, int64_t vocab) {
  // six workgroups per CU, of at least one block of 1024 runs of 8 each
  const int64_t runs = ceil_div(vocab, 8);
  int64_t parts = std::min<int64_t>(kTokenParts, ceil_div(6 * 256, rows));
  parts = std::max<int64_t>(1, std::min(parts, ceil_div(runs, 1024)));
  const int64_t per = ceil_div(runs, parts);
  return {(int)ceil_div(runs, per), (int)per};
}

mao_status launch_tokens(const TokenArgs& a, int dtype, hipStream_t s) {
  return dtype == MAO_BF16 ? forward_pick<bf16_t>(a, s) : forward_pick<float>(a, s);
}

mao_status launch_tokens_backward(const TokenBackArgs& a, int dtype, hipStream_t s) {
  if (dtype == MAO_BF16)
    return a.dx_dtype == MAO_BF16 ? backward_pick<bf16_t, bf16_t>(a, s)
                                  : backward_pick<bf16_t, float>(a, s);
  return a.dx_dtype == MAO_BF16 ? backward_pick<float, bf16_t>(a, s)
                                : backward_pick<float, float>(a, s);
}

mao_status launch_token_loss(const TokenBackArgs& a, int dtype, hipStream_t s) {
  return dtype == MAO_BF16 ? loss_pick<bf16_t>(a, s) : loss_pick<float>(a, s);
}

}  // namespace mao
