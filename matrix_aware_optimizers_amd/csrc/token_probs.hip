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
//
// One launch each, no workspace: a row belongs to a workgroup. Few rows are bounded by the call
// and the latency of one row, the rest by HBM (a copy of 1 GiB reaches 5.2 TB/s).
//
// Measured: forward bf16 16384 x 50304 269 us (6.1 TB/s), 4096 x 50304 with 20 alternatives 91
// (4.5), one row of 50304 6.6, with 20 alternatives 9.3; 77 rows 9.6; fp32 4096 x 50304 136 (6.1),
// with 20 alternatives 147 (5.6), one row 6.0 and 9.0. Backward bf16 8192 x 50304
// 270 us (6.1 TB/s), fp32 2045 x 50301 141 (5.8). Loss bf16 16384 x 50304 533 us (6.2 TB/s),
// 4096 x 128256 392 (5.4), 2048 x 256000 485 (4.3, or 6.5 with the second reading that bf16 rows
// beyond 196608 columns, fp32 ones beyond 98304, take), fp32 4096 x 50304 288 (5.7).
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

// Sums over the block's threads, in every thread. buf: 3 floats per wavefront, for one call.
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

template <int THREADS> struct TopShared {
  uint64_t list[kList];
  uint32_t group[64];
  uint32_t hist[256];
  uint32_t count, lines, limit, need;
  uint16_t line[THREADS];  // threads whose runs are looked through
};

// The `top` largest keys of a row, each handed to emit with its place in the order. m: the largest
// logit of this thread's runs, which `kept` holds if KEEP (R of them).
//
// The threads form 64 groups; the top-th largest of the groups' maxima is a limit that at least
// `top` logits reach and, of logits in no order, few more do. (All bits that the type has: with 16
// of them fp32 rows far from 0 sent thousands of logits past it, 1024 x 50304 around 4096 with 20
// alternatives 357 us for 37.) The runs of threads whose own maximum reaches it are looked through
// once more, by all threads. Where too many reach it (ties, rows in order), the exact limit is
// found by four histograms of 8 bits each, and of the logits equal to it the lowest tokens are
// taken. Masked logits are left out of that: where the others are fewer than `top`, the lowest
// masked tokens follow.
template <int THREADS>
__device__ __forceinline__ void group_maxima(float m, bool any, TopShared<THREADS>& sh) {
  constexpr int GROUP = THREADS / 64;
  uint32_t g = any ? ordered(m) : 0;
#pragma unroll
  for (int off = 1; off < GROUP; off <<= 1) g = max(g, (uint32_t)__shfl_xor((int)g, off, 64));
  if ((threadIdx.x & (GROUP - 1)) == 0) sh.group[threadIdx.x / GROUP] = g;
  if (threadIdx.x == 0) sh.count = sh.lines = 0;
}

// Hands the lowest `need` tokens (at most) whose logit is `equal` to emit, from place `at` on.
template <typename T, int THREADS, typename Emit>
__device__ void lowest_tokens(const T* x, int vocab, int runs, uint32_t equal, int at,
                              int need, TopShared<THREADS>& sh, Emit emit) {
  const int tid = threadIdx.x;
  int found = 0;
  for (int base = 0; found < need && base < runs; base += THREADS) {
    const int run = base + tid;
    uint32_t mine = 0;
    if (run < runs) {
      float v[8];
      load_logits(x, run, vocab, v);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (8 * run + i < vocab && ordered(v[i]) == equal) mine |= 1u << i;
    }
    // how many lie in the runs before this one
    int before = __popc(mine);
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int o = __shfl_up(before, off, 64);
      if ((tid & 63) >= off) before += o;
    }
    __syncthreads();
    if ((tid & 63) == 63) sh.group[tid >> 6] = (uint32_t)before;
    __syncthreads();
    before -= __popc(mine);
    int all = 0;
    for (int w = 0; w < THREADS / 64; ++w) {
      if (w < tid >> 6) before += (int)sh.group[w];
      all += (int)sh.group[w];
    }
    before += found;
    for (int i = 0; i < 8; ++i)
      if (mine >> i & 1) {
        if (before < need) emit(at + before, key_of(unordered(equal), 8 * run + i));
        ++before;
      }
    found += all;
  }
}

constexpr uint32_t kMasked = 0x007fffffu;  // ordered(-inf)

// After group_maxima and a barrier.
template <typename T, int THREADS, bool KEEP, int R, typename Emit>
__device__ __forceinline__ void select_top(const T* x, int vocab, int runs, int top, float m,
                                           const float (&kept)[R][8], TopShared<THREADS>& sh,
                                           Emit emit) {
  const int tid = threadIdx.x;
  uint32_t limit = 0;
  {
    const uint32_t g = sh.group[tid & 63];
#pragma unroll
    for (int bit = 31; bit >= (sizeof(T) == 2 ? 16 : 0); --bit) {
      const uint32_t higher = limit | 1u << bit;
      if (__popcll(__ballot(g >= higher)) >= top) limit = higher;
    }
  }
  limit = max(limit, kMasked + 1);
  auto offer = [&](const float (&v)[8], int run) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (8 * run + i < vocab && ordered(v[i]) >= limit) {
        const uint32_t at = atomicAdd(&sh.count, 1u);
        if (at < kList) sh.list[at] = key_of(v[i], 8 * run + i);
      }
    }
  };
  const bool reaches = tid < runs && ordered(m) >= limit;
  if constexpr (KEEP) {
    if (reaches) {
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (tid + r * THREADS < runs) offer(kept[r], tid + r * THREADS);
    }
  } else {
    if (reaches) sh.line[atomicAdd(&sh.lines, 1u)] = (uint16_t)tid;
    __syncthreads();
    // run r of thread line[l] for all r and l, four at a time
    const int lines = (int)sh.lines, all = lines * ((runs + THREADS - 1) / THREADS);
    for (int k0 = tid; k0 < all; k0 += 4 * THREADS) {
      float v[4][8];
      int run[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int k = k0 + u * THREADS, r = k / lines;
        run[u] = k < all ? r * THREADS + sh.line[k - r * lines] : runs;
        load_logits(x, run[u] < runs ? run[u] : 0, vocab, v[u]);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (run[u] < runs) offer(v[u], run[u]);
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
      for (int run = tid; run < runs; run += THREADS) {
        float v[8];
        load_logits(x, run, vocab, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t k = ordered(v[i]), bin = k >> shift & 255;
          const bool in = 8 * run + i < vocab && (shift == 24 || (k ^ prefix) >> (shift + 8) == 0);
          // lanes of one bin (equal logits, most often) add together
          const uint64_t in_lanes = __ballot(in);
          if (in_lanes == 0) continue;
          const int first = __ffsll((unsigned long long)in_lanes) - 1;
          const uint32_t one = (uint32_t)__builtin_amdgcn_readlane((int)bin, first);
          const uint64_t same = __ballot(in && bin == one);
          if ((tid & 63) == first) atomicAdd(&sh.hist[one], (uint32_t)__popcll(same));
          if (in && bin != one) atomicAdd(&sh.hist[bin], 1u);
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
    const int need = (int)sh.need, above = top - need;
    __syncthreads();
    if (tid == 0) sh.count = 0;
    __syncthreads();
    if (above > 0) {
      for (int run = tid; run < runs; run += THREADS) {
        float v[8];
        load_logits(x, run, vocab, v);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (8 * run + i < vocab && ordered(v[i]) > prefix)
            sh.list[atomicAdd(&sh.count, 1u)] = key_of(v[i], 8 * run + i);
      }
    }
    lowest_tokens<T, THREADS>(x, vocab, runs, prefix, above, need, sh, emit);
    __syncthreads();
  } else if ((int)sh.count < top) {
    // fewer than top that are not masked
    lowest_tokens<T, THREADS>(x, vocab, runs, kMasked, (int)sh.count, top - (int)sh.count, sh, emit);
  }
  // in order by counting the larger ones: keys are distinct
  const int n = (int)sh.count;
  for (int c = tid; c < n; c += THREADS) {
    const uint64_t mine = sh.list[c];
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) rank += sh.list[j] > mine;
    if (rank < top) emit(rank, mine);
  }
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

// A row per workgroup, in blocks of R runs a thread. KEEP: the row is one block.
template <typename T, int THREADS, bool ENT, bool TOP, bool KEEP>
__global__ __launch_bounds__(THREADS) void token_kernel(TokenArgs a) {
  constexpr int R = 4;
  __shared__ float buf[THREADS / 64][3];
  const int64_t row = blockIdx.x;
  const T* x = (const T*)a.x + row * a.ldx;
  const int runs = (a.vocab + 7) >> 3;
  Sums q;
  q.init();
  float v[R][8];
  int base = (int)threadIdx.x;
  do {
    Raw8<T> raw[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int run = base + r * THREADS;
      // past the end: the row's first run once more, replaced below
      raw[r].load_cut(x + 8 * (int64_t)(run < runs ? run : 0), a.vocab - (run < runs ? 8 * run : 0));
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int run = base + r * THREADS;
      raw[r].get(v[r]);
      const int valid = run < runs ? a.vocab - 8 * run : 0;
      if (valid < 8) cut_run(v[r], valid);
    }
    if (KEEP && runs <= R / 2 * THREADS)
      add_runs<ENT, R / 2>(q, (const float(&)[R / 2][8])v);
    else
      add_runs<ENT, R>(q, v);
    base += R * THREADS;
  } while (!KEEP && base < runs);
  if constexpr (TOP) {
    __shared__ TopShared<THREADS> sh;
    const float mine = q.m;
    group_maxima<THREADS>(mine, (int)threadIdx.x < runs, sh);
    if constexpr (THREADS == 64) __syncthreads();
    q = block_sums<THREADS>(q, buf);
    auto out = [&](int k, uint64_t key) { write_top(a, row, q, k, key); };
    if (q.s == q.s)
      select_top<T, THREADS, KEEP, R>(x, a.vocab, runs, a.top, mine, v, sh, out);
    else
      for (int k = threadIdx.x; k < a.top; k += THREADS) out(k, 0);
  } else {
    q = block_sums<THREADS>(q, buf);
  }
  if (threadIdx.x == 0) write_row<T>(a, row, q);
}

// Gradients work on pieces of 16 bytes: consecutive lanes read consecutive ones. (fp32 in
// runs of 8, of which each load takes every other 16 bytes: 2045 x 50301 167 us for 145, in the
// first form of the kernel.)
template <typename T> struct Piece {
  static constexpr int W = 16 / sizeof(T);
  u32x4 a;
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t row, int piece) {
    a = __builtin_amdgcn_raw_buffer_load_b128(row, piece * 16, 0, 0);
  }
  // the compiler may not carry values derived from here on across this point
  __device__ __forceinline__ void opaque() {
    asm volatile("" : "+v"(a[0]), "+v"(a[1]), "+v"(a[2]), "+v"(a[3]));
  }
  __device__ __forceinline__ void get(float (&v)[W]) const {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if (W == 4)
        v[i] = __uint_as_float(a[i]);
      else
        v[i] = __uint_as_float(i & 1 ? a[i >> 1] & 0xffff0000u : a[i >> 1] << 16);
    }
  }
};

// A row of results, written past the caches at every size: us, past them / through them, bf16, (with
// a reading of the gradient right after): loss 16 x 50304 8.9 / 8.9 (11.2 / 11.1), 256 x 50304 10.8 /
// 12.8 (21.5 / 21.1), 1024 x 50304 32.3 / 44.1 (78.5 / 77.2), 4096 x 50304 141 / 147 (310 / 301),
// 16384 x 8000 90 / 95 (203 / 194); gradient of log probabilities 16 x 50304 3.5 / 3.8 (7.1 / 7.1),
// 256 x 50304 6.8 / 10.3 (20.5 / 19.0), 16384 x 8000 75 / 93 (197 / 190). So the call gains up to a
// third, and a reader that follows at once pays it back and up to 10% of the two on top (1024 x
// 50304, gradient: 72.1 / 79.4): no size divides gain from loss.
template <int W> struct RowOut {
  char* p;
  int dtype, cols;
  __amdgpu_buffer_rsrc_t buf;  // its whole pieces
  __device__ __forceinline__ RowOut(void* base, int dt, int64_t ld, int row, int n)
      : dtype(dt), cols(n) {
    const int es = dt == MAO_BF16 ? 2 : 4;
    p = (char*)base + ld * es * row;
    buf = row_buffer(base, ld * es, row, n / W * W * es);
  }
  __device__ __forceinline__ void store(int piece, const float (&v)[W]) const {
    constexpr int NT = 2;
    if (dtype == MAO_BF16) {
      if constexpr (W == 8) {
        const u32x4 k = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                         pack_bf16x2(v[6], v[7])};
        __builtin_amdgcn_raw_buffer_store_b128(k, buf, piece * 16, 0, NT);
      } else {
        const u32x2 k = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        __builtin_amdgcn_raw_buffer_store_b64(k, buf, piece * 8, 0, NT);
      }
    } else {
#pragma unroll
      for (int i = 0; i < W; i += 4) {
        const u32x4 k = {__float_as_uint(v[i]), __float_as_uint(v[i + 1]), __float_as_uint(v[i + 2]),
                         __float_as_uint(v[i + 3])};
        __builtin_amdgcn_raw_buffer_store_b128(k, buf, piece * (W * 4) + i * 4, 0, NT);
      }
    }
    const int n = cols - W * piece;
    if (n > 0 && n < W) {
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (i < n) {
          if (dtype == MAO_BF16)
            ((bf16_t*)p)[W * piece + i] = f32_to_bf16(v[i]);
          else
            ((float*)p)[W * piece + i] = v[i];
        }
    }
  }
};

// Pieces a thread of the backward pass: 8192 x 50304 bf16 269 us with two, 291 with four, 299
// with one; 2045 x 50301 fp32 140, 145 and 141.
constexpr int kBackPieces = 2;

// The gradient, a segment of a row (kBackPieces a thread) per workgroup. ENT: the entropy's too.
template <typename T, int THREADS, bool ENT>
__global__ __launch_bounds__(THREADS) void token_backward_kernel(TokenBackArgs a) {
  constexpr int R = kBackPieces, W = Piece<T>::W;
  const uint32_t line = blockIdx.x / (uint32_t)a.parts;
  const int64_t row = line;
  const int part = (int)(blockIdx.x - line * (uint32_t)a.parts);
  const int lo = part * a.part_runs + (int)threadIdx.x, hi = (part + 1) * a.part_runs;
  const auto x = row_buffer(a.x, a.ldx * (int64_t)sizeof(T), (int)line, (a.vocab + W - 1) / W * 16);
  const RowOut<W> out(a.dx, a.dx_dtype, a.lddx, (int)line, a.vocab);
  Piece<T> raw[R];
#pragma unroll
  for (int r = 0; r < R; ++r) raw[r].load(x, lo + r * THREADS);
  const int64_t target = a.targets ? a.targets[row] : -1;
  const float m = a.stats[2 * row], log_s = a.stats[2 * row + 1];
  float dlp = a.dlogprob && target >= 0 ? a.dlogprob[row] : 0.f;
  if (target >= a.vocab && dlp != 0.f) dlp = NAN;
  const float dlse = a.dlse ? a.dlse[row] : 0.f, dl = dlse - dlp;
  const float de = ENT ? a.dentropy[row] : 0.f, h = ENT ? a.entropy[row] : 0.f;
  const bool empty = m == -INFINITY;
  if (empty) dlp = 0.f;
  const bool nothing = empty || (dlp == 0.f && dlse == 0.f && de == 0.f);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int piece = lo + r * THREADS;
    if (piece >= hi) break;
    float v[W], o[W];
    raw[r].get(v);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float y = (v[i] - m) - log_s, p = exp_hw(y);
      o[i] = p * (ENT ? dl - de * (fmaxf(y, -1e4f) + h) : dl);
    }
    if (nothing) {  // whatever the row holds
#pragma unroll
      for (int i = 0; i < W; ++i) o[i] = 0.f;
    }
    const int64_t at = target - W * (int64_t)piece;
    if (at >= 0 && at < W) {
#pragma unroll
      for (int i = 0; i < W; ++i) o[i] += i == (int)at ? dlp : 0.f;
    }
    out.store(piece, o);
  }
}

template <int W>
__device__ __forceinline__ void add_piece(Sums& q, float (&v)[W], int valid) {
  if (valid < W) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = i < valid ? v[i] : -INFINITY;
  }
  float c = max3(v[0], v[1], v[2]);
  c = max3(c, v[3], v[W - 1]);
  if constexpr (W == 8) {
    c = max3(c, v[4], v[5]);
    c = max3(c, v[6], c);
  }
  if (c > q.m) q.raise(c);
  float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < W; ++i) s[i & 3] += exp_hw(v[i] - q.m);
  q.s += (s[0] + s[1]) + (s[2] + s[3]);
}

// Log probability and the gradient of -w logprob, a row per workgroup. KEEP: the row stays in
// registers (R pieces a thread), else it is read twice. (Workgroups that go on to a next row and
// read it as they write, 1 to 4 of them at a time per place on the CUs: 610 to 617 us on
// 16384 x 50304 bf16, 540 with a workgroup for each row.)
template <typename T, int THREADS, int R, bool KEEP>
__global__ __launch_bounds__(THREADS) void token_loss_kernel(TokenBackArgs a) {
  constexpr int W = Piece<T>::W;
  __shared__ float buf[THREADS / 64][3];
  const int pieces = (a.vocab + W - 1) / W, tid = threadIdx.x, row = blockIdx.x;
  const int64_t target = a.targets[row];
  const bool live = target >= 0;  // else nothing of the row matters
  const int hit = live && target < a.vocab ? (int)target : -1;
  // a row that does not matter is not read
  const auto x = row_buffer(a.x, a.ldx * (int64_t)sizeof(T), row, live ? pieces * 16 : 0);
  const RowOut<W> out(a.dx, a.dx_dtype, a.lddx, row, a.vocab);
  Piece<T> raw[R];
  Sums q;
  q.init();
  for (int base = tid; base < pieces; base += THREADS * R) {
#pragma unroll
    for (int r = 0; r < R; ++r) raw[r].load(x, base + r * THREADS);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int piece = base + r * THREADS;
      if (piece < pieces) {
        float v[W];
        raw[r].get(v);
        add_piece<W>(q, v, a.vocab - W * piece);
      }
    }
    if (KEEP) break;
  }
  // dx may be x: a thread writes what it alone has read
  q = block_sums<THREADS>(q, buf);
  float w = a.weight && live ? a.weight[row] : 1.f;
  if (target >= a.vocab && w != 0.f) w = NAN;
  if (q.s == 0.f) w = 0.f;  // no finite logit
  const float scale = w / q.s;
  const bool nothing = !live || w == 0.f;
  if (a.logprob && hit < 0 && tid == 0) a.logprob[row] = live ? NAN : 0.f;
  auto finish = [&](Piece<T>& k, int piece) __attribute__((always_inline)) {
    float v[W];
    k.opaque();
    k.get(v);
    const int at = hit - W * piece;
    const bool here = hit >= 0 && at >= 0 && at < W;
    float xt = 0.f;
    if (here) {
#pragma unroll
      for (int i = 0; i < W; ++i) xt = i == at ? v[i] : xt;
    }
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = nothing ? 0.f : exp_hw(v[i] - q.m) * scale;
    if (here) {
      if (a.logprob) a.logprob[row] = log_prob(xt, q, q.s == 0.f ? 0.f : logf(q.s));
#pragma unroll
      for (int i = 0; i < W; ++i) v[i] -= i == at ? w : 0.f;
    }
    out.store(piece, v);
  };
  for (int base = tid; base < pieces; base += THREADS * R) {
    if (!KEEP) {
#pragma unroll
      for (int r = 0; r < R; ++r) raw[r].load(x, base + r * THREADS);
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (base + r * THREADS < pieces) finish(raw[r], base + r * THREADS);
    if (KEEP) break;
  }
}

template <typename T, int THREADS, bool KEEP>
mao_status forward_go(const TokenArgs& a, hipStream_t s) {
  const bool ent = a.entropy != nullptr, top = a.top != 0;
#define MAO_TOKEN(E, P) \
  hipLaunchKernelGGL((token_kernel<T, THREADS, E, P, KEEP>), dim3(a.rows), dim3(THREADS), 0, s, a)
  if (ent && top) MAO_TOKEN(true, true);
  else if (ent) MAO_TOKEN(true, false);
  else if (top) MAO_TOKEN(false, true);
  else MAO_TOKEN(false, false);
#undef MAO_TOKEN
  MAO_LAUNCH_CHECK();
  return MAO_OK;
}

// Threads of a row. Long rows, bf16, no alternatives / 20 of them, in us:
//   50304: 256 threads 7.4 / 11.8 (1 row), 20.6 / 28.0 (1024 rows); 512 threads 6.4 / 9.4, 20.1 /
//   26.0; 1024 threads 6.6 / 10.2, 24.1 / 39.2
//   20000: 256 threads 11.2 / 15.6 (1024 rows), 512 threads 13.2 / 18.8
// Above 65536, 512 threads and 1024, at 128 rows, 256 and 320 (a second row on some CUs):
//   65544: 8.0 / 11.2 and 7.5 / 11.1, 9.1 / 12.1 and 8.9 / 12.5, 13.0 / 16.7 and 13.1 / 20.3
//   128256: 12.9 / 17.0 and 11.8 / 15.6, 13.9 / 18.6 and 13.4 / 17.2, 21.4 / 27.2 and 21.5 / 28.8
//   256000: 23.4 / 29.4 and 20.8 / 25.2, 24.2 / 32.6 and 23.2 / 27.6, 41.2 / 50.1 and 42.2 / 50.2
//   (one row: 65544 7.1 / 10.0 and 6.8 / 10.4, 256000 20.3 / 24.7 and 18.8 / 22.7)
// A row over four workgroups and a second kernel to join them took 10 / 11.7 on one row of 50304 and
// gained nothing below 128256 columns or above 256 rows; one row of 256000, which a CU's
// arithmetic bounds, took 10 / 16 for 19 / 23. Left out: chosen here, for those sizes alone, it would
// cost the other calls nothing, and those two kernels more.
template <typename T>
mao_status forward_pick(const TokenArgs& a, hipStream_t s) {
  const int64_t runs = ceil_div(a.vocab, 8);
  if (runs <= 64 * 4) return forward_go<T, 64, true>(a, s);
  if (runs <= 256 * 4) return forward_go<T, 256, true>(a, s);
  if (runs <= 4096) return forward_go<T, 256, false>(a, s);
  // few very long rows: latency, a row has a CU to itself
  if (runs > 8192 && a.rows <= 256) return forward_go<T, 1024, false>(a, s);
  return forward_go<T, 512, false>(a, s);
}

template <typename T, int THREADS>
mao_status backward_go(TokenBackArgs a, hipStream_t s) {
  const int64_t pieces = ceil_div(a.vocab, Piece<T>::W);
  a.parts = (int)ceil_div(pieces, kBackPieces * THREADS);
  a.part_runs = (int)ceil_div(pieces, a.parts);
  const dim3 grid((uint32_t)((int64_t)a.rows * a.parts));
  if (a.dentropy)
    hipLaunchKernelGGL((token_backward_kernel<T, THREADS, true>), grid, dim3(THREADS), 0, s, a);
  else
    hipLaunchKernelGGL((token_backward_kernel<T, THREADS, false>), grid, dim3(THREADS), 0, s, a);
  MAO_LAUNCH_CHECK();
  return MAO_OK;
}

template <typename T>
mao_status backward_pick(const TokenBackArgs& a, hipStream_t s) {
  return a.vocab <= 64 * Piece<T>::W * kBackPieces ? backward_go<T, 64>(a, s)
                                                      : backward_go<T, 256>(a, s);
}

template <typename T, int THREADS, int R, bool KEEP>
mao_status loss_go(const TokenBackArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((token_loss_kernel<T, THREADS, R, KEEP>), dim3(a.rows), dim3(THREADS), 0, s, a);
  MAO_LAUNCH_CHECK();
  return MAO_OK;
}

template <typename T>
mao_status loss_pick(const TokenBackArgs& a, hipStream_t s) {
  const int64_t pieces = ceil_div(a.vocab, Piece<T>::W);
  if (pieces <= 64 * 4) return loss_go<T, 64, 4, true>(a, s);
  if (pieces <= 256 * 4) return loss_go<T, 256, 4, true>(a, s);
  if (pieces <= 512 * 4) return loss_go<T, 512, 4, true>(a, s);
  if (pieces <= 1024 * 4) return loss_go<T, 1024, 4, true>(a, s);
  if (pieces <= 1024 * 8) return loss_go<T, 1024, 8, true>(a, s);
  if (pieces <= 1024 * 16) return loss_go<T, 1024, 16, true>(a, s);
  if (pieces <= 1024 * 24) return loss_go<T, 1024, 24, true>(a, s);
  return loss_go<T, 1024, 4, false>(a, s);
}

}  // namespace

mao_status launch_tokens(const TokenArgs& a, int dtype, hipStream_t s) {
  return dtype == MAO_BF16 ? forward_pick<bf16_t>(a, s) : forward_pick<float>(a, s);
}

mao_status launch_tokens_backward(const TokenBackArgs& a, int dtype, hipStream_t s) {
  return dtype == MAO_BF16 ? backward_pick<bf16_t>(a, s) : backward_pick<float>(a, s);
}

mao_status launch_token_loss(const TokenBackArgs& a, int dtype, hipStream_t s) {
  return dtype == MAO_BF16 ? loss_pick<bf16_t>(a, s) : loss_pick<float>(a, s);
}

}  // namespace mao
