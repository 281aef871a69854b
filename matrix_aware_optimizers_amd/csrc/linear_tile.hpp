// The linear layer's products on matrix cores, with bias, activation, residual
// and the activation's slope applied as a result leaves.
//
//   forward            y  = act(x W^T + b) + res   A = x  (T x K), B = W (N x K)
//   input gradient     dx = (dy W) . act'(z) + add A = dy (T x N), B = W read K-major
//   weight gradient    dW = dy^T x (+ dW)          A = dy, B = x, both K-major
//
// "K-major": the reduction runs down the rows of the stored matrix. Nothing is
// transposed in memory: K-major bf16 tiles are read from LDS with the
// transposing read (ds_read_b64_tr_b16), fp32 ones by single elements, whose
// MFMA (32x32x2) takes one element per lane anyway.
//
// A workgroup of 4 wavefronts (2 x 2), or 8 (4 x 2) for the tiles of 256 rows,
// computes a BM x BN tile, each wavefront its share of it as 32 x 32 MFMA blocks,
// fp32 accumulation. K advances in
// slices of KSB bytes per row, copied global -> LDS without staging registers
// into a ring of NST stages. One barrier per slice: before it every wavefront
// has read its last fragments of slice k and waited for its loads of slice
// k + 1; after it the stage of slice k is refilled with slice k + NST while the
// fragments of k + 1 are read under the last MFMAs of k. Each stage is its own
// LDS object, so the compiler's waits stay exact.
//
// LDS layouts. A K-contiguous slice keeps KSB bytes per row, 16-byte chunks
// XOR-permuted by the row so that 16 consecutive rows' reads cover all banks.
// A K-major slice keeps one row per k, chunks XOR-permuted by the k row so that
// the four rows of a transposing read do.
//
// Rows and columns past M and N re-read valid storage; they feed outputs that
// are never stored. A partial last slice goes through registers with zero
// fill on both operands.
//
// Epilogue: each wavefront passes its blocks through a private piece of LDS, 32
// rows at a time and without workgroup barriers, so that bias, activation,
// residual and stores move 16-byte pieces and whole 128-byte lines of a bf16 row
// leave in one instruction.
//
// Few tiles: K is split over several workgroups per tile. Their fp32 partial
// results go to the workspace, and a second launch (linear_join.hip) adds them
// in a fixed order and finishes the result. No atomics anywhere.
//
// Bound: matrix cores for thousands of rows, plus a result's way out, which nothing
// hides: one workgroup of 256 x 256 tiles fills a CU, and every round ends in a burst
// of stores. Measured (MI355X, bf16, 16384 rows): 1536 -> 6144 without epilogue 278 us,
// 1110 TFLOP/s; keeping the pre-activation too adds 36 (201 MB written, 38 us at the
// copy rate), gelu_tanh 15 (9 beside the stores of both). Input gradient of 6144 ->
// 1536 271 us; reading int8 codes and relu's slope adds 25, gelu_tanh's 25 more. dW of
// 8191 rows 14336 -> 4096 840 us, 1146 TFLOP/s. The ROCm library's bare products on
// the same tensors: 214, 251 and 968 us (another card: 289, 275 and 856 against 226, 262
// and 985). Counters of the four products of 16384 and 8191 rows with their epilogues:
// matrix cores busy 44 to 55% of the time at 1.9 to 2.0 GHz, LDS active 20 to 25% of it
// (4 to 16% of that bank conflicts), L2 hit rate 72 to 79%, 1.0 to 1.9 TB/s past the L2:
// none is at its limit, the wavefronts wait. fp32, 4096 rows, 1536 -> 6144 and its two
// gradients: 617, 631 and 601 us, 80 to 84% of the fp32 matrix cores' 153 TFLOP/s.
#pragma once

#include "act.hpp"
#include "layers.hpp"
#include "linear.hpp"

namespace mao {

namespace {

typedef __attribute__((address_space(3))) void lds_void_t;
typedef __attribute__((address_space(1))) const void gbl_void_t;
typedef short lds_v4i16_t __attribute__((ext_vector_type(4), address_space(3)));

// s_waitcnt with vmcnt(n) and lgkmcnt(0)
template <int N>
__device__ __forceinline__ void wait_slice() {
  __builtin_amdgcn_s_waitcnt((N & 0xf) | (0x7 << 4) | ((N >> 4) << 14));
}

// s_waitcnt with lgkmcnt(0) alone
__device__ __forceinline__ void wait_lds() {
  __builtin_amdgcn_s_waitcnt(0xf | (0x7 << 4) | (0x3 << 14));
}

// What the epilogue does beyond D = acc + add.
// EPI_PARTIAL: fp32 partial results of a split product, which the join reads soon.
enum EpiKind { EPI_PLAIN, EPI_FORWARD, EPI_SLOPE, EPI_PARTIAL };

// A result line is written whole and not read again here: it should not push
// operand panels out of the L2 (16384 x 6144 x 1536 with gelu and its
// pre-activation kept 342 -> 330 us, 16384 x 1536 x 6144 271 -> 253 us).
__device__ __forceinline__ void store_once(void* p, const uint4& v) {
  typedef __attribute__((ext_vector_type(4))) uint32_t u32x4_t;
  const u32x4_t t = {v.x, v.y, v.z, v.w};
  __builtin_nontemporal_store(t, (u32x4_t*)p);
}

// Stores v[0 .. valid) (8 at most) at element off. A run cut by the last column
// goes out element by element, in a loop (rare, and short code matters here).
template <bool BF, bool ONCE = true>
__device__ __forceinline__ void put8(void* p, int dtype, int64_t off, const float (&v)[8],
                                     int valid) {
  if (BF || dtype == MAO_BF16) {
    uint4 k;
    k.x = pack_bf16x2(v[0], v[1]);
    k.y = pack_bf16x2(v[2], v[3]);
    k.z = pack_bf16x2(v[4], v[5]);
    k.w = pack_bf16x2(v[6], v[7]);
    bf16_t* d = (bf16_t*)p + off;
    if (valid >= 8) {
      store_once(d, k);
    } else {
#pragma unroll 1
      for (int i = 0; i < valid; ++i) {
        d[i] = (bf16_t)k.x;
        k.x = (k.x >> 16) | (k.y << 16);
        k.y = (k.y >> 16) | (k.z << 16);
        k.z = (k.z >> 16) | (k.w << 16);
        k.w >>= 16;
      }
    }
  } else {
    float* d = (float*)p + off;
    if (valid >= 8) {
      const uint4 a = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]),
                                 __float_as_uint(v[2]), __float_as_uint(v[3]));
      const uint4 b = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]),
                                 __float_as_uint(v[6]), __float_as_uint(v[7]));
      if constexpr (ONCE) {
        store_once(d, a);
        store_once(d + 4, b);
      } else {
        *(uint4*)d = a;
        *(uint4*)(d + 4) = b;
      }
    } else {
      float w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = v[i];
#pragma unroll 1
      for (int i = 0; i < valid; ++i) {
        d[i] = w[0];
#pragma unroll
        for (int k = 0; k < 7; ++k) w[k] = w[k + 1];
      }
    }
  }
}

// Eight values of a tensor, as loaded (BF: known to be bf16); of fewer valid ones the
// 16-byte pieces that hold one (as Raw8::load_cut).
template <bool BF> struct RawT {
  uint4 a, b[1];
  __device__ __forceinline__ void load(const void* p, int dtype, int64_t off, int valid) {
    if (BF || dtype == MAO_BF16) {
      a = *(const uint4*)((const bf16_t*)p + off);
    } else {
      a = *(const uint4*)((const float*)p + off);
      b[0] = *(const uint4*)((const float*)p + off + (valid > 4 ? 4 : 0));
    }
  }
  __device__ __forceinline__ void get(int dtype, float (&v)[8]) const {
    if (BF || dtype == MAO_BF16) {
      Raw8<bf16_t> r;
      r.a = a;
      r.get(v);
    } else {
      const uint32_t w[8] = {a.x, a.y, a.z, a.w, b[0].x, b[0].y, b[0].z, b[0].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
    }
  }
};

// Finishes a 32 x (32 JU) piece of a wavefront's result at (row0, col0). The
// blocks were computed transposed (MFMA rows are result columns), so a lane has
// four consecutive columns of one row per register group: 16-byte writes into
// the wavefront's own LDS piece `reg` (rows padded by 8 floats), from where each
// lane takes runs of 8 columns, 128 (JU = 2) or 192 bytes of a bf16 row together.
// The tensors that join are loaded, in the same runs, before the exchange. bias:
// LDS, from column col0. BF: every tensor but a checkpoint is bf16.
constexpr int piece_ld(int ju) { return 32 * ju + 8; }

template <EpiKind KIND, int ACT, bool BF, int JU>
__device__ __forceinline__ void finish(const f32x16_t* acc, float* reg, const LinProblem& P,
                                       const float* bias, int row0, int col0) {
  const LinEpilogue& e = P.e;
  constexpr int LD = piece_ld(JU), CPR = 4 * JU, IT = 2 * JU;
  constexpr bool SLOPE = KIND == EPI_SLOPE && ACT != MAO_ACT_NONE;
  const int lane = threadIdx.x & 63;
  const bool q8 = SLOPE && e.z_kind > MAO_BF16;
  struct Inputs {
    RawT<BF> z, a;
    int scale;
  };
  auto load = [&](int it, Inputs& t) __attribute__((always_inline)) {
    const int idx = it * 64 + lane, row = row0 + idx / CPR, col = col0 + 8 * (idx % CPR);
    if (row >= P.M || col >= P.N) return;
    if constexpr (SLOPE) {
      const int64_t off = (int64_t)row * e.ldzi + col;
      if (q8) {
        const uint2 w = *(const uint2*)((const uint8_t*)e.z_in + off);
        t.z.a.x = w.x;
        t.z.a.y = w.y;
        t.scale = e.z_scales[(int64_t)row * e.ldzs + (col >> 5)];
      } else {
        t.z.load(e.z_in, e.z_kind, off, P.N - col);
      }
    }
    if (e.add != nullptr)
      t.a.load(e.add, e.add_dtype, (int64_t)row * e.ldadd + col, P.N - col);
  };
  Inputs t0, t1;
  load(0, t0);
  load(1, t1);
  {
    float* d = reg + (lane & 31) * LD + 4 * (lane >> 5);
#pragma unroll
    for (int j = 0; j < JU; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *(float4*)(d + 32 * j + 8 * g) = make_float4(acc[j][4 * g], acc[j][4 * g + 1],
                                                     acc[j][4 * g + 2], acc[j][4 * g + 3]);
  }
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  // rolled: most launches run this code once per workgroup, from a cold
  // instruction cache
#pragma unroll 1
  for (int it = 0; it < IT; ++it) {
    const int idx = it * 64 + lane, rr = idx / CPR, cc = 8 * (idx % CPR);
    const int row = row0 + rr, col = col0 + cc, valid = P.N - col;
    const float4 lo = *(const float4*)(reg + rr * LD + cc);
    const float4 hi = *(const float4*)(reg + rr * LD + cc + 4);
    float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    const Inputs t = t0;
    t0 = t1;
    if (it + 2 < IT) load(it + 2, t1);
    if (row >= P.M || valid <= 0) continue;
    if constexpr (KIND == EPI_FORWARD) {
      const float4 b0 = *(const float4*)(bias + cc), b1 = *(const float4*)(bias + cc + 4);
      const float w[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] += w[k];
      if (e.z_out) put8<BF>(e.z_out, e.zo_dtype, (int64_t)row * e.ldzo + col, v, valid);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = act_value<ACT>(v[k]);
    }
    if constexpr (SLOPE) {
      float z[8];
      if (q8) {
        const float s = q8_scale_value(t.scale);
        const int fmt = e.z_kind == kXInt8 ? MAO_Q8_INT8 : MAO_Q8_E4M3;
        q8_decode4_any(fmt, t.z.a.x, s, z);
        q8_decode4_any(fmt, t.z.a.y, s, z + 4);
      } else {
        t.z.get(e.z_kind, z);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] *= act_slope<ACT>(z[k]);
    }
    if (e.add != nullptr) {
      float w[8];
      t.a.get(e.add_dtype, w);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] += w[k];
    }
    put8<BF, KIND != EPI_PARTIAL>(e.D, e.d_dtype, (int64_t)row * e.ldd + col, v, valid);
  }
  // the next piece overwrites reg: this one's reads are done
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
}

// All pieces of a wavefront, FM x FN blocks from (row0, col0).
template <EpiKind KIND, int ACT, bool BF, int JU, int FM, int FN>
__device__ __forceinline__ void finish_all(const f32x16_t (&acc)[FM][FN], float* reg,
                                           const LinProblem& P, const float* bias, int row0,
                                           int col0) {
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; j += JU)
      finish<KIND, ACT, BF, JU>(&acc[i][j], reg, P, bias + 32 * j, row0 + 32 * i, col0 + 32 * j);
}

// One contiguous piece of code per activation.
template <EpiKind KIND, bool BF, int JU, int FM, int FN>
__device__ __forceinline__ void finish_any(const f32x16_t (&acc)[FM][FN], float* reg,
                                           const LinProblem& P, const float* bias, int row0,
                                           int col0) {
#define MAO_FINISH(A) finish_all<KIND, A, BF, JU>(acc, reg, P, bias, row0, col0)
  if constexpr (KIND == EPI_PLAIN) {
    MAO_FINISH(MAO_ACT_NONE);
  } else {
    switch (P.e.act) {
      case MAO_ACT_RELU: MAO_FINISH(MAO_ACT_RELU); break;
      case MAO_ACT_GELU: MAO_FINISH(MAO_ACT_GELU); break;
      case MAO_ACT_GELU_TANH: MAO_FINISH(MAO_ACT_GELU_TANH); break;
      case MAO_ACT_SILU: MAO_FINISH(MAO_ACT_SILU); break;
      default: MAO_FINISH(MAO_ACT_NONE); break;
    }
  }
#undef MAO_FINISH
}

__device__ __forceinline__ float bias_at(const LinProblem& P, int col) {
  return P.e.bias != nullptr && col < P.N ? load1_any(P.e.bias, P.e.bias_dtype, col) : 0.f;
}

// Tile of a (tiles_m x tiles_n) grid: groups of 8 tile rows, so that tiles
// running together share operand panels.
__device__ __forceinline__ void tile_of(const LinArgs& a, int tile, int& tm, int& tn) {
  constexpr int G = 8;
  const int per_group = G * a.tiles_n;
  const int grp = tile / per_group;
  const int first = grp * G;
  const int gsz = min(G, a.tiles_m - first);
  const int in = tile - grp * per_group;
  tm = first + in % gsz;
  tn = in / gsz;
}

template <typename TIn, bool AKM, bool BKM, int BM_, int BN_, int WM_, int WN_, int KSB_, int NST_, int OCC_>
struct Cfg {
  using T = TIn;
  static constexpr bool akm = AKM, bkm = BKM;
  static constexpr int BM = BM_, BN = BN_, KSB = KSB_, NST = NST_, OCC = OCC_;
  static constexpr int WM = WM_, WN = WN_, WAVES = WM * WN, THREADS = 64 * WAVES;  // wavefront grid
  static constexpr int ES = (int)sizeof(TIn), EPC = 16 / ES, KS = KSB / ES, SUB = KSB / 32;
  static constexpr int FM = BM / (32 * WM), FN = BN / (32 * WN);
  static constexpr int AB = BM * KSB, BB = BN * KSB, STAGE = AB + BB;
  static constexpr int LA = AB / 16 / THREADS, LB = BB / 16 / THREADS;
  static constexpr int JU = FN % 2 == 0 ? 2 : FN;
  static constexpr int PIECE = 32 * piece_ld(JU) * 4;
  static_assert(AB % (16 * THREADS) == 0 && BB % (16 * THREADS) == 0, "whole loads per thread");
  static_assert(NST == 2 || NST == 3, "ring stages");
  static_assert(WAVES / 2 * PIECE + BN * 4 <= STAGE, "the epilogue's pieces and the bias fit the stages");
};

// XOR permutation of a K-contiguous row's 16-byte chunks (128 bytes per row).
__device__ __forceinline__ int swz_k(int row) { return (row >> 1) & 7; }
// XOR permutation of a K-major row's chunks (BX: tile rows of the operand).
template <int BX, int ES>
__device__ __forceinline__ int swz_m(int krow) {
  if (ES == 4) return ((krow >> 2) & 1) << 3;
  // rows of 384 or 128 bytes already alternate between the halves of the banks
  return BX == 192 || BX == 64 ? ((krow >> 1) & 1) << 2 : (krow & 3) << 2;
}

// Per-thread global sources of one operand's direct loads, and its LDS fragment
// offsets.
template <typename TIn, bool KM, int BX, int WX, int WAVES, int KSB, int NL>
struct Operand {
  static constexpr int ES = (int)sizeof(TIn), EPC = 16 / ES, F = BX / (32 * WX), SUB = KSB / 32;
  static constexpr int CPR = KM ? BX * ES / 16 : KSB / 16;  // chunks per LDS row
  const TIn* src[NL];
  int frag[KM ? F : SUB];

  __device__ __forceinline__ void init(const TIn* p, int64_t ld, int x0, int X, int w) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int h = lane >> 5, r32 = lane & 31;
#pragma unroll
    for (int q = 0; q < NL; ++q) {
      const int L = (q * WAVES + wave) * 64 + lane;
      const int r = L / CPR, slot = L % CPR;
      if constexpr (KM) {
        const int col = x0 + (slot ^ swz_m<BX, ES>(r)) * EPC;
        src[q] = p + (int64_t)r * ld + min(col, (X - 1) / EPC * EPC);
      } else {
        src[q] = p + (int64_t)min(x0 + r, X - 1) * ld + (slot ^ swz_k(r)) * EPC;
      }
    }
    if constexpr (!KM) {
      const int r = w * (BX / WX) + r32;
#pragma unroll
      for (int s = 0; s < SUB; ++s) frag[s] = r * KSB + (((2 * s + h) ^ swz_k(r)) << 4);
    } else if constexpr (ES == 2) {
      const int ti = lane & 15, tg = (lane >> 4) & 1;
      const int krow = 8 * h + (ti >> 2);
#pragma unroll
      for (int f = 0; f < F; ++f) {
        const int chunk = w * (BX / (8 * WX)) + 4 * f + 2 * tg + ((ti >> 1) & 1);
        frag[f] = krow * BX * 2 + ((chunk ^ swz_m<BX, ES>(krow)) << 4) + 8 * (ti & 1);
      }
    } else {
#pragma unroll
      for (int f = 0; f < F; ++f) {
        const int col = w * (BX / WX) + 32 * f + r32;
        frag[f] = 4 * h * BX * 4 + (((col >> 2) ^ (h << 3)) << 4) + 4 * (col & 3);
      }
    }
  }
  // slice starting at element k0 of the reduction
  __device__ __forceinline__ void issue(unsigned char* st, int64_t k0, int64_t ld) const {
    const int wave = threadIdx.x >> 6;
    const int64_t off = KM ? k0 * ld : k0;
#pragma unroll
    for (int q = 0; q < NL; ++q)
      __builtin_amdgcn_global_load_lds((gbl_void_t*)(src[q] + off),
                                       (lds_void_t*)(st + (q * WAVES + wave) * 1024), 16, 0, 0);
  }
  // partial slice [k0, kend): element by element, zero past kend
  __device__ __forceinline__ void stage_tail(unsigned char* st, const TIn* p, int64_t ld, int x0,
                                             int X, int64_t k0, int64_t kend) const {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll 1
    for (int q = 0; q < NL; ++q) {
      const int L = (q * WAVES + wave) * 64 + lane;
      const int r = L / CPR, slot = L % CPR;
      union {
        uint4 v;
        TIn e[EPC];
      } u;
      u.v = make_uint4(0, 0, 0, 0);
      if constexpr (KM) {
        const int64_t k = k0 + r;
        const int col = x0 + (slot ^ swz_m<BX, ES>(r)) * EPC;
        if (k < kend)
          for (int i = 0; i < EPC; ++i)
            if (col + i < X) u.e[i] = p[k * ld + col + i];
      } else {
        const int64_t k = k0 + (slot ^ swz_k(r)) * EPC;
        if (x0 + r < X)
          for (int i = 0; i < EPC; ++i)
            if (k + i < kend) u.e[i] = p[(int64_t)(x0 + r) * ld + k + i];
      }
      *(uint4*)(st + L * 16) = u.v;
    }
  }
  __device__ __forceinline__ uint4 read(const unsigned char* st, int s, int f) const {
    if constexpr (!KM) {
      return *(const uint4*)(st + frag[s] + f * 32 * KSB);
    } else if constexpr (ES == 2) {
      const unsigned char* q = st + frag[f] + s * 16 * BX * 2;
      const uint2 lo = __builtin_bit_cast(
          uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16_t*)(q)));
      const uint2 hi = __builtin_bit_cast(
          uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16_t*)(q + 4 * BX * 2)));
      return make_uint4(lo.x, lo.y, hi.x, hi.y);
    } else {
      const unsigned char* q = st + frag[f] + s * 8 * BX * 4;
      return make_uint4(*(const uint32_t*)q, *(const uint32_t*)(q + BX * 4),
                        *(const uint32_t*)(q + 2 * BX * 4), *(const uint32_t*)(q + 3 * BX * 4));
    }
  }
  static constexpr int reads = KM ? (ES == 2 ? 2 : 4) : 1;  // LDS reads per fragment
};

__device__ __forceinline__ uint32_t u4e(const uint4& v, int e) {
  return e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w;
}

template <typename C, EpiKind KIND, bool BF>
__global__ __launch_bounds__(C::THREADS, C::OCC) void linear_tile_kernel(LinArgs a) {
  using TIn = typename C::T;
  constexpr int FM = C::FM, FN = C::FN, SUB = C::SUB, NST = C::NST;
  constexpr int LPT = C::LA + C::LB;
  __shared__ __attribute__((aligned(16))) unsigned char st0[C::STAGE];
  __shared__ __attribute__((aligned(16))) unsigned char st1[C::STAGE];
  __shared__ __attribute__((aligned(16))) unsigned char st2[NST > 2 ? C::STAGE : 16];

  // Workgroups reach the 8 XCDs round-robin: each XCD takes a contiguous run of
  // the (split, tile) list, neighbours sharing panels in its L2.
  const int total = a.tiles * a.split;
  const int x = blockIdx.x & 7, base = total >> 3, rem = total & 7;
  const int local = x * base + min(x, rem) + (blockIdx.x >> 3);
  const int part = local / a.tiles, tile = local - part * a.tiles;
  int tm, tn;
  tile_of(a, tile, tm, tn);
  const LinProblem& P = a.p;
  const int m0 = tm * C::BM, n0 = tn * C::BN;
  const TIn* A = (const TIn*)P.A;
  const TIn* B = (const TIn*)P.B;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave / C::WN, wn = wave % C::WN;

  Operand<TIn, C::akm, C::BM, C::WM, C::WAVES, C::KSB, C::LA> oa;
  Operand<TIn, C::bkm, C::BN, C::WN, C::WAVES, C::KSB, C::LB> ob;
  oa.init(A, P.lda, m0, P.M, wm);
  ob.init(B, P.ldb, n0, P.N, wn);

  // the tile's bias, on its way during the main loop
  float bias_v = 0.f;
  if constexpr (KIND == EPI_FORWARD)
    if (a.split == 1) bias_v = bias_at(P, n0 + (int)threadIdx.x);

  // this workgroup's slices [s0, s1); the last slice of K may be partial
  const int s0 = (int)((int64_t)a.slices * part / a.split);
  const int s1 = (int)((int64_t)a.slices * (part + 1) / a.split);
  const bool tail = s1 == a.slices && P.K % C::KS != 0;
  const int nk = s1 - s0 - (tail ? 1 : 0);  // full slices

  f32x16_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;

  auto issue = [&](unsigned char* st, int k) __attribute__((always_inline)) {
    const int64_t k0 = (int64_t)(s0 + k) * C::KS;
    oa.issue(st, k0, P.lda);
    ob.issue(st + C::AB, k0, P.ldb);
  };
  auto read = [&](const unsigned char* st, int s, uint4 (&fa)[FM], uint4 (&fb)[FN])
                  __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < (FM > FN ? FM : FN); ++i) {
      if (i < FM) fa[i < FM ? i : 0] = oa.read(st, s, i);
      if (i < FN) fb[i < FN ? i : 0] = ob.read(st + C::AB, s, i);
    }
  };
  auto mma = [&](const uint4 (&fa)[FM], const uint4 (&fb)[FN]) __attribute__((always_inline)) {
    if constexpr (C::ES == 2) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
              __builtin_bit_cast(bf16x8_t, fb[j]), __builtin_bit_cast(bf16x8_t, fa[i]), acc[i][j],
              0, 0, 0);
    } else {
      // the four 2-deep steps run over all blocks in turn, so consecutive MFMAs
      // never accumulate into the same block
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(
                __uint_as_float(u4e(fb[j], e)), __uint_as_float(u4e(fa[i], e)), acc[i][j], 0, 0, 0);
    }
  };
  constexpr int NM = FM * FN * (C::ES == 2 ? 1 : 4);
  constexpr int NR = FM * decltype(oa)::reads + FN * decltype(ob)::reads;
  constexpr int RPM = (NR + NM - 1) / NM;
  constexpr int VPM = (LPT + NM - 1) / NM;
  // order inside a sub-step: operand reads (and direct loads) between MFMAs
  auto order = [&](bool loads) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < NM; ++q) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if (loads && q * VPM < LPT) __builtin_amdgcn_sched_group_barrier(0x020, VPM, 0);
      if (q * RPM < NR) __builtin_amdgcn_sched_group_barrier(0x100, RPM, 0);
    }
  };

  uint4 fa[2][FM], fb[2][FN];
  // Column sums of A (the bias gradient) on the way: slice g of the reduction is
  // summed by the workgroup whose tile column is g modulo the number of tile
  // columns, so every slice is summed once per tile row and the work is spread
  // evenly. A thread adds one 16-byte chunk of every RS-th k row of the slice.
  constexpr int ACH = C::BM * C::ES / 16, RS = C::THREADS / ACH, EPC = C::EPC;
  constexpr bool SUMS = KIND == EPI_PLAIN;
  float csum[SUMS ? EPC : 1];
  if constexpr (SUMS)
#pragma unroll
    for (int i = 0; i < EPC; ++i) csum[i] = 0.f;
  auto add_columns = [&](const unsigned char* st) __attribute__((always_inline)) {
    const int c = (int)threadIdx.x % ACH, r0 = (int)threadIdx.x / ACH;
    if (r0 >= RS) return;
#pragma unroll
    for (int r = 0; r < (C::KS + RS - 1) / RS; ++r) {
      const int kr = r0 + r * RS;
      if (C::KS % RS != 0 && kr >= C::KS) break;
      const uint4 q = *(const uint4*)(st + kr * C::BM * C::ES + ((c ^ swz_m<C::BM, C::ES>(kr)) << 4));
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (C::ES == 2) {
          csum[2 * i] += __uint_as_float(w[i] << 16);
          csum[2 * i + 1] += __uint_as_float(w[i] & 0xffff0000u);
        } else {
          csum[i] += __uint_as_float(w[i]);
        }
      }
    }
  };
  int next_sum = -1;  // this workgroup's next slice to sum, from s0
  if constexpr (SUMS)
    if (a.sums != nullptr) next_sum = (tn - s0 % a.tiles_n + a.tiles_n) % a.tiles_n;

  // slice k out of `cur`; `nxt` holds slice k + 1 (landing)
  auto step = [&](unsigned char* cur, const unsigned char* nxt, int k)
                  __attribute__((always_inline)) {
    if constexpr (SUMS) {
      if (k == next_sum) {
        add_columns(cur);
        next_sum += a.tiles_n;
      }
    }
#pragma unroll
    for (int s = 0; s + 1 < SUB; ++s) {
      read(cur, s + 1, fa[(s + 1) & 1], fb[(s + 1) & 1]);
      mma(fa[s & 1], fb[s & 1]);
      order(false);
      __builtin_amdgcn_sched_barrier(0);
    }
    // loads in flight here: slices k + 1 .. k + NST - 1, those below nk; the wait
    // leaves all but slice k + 1's
    if (NST == 2 || k + NST - 1 >= nk)
      wait_slice<0>();
    else
      wait_slice<(NST - 2) * LPT>();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (k + NST < nk) issue(cur, k + NST);
    if (k + 1 < nk) read(nxt, 0, fa[0], fb[0]);
    mma(fa[1], fb[1]);
    order(true);
    __builtin_amdgcn_sched_barrier(0);
  };

  if constexpr (C::WAVES == 8) {
    // Two wavefronts per SIMD take turns: while one multiplies a 16-deep step (bf16;
    // 8 deep in fp32), the other reads its fragments for its next step and issues
    // loads. The second group runs one barrier behind the first; every barrier ends
    // one group's reads and the other's products. Slice k + 1 is loaded during the
    // first two steps of slice k into the stage that both groups left a step ago.
    if (nk > 0) {
      issue(st0, 0);
      wait_slice<0>();
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      const int group = __builtin_amdgcn_readfirstlane(wave >> 2);
      if (group) __builtin_amdgcn_s_barrier();
      auto turn = [&](unsigned char* cur, unsigned char* nxt, int k) __attribute__((always_inline)) {
#pragma unroll
        for (int s = 0; s < SUB; ++s) {
          if constexpr (SUMS) {
            if (s == 0 && k == next_sum) {
              add_columns(cur);
              next_sum += a.tiles_n;
            }
          }
          __builtin_amdgcn_sched_barrier(0);
          read(cur, s, fa[0], fb[0]);
          if (s < 2 && k + 1 < nk) {
            const int64_t k0 = (int64_t)(s0 + k + 1) * C::KS;
            if (s == 0)
              oa.issue(nxt, k0, P.lda);
            else
              ob.issue(nxt + C::AB, k0, P.ldb);
          }
          // fragments are in; at the last step, so is this wavefront's part of
          // slice k + 1
          if (s == SUB - 1)
            wait_slice<0>();
          else
            wait_lds();
          __builtin_amdgcn_sched_barrier(0);
          asm volatile("" ::: "memory");
          __builtin_amdgcn_s_barrier();
          asm volatile("" ::: "memory");
          __builtin_amdgcn_s_setprio(1);
          mma(fa[0], fb[0]);
          __builtin_amdgcn_sched_barrier(0);
          __builtin_amdgcn_s_setprio(0);
          asm volatile("" ::: "memory");
          __builtin_amdgcn_s_barrier();
          asm volatile("" ::: "memory");
        }
      };
      int k = 0;
      for (; k + 2 <= nk; k += 2) {
        turn(st0, st1, k);
        turn(st1, st0, k + 1);
      }
      if (k < nk) turn(st0, st1, k);
      if (!group) __builtin_amdgcn_s_barrier();
    }
  } else if (nk > 0) {
    issue(st0, 0);
    if (nk > 1) issue(st1, 1);
    if (NST > 2 && nk > 2) issue(st2, 2);
    // wait for slice 0
    if (nk >= NST)
      wait_slice<(NST - 1) * LPT>();
    else
      wait_slice<0>();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    read(st0, 0, fa[0], fb[0]);
    __builtin_amdgcn_sched_barrier(0);
    int k = 0;
    if constexpr (NST == 2) {
      for (; k + 2 <= nk; k += 2) {
        step(st0, st1, k);
        step(st1, st0, k + 1);
      }
      if (k < nk) step(st0, st1, k);
    } else {
      for (; k + 3 <= nk; k += 3) {
        step(st0, st1, k);
        step(st1, st2, k + 1);
        step(st2, st0, k + 2);
      }
      if (k < nk) step(st0, st1, k);
      if (k + 1 < nk) step(st1, st2, k + 1);
    }
  }
  // every wavefront is past the last slice's barrier: no LDS reads or loads
  // are outstanding, the stages are free
  if (tail) {
    const int64_t k0 = (int64_t)(s1 - 1) * C::KS;
    oa.stage_tail(st0, A, P.lda, m0, P.M, k0, P.K);
    ob.stage_tail(st0 + C::AB, B, P.ldb, n0, P.N, k0, P.K);
    __syncthreads();
    if constexpr (SUMS)
      if (nk == next_sum) add_columns(st0);
#pragma unroll 1
    for (int s = 0; s < SUB; ++s) {
      // s is a run-time value here: fragment offsets by select, one copy of code
      uint4 ta[FM], tb[FN];
#pragma unroll
      for (int q = 0; q < SUB; ++q)
        if (s == q) read(st0, q, ta, tb);
      mma(ta, tb);
    }
    __syncthreads();
  }

  if constexpr (SUMS) {
    if (a.sums != nullptr) {  // join the RS row groups, in order
      float* js = (float*)st0;
      const int c = (int)threadIdx.x % ACH, r0 = (int)threadIdx.x / ACH;
      if (r0 < RS)
#pragma unroll
        for (int i = 0; i < EPC; ++i) js[r0 * C::BM + c * EPC + i] = csum[i];
      __syncthreads();
      if (threadIdx.x < C::BM && m0 + (int)threadIdx.x < P.M) {
        float t = 0.f;
#pragma unroll
        for (int r = 0; r < RS; ++r) t += js[r * C::BM + threadIdx.x];
        a.sums[((int64_t)part * a.tiles_n + tn) * P.M + m0 + threadIdx.x] = t;
      }
      __syncthreads();
    }
  }

  // The accumulators stay in AGPRs and are read value by value: as ordinary
  // registers the exchanges below, which overwrite their operands, would have
  // them all copied first, and spilled.
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) asm volatile("" : "+a"(acc[i][j]));

  float* reg = (float*)((wave < C::WAVES / 2 ? st0 : st1) + (wave % (C::WAVES / 2)) * C::PIECE);
  const int row0 = m0 + wm * (C::BM / C::WM), col0 = n0 + wn * (C::BN / C::WN);
  if (a.split > 1) {  // fp32 partial result, row-major like the result itself
    LinProblem q;
    q.M = P.M;
    q.N = P.N;
    q.e.D = a.part + (int64_t)part * P.M * a.ldpart;
    q.e.ldd = a.ldpart;
    q.e.d_dtype = MAO_F32;
    q.e.add = nullptr;
    finish_all<EPI_PARTIAL, MAO_ACT_NONE, false, C::JU>(acc, reg, q, nullptr, row0, col0);
    return;
  }
  float* bias = (float*)(st1 + C::STAGE - C::BN * 4);
  if constexpr (KIND == EPI_FORWARD) {
    if (threadIdx.x < C::BN) bias[threadIdx.x] = bias_v;
    __syncthreads();
  }
  finish_any<KIND, BF, C::JU>(acc, reg, P, bias + wn * (C::BN / C::WN), row0, col0);
}

template <typename C, EpiKind KIND, bool BF>
mao_status go(const LinArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((linear_tile_kernel<C, KIND, BF>), dim3(a.tiles * a.split), dim3(C::THREADS), 0, s,
                     a);
  MAO_LAUNCH_CHECK();
  return MAO_OK;
}

template <bool AKM, bool BKM, EpiKind KIND>
mao_status pick(int dtype, int cfg, bool bf, const LinArgs& a, hipStream_t s) {
  if (dtype == MAO_F32) {
    if (cfg == CFG_64x64) return go<Cfg<float, AKM, BKM, 64, 64, 2, 2, 128, 2, 4>, KIND, false>(a, s);
    return go<Cfg<float, AKM, BKM, 128, 128, 2, 2, 128, 2, 2>, KIND, false>(a, s);
  }
  constexpr bool BF = KIND != EPI_PLAIN;  // the weight gradient looks at its type
  switch (cfg) {
    case CFG_256x256: return go<Cfg<bf16_t, AKM, BKM, 256, 256, 4, 2, 128, 2, 2>, KIND, BF>(a, s);
    case CFG_256x192: return go<Cfg<bf16_t, AKM, BKM, 256, 192, 4, 2, 128, 2, 2>, KIND, BF>(a, s);
    case CFG_192x128: return go<Cfg<bf16_t, AKM, BKM, 192, 128, 2, 2, 128, 2, 2>, KIND, BF>(a, s);
  }
  if (cfg == CFG_64x64) return go<Cfg<bf16_t, AKM, BKM, 64, 64, 2, 2, 128, 3, 3>, KIND, false>(a, s);
  if (BF && bf) return go<Cfg<bf16_t, AKM, BKM, 128, 128, 2, 2, 128, 2, 2>, KIND, BF>(a, s);
  return go<Cfg<bf16_t, AKM, BKM, 128, 128, 2, 2, 128, 2, 2>, KIND, false>(a, s);
}

}  // namespace
}  // namespace mao
