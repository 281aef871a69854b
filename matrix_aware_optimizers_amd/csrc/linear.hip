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
// A workgroup of 4 wavefronts (2 x 2) computes a BM x BN tile, each wavefront
// (BM/2) x (BN/2) as 32 x 32 MFMA blocks, fp32 accumulation. K advances in
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
// Epilogue: a wavefront passes its accumulators through a private piece of LDS
// (32 rows x 64 columns at a time, no workgroup barrier) so that each lane
// finishes 8 consecutive columns: bias, activation, residual and stores all move
// whole 16-byte pieces, 128 bytes of a bf16 row together.
//
// Few tiles: K is split over several workgroups per tile. Their fp32 partial
// tiles go to the workspace, and a second launch adds them in a fixed order and
// runs the same epilogue. No atomics anywhere.
#include "act.hpp"
#include "layers.hpp"

#include <algorithm>

namespace mao {

namespace {

typedef __attribute__((address_space(3))) void lds_void_t;
typedef __attribute__((address_space(1))) const void gbl_void_t;
typedef short lds_v4i16_t __attribute__((ext_vector_type(4), address_space(3)));

constexpr int kThreads = 256;

// s_waitcnt with vmcnt(n) and lgkmcnt(0)
template <int N>
__device__ __forceinline__ void wait_slice() {
  __builtin_amdgcn_s_waitcnt((N & 0xf) | (0x7 << 4) | ((N >> 4) << 14));
}

struct LinArgs {
  LinProblem p;
  float* part;   // partial tiles (split > 1)
  int tiles_m, tiles_n, tiles, split, slices;
};

// What the epilogue does beyond D = acc + add.
enum EpiKind { EPI_PLAIN, EPI_FORWARD, EPI_SLOPE };

// Finishes one 32 x (32 JU) unit of a wavefront's result: acc -> wavefront-private
// LDS `reg` (rows padded by 8 floats) -> 8 columns per lane.
template <int JU>
constexpr int unit_ld() { return 32 * JU + 8; }

template <EpiKind KIND, int JU>
__device__ __forceinline__ void finish_unit(const f32x16_t* acc, float* reg, const LinProblem& P,
                                            int row0, int col0) {
  constexpr int LD = unit_ld<JU>();
  constexpr int CPR = 4 * JU;  // runs of 8 columns per row
  const int lane = threadIdx.x & 63, h = lane >> 5, r32 = lane & 31;
  const LinEpilogue& e = P.e;
#pragma unroll
  for (int j = 0; j < JU; ++j)
#pragma unroll
    for (int v = 0; v < 16; ++v)
      reg[(8 * (v >> 2) + 4 * h + (v & 3)) * LD + j * 32 + r32] = acc[j][v];
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll 1
  for (int it = 0; it < 2 * JU; ++it) {
    const int idx = it * 64 + lane;
    const int rr = idx / CPR, cc = idx % CPR;
    const int row = row0 + rr, col = col0 + 8 * cc;
    const float* s = reg + rr * LD + 8 * cc;
    const float4 lo = *(const float4*)s, hi = *(const float4*)(s + 4);
    if (row >= P.M || col >= P.N) continue;
    const int valid = P.N - col;
    float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    if constexpr (KIND == EPI_FORWARD) {
      if (e.bias) {
        float b[8];
        if (valid >= 8) {
          load8_any(e.bias, e.bias_dtype, col, b);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) b[i] = i < valid ? load1_any(e.bias, e.bias_dtype, col + i) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += b[i];
      }
      if (e.z_out) store8n_any(e.z_out, e.zo_dtype, (int64_t)row * e.ldzo + col, v, valid);
      act_apply(e.act, v);
    }
    if constexpr (KIND == EPI_SLOPE) {
      if (e.act != MAO_ACT_NONE) {
        float z[8];
        const int64_t off = (int64_t)row * e.ldzi + col;
        if (e.z_kind <= MAO_BF16) {
          load8_any(e.z_in, e.z_kind, off, z);
        } else {
          const uint2 q = *(const uint2*)((const uint8_t*)e.z_in + off);
          const float sc = q8_scale_value(e.z_scales[(int64_t)row * e.ldzs + (col >> 5)]);
          const int fmt = e.z_kind == kXInt8 ? MAO_Q8_INT8 : MAO_Q8_E4M3;
          q8_decode4_any(fmt, q.x, sc, z);
          q8_decode4_any(fmt, q.y, sc, z + 4);
        }
        act_slope_apply(e.act, z, v);
      }
    }
    if (e.add) {
      float w[8];
      load8_any(e.add, e.add_dtype, (int64_t)row * e.ldadd + col, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += w[i];
    }
    store8n_any(e.D, e.d_dtype, (int64_t)row * e.ldd + col, v, valid);
  }
  // the next unit overwrites reg: its reads above are done (values were used)
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
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

template <typename TIn, bool AKM, bool BKM, int BM_, int BN_, int KSB_, int NST_, int OCC_>
struct Cfg {
  using T = TIn;
  static constexpr bool akm = AKM, bkm = BKM;
  static constexpr int BM = BM_, BN = BN_, KSB = KSB_, NST = NST_, OCC = OCC_;
  static constexpr int ES = (int)sizeof(TIn), EPC = 16 / ES, KS = KSB / ES, SUB = KSB / 32;
  static constexpr int FM = BM / 64, FN = BN / 64;
  static constexpr int AB = BM * KSB, BB = BN * KSB, STAGE = AB + BB;
  static constexpr int LA = AB / 16 / kThreads, LB = BB / 16 / kThreads;
  static constexpr int JU = (FN % 2 == 0) ? 2 : 1;
  static constexpr int UNIT = 32 * unit_ld<JU>() * 4;
  static_assert(AB % (16 * kThreads) == 0 && BB % (16 * kThreads) == 0, "whole loads per thread");
  static_assert(2 * UNIT <= STAGE && NST >= 2, "epilogue pieces fit two per stage");
};

// XOR permutation of a K-contiguous row's 16-byte chunks.
template <int KSB>
__device__ __forceinline__ int swz_k(int row) {
  return KSB == 128 ? (row >> 1) & 7 : ((row >> 1) ^ (row >> 2)) & 3;
}
// XOR permutation of a K-major row's chunks (BX: tile rows of the operand).
template <int BX, int ES>
__device__ __forceinline__ int swz_m(int krow) {
  if (ES == 4) return ((krow >> 2) & 1) << 3;
  return BX == 192 ? ((krow >> 1) & 1) << 2 : (krow & 3) << 2;
}

// Per-thread global sources of one operand's direct loads, and its LDS fragment
// offsets.
template <typename TIn, bool KM, int BX, int KSB, int NL>
struct Operand {
  static constexpr int ES = (int)sizeof(TIn), EPC = 16 / ES, F = BX / 64, SUB = KSB / 32;
  static constexpr int CPR = KM ? BX * ES / 16 : KSB / 16;  // chunks per LDS row
  const TIn* src[NL];
  int frag[KM ? F : SUB];

  __device__ __forceinline__ void init(const TIn* p, int64_t ld, int x0, int X, int w) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int h = lane >> 5, r32 = lane & 31;
#pragma unroll
    for (int q = 0; q < NL; ++q) {
      const int L = (q * 4 + wave) * 64 + lane;
      const int r = L / CPR, slot = L % CPR;
      if constexpr (KM) {
        const int col = x0 + (slot ^ swz_m<BX, ES>(r)) * EPC;
        src[q] = p + (int64_t)r * ld + min(col, (X - 1) / EPC * EPC);
      } else {
        src[q] = p + (int64_t)min(x0 + r, X - 1) * ld + (slot ^ swz_k<KSB>(r)) * EPC;
      }
    }
    if constexpr (!KM) {
      const int r = w * (BX / 2) + r32;
#pragma unroll
      for (int s = 0; s < SUB; ++s) frag[s] = r * KSB + (((2 * s + h) ^ swz_k<KSB>(r)) << 4);
    } else if constexpr (ES == 2) {
      const int ti = lane & 15, tg = (lane >> 4) & 1;
      const int krow = 8 * h + (ti >> 2);
#pragma unroll
      for (int f = 0; f < F; ++f) {
        const int chunk = w * (BX / 16) + 4 * f + 2 * tg + ((ti >> 1) & 1);
        frag[f] = krow * BX * 2 + ((chunk ^ swz_m<BX, ES>(krow)) << 4) + 8 * (ti & 1);
      }
    } else {
#pragma unroll
      for (int f = 0; f < F; ++f) {
        const int col = w * (BX / 2) + 32 * f + r32;
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
                                       (lds_void_t*)(st + (q * 4 + wave) * 1024), 16, 0, 0);
  }
  // partial slice [k0, kend): element by element, zero past kend
  __device__ __forceinline__ void stage_tail(unsigned char* st, const TIn* p, int64_t ld, int x0,
                                             int X, int64_t k0, int64_t kend) const {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll 1
    for (int q = 0; q < NL; ++q) {
      const int L = (q * 4 + wave) * 64 + lane;
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
        const int64_t k = k0 + (slot ^ swz_k<KSB>(r)) * EPC;
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

template <typename C, EpiKind KIND>
__global__ __launch_bounds__(kThreads, C::OCC) void linear_tile_kernel(LinArgs a) {
  using TIn = typename C::T;
  constexpr int FM = C::FM, FN = C::FN, SUB = C::SUB, NST = C::NST;
  constexpr int LPT = C::LA + C::LB;
  __shared__ __attribute__((aligned(16))) unsigned char st0[C::STAGE];
  __shared__ __attribute__((aligned(16))) unsigned char st1[C::STAGE];
  __shared__ __attribute__((aligned(16))) unsigned char st2[NST > 2 ? C::STAGE : 16];
  __shared__ __attribute__((aligned(16))) unsigned char st3[NST > 3 ? C::STAGE : 16];

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
  const int wm = wave >> 1, wn = wave & 1;

  Operand<TIn, C::akm, C::BM, C::KSB, C::LA> oa;
  Operand<TIn, C::bkm, C::BN, C::KSB, C::LB> ob;
  oa.init(A, P.lda, m0, P.M, wm);
  ob.init(B, P.ldb, n0, P.N, wn);

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
              __builtin_bit_cast(bf16x8_t, fa[i]), __builtin_bit_cast(bf16x8_t, fb[j]), acc[i][j],
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
                __uint_as_float(u4e(fa[i], e)), __uint_as_float(u4e(fb[j], e)), acc[i][j], 0, 0, 0);
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
  // slice k out of `cur`; `nxt` holds slice k + 1 (landing)
  auto step = [&](unsigned char* cur, const unsigned char* nxt, int k)
                  __attribute__((always_inline)) {
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

  if (nk > 0) {
    issue(st0, 0);
    if (nk > 1) issue(st1, 1);
    if (NST > 2 && nk > 2) issue(st2, 2);
    if (NST > 3 && nk > 3) issue(st3, 3);
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
    } else if constexpr (NST == 3) {
      for (; k + 3 <= nk; k += 3) {
        step(st0, st1, k);
        step(st1, st2, k + 1);
        step(st2, st0, k + 2);
      }
      if (k < nk) step(st0, st1, k);
      if (k + 1 < nk) step(st1, st2, k + 1);
    } else {
      for (; k + 4 <= nk; k += 4) {
        step(st0, st1, k);
        step(st1, st2, k + 1);
        step(st2, st3, k + 2);
        step(st3, st0, k + 3);
      }
      if (k < nk) step(st0, st1, k);
      if (k + 1 < nk) step(st1, st2, k + 1);
      if (k + 2 < nk) step(st2, st3, k + 2);
    }
  }
  // every wavefront is past the last slice's barrier: no LDS reads or loads
  // are outstanding, the stages are free
  if (tail) {
    const int64_t k0 = (int64_t)(s1 - 1) * C::KS;
    oa.stage_tail(st0, A, P.lda, m0, P.M, k0, P.K);
    ob.stage_tail(st0 + C::AB, B, P.ldb, n0, P.N, k0, P.K);
    __syncthreads();
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

  if (a.split > 1) {
    float* w = a.part + ((int64_t)part * a.tiles + tile) * (C::BM * C::BN);
    w += (int64_t)wave * (C::BM * C::BN / 4);
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *(float4*)(w + (((i * FN + j) * 4 + g) * 64 + lane) * 4) =
              make_float4(acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2],
                          acc[i][j][4 * g + 3]);
    return;
  }
  float* reg = (float*)((wave < 2 ? st0 : st1) + (wave & 1) * C::UNIT);
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; j += C::JU)
      finish_unit<KIND, C::JU>(&acc[i][j], reg, P, m0 + wm * (C::BM / 2) + i * 32,
                               n0 + wn * (C::BN / 2) + j * 32);
}

// Adds the partial tiles of a split launch and finishes them: one wavefront per
// 32 x (32 JU) unit of a tile.
template <typename C, EpiKind KIND>
__global__ __launch_bounds__(64) void linear_join_kernel(LinArgs a) {
  constexpr int FM = C::FM, FN = C::FN, JU = C::JU;
  __shared__ __attribute__((aligned(16))) float reg[32 * unit_ld<JU>()];
  constexpr int UNITS = 4 * FM * (FN / JU);
  const int tile = blockIdx.x / UNITS, u = blockIdx.x % UNITS;
  const int wave = u / (FM * (FN / JU)), i = u / (FN / JU) % FM, j = u % (FN / JU) * JU;
  const int lane = threadIdx.x;
  int tm, tn;
  tile_of(a, tile, tm, tn);
  const float* w = a.part + (int64_t)tile * (C::BM * C::BN) + (int64_t)wave * (C::BM * C::BN / 4);
  f32x16_t acc[JU];
#pragma unroll
  for (int q = 0; q < JU; ++q)
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[q][v] = 0.f;
#pragma unroll 2
  for (int s = 0; s < a.split; ++s) {
    const float* ws = w + (int64_t)s * a.tiles * (C::BM * C::BN);
#pragma unroll
    for (int q = 0; q < JU; ++q)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const float4 t = *(const float4*)(ws + (((i * FN + j + q) * 4 + g) * 64 + lane) * 4);
        acc[q][4 * g] += t.x;
        acc[q][4 * g + 1] += t.y;
        acc[q][4 * g + 2] += t.z;
        acc[q][4 * g + 3] += t.w;
      }
  }
  const int wm = wave >> 1, wn = wave & 1;
  finish_unit<KIND, JU>(acc, reg, a.p, tm * C::BM + wm * (C::BM / 2) + i * 32,
                        tn * C::BN + wn * (C::BN / 2) + j * 32);
}

// How a product is cut: tile shape and K split.
struct Plan {
  int cfg, bm, bn, ks, split;
  int64_t tiles_m, tiles_n, slices;
  size_t ws;
};

enum { CFG_LARGE = 0, CFG_SMALL = 1 };

Plan make_plan(int dtype, int64_t M, int64_t N, int64_t K, int a_km, int b_km) {
  Plan p = {};
  (void)a_km;
  (void)b_km;
  const int ks = dtype == MAO_BF16 ? 64 : 32;
  auto cut = [&](int bm, int bn) {
    p.bm = bm;
    p.bn = bn;
    p.ks = ks;
    p.tiles_m = ceil_div(M, bm);
    p.tiles_n = ceil_div(N, bn);
    p.slices = ceil_div(K, ks);
  };
  p.cfg = CFG_SMALL;
  cut(128, 128);
  if (dtype == MAO_BF16 && ceil_div(M, 256) * ceil_div(N, 256) >= 192) {
    p.cfg = CFG_LARGE;
    cut(256, 256);
  }
  const int64_t tiles = p.tiles_m * p.tiles_n;
  // two workgroups per CU; a split adds a launch and its traffic, so it has to
  // at least double the workgroups and leave each four slices
  p.split = 1;
  if (p.cfg == CFG_SMALL && tiles < 256) {
    const int64_t s = std::min<int64_t>(512 / tiles, p.slices / 4);
    if (s >= 2) p.split = (int)s;
  }
  p.ws = p.split > 1 ? (size_t)tiles * p.split * p.bm * p.bn * 4 : 0;
  return p;
}

template <typename C, EpiKind KIND>
mao_status go(LinArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((linear_tile_kernel<C, KIND>), dim3(a.tiles * a.split), dim3(kThreads), 0, s,
                     a);
  MAO_LAUNCH_CHECK();
  if (a.split > 1) {
    constexpr int UNITS = 4 * C::FM * (C::FN / C::JU);
    hipLaunchKernelGGL((linear_join_kernel<C, KIND>), dim3(a.tiles * UNITS), dim3(64), 0, s, a);
    MAO_LAUNCH_CHECK();
  }
  return MAO_OK;
}

template <bool AKM, bool BKM, EpiKind KIND>
mao_status pick(int dtype, int cfg, LinArgs& a, hipStream_t s) {
  if (dtype == MAO_F32) return go<Cfg<float, AKM, BKM, 128, 128, 128, 2, 2>, KIND>(a, s);
  if (cfg == CFG_LARGE) return go<Cfg<bf16_t, AKM, BKM, 256, 256, 128, 2, 1>, KIND>(a, s);
  return go<Cfg<bf16_t, AKM, BKM, 128, 128, 128, 2, 2>, KIND>(a, s);
}

}  // namespace

size_t lin_workspace(int dtype, int64_t M, int64_t N, int64_t K, int a_km, int b_km) {
  return make_plan(dtype, M, N, K, a_km, b_km).ws;
}

mao_status launch_linear(int dtype, const LinProblem& p, void* ws, hipStream_t s) {
  const Plan pl = make_plan(dtype, p.M, p.N, p.K, p.a_km, p.b_km);
  LinArgs a = {};
  a.p = p;
  a.part = (float*)ws;
  a.tiles_m = (int)pl.tiles_m;
  a.tiles_n = (int)pl.tiles_n;
  a.tiles = (int)(pl.tiles_m * pl.tiles_n);
  a.split = pl.split;
  a.slices = (int)pl.slices;
  if (!p.a_km && !p.b_km) return pick<false, false, EPI_FORWARD>(dtype, pl.cfg, a, s);
  if (!p.a_km && p.b_km) return pick<false, true, EPI_SLOPE>(dtype, pl.cfg, a, s);
  return pick<true, true, EPI_PLAIN>(dtype, pl.cfg, a, s);
}

}  // namespace mao
