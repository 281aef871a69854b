// How the linear layer's products are cut into tiles and K splits.
#include "linear.hpp"

#include <algorithm>

namespace mao {

namespace {

// How a product is cut: tile shape and K split.
struct Plan {
  int cfg, split;
  int64_t tiles_m, tiles_n, slices;
  size_t ws;
};

// Tile shapes: workgroups that share a CU, TFLOP/s of a CU full of them (long K), the
// microseconds a workgroup takes to start and to finish its result, and the time of
// o = 1, 2, .. workgroups on a CU relative to a full one's.
struct Shape {
  int bm, bn, per_cu;
  double rate, ends, share[4];
};
const Shape kShapes[CFG_COUNT] = {
    {256, 256, 1, 5.54, 12.4, {1.0}},        {256, 192, 1, 4.79, 8.16, {1.0}},
    {192, 128, 2, 4.34, 9.61, {0.802, 1.0}}, {128, 128, 2, 4.01, 6.80, {0.907, 1.0}},
    {64, 64, 3, 2.03, 4.18, {0.556, 0.805, 1.0}},
};
const Shape kShapesF32[2] = {  // CFG_128x128, CFG_64x64
    {128, 128, 2, 0.476, 5.33, {0.511, 1.0}},
    {64, 64, 4, 0.546, 1.66, {0.339, 0.582, 0.799, 1.0}},
};
constexpr double kLastRound = 0.91;     // of a round's time for a last one nearly empty
constexpr double kJoinUs = 3.16;        // launch of the join
constexpr double kPartPerUs = 4.61e6;   // bytes of partial results written and read per us

// The cut with the shortest estimated time. Tiles run in rounds of 256 workgroups
// times those that share a CU; a last round that is not full is shorter too (the
// clock rises as CUs idle). With few tiles K is split: more workgroups, then a launch
// and one pass over the partial results.
//
// The constants are fitted to 888 products (296 drawn sizes, three layouts, both
// types, 65 to 16384 rows, operands mostly not in the L2), each timed on MI355X with
// the shapes and up to 14 splits. On sizes drawn apart, which they were not fitted
// to, the estimate's choice is 1.8% slower than the best one timed on average over
// 252 small and middle products and 28.8% at worst (dW of 2759 rows, 7689 -> 79: 29.2
// against 22.6 us), 1.4% and 12.4% over 48 products of 1e11 to 1e12
// multiply-adds. Constants fitted to 38 chosen sizes lost 1.2% on those and
// 4.1% (32.5% at worst) and 4.6% (22.2%) on these.
// The same draws on what a shape is worth, in bf16 products of 1e11 multiply-adds and
// more: without 256 x 192 tiles they lose 3.0% (sizes drawn apart) and 3.1% (sizes
// fitted to) instead of 1.4% and 2.0%; without 192 x 128 1.4% and 2.4%. 128 x 192
// beside it gained nothing and is not built.
Plan estimate_plan(int dtype, bool mixed, int64_t M, int64_t N, int64_t K) {
  const int ks = dtype == MAO_BF16 ? 64 : 32;
  const int slices = (int)ceil_div(K, ks);
  const double part_us = 8.0 * M * N / kPartPerUs;
  Plan best = {};
  double best_us = 0.0;
  for (int c = 0; c < CFG_COUNT; ++c) {
    // fp32 operands and mixed result types come with the small square tiles only
    if (c < CFG_128x128 && (dtype != MAO_BF16 || mixed)) continue;
    const Shape& h = dtype == MAO_BF16 ? kShapes[c] : kShapesF32[c - CFG_128x128];
    const int64_t tm = ceil_div(M, h.bm), tn = ceil_div(N, h.bn), tiles = tm * tn;
    const int slots = 256 * h.per_cu;
    const double slice_us = 2.0 * h.bm * h.bn * ks * h.per_cu / (h.rate * 1e6);
    // parts of at least two slices, no more than 32, and only where a round is
    // not full without them
    const int most = tiles >= slots
                         ? 1
                         : std::max(1, std::min({32, slices / 2, (int)ceil_div(2 * slots, tiles)}));
    for (int s = 1; s <= most; ++s) {
      const int64_t wgs = tiles * s, last = wgs % slots;
      const int here = (int)std::min<int64_t>(h.per_cu, ceil_div(wgs, 256));
      const double one = ((slices + s - 1) / s) * slice_us * h.share[here - 1] + h.ends;
      const double rounds = (double)(wgs / slots) +
                            (last ? kLastRound + (1.0 - kLastRound) * last / slots : 0.0);
      const double us = one * rounds + (s > 1 ? kJoinUs + part_us * s : 0.0);
      if (best_us == 0.0 || us < best_us) {
        best_us = us;
        best.cfg = c;
        best.split = s;
        best.tiles_m = tm;
        best.tiles_n = tn;
        best.slices = slices;
        best.ws = s > 1 ? (size_t)s * M * round_up(N, 8) * 4 : 0;
      }
    }
  }
  return best;
}

// The last cuts of this thread, by size: an estimate takes about a microsecond of
// host time, and a call needs it up to three times.
Plan make_plan(int dtype, bool mixed, int64_t M, int64_t N, int64_t K) {
  struct Entry {
    int64_t M, N, K;
    int type;
    Plan plan;
  };
  static thread_local Entry memo[16] = {};
  const int type = 1 + 2 * dtype + (mixed ? 1 : 0);  // 0: empty
  Entry& e = memo[(uint64_t)(M * 31 + N * 17 + K * 7 + type) % 16];
  if (e.type != type || e.M != M || e.N != N || e.K != K)
    e = Entry{M, N, K, type, estimate_plan(dtype, mixed, M, N, K)};
  return e.plan;
}

}  // namespace

LinCut lin_cut(int dtype, bool mixed, int64_t M, int64_t N, int64_t K) {
  const Plan pl = make_plan(dtype, mixed, M, N, K);
  return {kShapes[pl.cfg].bm, kShapes[pl.cfg].bn, pl.split};
}

size_t lin_workspace(int dtype, int64_t M, int64_t N, int64_t K) {
  // the caller may not know the result types yet
  if (dtype != MAO_BF16) return make_plan(dtype, false, M, N, K).ws;
  return std::max(make_plan(dtype, false, M, N, K).ws, make_plan(dtype, true, M, N, K).ws);
}

int lin_sum_rows(int dtype, int64_t M, int64_t N, int64_t K) {
  const Plan pl = make_plan(dtype, false, M, N, K);
  return (int)(pl.split * pl.tiles_n);
}

mao_status launch_linear(int dtype, const LinProblem& p, void* ws, float* sums, hipStream_t s) {
  // forward and input gradient: every tensor of the epilogue but a checkpoint is
  // bf16 (the weight gradient's kernels take either result type)
  const LinEpilogue& e = p.e;
  const bool bf = e.d_dtype == MAO_BF16 && (!e.z_out || e.zo_dtype == MAO_BF16) &&
                  (!e.add || e.add_dtype == MAO_BF16) && (!e.z_in || e.z_kind != MAO_F32);
  const Plan pl = make_plan(dtype, !p.a_km && !bf, p.M, p.N, p.K);
  LinArgs a = {};
  a.p = p;
  a.part = (float*)ws;
  a.ldpart = round_up(p.N, 8);
  a.sums = sums;
  a.tiles_m = (int)pl.tiles_m;
  a.tiles_n = (int)pl.tiles_n;
  a.tiles = (int)(pl.tiles_m * pl.tiles_n);
  a.split = pl.split;
  a.slices = (int)pl.slices;
  const bool slope = !p.a_km && p.b_km;
  if (!p.a_km && !p.b_km)
    MAO_TRY(linear_forward_tiles(dtype, pl.cfg, bf, a, s));
  else if (slope)
    MAO_TRY(linear_input_grad_tiles(dtype, pl.cfg, bf, a, s));
  else
    MAO_TRY(linear_weight_grad_tiles(dtype, pl.cfg, bf, a, s));
  return pl.split > 1 ? launch_linear_join(p, a.part, a.ldpart, pl.split, slope, s) : MAO_OK;
}

}  // namespace mao
