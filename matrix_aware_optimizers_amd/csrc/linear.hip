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

// Tile shapes: workgroups per CU, TFLOP/s of a CU full of them (bf16, long K) and
// the microseconds a workgroup takes to start and to finish its result.
struct Shape {
  int bm, bn, per_cu;
  double rate, ends;
};
const Shape kShapes[CFG_COUNT] = {
    {256, 256, 1, 5.43, 11.4}, {256, 192, 1, 4.95, 8.6}, {128, 192, 2, 5.2, 9.7},
    {192, 128, 2, 5.2, 9.1},   {128, 128, 2, 4.2, 6.9},  {64, 64, 3, 2.5, 4.9},
};
constexpr double kF32Rate[2] = {0.485, 0.53};  // 128 x 128 and 64 x 64 tiles

// The cut with the shortest estimated time. Tiles run in rounds of 256 workgroups
// times those that share a CU; a last round that is not full is shorter too (the
// clock rises as CUs idle). Of p workgroups that fit a CU, o take the square root
// of o / p of the time of p. With few tiles K is split: more workgroups, then a launch and one pass
// over the partial results.
//
// The constants minimise the loss over 117 products (three layouts, both types, 77
// to 16384 rows, K from 200 to 16384, operands not in the L2) timed with every shape
// and up to 14 splits on MI355X: the estimate's choice is 2% slower than the best
// one on average, 15% at worst (512 x 4096 x 4096, 40 against 35 us).
Plan estimate_plan(int dtype, bool mixed, int64_t M, int64_t N, int64_t K) {
  // sqrt(o / p) for o = 1 .. p
  static const double kShare[5][4] = {
      {}, {1.0}, {0.707, 1.0}, {0.577, 0.816, 1.0}, {0.5, 0.707, 0.866, 1.0}};
  const int ks = dtype == MAO_BF16 ? 64 : 32;
  const int slices = (int)ceil_div(K, ks);
  const double part_us = 8.0 * M * N / 1e7;
  Plan best = {};
  double best_us = 0.0;
  for (int c = 0; c < CFG_COUNT; ++c) {
    // fp32 operands and mixed result types come with the small square tiles only
    if (c < CFG_128x128 && (dtype != MAO_BF16 || mixed)) continue;
    const Shape& h = kShapes[c];
    const int64_t tm = ceil_div(M, h.bm), tn = ceil_div(N, h.bn), tiles = tm * tn;
    const int per_cu = dtype != MAO_BF16 && c == CFG_64x64 ? 4 : h.per_cu;
    const int slots = 256 * per_cu;
    const double rate = (dtype != MAO_BF16 ? kF32Rate[c == CFG_64x64] : h.rate) * 1e6 / per_cu;
    const double slice_us = 2.0 * h.bm * h.bn * ks / rate;
    // parts of at least two slices, no more than 32, and only where a round is
    // not full without them
    const int most = tiles >= slots
                         ? 1
                         : std::max(1, std::min({32, slices / 2, (int)ceil_div(2 * slots, tiles)}));
    for (int s = 1; s <= most; ++s) {
      double one = ((slices + s - 1) / s) * slice_us, rounds;
      if (s == 1 && tiles >= slots) {
        const int64_t last = tiles % slots;
        rounds = (double)(tiles / slots) + (last ? 0.7 + 0.3 * last / slots : 0.0);
      } else {
        const int wgs = (int)tiles * s, last = wgs % slots;
        one *= kShare[per_cu][std::min(per_cu, (wgs + 255) / 256) - 1];
        rounds = wgs / slots + (last ? 0.7 + 0.3 * last / slots : 0.0);
      }
      const double us = (one + h.ends) * rounds + (s > 1 ? 4.8 + part_us * s : 0.0);
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
