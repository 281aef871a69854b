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

constexpr int kSlots = 512;  // workgroups resident at once: two per CU

// The cut with the shortest estimated time. Two workgroups share a CU, so tiles
// run in rounds of 512; a workgroup alone on its CU runs 1.7 times as fast. With few
// tiles K is split: more workgroups, each part followed by one pass over the
// partial tiles (written and read once) and a launch. Rates of the estimate
// (bf16: 16384 x 6144 x 1536 and 6144 x 1536 x 16384 on MI355X): 128 x 192 and
// 192 x 128 tiles 4.1 TFLOP/s per CU, 128 x 128 tiles 3.6 (they read 20% more
// operand bytes per flop); fp32 0.5; partial results 4 TB/s; 3 us to start and end
// a workgroup, 4 us for the second launch.
Plan make_plan(int dtype, bool mixed, int64_t M, int64_t N, int64_t K) {
  static const int shape[3][2] = {{128, 192}, {192, 128}, {128, 128}};
  const int ks = dtype == MAO_BF16 ? 64 : 32;
  const int64_t slices = ceil_div(K, ks);
  Plan best = {};
  double best_us = 0.0;
  for (int c = 0; c < 3; ++c) {
    // fp32 operands and mixed result types come with the square tile only
    if (c != CFG_128x128 && (dtype != MAO_BF16 || mixed)) continue;
    const int bm = shape[c][0], bn = shape[c][1];
    const int64_t tm = ceil_div(M, bm), tn = ceil_div(N, bn), tiles = tm * tn;
    const double rate = (dtype != MAO_BF16 ? 0.5 : c == CFG_128x128 ? 3.6 : 4.1) * 0.5e6;
    const double slice_us = 2.0 * bm * bn * ks / rate;
    // parts of at least two slices, no more than 32, and only where a round is
    // not full without them
    const int64_t most = tiles >= kSlots ? 1 : std::min<int64_t>({32, slices / 2, ceil_div(2 * kSlots, tiles)});
    for (int64_t s = 1; s <= std::max<int64_t>(1, most); ++s) {
      const int64_t wgs = tiles * s;
      const double alone = wgs <= kSlots / 2 ? 1.0 / 1.7 : 1.0;
      double us = (double)ceil_div(wgs, kSlots) * (ceil_div(slices, s) * slice_us * alone + 3.0);
      if (s > 1) us += 4.0 + 8.0 * s * M * N / 4e6;
      if (best_us == 0.0 || us < best_us) {
        best_us = us;
        best.cfg = c;
        best.split = (int)s;
        best.tiles_m = tm;
        best.tiles_n = tn;
        best.slices = slices;
        best.ws = s > 1 ? (size_t)s * M * round_up(N, 8) * 4 : 0;
      }
    }
  }
  return best;
}

}  // namespace

size_t lin_workspace(int dtype, int64_t M, int64_t N, int64_t K) {
  // the caller may not know the result types yet
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
  const Plan pl = make_plan(dtype, !(p.a_km && p.b_km) && !bf, p.M, p.N, p.K);
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
