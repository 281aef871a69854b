// Launch arguments shared by the linear layer's three products.
#pragma once

#include "layers.hpp"

namespace mao {

struct LinArgs {
  LinProblem p;
  float* part;     // fp32 partial results [split][M][ldpart] (split > 1)
  int64_t ldpart;
  float* sums;     // weight gradient: partial column sums of A [split * tiles_n][M], or nullptr
  int tiles_m, tiles_n, tiles, split, slices;
};

// Adds a.split partial results and finishes them (linear_join.hip).
mao_status launch_linear_join(const LinProblem& p, const float* part, int64_t ldpart, int split,
                              bool slope, hipStream_t s);

// Tile configurations (linear_tile.hpp).
enum { CFG_256x256 = 0, CFG_256x192, CFG_192x128, CFG_128x128, CFG_64x64, CFG_COUNT };

// One translation unit per product: linear_fwd.hip, linear_dx.hip, linear_dw.hip.
// bf: every tensor of the epilogue but a checkpoint is bf16.
mao_status linear_forward_tiles(int dtype, int cfg, bool bf, const LinArgs& a, hipStream_t s);
mao_status linear_input_grad_tiles(int dtype, int cfg, bool bf, const LinArgs& a, hipStream_t s);
mao_status linear_weight_grad_tiles(int dtype, int cfg, bool bf, const LinArgs& a, hipStream_t s);

}  // namespace mao
