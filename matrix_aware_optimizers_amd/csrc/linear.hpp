// Launch arguments shared by the linear layer's three products.
#pragma once

#include "layers.hpp"

namespace mao {

struct LinArgs {
  LinProblem p;
  float* part;   // partial tiles (split > 1)
  int tiles_m, tiles_n, tiles, split, slices;
};

// Tile configurations (linear_tile.hpp).
enum { CFG_128x192 = 0, CFG_192x128 = 1, CFG_128x128 = 2 };

// One translation unit per product: linear_fwd.hip, linear_dx.hip, linear_dw.hip.
// bf: every tensor of the epilogue but a checkpoint is bf16.
mao_status linear_forward_tiles(int dtype, int cfg, bool bf, const LinArgs& a, hipStream_t s);
mao_status linear_input_grad_tiles(int dtype, int cfg, bool bf, const LinArgs& a, hipStream_t s);
mao_status linear_weight_grad_tiles(int dtype, int cfg, bool bf, const LinArgs& a, hipStream_t s);

}  // namespace mao
