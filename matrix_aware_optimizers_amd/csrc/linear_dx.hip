// dx = (dy W) . act'(z) + add: the tile kernels of this product.
#include "linear_tile.hpp"

namespace mao {

mao_status linear_input_grad_tiles(int dtype, int cfg, bool bf, const LinArgs& a, hipStream_t s) {
  return pick<false, true, EPI_SLOPE>(dtype, cfg, bf, a, s);
}

}  // namespace mao
