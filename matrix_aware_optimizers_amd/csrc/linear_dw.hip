// dW = dy^T x (+ dW): the tile kernels of this product.
#include "linear_tile.hpp"

namespace mao {

mao_status linear_weight_grad_tiles(int dtype, int cfg, bool bf, const LinArgs& a, hipStream_t s) {
  return pick<true, true, EPI_PLAIN>(dtype, cfg, bf, a, s);
}

}  // namespace mao
