// y = act(x W^T + b) + res: the tile kernels of this product.
#include "linear_tile.hpp"

namespace mao {

mao_status linear_forward_tiles(int dtype, int cfg, bool bf, const LinArgs& a, hipStream_t s) {
  return pick<false, false, EPI_FORWARD>(dtype, cfg, bf, a, s);
}

}  // namespace mao
