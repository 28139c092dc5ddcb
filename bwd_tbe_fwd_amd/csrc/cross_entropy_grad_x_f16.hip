// Cross entropy, the rows' gradient, fp16.
#include "cross_entropy_tile.h"

namespace tbe {
template <>
tbe_status ce_launch_grad_x<1>(const CeArgs& a, int tile, hipStream_t s) {
  return ce_grad<1, true>(a, tile, s);
}
}  // namespace tbe
