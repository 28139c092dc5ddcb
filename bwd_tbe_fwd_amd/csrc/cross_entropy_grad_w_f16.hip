// Cross entropy, the weights' gradient, fp16.
#include "cross_entropy_tile.h"

namespace tbe {
template <>
tbe_status ce_launch_grad_w<1>(const CeArgs& a, int tile, hipStream_t s) {
  return ce_grad<1, false>(a, tile, s);
}
}  // namespace tbe
