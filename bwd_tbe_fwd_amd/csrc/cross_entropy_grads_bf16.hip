// Cross entropy, the gradients' products, bf16.
#include "cross_entropy_tile.h"

namespace tbe {
template <>
tbe_status ce_launch_grads<2>(const CeArgs& x, int x_tile, const CeArgs& w, int w_tile, hipStream_t s) {
  return ce_grads<2>(x, x_tile, w, w_tile, s);
}
}  // namespace tbe
