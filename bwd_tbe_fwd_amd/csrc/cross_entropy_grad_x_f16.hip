// Cross entropy, the rows' gradient, fp16.
#include "cross_entropy_tile.h"

namespace tbe {
template <>
tbe_status ce_launch_grad_x<1>(const CeArgs& a, int tile, bool direct, hipStream_t s) {
  return direct ? ce_grad<1, true, true>(a, tile, s) : ce_grad<1, true, false>(a, tile, s);
}
}  // namespace tbe
