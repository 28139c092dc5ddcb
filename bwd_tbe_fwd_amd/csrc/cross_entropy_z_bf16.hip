// Cross entropy, the logits backward, bf16.
#include "cross_entropy_tile.h"

namespace tbe {
template <>
tbe_status ce_launch_z<2>(const CeArgs& a, int tile, hipStream_t s) {
  return ce_logits<2, true>(a, tile, s);
}
}  // namespace tbe
