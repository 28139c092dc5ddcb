// Cross entropy, the logits forward, bf16.
#include "cross_entropy_tile.h"

namespace tbe {
template <>
tbe_status ce_launch_forward<2>(const CeArgs& a, int tile, bool direct, hipStream_t s) {
  return direct ? ce_logits<2, false, true>(a, tile, s) : ce_logits<2, false, false>(a, tile, s);
}
}  // namespace tbe
