// Cross entropy, the logits forward, fp16.
#include "cross_entropy_tile.h"

namespace tbe {
template <>
tbe_status ce_launch_forward<1>(const CeArgs& a, int tile, bool direct, hipStream_t s) {
  return direct ? ce_logits<1, false, true>(a, tile, s) : ce_logits<1, false, false>(a, tile, s);
}
}  // namespace tbe
