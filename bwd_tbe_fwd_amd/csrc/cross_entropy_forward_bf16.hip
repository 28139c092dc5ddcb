// Cross entropy, the logits forward, bf16.
#include "cross_entropy_tile.h"

namespace tbe {
template <>
tbe_status ce_launch_forward<2>(const CeArgs& a, int tile, bool direct, hipStream_t s) {
  // few rows and weights that do not start on 16 bytes: through registers, where copying the weights would cost more
  if (!direct) return ce_launch(ce_logits_kernel<2, false, 64, 64, 2, 2, false>, "ce_logits", 256, ce_tiles(a.rows, 64, a.items, 64), s, a);
  return ce_logits<2, false>(a, tile, s);
}
}  // namespace tbe
