// Cross entropy, the logits of narrow rows backward, bf16.
#include "cross_entropy_narrow.h"

namespace tbe {
template <>
tbe_status ce_launch_narrow_z<2>(const CeArgs& a, bool few, hipStream_t s) {
  return ce_narrow<2, true>(a, few, s);
}
}  // namespace tbe
