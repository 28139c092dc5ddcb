// Cross entropy, the gradients of narrow rows, bf16.
#include "cross_entropy_fused.h"

namespace tbe {
template <>
tbe_status ce_launch_fused<2>(const CeArgs& a, bool x, hipStream_t s) {
  return x ? ce_fused<2, true, false>(a, s) : a.bias_part ? ce_fused<2, false, true>(a, s) : ce_fused<2, false, false>(a, s);
}
}  // namespace tbe
