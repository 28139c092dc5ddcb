// Cross entropy, the gradients of narrow rows, fp16.
#include "cross_entropy_fused.h"

namespace tbe {
template <>
tbe_status ce_launch_fused<1>(const CeArgs& a, bool x, hipStream_t s) {
  return x ? ce_fused<1, true, false>(a, s) : a.bias_part ? ce_fused<1, false, true>(a, s) : ce_fused<1, false, false>(a, s);
}
}  // namespace tbe
