// Scaled lookup, the backward's sums of fp32 gradients.
#include "lookup.h"

namespace tbe {
template <>
tbe_status launch_lookup_sum<0>(const LookupGradArgs& a, int table_dtype, int lanes, dim3 grid, hipStream_t s) {
  return lookup_sum<0>(a, table_dtype, lanes, grid, s);
}
}  // namespace tbe
