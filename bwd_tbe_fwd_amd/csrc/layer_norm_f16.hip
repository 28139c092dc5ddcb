// Layer norm kernels for x of type f16.
#include "layer_norm.h"

namespace tbe {
TBE_NORM_TYPE(1)
}  // namespace tbe
