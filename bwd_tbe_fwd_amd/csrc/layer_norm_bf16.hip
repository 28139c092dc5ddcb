// Layer norm kernels for x of type bf16.
#include "layer_norm.h"

namespace tbe {
TBE_NORM_TYPE(2)
}  // namespace tbe
