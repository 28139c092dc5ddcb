// Layer norm kernels for x of type f32.
#include "layer_norm.h"

namespace tbe {
TBE_NORM_TYPE(0)
}  // namespace tbe
