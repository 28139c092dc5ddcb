// Grouped linear layers, backward by weight, bf16.
#include "grouped_launch.h"

TBE_GROUPED(2, kBackwardWeight)
