// Grouped linear layers, backward by weight, f16.
#include "grouped_launch.h"

TBE_GROUPED(1, kBackwardWeight)
