// Grouped linear layers, backward by input, f16.
#include "grouped_launch.h"

TBE_GROUPED(1, kBackwardInput)
