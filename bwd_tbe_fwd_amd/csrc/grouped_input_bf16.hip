// Grouped linear layers, backward by input, bf16.
#include "grouped_launch.h"

TBE_GROUPED(2, kBackwardInput)
