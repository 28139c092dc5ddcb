// Grouped linear layers, forward, bf16.
#include "grouped_launch.h"

TBE_GROUPED(2, kForward)
