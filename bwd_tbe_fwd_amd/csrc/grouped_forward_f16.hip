// Grouped linear layers, forward, f16.
#include "grouped_launch.h"

TBE_GROUPED(1, kForward)
