// The fp32 kernels of linear_forward.
#define LINEAR_T float
#include "linear_tile.h"
