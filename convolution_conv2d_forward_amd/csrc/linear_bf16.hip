// The bf16 kernels of linear_forward.
#define LINEAR_T bf16
#include "linear_tile.h"
