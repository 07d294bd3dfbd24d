// The fp32 kernels of attention_forward for many rows.
#define ATTENTION_T float
#include "attention_tile.h"
