// The kernels of paged_attention for many rows: fp32, its own pages.
#define PAGED_T float
#define PAGED_E4 false
#include "paged_tile.h"
