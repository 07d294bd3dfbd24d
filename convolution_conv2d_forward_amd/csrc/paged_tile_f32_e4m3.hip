// The kernels of paged_attention for many rows: fp32, E4M3 pages.
#define PAGED_T float
#define PAGED_E4 true
#include "paged_tile.h"
