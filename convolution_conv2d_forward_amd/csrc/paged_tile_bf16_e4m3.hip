// The kernels of paged_attention for many rows: bf16, E4M3 pages.
#define PAGED_T bf16
#define PAGED_E4 true
#include "paged_tile.h"
