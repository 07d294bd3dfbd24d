// The kernels of paged_attention for many rows: bf16, its own pages.
#define PAGED_T bf16
#define PAGED_E4 false
#include "paged_tile.h"
