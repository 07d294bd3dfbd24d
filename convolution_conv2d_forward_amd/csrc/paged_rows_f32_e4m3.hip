// The kernels of paged_attention for few rows: fp32, E4M3 pages.
#define PAGED_T float
#define PAGED_E4 true
#include "paged_rows.h"
