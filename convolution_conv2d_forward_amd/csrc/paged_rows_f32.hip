// The kernels of paged_attention for few rows: fp32, its own pages.
#define PAGED_T float
#define PAGED_E4 false
#include "paged_rows.h"
