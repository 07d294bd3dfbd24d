// The bf16 kernels of attention_forward for many rows.
#define ATTENTION_T bf16
#include "attention_tile.h"
