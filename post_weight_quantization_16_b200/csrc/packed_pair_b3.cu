// packed_pair_b3.cu — the CTA-pair kernels of 3-bit codes.
#define PACKED_BITS 3
#include "packed_pair_inst.cuh"
