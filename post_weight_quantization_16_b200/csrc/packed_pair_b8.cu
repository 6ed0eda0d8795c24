// packed_pair_b8.cu — the CTA-pair kernels of 8-bit codes.
#define PACKED_BITS 8
#include "packed_pair_inst.cuh"
