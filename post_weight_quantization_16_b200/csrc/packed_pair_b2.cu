// packed_pair_b2.cu — the CTA-pair kernels of 2-bit codes.
#define PACKED_BITS 2
#include "packed_pair_inst.cuh"
