// packed_pair_b4.cu — the CTA-pair kernels of 4-bit codes.
#define PACKED_BITS 4
#include "packed_pair_inst.cuh"
