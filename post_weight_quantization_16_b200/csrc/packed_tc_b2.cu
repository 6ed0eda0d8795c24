// packed_tc_b2.cu — the tensor-core kernels of 2-bit codes.
#define PACKED_BITS 2
#include "packed_tc_inst.cuh"
