// packed_tc_b3.cu — the tensor-core kernels of 3-bit codes.
#define PACKED_BITS 3
#include "packed_tc_inst.cuh"
