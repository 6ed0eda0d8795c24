// packed_tc_b4.cu — the tensor-core kernels of 4-bit codes.
#define PACKED_BITS 4
#include "packed_tc_inst.cuh"
