// packed_tc_b8.cu — the tensor-core kernels of 8-bit codes.
#define PACKED_BITS 8
#include "packed_tc_inst.cuh"
