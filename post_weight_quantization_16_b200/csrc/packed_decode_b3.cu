// packed_decode_b3.cu — the decode kernels of 3-bit codes.
#define PACKED_BITS 3
#include "packed_decode_inst.cuh"
