// packed_decode_b8.cu — the decode kernels of 8-bit codes.
#define PACKED_BITS 8
#include "packed_decode_inst.cuh"
