// packed_decode_b2.cu — the decode kernels of 2-bit codes.
#define PACKED_BITS 2
#include "packed_decode_inst.cuh"
