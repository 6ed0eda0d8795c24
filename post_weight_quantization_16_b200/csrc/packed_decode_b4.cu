// packed_decode_b4.cu — the decode kernels of 4-bit codes.
#define PACKED_BITS 4
#include "packed_decode_inst.cuh"
