// packed_grad.cuh — the elementwise passes around the gradient's product: dz = dY act'(Z) in the
// product's operand form, its column sums (the bias's gradient), and dX from sweep to original order.
#pragma once

#include "packed_decode.cuh"

namespace gptq {

__device__ __forceinline__ float act_grad(float z, int act) {
  if (act == ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
  if (act == ACT_GELU)
    return 0.5f * erfcf(z * -0.70710678118654752f) + z * expf(-0.5f * z * z) * 0.39894228040143268f;
  if (act == ACT_SILU) {
    const float s = 1.0f / (1.0f + expf(-z));
    return s * (1.0f + z * (1.0f - s));
  }
  return 1.0f;
}

// One block per token.  scale_t = 2^e with the largest |dY| of the token in [2^(e+13), 2^(e+14))
// (e clamped to [-100, 100]; 1 for a token without a finite, nonzero value), then hi + lo = dz /
// scale_t in fp16 (lo null: hi alone).  Rows of ldz elements.
template <bool BF>
__global__ void __launch_bounds__(256) act_grad_kernel(const uint16_t* __restrict__ dY, int64_t ld_dy,
                                                       const uint16_t* __restrict__ Z, int m, int act,
                                                       uint16_t* __restrict__ hi, uint16_t* __restrict__ lo,
                                                       int64_t ldz, float* __restrict__ token_scale) {
  __shared__ float wmax[8];
  griddep_wait();
  griddep_launch_dependents();
  const size_t t = blockIdx.x;
  const uint16_t* dy = dY + t * ld_dy;
  const uint16_t* z = Z ? Z + t * m : nullptr;
  float mx = 0.0f;
  for (int r = threadIdx.x; r < m; r += 256) mx = fmaxf(mx, fabsf(h2f<BF>(dy[r])));
#pragma unroll
  for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) mx = fmaxf(mx, wmax[w]);
  int e = 0;
  if (mx > 0.0f && mx < INFINITY) e = min(100, max(-100, ilogbf(mx) - 13));
  const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  if (threadIdx.x == 0) token_scale[t] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
  for (int r = threadIdx.x; r < m; r += 256) {
    float v = h2f<BF>(dy[r]) * inv;
    if (z) v *= act_grad(h2f<BF>(z[r]), act);
    const uint16_t h = f2h<false>(v);
    hi[t * ldz + r] = h;
    if (lo) lo[t * ldz + r] = f2h<false>(v - h2f<false>(h));
  }
}

// dbias[r] = sum over tokens of dY act'(Z), in fp32.  A block takes 128 columns and, as one of a
// cluster of eight, every eighth stripe of tokens; sums meet in a fixed order.
constexpr int DBIAS_CLUSTER = 8;
template <bool BF>
__global__ void __launch_bounds__(256) dbias_kernel(const uint16_t* __restrict__ dY, int64_t ld_dy,
                                                    const uint16_t* __restrict__ Z, int T, int m, int act,
                                                    float* __restrict__ dbias) {
  __shared__ float part[8][128];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int c0 = static_cast<int>(blockIdx.x) / DBIAS_CLUSTER * 128;
  float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int t = rank * 8 + warp; t < T; t += 8 * DBIAS_CLUSTER) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = c0 + lane + 32 * j;
      if (c < m) {
        float v = h2f<BF>(dY[static_cast<size_t>(t) * ld_dy + c]);
        if (Z) v *= act_grad(h2f<BF>(Z[static_cast<size_t>(t) * m + c]), act);
        sum[j] += v;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) part[warp][lane + 32 * j] = sum[j];
  __syncthreads();
  if (threadIdx.x < 128) {
    float v = part[0][threadIdx.x];
#pragma unroll
    for (int w = 1; w < 8; ++w) v += part[w][threadIdx.x];
    part[0][threadIdx.x] = v;
  }
  cluster_sync();
  if (rank == 0 && threadIdx.x < 128 && c0 + threadIdx.x < m) {
    float v = 0.0f;
    for (int o = 0; o < DBIAS_CLUSTER; ++o) v += ld_dsmem_f(mapa_shared(smem_u32(&part[0][threadIdx.x]), o));
    dbias[c0 + threadIdx.x] = v;
  }
  cluster_sync();
}

// out[t][perm[k]] = in[t][k]: the row is scattered in shared memory and leaves in order.
__global__ void __launch_bounds__(256) unpermute_kernel(const uint16_t* __restrict__ in, int n,
                                                        const int32_t* __restrict__ perm, uint16_t* __restrict__ out,
                                                        int64_t ld_out) {
  extern __shared__ uint16_t up_row[];
  griddep_wait();
  griddep_launch_dependents();
  const size_t t = blockIdx.x;
  for (int k = threadIdx.x * 4; k < n; k += 1024) {
    const int4 i = *reinterpret_cast<const int4*>(perm + k);
    const ushort4 v = *reinterpret_cast<const ushort4*>(in + t * n + k);
    up_row[i.x] = v.x;
    up_row[i.y] = v.y;
    up_row[i.z] = v.z;
    up_row[i.w] = v.w;
  }
  __syncthreads();
  uint16_t* d = out + t * ld_out;
  if (ld_out % 2 == 0 && (reinterpret_cast<uintptr_t>(out) & 3u) == 0) {
    for (int k = threadIdx.x; k < n / 2; k += 256)
      reinterpret_cast<uint32_t*>(d)[k] = reinterpret_cast<const uint32_t*>(up_row)[k];
  } else {
    for (int k = threadIdx.x; k < n; k += 256) d[k] = up_row[k];
  }
}

}  // namespace gptq
