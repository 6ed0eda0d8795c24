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
    const float s = __fdividef(1.0f, 1.0f + __expf(-z));  // (the result is rounded to 16 bits or summed)
    return s * (1.0f + z * (1.0f - s));
  }
  return 1.0f;
}

// Four 16-bit values from p (vec: p is 8-byte aligned and all four exist).
__device__ __forceinline__ void load4(const uint16_t* p, bool vec, int left, uint16_t (&v)[4]) {
  if (vec) {
    const ushort4 x = *reinterpret_cast<const ushort4*>(p);
    v[0] = x.x;
    v[1] = x.y;
    v[2] = x.z;
    v[3] = x.w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = j < left ? p[j] : static_cast<uint16_t>(0);
  }
}

// One block per token.  scale_t = 2^e with the largest |dY| of the token in [2^(e+13), 2^(e+14))
// (e clamped to [-100, 100]; 1 for a token without a finite, nonzero value), then hi + lo = dz /
// scale_t in fp16 (lo null: hi alone).  Rows of ldz (a multiple of 8) elements; the second pass finds
// dY in the caches.  vec: rows of dY and Z allow 8-byte accesses.
template <bool BF>
__global__ void __launch_bounds__(512) act_grad_kernel(const uint16_t* __restrict__ dY, int64_t ld_dy,
                                                       const uint16_t* __restrict__ Z, int m, int act, int vec,
                                                       uint16_t* __restrict__ hi, uint16_t* __restrict__ lo,
                                                       int64_t ldz, float* __restrict__ token_scale) {
  __shared__ float wmax[16];
  griddep_wait();
  griddep_launch_dependents();
  const size_t t = blockIdx.x;
  const uint16_t* dy = dY + t * ld_dy;
  const uint16_t* z = Z ? Z + t * m : nullptr;
  float mx = 0.0f;
#pragma unroll 4
  for (int r = threadIdx.x * 4; r < m; r += 2048) {
    uint16_t v[4];
    load4(dy + r, vec && r + 4 <= m, m - r, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) mx = fmaxf(mx, fabsf(h2f<BF>(v[j])));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 16; ++w) mx = fmaxf(mx, wmax[w]);
  int e = 0;
  if (mx > 0.0f && mx < INFINITY) e = min(100, max(-100, ilogbf(mx) - 13));
  const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  if (threadIdx.x == 0) token_scale[t] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll 2
  for (int r = threadIdx.x * 4; r < m; r += 2048) {
    uint16_t v[4], zv[4], h[4], l[4];
    load4(dy + r, vec && r + 4 <= m, m - r, v);
    if (z) load4(z + r, vec && r + 4 <= m, m - r, zv);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float x = h2f<BF>(v[j]) * inv;
      if (z) x *= act_grad(h2f<BF>(zv[j]), act);
      h[j] = f2h<false>(x);
      l[j] = f2h<false>(x - h2f<false>(h[j]));
    }
    // (rows are padded to a multiple of 8: a whole group of four always has room)
    *reinterpret_cast<ushort4*>(hi + t * ldz + r) = make_ushort4(h[0], h[1], h[2], h[3]);
    if (lo) *reinterpret_cast<ushort4*>(lo + t * ldz + r) = make_ushort4(l[0], l[1], l[2], l[3]);
  }
}

// dbias[r] = sum over tokens of dY act'(Z), in fp32.  A block takes 128 columns, a lane four of them
// and a warp every DBIAS_WARPS-th token of its block's stripe; the eight blocks of a cluster take the
// stripes; sums meet in a fixed order.
constexpr int DBIAS_CLUSTER = 8, DBIAS_WARPS = 16;
template <bool BF>
__global__ void __launch_bounds__(DBIAS_WARPS * 32) dbias_kernel(const uint16_t* __restrict__ dY, int64_t ld_dy,
                                                                 const uint16_t* __restrict__ Z, int T, int m, int act,
                                                                 int vec, float* __restrict__ dbias) {
  __shared__ float part[DBIAS_WARPS][128];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int c = static_cast<int>(blockIdx.x) / DBIAS_CLUSTER * 128 + lane * 4, left = m - c;
  const bool whole = vec && left >= 4;
  float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (left > 0) {
#pragma unroll 4
    for (int t = rank * DBIAS_WARPS + warp; t < T; t += DBIAS_WARPS * DBIAS_CLUSTER) {
      uint16_t v[4], z[4];
      load4(dY + static_cast<size_t>(t) * ld_dy + c, whole, left, v);
      if (Z) load4(Z + static_cast<size_t>(t) * m + c, whole, left, z);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float x = h2f<BF>(v[j]);
        sum[j] += Z ? x * act_grad(h2f<BF>(z[j]), act) : x;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) part[warp][lane * 4 + j] = sum[j];
  __syncthreads();
  if (threadIdx.x < 128) {
    float v = part[0][threadIdx.x];
#pragma unroll
    for (int w = 1; w < DBIAS_WARPS; ++w) v += part[w][threadIdx.x];
    part[0][threadIdx.x] = v;
  }
  cluster_sync();
  const int col = static_cast<int>(blockIdx.x) / DBIAS_CLUSTER * 128 + static_cast<int>(threadIdx.x);
  if (rank == 0 && threadIdx.x < 128 && col < m) {
    float v = 0.0f;
    for (int o = 0; o < DBIAS_CLUSTER; ++o) v += ld_dsmem_f(mapa_shared(smem_u32(&part[0][threadIdx.x]), o));
    dbias[col] = v;
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
