// packed_grad.cuh — the elementwise passes around the gradient's product: dz = dY act'(Z) in the
// product's operand form, its column sums (the bias's gradient), and dX from sweep to original order.
#pragma once

#include "packed_decode.cuh"

namespace gptq {

// act'(z), off by less than 2^-20 of its largest value, 1.13, and far from its zero by less than 2^-18 of
// itself: dz keeps 11 bits (22 in two parts), and what the bias's gradient sums is off by no more than the
// rest of its terms.  (With the epilogue's form of SiLU's power the bias's pass takes 3 us more of 58.)
template <int ACT>
__device__ __forceinline__ float act_grad(float z) {
  if (ACT == ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
  if (ACT == ACT_GELU)
    return 0.5f * erfcf(z * -0.70710678118654752f) + z * expf(-0.5f * z * z) * 0.39894228040143268f;
  if (ACT == ACT_SILU) {
    const float s = __fdividef(1.0f, 1.0f + __expf(-z));
    return s * (1.0f + z * (1.0f - s));
  }
  return 1.0f;
}

// Eight 16-bit values from p as four words (vec: p is 16-byte aligned and all eight exist).
__device__ __forceinline__ uint4 load8(const uint16_t* p, bool vec, int left) {
  if (vec) return *reinterpret_cast<const uint4*>(p);
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w[j] = (2 * j < left ? p[2 * j] : 0u) | (2 * j + 1 < left ? static_cast<uint32_t>(p[2 * j + 1]) << 16 : 0u);
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// Value j (0 .. 7) of the eight.
template <bool BF>
__device__ __forceinline__ float at8(const uint4& v, int j) {
  const uint32_t w = j < 2 ? v.x : j < 4 ? v.y : j < 6 ? v.z : v.w;
  return h2f<BF>(static_cast<uint16_t>((j & 1) ? w >> 16 : w & 0xFFFFu));
}

// Exponents of the blocks of 128 columns of W: (u - z) s 2^e lies below 2^15 for every row, and the largest
// scale's weights near it, so that the product's fp16 weights keep 11 significant bits down to 2^-29 of
// the block's largest, whatever the layer's scales are (a scale of 1e-7 would leave its codes in fp16's
// subnormals, one of 1e4 above its largest value).  Slabs of rows, read as they lie, a block each, with some
// eight scales a thread in flight; the product's kernel takes the least of a column block's `slabs`
// exponents.  Scales that are not finite do not count.  (Where these blocks are a launch of their own, 17
// tokens' fp16 gradient through 4096 x 4096 takes 15 us, 12 without exponents, and 32 tokens' of 152064 rows
// 205, not 194.  By blocks of 128 columns, each row's groups another 32-byte sector, they took 17 and 274.)
struct SlabArgs {
  const float* scales;
  int G, per, bits, chunks, slabs;  // per: groups of 128 columns, 1, 2 or 4
  GroupIndex gi;
  int* exponent;  // [chunks][slabs]
};
__device__ __forceinline__ void slab_exponents(const SlabArgs& p, int m, int slab) {
  __shared__ unsigned largest[512];  // by column block, or by group where that is wider (bits of a float >= 0)
  const int t = threadIdx.x, shift = p.per == 4 ? 2 : p.per - 1;
  largest[t] = 0u;
  __syncthreads();
  const int r0 = static_cast<int>(static_cast<int64_t>(m) * slab / p.slabs),
            r1 = static_cast<int>(static_cast<int64_t>(m) * (slab + 1) / p.slabs);
  const int width = min(p.G, 512), at_once = 512 / width, sub = t / width;  // rows at a time; this thread's
  if (sub < at_once) {
    for (int c = t % width; c < p.G; c += width) {
      float mx = 0.0f;
      for (int r = r0 + sub; r < r1; r += 8 * at_once) {
        float a[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          a[j] = r + j * at_once < r1 ? fabsf(__ldg(p.scales + static_cast<size_t>(r + j * at_once) * p.G + c)) : 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) mx = fmaxf(mx, a[j] < INFINITY ? a[j] : 0.0f);
      }
      unsigned bits = __float_as_uint(mx);
      if (p.G == 1) bits = __reduce_max_sync(0xffffffffu, bits);
      if (p.G > 1 || (t & 31) == 0) atomicMax(&largest[c >> shift], bits);
    }
  }
  __syncthreads();
  for (int k = t; k < p.chunks; k += 512) {
    // (a subnormal scale counts as 2^-127)
    const int ilog = static_cast<int>(largest[p.per > 1 ? k : group_of<128>(p.gi, k, 0)] >> 23) - 127;
    p.exponent[k * p.slabs + slab] = min(126, 14 - p.bits - ilog);
  }
}

// The first blocks: the weights' exponents.  Then one block per token (the grid has none when dY itself is
// the operand).  scale_t = 2^e with the largest finite |dz| of the token, dz = dY act'(Z), in
// [2^(e+13), 2^(e+14)) (e clamped to [-126, 126], where both scale_t and its inverse are normal; 1 for a
// token without a finite, nonzero value), then hi + lo = dz / scale_t in fp16 (lo null: hi alone).  (The
// largest |dY| would not do: an outlier that act' masks would push what is left into fp16's subnormals.)
// Rows of ldz (a multiple of 8) elements.  A thread keeps its first KEPT eights of dz in registers: 1 for
// rows of up to 4096 values, else 3, where 12288 are read and act' evaluated once; what is beyond is
// computed again.  vec: rows of dY and Z allow 16-byte accesses.  4096 x 11008 values with SiLU: 53 us
// (5.1 TB/s; 67 where each load waited for the one before it).
template <bool BF, int ACT, int KEPT>
__global__ void __launch_bounds__(512) act_grad_kernel(const uint16_t* __restrict__ dY, int64_t ld_dy,
                                                       const uint16_t* __restrict__ Z, int m, int vec,
                                                       uint16_t* __restrict__ hi, uint16_t* __restrict__ lo,
                                                       int64_t ldz, float2* __restrict__ token_scale,
                                                       const SlabArgs w) {
  __shared__ float wmax[16];
  griddep_wait();
  griddep_launch_dependents();
  if (static_cast<int>(blockIdx.x) < w.slabs) {
    slab_exponents(w, m, static_cast<int>(blockIdx.x));
    return;
  }
  const size_t t = blockIdx.x - w.slabs;
  const uint16_t* dy = dY + t * ld_dy;
  const uint16_t* z = Z + t * m;
  // Eight values of dz; of bf16 and a slope that exceeds 1, halved: dz may lie above fp32's largest.
  constexpr int HALVED = BF && (ACT == ACT_GELU || ACT == ACT_SILU) ? 1 : 0;
  auto eight = [&](const uint4& v, const uint4& zv, float (&x)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float d = HALVED ? 0.5f * at8<BF>(v, j) : at8<BF>(v, j);
      x[j] = d * (ACT != ACT_NONE ? act_grad<ACT>(at8<BF>(zv, j)) : 1.0f);
    }
  };
  auto load = [&](int r, bool whole, uint4& v, uint4& zv) {
    v = load8(dy + r, whole, m - r);
    if (ACT != ACT_NONE) zv = load8(z + r, whole, m - r);
  };
  float mx = 0.0f;
  auto largest = [&](const float (&x)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float a = fabsf(x[j]);
      mx = fmaxf(mx, a < INFINITY ? a : 0.0f);
    }
  };
  float kept[KEPT][8];
  {
    uint4 v[KEPT], zv[KEPT];
    // (the wide loads first, all in flight together)
#pragma unroll
    for (int k = 0; k < KEPT; ++k) {
      const int r = static_cast<int>(threadIdx.x) * 8 + k * 4096;
      v[k] = zv[k] = make_uint4(0u, 0u, 0u, 0u);
      if (vec && r + 8 <= m) load(r, true, v[k], zv[k]);
    }
#pragma unroll
    for (int k = 0; k < KEPT; ++k) {
      const int r = static_cast<int>(threadIdx.x) * 8 + k * 4096;
      if (r < m) {
        if (!(vec && r + 8 <= m)) load(r, false, v[k], zv[k]);
        eight(v[k], zv[k], kept[k]);
        largest(kept[k]);
      }
    }
  }
  for (int r = threadIdx.x * 8 + KEPT * 4096; r < m; r += 4096) {
    uint4 v, zv = {};
    float x[8];
    load(r, vec && r + 8 <= m, v, zv);
    eight(v, zv, x);
    largest(x);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 16; ++w) mx = fmaxf(mx, wmax[w]);
  int e = 0;
  if (mx > 0.0f) e = min(126, max(-126, ilogbf(mx) - 13));
  const float inv = pow2(-e);
  if (threadIdx.x == 0) token_scale[t] = pow2_halves(e + HALVED);
  auto store = [&](int r, float (&x)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] *= inv;
    // (rows are padded to a multiple of 8: a whole group always has room)
    const uint4 h = make_uint4(pack2<false>(x[0], x[1]), pack2<false>(x[2], x[3]), pack2<false>(x[4], x[5]),
                               pack2<false>(x[6], x[7]));
    *reinterpret_cast<uint4*>(hi + t * ldz + r) = h;
    if (lo) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] -= at8<false>(h, j);
      *reinterpret_cast<uint4*>(lo + t * ldz + r) = make_uint4(
          pack2<false>(x[0], x[1]), pack2<false>(x[2], x[3]), pack2<false>(x[4], x[5]), pack2<false>(x[6], x[7]));
    }
  };
#pragma unroll
  for (int k = 0; k < KEPT; ++k) {
    const int r = static_cast<int>(threadIdx.x) * 8 + k * 4096;
    if (r < m) store(r, kept[k]);
  }
  for (int r = threadIdx.x * 8 + KEPT * 4096; r < m; r += 4096) {
    uint4 v, zv = {};
    float x[8];
    load(r, vec && r + 8 <= m, v, zv);
    eight(v, zv, x);
    store(r, x);
  }
}

// dbias[r] = sum over tokens of dY act'(Z), in fp32.  A block takes 256 columns, a lane eight of them
// and a warp every DBIAS_WARPS-th token of its block's stripe; the eight blocks of a cluster take the
// stripes; sums meet in a fixed order.  (One pass that also writes dz, with the sums in registers, was
// slower: 237 us against 88 + 84 on 4096 x 11008 values, too few loads in flight; 53 + 58 since, 3.1 TB/s
// here: act' by the special functions.)
constexpr int DBIAS_CLUSTER = 8, DBIAS_WARPS = 8, DBIAS_COLS = 256;
template <bool BF, int ACT>
__global__ void __launch_bounds__(DBIAS_WARPS * 32) dbias_kernel(const uint16_t* __restrict__ dY, int64_t ld_dy,
                                                                 const uint16_t* __restrict__ Z, int T, int m, int vec,
                                                                 float* __restrict__ dbias,
                                                                 int* __restrict__ status) {
  __shared__ float part[DBIAS_WARPS][DBIAS_COLS];
  griddep_wait();
  griddep_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0) *status = 0;  // (the only launch when dX is not asked for)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int c0 = static_cast<int>(blockIdx.x) / DBIAS_CLUSTER * DBIAS_COLS, c = c0 + lane * 8, left = m - c;
  const bool whole = vec && left >= 8;
  float sum[8] = {};
  if (left > 0) {
#pragma unroll 4
    for (int t = rank * DBIAS_WARPS + warp; t < T; t += DBIAS_WARPS * DBIAS_CLUSTER) {
      const uint4 v = load8(dY + static_cast<size_t>(t) * ld_dy + c, whole, left);
      uint4 zv = {};
      if (ACT != ACT_NONE) zv = load8(Z + static_cast<size_t>(t) * m + c, whole, left);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        sum[j] += ACT != ACT_NONE ? at8<BF>(v, j) * act_grad<ACT>(at8<BF>(zv, j)) : at8<BF>(v, j);
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) part[warp][lane * 8 + j] = sum[j];
  __syncthreads();
  float v = part[0][threadIdx.x];
#pragma unroll
  for (int w = 1; w < DBIAS_WARPS; ++w) v += part[w][threadIdx.x];
  part[0][threadIdx.x] = v;
  cluster_sync();
  const int col = c0 + static_cast<int>(threadIdx.x);
  if (rank == 0 && col < m) {
    v = 0.0f;
    for (int o = 0; o < DBIAS_CLUSTER; ++o) v += ld_dsmem_f(mapa_shared(smem_u32(&part[0][threadIdx.x]), o));
    dbias[col] = v;
  }
  cluster_sync();
}
static_assert(DBIAS_COLS == DBIAS_WARPS * 32, "a column per thread");

// out[t][perm[k]] = in[t][k]: the row is scattered in shared memory and leaves in order.  4096 x 4096
// values: 16 us (4.2 TB/s).
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
