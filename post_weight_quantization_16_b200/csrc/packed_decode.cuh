// packed_decode.cuh — products of packed weights with a few tokens: the linear layer for decoding
// (linear_decode_kernel) and the two products of the mixture-of-experts layer (moe_gate_up_kernel,
// moe_down_kernel).
//
//     y[t][r] = sum over groups G of  s[r][G] * ( sum over k in G of (u[r][k] - z[r][G]) x[t][k] )
//
// u - z is a small integer and exact in fp16 and bf16, and a product of two 16-bit values is exact
// in fp32, so the only roundings of a group's inner sum are those of its fp32 accumulation; the
// scale multiplies the group's sum in fp32.  No weight is rounded to 16 bits.
//
// What bounds it: the packed codes are read once (HBM).  A weight costs 0.5 byte at 4 bits, so at
// the card's copy rate an SM has to unpack about 46 weights a cycle with 128 lanes: at most 2.8
// instructions a weight in all.  Unpacking a word of eight 4-bit codes therefore takes pairs of
// codes (i, i + 4) with one logical operation each (the mask and the exponent of 1024 or 128 in one
// lop3) and one packed subtraction or fused multiply-add; the pair order is matched on the
// activations' side by byte permutes, once per token tile.
//
// One warp owns 16 * RT weight rows and a range of 128-column chunks; mma.sync m16n8k16 takes the
// weights as the 16-row operand and eight tokens as the columns.  The order of k inside an MMA is
// free as long as both operands agree: the lane of quad position q owns GU / 4 consecutive columns
// of every unit of GU = min(group, 128) columns, so codes arrive as 16-byte loads straight from the
// framework's row format (no repacking, no shared memory) and a unit never mixes two groups.
// The block's warps and the blocks of a cluster split k; partial sums meet in shared memory and
// over distributed shared memory in a fixed order, so results are deterministic and need no
// workspace.  tcgen05 is not used here: with at most 16 tokens its operand would have to pass
// through shared memory, which costs more than the product itself.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "sm100_ptx.cuh"

namespace gptq {

// ------------------------------------------------------------------------------------------
// activations of the epilogues
// ------------------------------------------------------------------------------------------
enum : int { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_SILU = 3 };

__device__ __forceinline__ float act_apply(float z, int act) {
  if (act == ACT_RELU) return z > 0.0f ? z : 0.0f;
  if (act == ACT_GELU) return 0.5f * z * erfcf(z * -0.70710678118654752f);  // z times the normal CDF
  if (act == ACT_SILU) return z / (1.0f + expf(-z));
  return z;
}

// ------------------------------------------------------------------------------------------
// 16-bit types
// ------------------------------------------------------------------------------------------
template <bool BF>
__device__ __forceinline__ float h2f(uint16_t v) {
  if (BF) return __uint_as_float(static_cast<uint32_t>(v) << 16);
  return __half2float(__ushort_as_half(v));
}
template <bool BF>
__device__ __forceinline__ uint16_t f2h(float v) {
  if (BF) return __bfloat16_as_ushort(__float2bfloat16_rn(v));
  return __half_as_ushort(__float2half_rn(v));
}
template <bool BF>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if (BF) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <bool BF>
__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
  if (BF) {
    const __nv_bfloat162 v =
        __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t fma2_f16(uint32_t a, uint32_t b, uint32_t c) {
  const __half2 v = __hfma2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b),
                            *reinterpret_cast<const __half2*>(&c));
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <bool BF>
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  if (BF)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// ------------------------------------------------------------------------------------------
// unpacking: eight consecutive codes -> four pairs (u_i - z, u_{i+4} - z), i = 0 .. 3, exact
// ------------------------------------------------------------------------------------------
// What a row's zero-point has to be subtracted as.  fp16 with 4 bits: codes in the upper nibble
// of a byte stay there (1024 + 16 u) and the fused multiply-add by 1/16 brings them down.
struct ZeroTerm {
  uint32_t a, b;  // packed pairs; 8-bit codes with bf16: a is 2^23 + z in fp32
};
template <int BITS, bool BF>
__device__ __forceinline__ ZeroTerm zero_term(float z) {
  ZeroTerm t;
  if (BITS == 8 && BF) {
    t.a = __float_as_uint(8388608.0f + z);
    t.b = 0;
  } else if (BF) {
    t.a = pack2<true>(128.0f + z, 128.0f + z);
    t.b = 0;
  } else {
    t.a = pack2<false>(1024.0f + z, 1024.0f + z);
    t.b = BITS == 4 ? pack2<false>(-64.0f - z, -64.0f - z) : 0u;
  }
  return t;
}

// v: the block's codes in its low 8 * BITS bits (8-bit codes: v holds codes 0-3, v1 codes 4-7).
template <int BITS, bool BF>
__device__ __forceinline__ void unpack8(uint32_t v, uint32_t v1, const ZeroTerm& zt, uint32_t (&p)[4]) {
  constexpr uint32_t magic = BF ? 0x43004300u : 0x64006400u;  // 128 or 1024 in both halves
  if (BITS == 8) {
    if (BF) {
      // 128 + u does not fit bf16's eight significant bits: through fp32 under the exponent of 2^23
      const float zm = __uint_as_float(zt.a);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float lo = __uint_as_float(__byte_perm(v, 0x4B000000u, 0x7540u + i)) - zm;
        const float hi = __uint_as_float(__byte_perm(v1, 0x4B000000u, 0x7540u + i)) - zm;
        p[i] = pack2<true>(lo, hi);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t t = __byte_perm(v, v1, 0x0400u + 0x0101u * i);  // bytes: v.i, -, v1.i, -
        p[i] = sub2<false>((t & 0x00FF00FFu) | magic, zt.a);
      }
    }
  } else if (BITS == 4 && !BF) {
    constexpr uint32_t sixteenth = 0x2C002C00u;  // 1/16 in both halves
    const uint32_t w8 = v >> 8;
    p[0] = sub2<false>((v & 0x000F000Fu) | magic, zt.a);
    p[1] = fma2_f16((v & 0x00F000F0u) | magic, sixteenth, zt.b);
    p[2] = sub2<false>((w8 & 0x000F000Fu) | magic, zt.a);
    p[3] = fma2_f16((w8 & 0x00F000F0u) | magic, sixteenth, zt.b);
  } else {
    constexpr uint32_t m1 = (1u << BITS) - 1u, mask = m1 | (m1 << 16);
    uint32_t c = v;  // codes 0-3 from bit 0, codes 4-7 from bit 16
    if (BITS == 3) c = (v & 0x00000FFFu) | ((v << 4) & 0x0FFF0000u);
    if (BITS == 2) c = __byte_perm(v, 0u, 0x4140u);
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = sub2<BF>(((c >> (BITS * i)) & mask) | magic, zt.a);
  }
}

// ------------------------------------------------------------------------------------------
// a lane's share of one 128-column chunk of one packed row
// ------------------------------------------------------------------------------------------
__device__ __forceinline__ uint32_t ldg32(const uint32_t* p) { return __ldg(p); }
__device__ __forceinline__ uint2 ldg64(const uint32_t* p) { return __ldg(reinterpret_cast<const uint2*>(p)); }
__device__ __forceinline__ uint4 ldg128(const uint32_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <int BITS, int GU>
struct RawChunk {
  static constexpr int UNITS = 128 / GU;
  static constexpr int BLOCKS = GU / 32;  // blocks of eight codes a lane owns in a unit
  // words a lane keeps per unit: 3-bit codes of narrow units do not start on word boundaries
  static constexpr int WPU = GU == 128 ? BITS
                             : GU == 64 ? (BITS == 3 ? 2 : BITS / 2)
                                        : (BITS == 8 ? 2 : BITS == 3 ? 2 : 1);
  uint32_t w[UNITS * WPU];

  // base: the row's words of this chunk
  __device__ __forceinline__ void load(const uint32_t* base, int q) {
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      const uint32_t* ub = base + u * (GU * BITS / 32);
      uint32_t* d = w + u * WPU;
      if (BITS == 3) {
        if (GU == 128) {
#pragma unroll
          for (int j = 0; j < WPU; ++j) d[j] = ldg32(ub + 3 * q + j);
        } else {
          const int i = GU == 64 ? (3 * q) >> 1 : (24 * q) >> 5;
          d[0] = ldg32(ub + i);
          d[1 % WPU] = ldg32(ub + (GU == 64 ? i + 1 : min(i + 1, 2)));
        }
      } else if (BITS == 2 && GU == 32) {
        d[0] = __ldg(reinterpret_cast<const uint16_t*>(ub) + q);
      } else if (WPU % 4 == 0) {
#pragma unroll
        for (int j = 0; j < WPU / 4; ++j) {
          const uint4 x = ldg128(ub + q * WPU + 4 * j);
          d[4 * j] = x.x;
          d[(4 * j + 1) % WPU] = x.y;
          d[(4 * j + 2) % WPU] = x.z;
          d[(4 * j + 3) % WPU] = x.w;
        }
      } else if (WPU == 2) {
        const uint2 x = ldg64(ub + q * 2);
        d[0] = x.x;
        d[1 % WPU] = x.y;
      } else {
        d[0] = ldg32(ub + q);
      }
    }
  }

  // block b of unit u: its codes in the low bits of v (8-bit: codes 4-7 in v1)
  __device__ __forceinline__ void block(int u, int b, int q, uint32_t& v, uint32_t& v1) const {
    const uint32_t* d = w + u * WPU;
    v1 = 0;
    if (BITS == 8) {
      v = d[(2 * b) % WPU];
      v1 = d[(2 * b + 1) % WPU];
    } else if (BITS == 4) {
      v = d[b % WPU];
    } else if (BITS == 2) {
      v = (GU == 32) ? d[0] : ((b & 1) ? d[(b >> 1) % WPU] >> 16 : d[(b >> 1) % WPU]);
    } else if (GU == 128) {
      v = b == 0 ? d[0]
                 : b == 1 ? __funnelshift_r(d[0], d[1 % WPU], 24)
                          : b == 2 ? __funnelshift_r(d[1 % WPU], d[2 % WPU], 16) : d[2 % WPU] >> 8;
    } else if (GU == 64) {
      const int sh = (q & 1) * 16;
      const uint32_t lo = __funnelshift_r(d[0], d[1 % WPU], sh);
      v = b == 0 ? lo : __funnelshift_r(lo, d[1 % WPU] >> sh, 24);
    } else {
      v = __funnelshift_r(d[0], d[1 % WPU], (24 * q) & 31);
    }
  }
};

// ------------------------------------------------------------------------------------------
// the stream of a warp: 16 * RT rows x NT * 8 tokens over chunks [c0, c1)
// ------------------------------------------------------------------------------------------
struct GroupIndex {
  int units_per_chunk_shift;  // group < 128: log2(128 / group) groups in a chunk, else 0
  int div;                    // group >= 128: chunks per group
  uint32_t magic;             // ceil(2^32 / div), exact for chunk < 2^14 and div <= 2^14
};
// Index of the group of unit u in chunk c.
template <int GU>
__device__ __forceinline__ int group_of(const GroupIndex& gi, int c, int u) {
  if (GU < 128) return c * (128 / GU) + u;
  return gi.div == 1 ? c : static_cast<int>(__umulhi(static_cast<uint32_t>(c), gi.magic));
}

template <int BITS, bool BF, int GU, int NT, int RT>
struct Stream {
  using Raw = RawChunk<BITS, GU>;
  static constexpr int UNITS = Raw::UNITS, BLOCKS = Raw::BLOCKS;
  static constexpr int DEPTH = 2;  // chunks whose codes are in flight

  struct Stage {
    Raw raw[RT][2];
    float s[RT][2][UNITS], z[RT][2][UNITS];
  };

  const uint32_t* code[RT][2];  // rows g and g + 8 of each 16-row tile
  const float* scale[RT][2];
  ptrdiff_t zoff;               // zeros - scales (elements)
  GroupIndex gi;
  int q;

  __device__ __forceinline__ void fetch(Stage& st, int c) const {
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        st.raw[r][h].load(code[r][h] + static_cast<size_t>(c) * (4 * BITS), q);
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
          const float* sp = scale[r][h] + group_of<GU>(gi, c, u);
          st.s[r][h][u] = __ldg(sp);
          st.z[r][h][u] = __ldg(sp + zoff);
        }
      }
  }

  __device__ __forceinline__ void compute(const Stage& st, int c, const uint16_t* const (&x)[NT],
                                          float (&acc)[RT][NT][4]) const {
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      float sum[RT][NT][4];
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) sum[r][t][j] = 0.0f;
      ZeroTerm zt[RT][2];
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h) zt[r][h] = zero_term<BITS, BF>(st.z[r][h][u]);
#pragma unroll
      for (int b = 0; b < BLOCKS; ++b) {
        uint32_t xb[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const uint4 v = *reinterpret_cast<const uint4*>(x[t] + c * 128 + u * GU + q * (GU / 4) + b * 8);
          xb[t][0] = __byte_perm(v.x, v.z, 0x5410);
          xb[t][1] = __byte_perm(v.x, v.z, 0x7632);
          xb[t][2] = __byte_perm(v.y, v.w, 0x5410);
          xb[t][3] = __byte_perm(v.y, v.w, 0x7632);
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          uint32_t pa[4], pb[4], v, v1;
          st.raw[r][0].block(u, b, q, v, v1);
          unpack8<BITS, BF>(v, v1, zt[r][0], pa);
          st.raw[r][1].block(u, b, q, v, v1);
          unpack8<BITS, BF>(v, v1, zt[r][1], pb);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            mma_16816<BF>(sum[r][t], pa[0], pb[0], pa[1], pb[1], xb[t][0], xb[t][1]);
            mma_16816<BF>(sum[r][t], pa[2], pb[2], pa[3], pb[3], xb[t][2], xb[t][3]);
          }
        }
      }
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          acc[r][t][0] = fmaf(st.s[r][0][u], sum[r][t][0], acc[r][t][0]);
          acc[r][t][1] = fmaf(st.s[r][0][u], sum[r][t][1], acc[r][t][1]);
          acc[r][t][2] = fmaf(st.s[r][1][u], sum[r][t][2], acc[r][t][2]);
          acc[r][t][3] = fmaf(st.s[r][1][u], sum[r][t][3], acc[r][t][3]);
        }
    }
  }

  __device__ __forceinline__ void prologue(Stage (&st)[DEPTH], int c0, int c1) const {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
      if (c0 + d < c1) fetch(st[d], c0 + d);
  }
  __device__ __forceinline__ void run(Stage (&st)[DEPTH], int c0, int c1, const uint16_t* const (&x)[NT],
                                      float (&acc)[RT][NT][4]) const {
    for (int c = c0; c < c1; c += DEPTH) {
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) {
        if (c + d < c1) {
          compute(st[d], c + d, x, acc);
          if (c + d + DEPTH < c1) fetch(st[d], c + d + DEPTH);
        }
      }
    }
  }
};

// ------------------------------------------------------------------------------------------
// cluster helpers
// ------------------------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_nctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ float4 ld_dsmem_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ float ld_dsmem_f(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}

// ------------------------------------------------------------------------------------------
// the linear layer for few tokens
// ------------------------------------------------------------------------------------------
constexpr int DEC_WARPS = 8;  // warps of a block: they split k

struct LinearDecodeArgs {
  const uint16_t* X;  // [T x n], sweep order
  int64_t ldx;
  const uint32_t* codes;
  const float *scales, *zeros;
  int T, m, chunks, G;
  GroupIndex gi;
  const uint16_t *bias, *residual;
  int64_t ld_res, ldy;
  void* Y;
  uint16_t* preact;  // [T x m] or null
  int act, y_fp32;
  int early;    // 1: the launch before this one belongs to the same call, so weights may be read before it ends
  int* status;  // cleared (this kernel waits on nothing)
};

template <int BITS, bool BF, int GU, int NT, int RT>
__global__ void __launch_bounds__(DEC_WARPS * 32) linear_decode_kernel(const LinearDecodeArgs p) {
  __shared__ float4 red[DEC_WARPS][RT * NT * 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int cs = static_cast<int>(cluster_nctarank()), rank = static_cast<int>(cluster_ctarank());
  const int row0 = static_cast<int>(blockIdx.x) / cs * (16 * RT);
  const int tok0 = static_cast<int>(blockIdx.y) * (8 * NT);
  Stream<BITS, BF, GU, NT, RT> s;
  s.q = q;
  s.gi = p.gi;
  s.zoff = p.zeros - p.scales;
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = min(row0 + 16 * r + 8 * h + g, p.m - 1);  // rows past m repeat the last one, unstored
      s.code[r][h] = p.codes + static_cast<size_t>(row) * p.chunks * (4 * BITS);
      s.scale[r][h] = p.scales + static_cast<size_t>(row) * p.G;
    }
  const int slice = rank * DEC_WARPS + warp, slices = cs * DEC_WARPS;
  const int c0 = static_cast<int>(static_cast<int64_t>(p.chunks) * slice / slices);
  const int c1 = static_cast<int>(static_cast<int64_t>(p.chunks) * (slice + 1) / slices);
  typename Stream<BITS, BF, GU, NT, RT>::Stage st[Stream<BITS, BF, GU, NT, RT>::DEPTH];
  if (!p.early) griddep_wait();
  s.prologue(st, c0, c1);
  if (p.early) griddep_wait();
  griddep_launch_dependents();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.status = 0;
  const uint16_t* x[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) x[t] = p.X + static_cast<size_t>(min(tok0 + 8 * t + g, p.T - 1)) * p.ldx;
  float acc[RT][NT][4];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[r][t][j] = 0.0f;
  s.run(st, c0, c1, x, acc);
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t)
      red[warp][(r * NT + t) * 32 + lane] = make_float4(acc[r][t][0], acc[r][t][1], acc[r][t][2], acc[r][t][3]);
  __syncthreads();
  // the block's warps in order, then the cluster's blocks in order
  constexpr int ITEMS = RT * NT * 32;
  for (int i = threadIdx.x; i < ITEMS; i += DEC_WARPS * 32) {
    float4 v = red[0][i];
#pragma unroll
    for (int w = 1; w < DEC_WARPS; ++w) {
      const float4 o = red[w][i];
      v.x += o.x;
      v.y += o.y;
      v.z += o.z;
      v.w += o.w;
    }
    red[0][i] = v;
  }
  if (cs > 1) {
    cluster_sync();
  } else {
    __syncthreads();
  }
  if (rank == 0) {
    for (int i = threadIdx.x; i < ITEMS; i += DEC_WARPS * 32) {
      float4 v = red[0][i];
      for (int o = 1; o < cs; ++o) {
        const float4 w = ld_dsmem_f4(mapa_shared(smem_u32(&red[0][i]), o));
        v.x += w.x;
        v.y += w.y;
        v.z += w.z;
        v.w += w.w;
      }
      const int l = i & 31, t = (i >> 5) % NT, r = (i >> 5) / NT;
      const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int row = row0 + 16 * r + (l >> 2) + 8 * (j >> 1);
        const int tok = tok0 + 8 * t + 2 * (l & 3) + (j & 1);
        if (row < p.m && tok < p.T) {
          float z = e[j];
          if (p.bias) z += h2f<BF>(p.bias[row]);
          if (p.preact) p.preact[static_cast<size_t>(tok) * p.m + row] = f2h<BF>(z);
          float y = act_apply(z, p.act);
          if (p.residual) y += h2f<BF>(p.residual[static_cast<size_t>(tok) * p.ld_res + row]);
          if (p.y_fp32)
            static_cast<float*>(p.Y)[static_cast<size_t>(tok) * p.ldy + row] = y;
          else
            static_cast<uint16_t*>(p.Y)[static_cast<size_t>(tok) * p.ldy + row] = f2h<BF>(y);
        }
      }
    }
  }
  if (cs > 1) cluster_sync();  // no block leaves while its sums may still be read
}

// ------------------------------------------------------------------------------------------
// the mixture-of-experts products
// ------------------------------------------------------------------------------------------
constexpr int MOE_MAX_T = 128;      // "few tokens": the down product keeps a row of sums per token in shared memory
constexpr int MOE_MAX_E = 256;
constexpr int MOE_MAX_TOPK = 16;

// The routing of one call (workspace): the experts that got tokens, in ascending order, and their
// (token, choice) pairs, ascending inside an expert.
struct MoePlan {
  int* active;        // [1]
  int* expert;        // [E] expert of slot s
  int* begin;         // [E] first list position of slot s
  int* count;         // [E] pairs of slot s
  int* pair;          // [T * top_k] pair (token * top_k + choice) at list position i
  float* weight;      // [T * top_k] its routing weight
};

struct MoeArgs {
  const uint16_t* X;  // gathered: [T * top_k x H] in list order and the expert's sweep order; else [T x H]
  int64_t ldx;
  int gathered;
  MoePlan plan;
  int T, E, top_k, H, I;
  const uint32_t *gu_codes, *dn_codes;
  const float *gu_scales, *gu_zeros, *dn_scales, *dn_zeros;
  int gu_G, dn_G;
  GroupIndex gu_gi, dn_gi;
  int act;
  uint16_t* h;  // [T * top_k x I], list order
  const uint16_t* residual;
  int64_t ld_res, ldy;
  uint16_t* Y;
};

// h = act(x Wg^T) * (x Wu^T), rounded to the activations' type (the operand type of the second
// product).  Grid (I / (8 RT), slots): a block's 16-row tiles hold eight gate rows and, as rows
// 8-15, the same eight up rows, so both halves of an h value end up in one lane.
template <int BITS, bool BF, int GU, int NT, int RT>
__global__ void __launch_bounds__(DEC_WARPS * 32) moe_gate_up_kernel(const MoeArgs p) {
  __shared__ float4 red[DEC_WARPS][RT * NT * 32];
  griddep_wait();
  griddep_launch_dependents();
  const int slot = static_cast<int>(blockIdx.y);
  if (slot >= *p.plan.active) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int e = p.plan.expert[slot], begin = p.plan.begin[slot], count = p.plan.count[slot];
  const int i0 = static_cast<int>(blockIdx.x) * (8 * RT);
  const int chunks = p.H / 128;
  Stream<BITS, BF, GU, NT, RT> s;
  s.q = q;
  s.gi = p.gu_gi;
  s.zoff = p.gu_zeros - p.gu_scales;
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const size_t row = static_cast<size_t>(e) * 2 * p.I + static_cast<size_t>(h) * p.I + (i0 + 8 * r + g);
      s.code[r][h] = p.gu_codes + row * chunks * (4 * BITS);
      s.scale[r][h] = p.gu_scales + row * p.gu_G;
    }
  const int c0 = chunks * warp / DEC_WARPS, c1 = chunks * (warp + 1) / DEC_WARPS;
  for (int b0 = 0; b0 < count; b0 += 8 * NT) {
    typename Stream<BITS, BF, GU, NT, RT>::Stage st[Stream<BITS, BF, GU, NT, RT>::DEPTH];
    s.prologue(st, c0, c1);
    const uint16_t* x[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int i = begin + min(b0 + 8 * t + g, count - 1);
      x[t] = p.X + static_cast<size_t>(p.gathered ? i : p.plan.pair[i] / p.top_k) * p.ldx;
    }
    float acc[RT][NT][4];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[r][t][j] = 0.0f;
    s.run(st, c0, c1, x, acc);
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int t = 0; t < NT; ++t)
        red[warp][(r * NT + t) * 32 + lane] = make_float4(acc[r][t][0], acc[r][t][1], acc[r][t][2], acc[r][t][3]);
    __syncthreads();
    for (int i = threadIdx.x; i < RT * NT * 32; i += DEC_WARPS * 32) {
      float4 v = red[0][i];
#pragma unroll
      for (int w = 1; w < DEC_WARPS; ++w) {
        const float4 o = red[w][i];
        v.x += o.x;
        v.y += o.y;
        v.z += o.z;
        v.w += o.w;
      }
      const int l = i & 31, t = (i >> 5) % NT, r = (i >> 5) / NT;
      const int col = i0 + 8 * r + (l >> 2), n0 = b0 + 8 * t + 2 * (l & 3);
      if (n0 < count) p.h[static_cast<size_t>(begin + n0) * p.I + col] = f2h<BF>(act_apply(v.x, p.act) * v.z);
      if (n0 + 1 < count) p.h[static_cast<size_t>(begin + n0 + 1) * p.I + col] = f2h<BF>(act_apply(v.y, p.act) * v.w);
    }
    __syncthreads();
  }
}

// y = sum over the token's experts of weight * h Wd^T, + residual.  A block owns 16 RT output
// rows of every expert: its warps (and the cluster's blocks) split the list of (slot, chunk)
// evenly, each adding its share of every expert into its own row of sums per token in shared
// memory; the shares meet in a fixed order.  One pass, no sums in global memory, no atomics.
template <int BITS, bool BF, int GU, int NT, int RT>
__global__ void __launch_bounds__(DEC_WARPS * 32) moe_down_kernel(const MoeArgs p) {
  extern __shared__ float ysum[];  // [DEC_WARPS][T][16 RT]
  constexpr int ROWS = 16 * RT;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int cs = static_cast<int>(cluster_nctarank()), rank = static_cast<int>(cluster_ctarank());
  const int row0 = static_cast<int>(blockIdx.x) / cs * ROWS;
  float* mine = ysum + static_cast<size_t>(warp) * p.T * ROWS;
  for (int i = lane; i < p.T * ROWS; i += 32) mine[i] = 0.0f;
  __syncwarp();
  griddep_wait();
  griddep_launch_dependents();
  const int chunks = p.I / 128;
  const int64_t total = static_cast<int64_t>(*p.plan.active) * chunks;
  const int slice = rank * DEC_WARPS + warp, slices = cs * DEC_WARPS;
  const int64_t w0 = total * slice / slices, w1 = total * (slice + 1) / slices;
  Stream<BITS, BF, GU, NT, RT> s;
  s.q = q;
  s.gi = p.dn_gi;
  s.zoff = p.dn_zeros - p.dn_scales;
  for (int64_t w = w0; w < w1;) {
    const int slot = static_cast<int>(w / chunks);
    const int c0 = static_cast<int>(w - static_cast<int64_t>(slot) * chunks);
    const int c1 = static_cast<int>(min(static_cast<int64_t>(chunks), c0 + (w1 - w)));
    w += c1 - c0;
    const int e = p.plan.expert[slot], begin = p.plan.begin[slot], count = p.plan.count[slot];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int rr = min(row0 + 16 * r + 8 * h + g, p.H - 1);
        const size_t row = static_cast<size_t>(e) * p.H + rr;
        s.code[r][h] = p.dn_codes + row * chunks * (4 * BITS);
        s.scale[r][h] = p.dn_scales + row * p.dn_G;
      }
    for (int b0 = 0; b0 < count; b0 += 8 * NT) {
      typename Stream<BITS, BF, GU, NT, RT>::Stage st[Stream<BITS, BF, GU, NT, RT>::DEPTH];
      s.prologue(st, c0, c1);
      const uint16_t* x[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t)
        x[t] = p.h + static_cast<size_t>(begin + min(b0 + 8 * t + g, count - 1)) * p.I;
      float acc[RT][NT][4];
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[r][t][j] = 0.0f;
      s.run(st, c0, c1, x, acc);
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int i = b0 + 8 * t + 2 * q + j;
          if (i < count) {
            const float wt = p.plan.weight[begin + i];
            float* y = mine + static_cast<size_t>(p.plan.pair[begin + i] / p.top_k) * ROWS + g;
#pragma unroll
            for (int r = 0; r < RT; ++r) {
              y[16 * r] = fmaf(wt, acc[r][t][j], y[16 * r]);
              y[16 * r + 8] = fmaf(wt, acc[r][t][2 + j], y[16 * r + 8]);
            }
          }
        }
      __syncwarp();
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.T * ROWS; i += DEC_WARPS * 32) {
    float v = ysum[i];
#pragma unroll
    for (int k = 1; k < DEC_WARPS; ++k) v += ysum[static_cast<size_t>(k) * p.T * ROWS + i];
    ysum[i] = v;
  }
  if (cs > 1) {
    cluster_sync();
  } else {
    __syncthreads();
  }
  if (rank == 0) {
    for (int i = threadIdx.x; i < p.T * ROWS; i += DEC_WARPS * 32) {
      float v = ysum[i];
      for (int o = 1; o < cs; ++o) v += ld_dsmem_f(mapa_shared(smem_u32(&ysum[i]), o));
      const int tok = i / ROWS, row = row0 + i % ROWS;
      if (row < p.H) {
        if (p.residual) v += h2f<BF>(p.residual[static_cast<size_t>(tok) * p.ld_res + row]);
        p.Y[static_cast<size_t>(tok) * p.ldy + row] = f2h<BF>(v);
      }
    }
  }
  if (cs > 1) cluster_sync();
}

// ------------------------------------------------------------------------------------------
// launches, one translation unit per code width (packed_decode_inst.cuh)
// ------------------------------------------------------------------------------------------
struct DecodeLaunch {
  bool bf16;
  int unit;      // 32, 64 or 128
  int nt, rt;    // (1, 1) or (2, 2)
  int cluster;   // blocks that split k
  int device;
  cudaStream_t stream;
};

template <int BITS>
cudaError_t launch_linear_decode(const DecodeLaunch& l, const LinearDecodeArgs& a);
template <int BITS>
cudaError_t launch_moe_gate_up(const DecodeLaunch& l, const MoeArgs& a, int slots);
template <int BITS>
cudaError_t launch_moe_down(const DecodeLaunch& l, const MoeArgs& a);

// A launch that may overlap the end of the kernel before it (every kernel here waits for that
// kernel before it touches what it wrote).
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, int cluster, cudaStream_t stream,
                       Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// Raise a kernel's dynamic shared-memory limit to `smem` once per device.
template <typename K>
cudaError_t raise_smem_limit(std::atomic<uint64_t>& done, int device, K kernel, int smem) {
  const uint64_t bit = uint64_t(1) << (device & 63);
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

}  // namespace gptq
