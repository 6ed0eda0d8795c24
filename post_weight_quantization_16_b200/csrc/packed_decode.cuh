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
// mma.sync m16n8k16 takes the weights as the 16-row operand and eight tokens as the columns; the
// order of k inside an MMA is free as long as both operands agree: the lane of quad position q owns
// GU / 4 consecutive columns of every unit of GU = min(group, 128) columns, so a unit never mixes
// two groups and a lane's codes are one 16-byte word group of the framework's row format (no
// repacking).  A block owns 128 rows (a warp 16) and a range of 128-column chunks.  One producer
// lane streams the codes by TMA, and the activations by bulk copies, through a ring of shared-memory
// stages deep enough to cover HBM's latency; the activations come in "fragment order" (below), which
// a small kernel lays out first, so that a warp reads them as conflict-free 16-byte words that are
// the MMA operand as they stand.  The blocks of a cluster split k; their sums meet over distributed
// shared memory in a fixed order, so results are deterministic.  tcgen05 is not used here: with
// this few tokens its operand would have to pass through shared memory once more, which costs more
// than the product.
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

// One form each for all kernels, so that a value does not depend on the number of tokens, and short: the
// CTA-pair kernel's epilogue holds 128 of them a thread, unrolled, and longer code costs it more than its
// operations do (2048 tokens through 11008 x 4096 with SiLU: 294 us with expf, 263 with these, 254 with a plain
// __expf whose error grows with |z|).
__device__ __forceinline__ float ex2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_ftz(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// -(hi + lo) log2 e = y + r with y in fp32 and r the rest, log2 e in two parts: an exponent's own rounding,
// 2^-24 of some 100, would be an error of 2^-17 of the power.
constexpr float kLog2e = 1.44269502f, kLog2eLow = 1.92596303e-8f, kLn2 = 0.693147182f;
__device__ __forceinline__ float2 minus_log2e(float hi) {
  const float y = -kLog2e * hi;
  return make_float2(y, fmaf(-kLog2eLow, hi, fmaf(-kLog2e, hi, -y)));
}
// SiLU, z / (1 + e^-z): relative error below 2^-20 (0 for z below -87.3).  Past 88 either way the power
// changes nothing, and its exponent's rest would not be a number.
__device__ __forceinline__ float silu(float z) {
  const float2 x = minus_log2e(fminf(fmaxf(z, -88.0f), 88.0f));
  const float p = ex2_ftz(x.x), e = fmaf(p, x.y * kLn2, p);
  return z * rcp_ftz(1.0f + e);
}
// GELU, z times the normal distribution function: relative error below 2^-19 (0 where e^(-z^2 / 2) is below
// 2^-126, z < -13.2).  The tail beyond |z| by the complementary error function's Chebyshev fit of Numerical
// Recipes, t e^(q(t) - x^2) with a relative error below 1.2e-7 for every x = |z| / sqrt 2; the rounding errors
// of the square and of its exponent go into the second power.
__device__ __forceinline__ float gelu(float z) {
  const float a = fminf(fabsf(z), 20.0f), square = a * a, low = fmaf(a, a, -square);
  const float t = rcp_ftz(1.0f + 0.35355339059327376f * a);
  float q = 0.17087277f;
  q = fmaf(t, q, -0.82215223f);
  q = fmaf(t, q, 1.48851587f);
  q = fmaf(t, q, -1.13520398f);
  q = fmaf(t, q, 0.27886807f);
  q = fmaf(t, q, -0.18628806f);
  q = fmaf(t, q, 0.09678418f);
  q = fmaf(t, q, 0.37409196f);
  q = fmaf(t, q, 1.00002368f);
  q = fmaf(t, q, -1.26551223f);
  const float2 x = minus_log2e(0.5f * square);
  const float r = fmaf(-0.5f * kLog2e, low, x.y);
  const float c = 0.5f * t * (ex2_ftz(x.x) * ex2_ftz(fmaf(kLog2e, q, r)));
  return z * (z < 0.0f ? c : 1.0f - c);
}
__device__ __forceinline__ float act_apply(float z, int act) {
  if (act == ACT_RELU) return z > 0.0f ? z : 0.0f;
  if (act == ACT_GELU) return gelu(z);
  if (act == ACT_SILU) return silu(z);
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
// 2^e for |e| <= 126, and as two factors for |e| <= 252
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }
__device__ __forceinline__ float2 pow2_halves(int e) { return make_float2(pow2(e >> 1), pow2(e - (e >> 1))); }
__device__ __forceinline__ uint32_t fma2_f16(uint32_t a, uint32_t b, uint32_t c) {
  const __half2 v = __hfma2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b),
                            *reinterpret_cast<const __half2*>(&c));
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Bounded wait of a whole warp: all lanes test the barrier together and take one decision, so that the warp
// stays converged (the MMAs and tensor-memory loads that follow are warp-wide instructions).
__device__ __forceinline__ bool warp_wait_uniform(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if ((i & 255u) == 0) {
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      const bool late = now - t0 > kWaitLimitNs;
      if (__any_sync(0xffffffffu, late)) *abort_flag = 1;
      if (__any_sync(0xffffffffu, late || *abort_flag)) return false;
    }
  }
}

// (for barriers that a peer block arrives on)
__device__ __forceinline__ bool warp_wait_uniform_cl(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  if (__all_sync(0xffffffffu, mbar_try_wait_cl(bar, parity))) return true;
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    if (__all_sync(0xffffffffu, mbar_try_wait_cl(bar, parity))) return true;
    if ((i & 255u) == 0) {
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      const bool late = now - t0 > kWaitLimitNs;
      if (__any_sync(0xffffffffu, late)) *abort_flag = 1;
      if (__any_sync(0xffffffffu, late || *abort_flag)) return false;
    }
  }
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

// The same with a zero addend (the first product of a sum).
template <bool BF>
__device__ __forceinline__ void mma_16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                uint32_t b0, uint32_t b1) {
  if (BF)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
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
// a lane's share of one 128-column chunk of one packed row (shared memory)
// ------------------------------------------------------------------------------------------
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
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

  // base: shared-memory address of the row's 16 * BITS bytes of this chunk
  __device__ __forceinline__ void load(uint32_t base, int q) {
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      const uint32_t ub = base + u * (GU * BITS / 8);
      uint32_t* d = w + u * WPU;
      if (BITS == 3) {
        if (GU == 128) {
#pragma unroll
          for (int j = 0; j < WPU; ++j) d[j] = lds32(ub + 4 * (3 * q + j));
        } else {
          const int i = GU == 64 ? (3 * q) >> 1 : (24 * q) >> 5;
          d[0] = lds32(ub + 4 * i);
          d[1 % WPU] = lds32(ub + 4 * (GU == 64 ? i + 1 : min(i + 1, 2)));
        }
      } else if (BITS == 2 && GU == 32) {
        d[0] = lds32(ub + 4 * (q >> 1)) >> (16 * (q & 1));
      } else if (WPU % 4 == 0) {
#pragma unroll
        for (int j = 0; j < WPU / 4; ++j) {
          const uint4 x = lds128(ub + 4 * (q * WPU + 4 * j));
          d[4 * j] = x.x;
          d[(4 * j + 1) % WPU] = x.y;
          d[(4 * j + 2) % WPU] = x.z;
          d[(4 * j + 3) % WPU] = x.w;
        }
      } else if (WPU == 2) {
        const uint2 x = lds64(ub + 8 * q);
        d[0] = x.x;
        d[1 % WPU] = x.y;
      } else {
        d[0] = lds32(ub + 4 * q);
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
// activations in fragment order
// ------------------------------------------------------------------------------------------
// A tile is eight tokens.  Of every 128-column chunk it takes FRAG_BYTES = 2 KB: four blocks x 32
// lanes x 16 bytes; lane (token n, quad position q) of block kb holds the eight columns
// frag_column(kb, q) .. + 7 in the pair order (0, 4), (1, 5), (2, 6), (3, 7) of unpack8.
constexpr int FRAG_BYTES = 2048;

// First column (within the chunk) of block kb (0 .. 3) of quad position q for units of gu columns.
__device__ __forceinline__ int frag_column(int gu, int kb, int q) {
  if (gu == 128) return q * 32 + kb * 8;
  if (gu == 64) return (kb >> 1) * 64 + q * 16 + (kb & 1) * 8;
  return kb * 32 + q * 8;
}
// Offset, in 16-bit values inside the chunk's FRAG_BYTES, of column c of token n.
__device__ __forceinline__ int frag_offset(int gu, int n, int c) {
  int kb, q;
  if (gu == 128) {
    q = c >> 5;
    kb = (c >> 3) & 3;
  } else if (gu == 64) {
    q = (c >> 4) & 3;
    kb = ((c >> 6) << 1) | ((c >> 3) & 1);
  } else {
    q = (c >> 3) & 3;
    kb = c >> 5;
  }
  const int i = c & 7;
  return (kb * 32 + n * 4 + q) * 8 + 2 * (i & 3) + (i >> 2);
}
// The 16 bytes of one lane from a token's row: eight columns from `col`, through perm if there is one.
__device__ __forceinline__ uint4 frag_gather(const uint16_t* row, const int32_t* perm, int col) {
  uint4 v;
  if (perm) {
    const int4 a = *reinterpret_cast<const int4*>(perm + col), b = *reinterpret_cast<const int4*>(perm + col + 4);
    v.x = static_cast<uint32_t>(row[a.x]) | (static_cast<uint32_t>(row[b.x]) << 16);
    v.y = static_cast<uint32_t>(row[a.y]) | (static_cast<uint32_t>(row[b.y]) << 16);
    v.z = static_cast<uint32_t>(row[a.z]) | (static_cast<uint32_t>(row[b.z]) << 16);
    v.w = static_cast<uint32_t>(row[a.w]) | (static_cast<uint32_t>(row[b.w]) << 16);
  } else {
    const uint4 r = *reinterpret_cast<const uint4*>(row + col);
    v.x = __byte_perm(r.x, r.z, 0x5410);
    v.y = __byte_perm(r.x, r.z, 0x7632);
    v.z = __byte_perm(r.y, r.w, 0x5410);
    v.w = __byte_perm(r.y, r.w, 0x7632);
  }
  return v;
}

// ------------------------------------------------------------------------------------------
// the stream of a block: 128 rows x up to NT tiles of tokens over ranges of chunks
// ------------------------------------------------------------------------------------------
struct GroupIndex {
  int div;         // group >= 128: chunks per group
  uint32_t magic;  // ceil(2^32 / div), exact for chunk < 2^14 and div <= 2^14
};
// Index of the group of unit u in chunk c.
template <int GU>
__device__ __forceinline__ int group_of(const GroupIndex& gi, int c, int u) {
  if (GU < 128) return c * (128 / GU) + u;
  return gi.div == 1 ? c : static_cast<int>(__umulhi(static_cast<uint32_t>(c), gi.magic));
}

constexpr int DEC_WARPS = 8;                        // consumer warps: 16 rows each
constexpr int DEC_ROWS = 16 * DEC_WARPS;            // rows of a block
constexpr int DEC_THREADS = (DEC_WARPS + 1) * 32;   // and the producer warp
constexpr int DEC_MAX_STAGES = 12;
constexpr int DEC_SMEM = 94 * 1024;                 // ring of a block at most: two blocks per SM

__host__ __device__ constexpr int dec_code_bytes(int bits) { return DEC_ROWS * 16 * bits; }
__host__ __device__ constexpr int dec_stage_bytes(int bits, int nt) { return dec_code_bytes(bits) + nt * FRAG_BYTES; }
__host__ __device__ constexpr int dec_stages(int bits, int nt, int smem) {
  const int s = smem / dec_stage_bytes(bits, nt);
  return s > DEC_MAX_STAGES ? DEC_MAX_STAGES : s;
}
__host__ __device__ constexpr int dec_ring_bytes(int bits, int nt, int smem) {
  return 128 + dec_stages(bits, nt, smem) * dec_stage_bytes(bits, nt);
}

// Start of the dynamic shared memory at the next multiple of 128 bytes.
__device__ __forceinline__ uint8_t* align128(uint8_t* raw) {
  const uint32_t a = smem_u32(raw);
  return raw + (((a + 127u) & ~127u) - a);
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// A range of chunks of one weight matrix and the activations it meets.
struct Segment {
  int row_a, row_b;     // tensor-map rows of the stage's rows 0-63 and 64-127
  int c0, c1;           // chunks
  int tiles;            // token tiles, 1 .. NT
  const uint8_t* x;     // fragment order, [chunk][tiles][FRAG_BYTES]
};

// XL: the activations of the block's chunks are laid out in shared memory by its own consumer warps
// before the loop (few tokens: no launch of its own, no copies in the ring); NT is 1 then.
template <int BITS, bool BF, int GU, int NT, bool XL>
struct Ring {
  using Raw = RawChunk<BITS, GU>;
  static constexpr int UNITS = Raw::UNITS, BLOCKS = Raw::BLOCKS;
  static constexpr int STAGE = dec_stage_bytes(BITS, XL ? 0 : NT), CODES = dec_code_bytes(BITS);
  static_assert(!XL || NT == 1, "local activations: one tile");

  uint32_t base, full, empty;  // shared-memory addresses: stages, barriers
  int stages;
  volatile int* abort_flag;

  // Position in the ring: stage and the parity of its use.
  struct Cursor {
    int s = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void next(int stages) {
      if (++s == stages) {
        s = 0;
        ph ^= 1u;
      }
    }
  };

  __device__ __forceinline__ void init(uint32_t smem_base, int n, uint64_t* bars, int* flag) {
    stages = n;
    base = smem_base;
    full = smem_u32(bars);
    empty = full + 8 * stages;
    abort_flag = flag;
    if (threadIdx.x == 0) {
      for (int s = 0; s < stages; ++s) {
        mbar_init(full + 8 * s, 1);
        mbar_init(empty + 8 * s, DEC_WARPS);
      }
      *flag = 0;
      fence_mbar_init();
    }
    __syncthreads();
  }

  // Producer (one lane).  `it` counts stages over all segments of the block.
  __device__ __forceinline__ bool codes(const CUtensorMap* map, const Segment& g, int c, int it) const {
    const int s = it % stages;
    if (!mbar_wait_bounded(empty + 8 * s, (static_cast<uint32_t>(it / stages) & 1u) ^ 1u, abort_flag)) return false;
    const uint32_t fb = full + 8 * s, st = base + s * STAGE;
    mbar_arrive_expect_tx(fb, static_cast<uint32_t>(CODES + (XL ? 0 : g.tiles * FRAG_BYTES)));
    tma_load_2d(st, map, fb, c * (4 * BITS), g.row_a);
    tma_load_2d(st + CODES / 2, map, fb, c * (4 * BITS), g.row_b);
    return true;
  }
  __device__ __forceinline__ void acts(const Segment& g, int c, int it) const {
    if (XL) return;
    const int s = it % stages;
    bulk_load(base + s * STAGE + CODES, g.x + static_cast<size_t>(c) * g.tiles * FRAG_BYTES,
              static_cast<uint32_t>(g.tiles * FRAG_BYTES), full + 8 * s);
  }
  // No copy may be in flight when the block leaves.
  __device__ __forceinline__ void drain(int issued) const {
    for (int i = max(0, issued - stages); i < issued; ++i)
      mbar_wait_drain(full + 8 * (i % stages), static_cast<uint32_t>(i / stages) & 1u);
  }

  // Local activations: pieces [chunk][block][token][quad position] of 16 bytes.
  uint32_t xs;   // shared-memory address
  int xtok;      // tokens in them, 1 .. 8
  template <typename RowOf>
  __device__ __forceinline__ void lay_out(uint4* dst, int c0, int c1, int tokens, const int32_t* perm, RowOf&& row_of) {
    xs = smem_u32(dst);
    xtok = tokens;
    const int pieces = (c1 - c0) * 16 * tokens;
    for (int i = threadIdx.x; i < pieces; i += DEC_WARPS * 32) {
      const int q = i & 3, n = (i >> 2) % tokens, ck = (i >> 2) / tokens;
      dst[i] = frag_gather(row_of(n), perm, (c0 + (ck >> 2)) * 128 + frag_column(GU, ck & 3, q));
    }
    asm volatile("bar.sync 1, %0;" ::"n"(DEC_WARPS * 32) : "memory");  // the consumer warps
  }

  // Consumer warp.  A lane fetches one of the four parameter rows of its quad's two weight rows:
  // q = 0 scales of row a, 1 its zero-points, 2 and 3 those of row b; four units (a window) at a time,
  // one window ahead; shuffles spread them.  The 32 lanes' addresses lie in 32 cache lines whatever a
  // load's width, and the L1's tag lookups for them are what a load costs: with one load of 16 bytes
  // instead of four of 4 the gate and up product of 64 experts took 56 us, not 65 (3 bits, groups of
  // 64), and that of eight large ones 139, not 158.
  const float* param;
  int pitch;  // units of a parameter row
  int vec;    // values that a load can take by the rows' alignment: 4, 2 or 1
  GroupIndex gi;
  // Units 4 w .. 4 w + 3 of the rows; chunks c0 .. c1 - 1 are wanted.
  __device__ __forceinline__ void window(float (&v)[4], int w, int c0, int c1) const {
    if (UNITS > 1 || gi.div == 1) {
      const float* at = param + 4 * w;
      if (vec == 4) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(at));
        v[0] = x.x;
        v[1] = x.y;
        v[2] = x.z;
        v[3] = x.w;
      } else if (vec == 2) {
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          if (4 * w + j < pitch) {
            const float2 x = __ldg(reinterpret_cast<const float2*>(at + j));
            v[j] = x.x;
            v[j + 1] = x.y;
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (4 * w + j < pitch) v[j] = __ldg(at + j);
      }
    } else {  // a group of several chunks: one load
      int of = -1;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int g = group_of<GU>(gi, min(max(4 * w + j, c0), c1 - 1), 0);
        v[j] = j > 0 && g == of ? v[j > 0 ? j - 1 : 0] : __ldg(param + g);
        of = g;
      }
    }
  }

  // acc[t] += the warp's 16 rows x tile t over chunks [c0, c1), TL tiles; offa, offb: byte offsets
  // of the lane's two rows in a stage.  False when a wait ran out.
  template <int TL>
  __device__ __forceinline__ bool consume(int c0, int c1, uint32_t offa, uint32_t offb, int lane, Cursor& cur,
                                          float (&acc)[NT][4]) const {
    constexpr int PER = 4 / UNITS;  // chunks of a window
    const int q = lane & 3, src = lane & 28;
    uint32_t xat = XL ? xs + static_cast<uint32_t>((min(lane >> 2, xtok - 1) * 4 + q) * 16) : 0u;
    const uint32_t xstep = XL ? static_cast<uint32_t>(xtok * 64) : 0u;
    const int w1 = (c1 + PER - 1) / PER;
    float next[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    window(next, c0 / PER, c0, c1);
    for (int w = c0 / PER; w < w1; ++w) {
      float now[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) now[j] = next[j];
      if (w + 1 < w1) window(next, w + 1, c0, c1);
#pragma unroll
      for (int jj = 0; jj < PER; ++jj) {
        if (w * PER + jj >= c0 && w * PER + jj < c1) {
          if (!warp_wait_uniform(full + 8 * cur.s, cur.ph, abort_flag)) return false;
          const uint32_t st = base + cur.s * STAGE;
          Raw ra, rb;
          ra.load(st + offa, q);
          rb.load(st + offb, q);
#pragma unroll
          for (int u = 0; u < UNITS; ++u) {
            float sum[TL][4];
            const float pv = now[(jj * UNITS + u) % 4];
            const float s_a = __shfl_sync(0xffffffffu, pv, src), s_b = __shfl_sync(0xffffffffu, pv, src | 2);
            const ZeroTerm za = zero_term<BITS, BF>(__shfl_sync(0xffffffffu, pv, src | 1)),
                           zb = zero_term<BITS, BF>(__shfl_sync(0xffffffffu, pv, src | 3));
#pragma unroll
            for (int b = 0; b < BLOCKS; ++b) {
              uint32_t pa[4], pb[4], v, v1;
              ra.block(u, b, q, v, v1);
              unpack8<BITS, BF>(v, v1, za, pa);
              rb.block(u, b, q, v, v1);
              unpack8<BITS, BF>(v, v1, zb, pb);
#pragma unroll
              for (int t = 0; t < TL; ++t) {
                const uint4 x = lds128(XL ? xat : st + CODES + t * FRAG_BYTES + (u * BLOCKS + b) * 512 + lane * 16);
                if (b == 0)
                  mma_16816_first<BF>(sum[t], pa[0], pb[0], pa[1], pb[1], x.x, x.y);
                else
                  mma_16816<BF>(sum[t], pa[0], pb[0], pa[1], pb[1], x.x, x.y);
                mma_16816<BF>(sum[t], pa[2], pb[2], pa[3], pb[3], x.z, x.w);
              }
              if (XL) xat += xstep;
            }
#pragma unroll
            for (int t = 0; t < TL; ++t) {
              acc[t][0] = fmaf(s_a, sum[t][0], acc[t][0]);
              acc[t][1] = fmaf(s_a, sum[t][1], acc[t][1]);
              acc[t][2] = fmaf(s_b, sum[t][2], acc[t][2]);
              acc[t][3] = fmaf(s_b, sum[t][3], acc[t][3]);
            }
          }
          // The stage's loads have to be done, not only issued, before it is given back: with 16 warps'
          // loads queued, the copy that refills it was seen to overtake them where only the arrival
          // stood here (run-to-run differences; none with the fence, which costs 1 %).
          asm volatile("fence.acq_rel.cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(empty + 8 * cur.s);
          cur.next(stages);
        }
      }
    }
    return true;
  }
  // The same for a number of tiles known at run time (1 .. NT): loops without conditions inside.
  __device__ __forceinline__ bool consume_tiles(int tiles, int c0, int c1, uint32_t offa, uint32_t offb, int lane,
                                                Cursor& cur, float (&acc)[NT][4]) const {
    if (NT == 1 || tiles == 1) return consume<1>(c0, c1, offa, offb, lane, cur, acc);
    if (NT == 2 || tiles == 2) return consume<(NT < 2 ? NT : 2)>(c0, c1, offa, offb, lane, cur, acc);
    if (tiles == 3) return consume<(NT < 3 ? NT : 3)>(c0, c1, offa, offb, lane, cur, acc);
    return consume<NT>(c0, c1, offa, offb, lane, cur, acc);
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
// Measured, 4 bits: one token through 4096 x 4096 in act-order 7.8 us (1.2 TB/s), sixteen through
// 4096 x 11008 22 us (1.2 TB/s).  The first is a launch, one trip to memory, a few chunks and the
// cluster's sums, one after the other; the stream alone of the second (no unpacking, no products)
// takes 12 us, and the rest is the instructions of 16 tokens' products with 16 warps an SM.
constexpr int DEC_LOCAL_BYTES = 32 * 1024;  // local activations of a block at most

struct LinearDecodeArgs {
  const uint8_t* x;  // fragment order, [chunk][tiles][FRAG_BYTES] (not with local activations)
  const uint16_t* X;  // local activations: the caller's [T x n], and its order
  int64_t ldx;
  const int32_t* perm;
  const float *scales, *zeros;
  int stages;  // of the ring
  int T, tiles, m, chunks, G, vec;
  GroupIndex gi;
  const uint16_t *bias, *residual;
  int64_t ld_res, ldy;
  void* Y;
  uint16_t* preact;  // [T x m] or null
  int act, y_fp32;
  int* status;
};

template <int BITS, bool BF, int GU, int NT, bool XL>
__global__ void __launch_bounds__(DEC_THREADS)
    linear_decode_kernel(const __grid_constant__ CUtensorMap codes_map, const LinearDecodeArgs p) {
  extern __shared__ uint8_t dec_smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * DEC_MAX_STAGES];
  __shared__ int abort_flag;
  __shared__ float4 red[DEC_WARPS * NT * 32];
  uint8_t* dec_smem = align128(dec_smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int cs = static_cast<int>(cluster_nctarank()), rank = static_cast<int>(cluster_ctarank());
  const int row0 = static_cast<int>(blockIdx.x) / cs * DEC_ROWS;
  Ring<BITS, BF, GU, NT, XL> r;
  r.init(smem_u32(dec_smem), p.stages, bars, &abort_flag);
  Segment sg;
  sg.row_a = row0;
  sg.row_b = row0 + 64;
  sg.c0 = p.chunks * rank / cs;
  sg.c1 = p.chunks * (rank + 1) / cs;
  sg.tiles = p.tiles;
  sg.x = p.x;
  if (XL) {
    griddep_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;
  }
  if (warp == DEC_WARPS) {
    if (lane == 0) {
      const int n = sg.c1 - sg.c0, ahead = min(r.stages, n);
      int it = 0;
      // the launch before this one laid out x and had waited for all earlier work: the weights can
      // be read before it ends, x cannot
      for (; it < ahead; ++it) r.codes(&codes_map, sg, sg.c0 + it, it);
      if (!XL) griddep_wait();
      for (int i = 0; i < ahead; ++i) r.acts(sg, sg.c0 + i, i);
      for (; it < n; ++it) {
        if (!r.codes(&codes_map, sg, sg.c0 + it, it)) break;
        r.acts(sg, sg.c0 + it, it);
      }
      r.drain(it);
    }
    griddep_launch_dependents();
  } else {
    float acc[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[t][j] = 0.0f;
    const int ra = warp * 16 + g, rb = ra + 8;
    // (rows past m repeat the last one's parameters, unstored)
    r.param = ((q & 1) ? p.zeros : p.scales) + static_cast<size_t>(min(row0 + ((q & 2) ? rb : ra), p.m - 1)) * p.G;
    r.pitch = p.G;
    r.vec = p.vec;
    r.gi = p.gi;
    if (XL)
      r.lay_out(reinterpret_cast<uint4*>(dec_smem + p.stages * dec_stage_bytes(BITS, 0)), sg.c0, sg.c1, p.T, p.perm,
                [&](int n) { return p.X + n * p.ldx; });
    typename Ring<BITS, BF, GU, NT, XL>::Cursor cur;
    r.template consume<NT>(sg.c0, sg.c1, ra * (16 * BITS), rb * (16 * BITS), lane, cur, acc);
    if (!XL) griddep_wait();  // (the residual and the outputs are touched from here on)
#pragma unroll
    for (int t = 0; t < NT; ++t)
      red[(warp * NT + t) * 32 + lane] = make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
  }
  if (cs > 1) {
    cluster_sync();
  } else {
    __syncthreads();
  }
  // the cluster's blocks in order; each block finishes its share of the items
  constexpr int ITEMS = DEC_WARPS * NT * 32;
  for (int i = rank * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x); i < ITEMS && !abort_flag;
       i += cs * static_cast<int>(blockDim.x)) {
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int o = 0; o < cs; ++o) {
      const float4 w = cs > 1 ? ld_dsmem_f4(mapa_shared(smem_u32(&red[i]), o)) : red[i];
      v.x += w.x;
      v.y += w.y;
      v.z += w.z;
      v.w += w.w;
    }
    const int l = i & 31, t = (i >> 5) % NT, w = (i >> 5) / NT;
    const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = row0 + 16 * w + (l >> 2) + 8 * (j >> 1);
      const int tok = 8 * t + 2 * (l & 3) + (j & 1);
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
  if (cs > 1) cluster_sync();  // no block leaves while its sums may still be read
  if (threadIdx.x == 0 && abort_flag) atomicOr(p.status, ST_TIMEOUT);
}

// ------------------------------------------------------------------------------------------
// the mixture-of-experts products
// ------------------------------------------------------------------------------------------
constexpr int MOE_MAX_T = 128;      // "few tokens": the down product keeps a row of sums per token in shared memory
constexpr int MOE_MAX_E = 256;
constexpr int MOE_MAX_TOPK = 16;
constexpr float MOE_HIGH_UP = 268435456.0f, MOE_HIGH_DOWN = 1.0f / MOE_HIGH_UP;  // 2^28

// The routing of one call (workspace).  The (token, choice) pairs are listed by expert, ascending
// inside an expert; a segment is up to 8 NT consecutive pairs of one expert.  Its tiles of eight
// pairs follow those of the segments before it.
struct MoePlan {
  int* segments;   // [1]
  int* expert;     // [segments]
  int* begin;      // [segments] first list position
  int* count;      // [segments] pairs
  int* tile0;      // [segments] tiles of the segments before it
  int* high;       // [segments] 1: some h of the segment is past fp16 and lies in h_high
  int* tiles;      // [1] all tiles
  int* tile_seg;   // [tiles] segment of a tile
  int* pair;       // [T * top_k] pair (token * top_k + choice) at a list position
  float* weight;   // [T * top_k] its routing weight
};

struct MoeArgs {
  const uint8_t* x;  // fragment order: segment s at tile0[s] * (H / 128) * FRAG_BYTES, [chunk][tiles][FRAG_BYTES]
  const uint16_t* X;  // local activations: the caller's [T x H], and the experts' orders
  int64_t ldx;
  const int32_t* perm;
  MoePlan plan;
  int stages;      // of the ring
  int T, E, top_k, H, I;
  const float *gu_scales, *gu_zeros, *dn_scales, *dn_zeros;
  int gu_G, dn_G, gu_vec, dn_vec;
  GroupIndex gu_gi, dn_gi;
  int act, dn_unit;
  uint8_t* h;  // fragment order, as x with I / 128 chunks
  uint8_t* h_high;  // fp16: h 2^-28 of the values that are past fp16's largest, 0 for the others
  int splits;      // of the down product's list, beyond the cluster's
  float* partial;  // splits > 1: [splits][T][H]
  int* tickets;    // and a count per block of a split, zero before the call's down product
  const uint16_t* residual;
  int64_t ld_res, ldy;
  uint16_t* Y;
  int* status;
};

// h = act(x Wg^T) * (x Wu^T), rounded to the activations' type (the operand type of the second
// product).  In fp16 a value that would round to infinity (65520 and above: a gated product has such
// outliers, while Y, after the down weights, is small) goes into a second operand times 2^-28, which holds
// up to 1.7e13 with all its 11 bits; the down product takes that operand too for segments that have one.
// Grid (I / 64 * cluster, segments): a block's stage holds 64 gate rows and the same 64
// up rows; a warp takes eight of each as rows 0-7 and 8-15 of its MMA, so both halves of an h value
// end up in one lane.  Measured: 48 tokens, two of eight experts of 4096 x 11008, 139 us (2.6 TB/s);
// 33 tokens, 8 of 64 experts of 2048 x 768 with 3 bits, 57 us.  The stream alone takes 67 and 25 us,
// without the unpacking and the products 108 and 41: instruction issue and latency with 16 to 24 warps
// an SM, no single pipe (the fullest, the integer one, is busy for half of the time).
template <int BITS, bool BF, int GU, int NT, bool XL>
__global__ void __launch_bounds__(DEC_THREADS)
    moe_gate_up_kernel(const __grid_constant__ CUtensorMap codes_map, const MoeArgs p) {
  extern __shared__ uint8_t dec_smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * DEC_MAX_STAGES];
  __shared__ int abort_flag;
  __shared__ float4 red[DEC_WARPS * NT * 32];
  uint8_t* dec_smem = align128(dec_smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int cs = static_cast<int>(cluster_nctarank()), rank = static_cast<int>(cluster_ctarank());
  Ring<BITS, BF, GU, NT, XL> r;
  r.init(smem_u32(dec_smem), p.stages, bars, &abort_flag);
  griddep_wait();
  griddep_launch_dependents();
  const int seg = static_cast<int>(blockIdx.y);
  if (seg >= *p.plan.segments) return;  // (the whole cluster)
  const int e = p.plan.expert[seg], count = p.plan.count[seg], tile0 = p.plan.tile0[seg];
  const int i0 = static_cast<int>(blockIdx.x) / cs * 64;
  const int chunks = p.H / 128;
  Segment sg;
  sg.row_a = e * 2 * p.I + i0;
  sg.row_b = sg.row_a + p.I;
  sg.c0 = chunks * rank / cs;
  sg.c1 = chunks * (rank + 1) / cs;
  sg.tiles = (count + 7) / 8;
  sg.x = p.x + static_cast<size_t>(tile0) * chunks * FRAG_BYTES;
  if (warp == DEC_WARPS) {
    if (lane == 0) {
      int it = 0;
      for (; it < sg.c1 - sg.c0; ++it) {
        if (!r.codes(&codes_map, sg, sg.c0 + it, it)) break;
        r.acts(sg, sg.c0 + it, it);
      }
      r.drain(it);
    }
  } else {
    float acc[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[t][j] = 0.0f;
    const int ra = warp * 8 + g;
    r.param = ((q & 1) ? p.gu_zeros : p.gu_scales) + static_cast<size_t>(((q & 2) ? sg.row_b : sg.row_a) + ra) * p.gu_G;
    r.pitch = p.gu_G;
    r.vec = p.gu_vec;
    r.gi = p.gu_gi;
    if (XL)
      r.lay_out(reinterpret_cast<uint4*>(dec_smem + p.stages * dec_stage_bytes(BITS, 0)), sg.c0, sg.c1, count,
                p.perm ? p.perm + static_cast<size_t>(e) * p.H : nullptr,
                [&](int n) { return p.X + p.plan.pair[p.plan.begin[seg] + n] / p.top_k * p.ldx; });
    typename Ring<BITS, BF, GU, NT, XL>::Cursor cur;
    r.consume_tiles(sg.tiles, sg.c0, sg.c1, ra * (16 * BITS), (ra + 64) * (16 * BITS), lane, cur, acc);
#pragma unroll
    for (int t = 0; t < NT; ++t)
      red[(warp * NT + t) * 32 + lane] = make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
  }
  if (cs > 1) {
    cluster_sync();
  } else {
    __syncthreads();
  }
  constexpr int ITEMS = DEC_WARPS * NT * 32;
  const size_t h_at = static_cast<size_t>(tile0) * (p.I / 128) * FRAG_BYTES;
  uint16_t *h = reinterpret_cast<uint16_t*>(p.h + h_at), *h_high = reinterpret_cast<uint16_t*>(p.h_high + h_at);
  for (int i = rank * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x); i < ITEMS && !abort_flag;
       i += cs * static_cast<int>(blockDim.x)) {
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int o = 0; o < cs; ++o) {
      const float4 w = cs > 1 ? ld_dsmem_f4(mapa_shared(smem_u32(&red[i]), o)) : red[i];
      v.x += w.x;
      v.y += w.y;
      v.z += w.z;
      v.w += w.w;
    }
    const int l = i & 31, t = (i >> 5) % NT, w = (i >> 5) / NT;
    const int col = i0 + 8 * w + (l >> 2), n = 2 * (l & 3);
    if (t < sg.tiles) {
      const size_t at = (static_cast<size_t>(col >> 7) * sg.tiles + t) * (FRAG_BYTES / 2);
      const float hv[2] = {act_apply(v.x, p.act) * v.z, act_apply(v.y, p.act) * v.w};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const size_t o = at + frag_offset(p.dn_unit, n + j, col & 127);
        const bool high = !BF && fabsf(hv[j]) >= 65520.0f;
        h[o] = f2h<BF>(high ? 0.0f : hv[j]);
        if (!BF) {
          h_high[o] = f2h<BF>(high ? hv[j] * MOE_HIGH_DOWN : 0.0f);
          if (high) p.plan.high[seg] = 1;
        }
      }
    }
  }
  if (cs > 1) cluster_sync();
  if (threadIdx.x == 0 && abort_flag) atomicOr(p.status, ST_TIMEOUT);
}

// y = sum over the token's experts of weight * h Wd^T, + residual.  A block owns 128 output rows of
// every expert and, in a cluster, an even share of the list of (segment, chunk); each segment's
// sums are added, times the routing weight, into a row per token in shared memory (a warp owns its
// 16 columns of it); the shares meet over the cluster in a fixed order.  Where the row tiles and
// clusters of eight leave SMs idle, grid.y splits the list further: each split's block leaves its
// sums in `partial`, and the last of them to come adds all in their order, so the result does not
// depend on which it was (33 tokens over 64 experts: 41 us against 63 on the 64 SMs that 16 clusters of
// eight are packed on; clusters of 16 gained half as much).  88 us for the 48 tokens above.
template <int BITS, bool BF, int GU, int NT>
__global__ void __launch_bounds__(DEC_THREADS)
    moe_down_kernel(const __grid_constant__ CUtensorMap codes_map, const MoeArgs p) {
  extern __shared__ uint8_t dec_smem_raw[];  // ring, then float [T][DEC_ROWS]
  __shared__ __align__(8) uint64_t bars[2 * DEC_MAX_STAGES];
  __shared__ int abort_flag, last;
  uint8_t* dec_smem = align128(dec_smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int cs = static_cast<int>(cluster_nctarank()), rank = static_cast<int>(cluster_ctarank());
  const int row0 = static_cast<int>(blockIdx.x) / cs * DEC_ROWS;
  float* ysum = reinterpret_cast<float*>(dec_smem + p.stages * dec_stage_bytes(BITS, NT));
  for (int i = threadIdx.x; i < p.T * DEC_ROWS; i += DEC_THREADS) ysum[i] = 0.0f;
  Ring<BITS, BF, GU, NT, false> r;
  r.init(smem_u32(dec_smem), p.stages, bars, &abort_flag);
  griddep_wait();
  griddep_launch_dependents();
  const int chunks = p.I / 128;
  const int total = *p.plan.segments * chunks;
  const int share = static_cast<int>(blockIdx.y) * cs + rank, shares = p.splits * cs;
  const int w0 = static_cast<int>(static_cast<int64_t>(total) * share / shares);
  const int w1 = static_cast<int>(static_cast<int64_t>(total) * (share + 1) / shares);
  auto segment_at = [&](int w, int& seg) {
    Segment sg;
    seg = w / chunks;
    sg.c0 = w - seg * chunks;
    sg.c1 = min(chunks, sg.c0 + (w1 - w));
    sg.row_a = p.plan.expert[seg] * p.H + row0;
    sg.row_b = sg.row_a + 64;
    sg.tiles = (p.plan.count[seg] + 7) / 8;
    sg.x = p.h + static_cast<size_t>(p.plan.tile0[seg]) * chunks * FRAG_BYTES;
    return sg;
  };
  if (warp == DEC_WARPS) {
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int w = w0; w < w1 && ok;) {
        int seg;
        Segment sg = segment_at(w, seg);
        for (int high = BF ? 0 : p.plan.high[seg]; high >= 0 && ok; --high) {
          if (high) sg.x += p.h_high - p.h;
          for (int c = sg.c0; c < sg.c1; ++c, ++it) {
            if (!r.codes(&codes_map, sg, c, it)) {
              ok = false;
              break;
            }
            r.acts(sg, c, it);
          }
          if (high) sg.x -= p.h_high - p.h;
        }
        w += sg.c1 - sg.c0;
      }
      r.drain(it);
    }
  } else {
    typename Ring<BITS, BF, GU, NT, false>::Cursor cur;
    r.pitch = p.dn_G;
    r.vec = p.dn_vec;
    r.gi = p.dn_gi;
    const int ra = warp * 16 + g, rb = ra + 8;
    int high = -1;  // 1 while a segment's high operand comes, 0 for h itself, -1 before a segment
    for (int w = w0; w < w1;) {
      int seg;
      const Segment sg = segment_at(w, seg);
      if (high < 0) high = BF ? 0 : p.plan.high[seg];
      float acc[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[t][j] = 0.0f;
      r.param = ((q & 1) ? p.dn_zeros : p.dn_scales) + static_cast<size_t>(sg.row_a + ((q & 2) ? rb : ra)) * p.dn_G;
      if (!r.consume_tiles(sg.tiles, sg.c0, sg.c1, ra * (16 * BITS), rb * (16 * BITS), lane, cur, acc)) break;
      const int begin = p.plan.begin[seg], count = p.plan.count[seg];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int i = 8 * t + 2 * q + j;
          if (i < count) {
            const float wt = p.plan.weight[begin + i] * (high ? MOE_HIGH_UP : 1.0f);
            float* y = ysum + p.plan.pair[begin + i] / p.top_k * DEC_ROWS + ra;
            y[0] = fmaf(wt, acc[t][j], y[0]);
            y[8] = fmaf(wt, acc[t][2 + j], y[8]);
          }
        }
      __syncwarp();
      if (--high < 0) w += sg.c1 - sg.c0;
    }
  }
  if (cs > 1) {
    cluster_sync();
  } else {
    __syncthreads();
  }
  const int first = rank * DEC_THREADS + static_cast<int>(threadIdx.x), stride = cs * DEC_THREADS;
  auto finish = [&](int i, float v) {
    const int tok = i / DEC_ROWS, row = row0 + i % DEC_ROWS;
    if (p.residual) v += h2f<BF>(p.residual[static_cast<size_t>(tok) * p.ld_res + row]);
    p.Y[static_cast<size_t>(tok) * p.ldy + row] = f2h<BF>(v);
  };
  // (rows of `partial` hold T * H sums)
  auto at = [&](int split, int i) {
    return p.partial + (static_cast<size_t>(split) * p.T + i / DEC_ROWS) * p.H + row0 + i % DEC_ROWS;
  };
  for (int i = first; i < p.T * DEC_ROWS && !abort_flag; i += stride) {
    float v = 0.0f;
    for (int o = 0; o < cs; ++o) v += cs > 1 ? ld_dsmem_f(mapa_shared(smem_u32(&ysum[i]), o)) : ysum[i];
    if (p.splits == 1)
      finish(i, v);
    else
      __stcg(at(static_cast<int>(blockIdx.y), i), v);
  }
  if (p.splits > 1) {
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(p.tickets + blockIdx.x, 1) == p.splits - 1;
    __syncthreads();
    if (last) {
      __threadfence();
      for (int i = first; i < p.T * DEC_ROWS && !abort_flag; i += stride) {
        float v = 0.0f;
        for (int o = 0; o < p.splits; ++o) v += __ldcg(at(o, i));
        finish(i, v);
      }
    }
  }
  if (cs > 1) cluster_sync();
  if (threadIdx.x == 0 && abort_flag) atomicOr(p.status, ST_TIMEOUT);
}

// ------------------------------------------------------------------------------------------
// launches, one translation unit per code width (packed_decode_inst.cuh)
// ------------------------------------------------------------------------------------------
struct DecodeLaunch {
  bool bf16;
  int unit;      // 32, 64 or 128
  int nt;        // tiles a block holds sums for: 1, 2 or 4
  int local;     // tokens whose activations the blocks lay out themselves (nt = 1), 0: none
  int chunks;    // chunks of a block at most (local)
  int cluster;   // blocks that split k
  int ring;      // bytes of the ring at most
  int device;
  cudaStream_t stream;
};

template <int BITS>
cudaError_t launch_linear_decode(const DecodeLaunch& l, const CUtensorMap& codes, LinearDecodeArgs& a);
template <int BITS>
cudaError_t launch_moe_gate_up(const DecodeLaunch& l, const CUtensorMap& codes, MoeArgs& a, int segments);
template <int BITS>
cudaError_t launch_moe_down(const DecodeLaunch& l, const CUtensorMap& codes, MoeArgs& a);

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
