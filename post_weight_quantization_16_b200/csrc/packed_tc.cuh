// packed_tc.cuh — products of packed weights with 17 to 128 tokens on the sm_100a tensor cores
// (tcgen05), and with more where the CTA-pair kernel would leave SMs idle: the linear layer
// (BWD = false) and its gradient (BWD = true).
//
// Forward, one block = 128 weight rows (the MMA's M) x TN tokens (its N) over a range of k:
//     y[t][r] = sum over groups G of  s[r][G] * ( sum over k in G of (u[r][k] - z[r][G]) x[t][k] )
// The A operand is the exact integer u - z; a unit of min(group, 128) columns is accumulated in one
// of two tensor-memory buffers and drained into fp32 registers with one fused multiply-add by the
// row's scale.  So weights are never rounded to 16 bits, and no sum on the tensor cores is longer
// than 128 terms (their accumulation truncates; the registers' additions round to nearest).
//   warp 0        activations by TMA (128-byte swizzle)
//   warp 3        codes by TMA (no swizzle)
//   warp 1        tensor-memory allocation and MMA issue (one lane)
//   warps 4-19    unpack codes into the swizzled operand tile: four groups of four warps, each its half
//                 of every other chunk (two groups, each its half of every chunk, left the 500 tokens'
//                 gradient below at 43 us: a warp's chain of waits, loads and stores was the bound)
//   warps 20-27   drain: lane = weight row, each warp half of the tokens
// Operands move in steps of 64 along k through a ring deep enough to hide the hand-over between the
// unpack warps and the MMA (about 2700 cycles there and back).  Cost of a 128-column chunk at TN =
// 128: the MMAs take 512 cycles, unpacking about 320 of the integer pipes, the drain 128: all three
// overlap.  The blocks of a cluster split k when there are few tiles; their sums meet over
// distributed shared memory in a fixed order, in the epilogue that also adds the bias, applies the
// activation and adds the residual: one launch, deterministic.  77 tokens through 11008 x 4096 with 3
// bits take 38 us (the bytes and the products would take 4): 32 chunks of unpacking, hand-over and drain
// one behind the other in 86 blocks; 500 tokens' gradient through 4096 x 4096 39 us with its two other
// launches, 32 here.
//
// Gradient: dX[t][perm[k]] = scale_t * sum over rows r of W16[r][k] * dz[t][r],
//     W16 = fp16( fp32(u - z) * s * 2^e ) / 2^e,   dz[t][r] = dY[t][r] act'(Z[t][r]) / scale_t  in fp16
// The sum runs over the rows, across which the scale varies, so the weights enter as rounded to fp16's 11
// significant bits, and both operands are fp16 whatever the type of the activations: bf16 operands
// would lose three more bits of each.  e is one exponent per 128 columns, from their largest scale
// (packed_grad.cuh), and scale_t a power of two per token that puts the token's largest dz at 2^13 or
// above, so layers of any scale and the range of bf16 gradients fit; both are undone in fp32.
// With fp16 activations and a smooth act' the rounding of dz would be as large as that of dX
// itself: dz then comes as a sum of two fp16 values and the rows are gone through twice.  A block
// owns 128 columns of W: its operand is read transposed (MN-major) straight from the row-wise
// unpacked tile, and everything accumulates in one tensor-memory buffer.
#pragma once

#include "packed_decode.cuh"

namespace gptq {

constexpr int TC_BM = 128;                    // weight rows of a block
constexpr int TC_BK = 128;                    // columns of a chunk (two 64-column swizzle atoms)
constexpr int TC_THREADS = 28 * 32;
constexpr int TC_MAX_TN = 128;
constexpr int TC_STEP_A = 128 * 128;          // an unpacked step: 128 x 64 values
constexpr int TC_STEPS_MAX = 8;
// Register split (setmaxnreg): 128 * (40 + 4 * 56 + 2 * 120) = 64512, what 896 threads of 72 start with.
constexpr int TC_REGS_MISC = 40, TC_REGS_UNPACK = 56, TC_REGS_DRAIN = 120;
static_assert(TC_REGS_MISC + 4 * TC_REGS_UNPACK + 2 * TC_REGS_DRAIN <= 7 * 72, "register split");

__host__ __device__ constexpr int tc_code_bytes(int bits) { return TC_BM * TC_BK * bits / 8; }
__host__ __device__ constexpr int tc_code_chunks(int bits) { return bits == 8 ? 2 : 3; }  // in flight
__host__ __device__ constexpr int tc_steps(int tn) { return tn == 128 ? 6 : TC_STEPS_MAX; }  // in flight (even)
__host__ __device__ constexpr int tc_smem_bytes(int tn, int bits) {
  return 1024 + tc_steps(tn) * (TC_STEP_A + tn * 128) + tc_code_chunks(bits) * tc_code_bytes(bits) + 512;
}
static_assert(tc_smem_bytes(128, 8) <= 227 * 1024 && tc_smem_bytes(128, 4) <= 227 * 1024, "shared memory");

struct LinearTcArgs {
  int T, m, chunks, G, tn;
  GroupIndex gi;
  const float *scales, *zeros;
  const uint16_t *bias, *residual;
  int64_t ld_res, ldy;
  void* Y;
  uint16_t* preact;
  int act, y_fp32;
  int vec;  // 1: Y, residual and preact allow 4-element accesses at rows that are multiples of 4
  int* status;
};

// The 2 * BITS code words of half row h (64 columns) of tile row r, from a [128][16 * BITS bytes]
// tile.  16-byte loads start at a chunk rotated by the row, so that the lanes of a quarter warp
// touch distinct banks.
template <int BITS>
__device__ __forceinline__ void load_half_row(const uint8_t* tile, int r, int h, uint32_t (&w)[2 * BITS]) {
  const uint8_t* cw = tile + r * (16 * BITS) + h * (8 * BITS);
  if (BITS == 2) {
    const uint4 v = *reinterpret_cast<const uint4*>(cw);
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
  } else if (BITS == 3) {
#pragma unroll
    for (int j = 0; j < BITS; ++j) {
      const uint2 v = *reinterpret_cast<const uint2*>(cw + 8 * j);
      w[2 * j] = v.x;
      w[2 * j + 1] = v.y;
    }
  } else {
    constexpr int NCH = BITS / 2;
    const int rot = BITS == 4 ? ((r >> 1) & 1) : (r & 3);
    uint4 v[NCH];
#pragma unroll
    for (int j = 0; j < NCH; ++j) v[j] = *reinterpret_cast<const uint4*>(cw + 16 * ((j + rot) & (NCH - 1)));
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const uint4 x = rot == 0   ? v[c]
                      : rot == 1 ? v[(c + NCH - 1) & (NCH - 1)]
                      : rot == 2 ? v[(c + NCH - 2) & (NCH - 1)]
                                 : v[(c + NCH - 3) & (NCH - 1)];
      w[4 * c] = x.x;
      w[4 * c + 1] = x.y;
      w[4 * c + 2] = x.z;
      w[4 * c + 3] = x.w;
    }
  }
}

// Block c (eight codes) of a half row: codes in the low bits of v (8-bit: codes 4-7 in v1).
template <int BITS>
__device__ __forceinline__ void half_row_block(const uint32_t (&w)[2 * BITS], int c, uint32_t& v, uint32_t& v1) {
  v1 = 0;
  if (BITS == 8) {
    v = w[(2 * c) % (2 * BITS)];
    v1 = w[(2 * c + 1) % (2 * BITS)];
  } else if (BITS == 4) {
    v = w[c % (2 * BITS)];
  } else if (BITS == 2) {
    v = (c & 1) ? w[(c >> 1) % (2 * BITS)] >> 16 : w[(c >> 1) % (2 * BITS)];
  } else {
    const int bit = 24 * c, i = bit >> 5, sh = bit & 31;
    v = sh <= 8 ? w[i % (2 * BITS)] >> sh : __funnelshift_r(w[i % (2 * BITS)], w[(i + 1) % (2 * BITS)], sh);
  }
}

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// Four outputs (rows row .. row + 3 of token tok) of the epilogue.
template <bool BF>
__device__ __forceinline__ void linear_epilogue4(const LinearTcArgs& p, int tok, int row, float4 v) {
  float z[4] = {v.x, v.y, v.z, v.w};
  const int cnt = min(4, p.m - row);
  if (p.bias) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < cnt) z[j] += h2f<BF>(p.bias[row + j]);
  }
  const bool vec = p.vec && cnt == 4;
  if (p.preact) {
    uint16_t* d = p.preact + static_cast<size_t>(tok) * p.m + row;
    if (vec) {
      *reinterpret_cast<uint2*>(d) = make_uint2(pack2<BF>(z[0], z[1]), pack2<BF>(z[2], z[3]));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < cnt) d[j] = f2h<BF>(z[j]);
    }
  }
  if (p.act != ACT_NONE) {
#pragma unroll
    for (int j = 0; j < 4; ++j) z[j] = act_apply(z[j], p.act);
  }
  if (p.residual) {
    const uint16_t* s = p.residual + static_cast<size_t>(tok) * p.ld_res + row;
    if (vec) {
      const ushort4 r = *reinterpret_cast<const ushort4*>(s);
      z[0] += h2f<BF>(r.x);
      z[1] += h2f<BF>(r.y);
      z[2] += h2f<BF>(r.z);
      z[3] += h2f<BF>(r.w);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < cnt) z[j] += h2f<BF>(s[j]);
    }
  }
  if (p.y_fp32) {
    float* d = static_cast<float*>(p.Y) + static_cast<size_t>(tok) * p.ldy + row;
    if (vec) {
      *reinterpret_cast<float4*>(d) = make_float4(z[0], z[1], z[2], z[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < cnt) d[j] = z[j];
    }
  } else {
    uint16_t* d = static_cast<uint16_t*>(p.Y) + static_cast<size_t>(tok) * p.ldy + row;
    if (vec) {
      *reinterpret_cast<uint2*>(d) = make_uint2(pack2<BF>(z[0], z[1]), pack2<BF>(z[2], z[3]));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < cnt) d[j] = f2h<BF>(z[j]);
    }
  }
}

// Eight codes -> their fp16 weights, adjacent pairs in order.  f + nzm is u - z exactly (2^23 + u
// minus 2^23 + z), times s rounded to nearest in fp32, then to nearest fp16.
template <int BITS>
__device__ __forceinline__ void dequant8(uint32_t v, uint32_t v1, float2 nzm, float2 ss, uint32_t (&out)[4]) {
  uint32_t f[8];
  if (BITS == 4) {
    const uint32_t ev = v & 0x0F0F0F0Fu, od = (v >> 4) & 0x0F0F0F0Fu;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __byte_perm(ev, 0x4B000000u, 0x7540u + i);
      f[2 * i + 1] = __byte_perm(od, 0x4B000000u, 0x7540u + i);
    }
  } else if (BITS == 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __byte_perm(i < 4 ? v : v1, 0x4B000000u, 0x7540u + (i & 3));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = ((v >> (BITS * i)) & ((1u << BITS) - 1u)) | 0x4B000000u;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 d = __fmul2_rn(
        __fadd2_rn(make_float2(__uint_as_float(f[2 * i]), __uint_as_float(f[2 * i + 1])), nzm), ss);
    out[i] = pack2<false>(d.x, d.y);
  }
}

template <int REGS>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}
template <int REGS>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
}
// Position in a ring of n stages.
struct RingAt {
  int s = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next(int n) {
    if (++s == n) {
      s = 0;
      ph ^= 1u;
    }
  }
};

struct GradOut {
  const float2* token_scale;  // [T], powers of two as products of two, or null (1)
  const int* exponent;       // [n / 128][slabs]: the weights of these columns are multiplied by 2^(the least of them)
  int slabs;
  uint16_t* dX;              // [T x n], sweep order
  int64_t lddx;
  int n, vec;  // vec: dX allows 8-byte accesses
};

// The exponent of 128 columns is the least of the warp's lanes' parts.
__device__ __forceinline__ int exponent_part(const GradOut& go, int chunk, int lane) {
  int e = 126;
  if (lane < go.slabs) e = go.exponent[chunk * go.slabs + lane];
  for (int i = lane + 32; i < go.slabs; i += 32) e = min(e, go.exponent[chunk * go.slabs + i]);
  return e;
}
__device__ __forceinline__ int column_exponent(const GradOut& go, int chunk, int lane) {
  return __reduce_min_sync(0xffffffffu, exponent_part(go, chunk, lane));
}
// v times the token's scale over the weights' 2^e: both in two halves, as the two together may lie past the
// exponents of fp32 while the result does not.
struct Unscale {
  float a, b;
  __device__ __forceinline__ Unscale(float2 token_scale, float2 weights)
      : a(token_scale.x * weights.x), b(token_scale.y * weights.y) {}
  __device__ __forceinline__ float operator()(float v) const { return v * a * b; }
};

// Forward: lin holds everything, `chunks` are 128-column chunks of k.  Gradient: lin holds T, m, G,
// gi, scales, zeros, tn and status; `chunks` are 128-row chunks, gone through `parts` times (dz, then
// its low part).
template <int BITS, bool BF, int GU, bool BWD>
__global__ void __launch_bounds__(TC_THREADS, 1)
    packed_tc_kernel(const __grid_constant__ CUtensorMap codes_map, const __grid_constant__ CUtensorMap x_map,
                     const __grid_constant__ CUtensorMap xlo_map, const LinearTcArgs p, const GradOut go,
                     const int parts) {
  constexpr int UNITS = 128 / GU, SC = tc_code_chunks(BITS), CODES = tc_code_bytes(BITS);
  extern __shared__ uint8_t tc_smem_raw[];
  const uint32_t raw_s = smem_u32(tc_smem_raw);
  uint8_t* smem = tc_smem_raw + (((raw_s + 1023u) & ~1023u) - raw_s);
  const uint32_t sbase = smem_u32(smem);
  const int tn = p.tn, NS = tc_steps(tn), xb = tn * 128;
  const uint32_t a_base = sbase, x_base = a_base + NS * TC_STEP_A, c_base = x_base + NS * xb,
                 bar_full = c_base + SC * CODES, bar_empty = bar_full + 8 * TC_STEPS_MAX,
                 bar_cfull = bar_empty + 8 * TC_STEPS_MAX, bar_cempty = bar_cfull + 8 * SC, bar_tfull = bar_cempty + 8 * SC,
                 bar_tempty = bar_tfull + 16, bar_drain = bar_tempty + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + (bar_drain + 8 - sbase));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  // (a shuffled warp index is known to be uniform: operands of the MMAs stay in uniform registers)
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int cs = static_cast<int>(cluster_nctarank()), rank = static_cast<int>(cluster_ctarank());
  const int mt = static_cast<int>(blockIdx.x) / cs;  // tile of 128 rows of W, or of 128 columns (gradient)
  const int t0 = static_cast<int>(blockIdx.y) * tn;
  // this block's part of the reduction, in chunks; the gradient's second part follows the first
  const int ch0 = static_cast<int>(static_cast<int64_t>(p.chunks) * rank / cs);
  const int nch = static_cast<int>(static_cast<int64_t>(p.chunks) * (rank + 1) / cs) - ch0;
  const int nk = nch * parts;
  const uint32_t tmem_cols = static_cast<uint32_t>(2 * tn);

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(bar_full + 8 * s, 5);  // the activations and a group of unpack warps
      mbar_init(bar_empty + 8 * s, 1);
    }
    for (int s = 0; s < SC; ++s) {
      mbar_init(bar_cfull + 8 * s, 1);
      mbar_init(bar_cempty + 8 * s, 8);
    }
    for (int j = 0; j < 2; ++j) {
      mbar_init(bar_tfull + 8 * j, 1);
      mbar_init(bar_tempty + 8 * j, 8);
    }
    mbar_init(bar_drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), tmem_cols);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&codes_map);
    tma_prefetch_desc(&x_map);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  griddep_wait();
  griddep_launch_dependents();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) atomicExch(p.status, 0);

  if (warp < 4) {
    regs_dec<TC_REGS_MISC>();
    if (warp == 0 && lane == 0) {
      // ---------------- activations ----------------
      RingAt r;
      int issued = 0;
      for (int i = 0; i < 2 * nk; ++i) {
        if (!mbar_wait_bounded(bar_empty + 8 * r.s, r.ph ^ 1u, abort_flag)) break;
        const bool low = BWD && i >= 2 * nch;
        mbar_arrive_expect_tx(bar_full + 8 * r.s, static_cast<uint32_t>(xb));
        tma_load_2d(x_base + r.s * xb, low ? &xlo_map : &x_map, bar_full + 8 * r.s,
                    ch0 * 128 + (low ? i - 2 * nch : i) * 64, t0);
        r.next(NS);
        ++issued;
      }
      for (int i = max(0, issued - NS); i < issued; ++i)
        mbar_wait_drain(bar_full + 8 * (i % NS), static_cast<uint32_t>(i / NS) & 1u);
    } else if (warp == 3 && lane == 0) {
      // ---------------- codes ----------------
      RingAt r;
      int issued = 0;
      for (int i = 0; i < nk; ++i) {
        if (!mbar_wait_bounded(bar_cempty + 8 * r.s, r.ph ^ 1u, abort_flag)) break;
        const int c = ch0 + (BWD && i >= nch ? i - nch : i);
        mbar_arrive_expect_tx(bar_cfull + 8 * r.s, CODES);
        tma_load_2d(c_base + r.s * CODES, &codes_map, bar_cfull + 8 * r.s, (BWD ? mt : c) * (4 * BITS),
                    (BWD ? c : mt) * 128);
        r.next(SC);
        ++issued;
      }
      for (int i = max(0, issued - SC); i < issued; ++i)
        mbar_wait_drain(bar_cfull + 8 * (i % SC), static_cast<uint32_t>(i / SC) & 1u);
    } else if (warp == 1) {
      // ---------------- MMA: the whole warp runs the loop, one lane issues ----------------
      const bool issue = elect_one_sync();
      const uint32_t fmt = (BF && !BWD) ? 1u : 0u;
      const uint32_t idesc = idesc_make(fmt, fmt, BWD ? 1u : 0u, 0u, TC_BM, static_cast<uint32_t>(tn));
      // forward: K-major; gradient: MN-major, 16 rows = two 8-row atoms, 64-column halves 8 KB apart
      const uint64_t ad0 = BWD ? sdesc_sw128(a_base, TC_STEP_A / 2, 1024) : sdesc_sw128(a_base, 16, 1024);
      const uint64_t bd0 = sdesc_sw128(x_base, 16, 1024);
      constexpr uint32_t A_SLICE = (BWD ? 2048 : 32) >> 4, B_SLICE = 32 >> 4;
      constexpr int SUB = (!BWD && GU == 32) ? 2 : 1;  // accumulation units of a step
      RingAt x, t;
      bool ok = true;
      for (int i = 0; i < nk && ok; ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!warp_wait_uniform(bar_full + 8 * x.s, x.ph, abort_flag)) {
            ok = false;
            break;
          }
          const uint64_t ad = ad0 + static_cast<uint32_t>(x.s * (TC_STEP_A >> 4)),
                         bd = bd0 + static_cast<uint32_t>(x.s * (xb >> 4));
#pragma unroll
          for (int u = 0; u < SUB; ++u) {
            const bool first = BWD ? (h == 0 && i == 0) : (GU < 128 || h == 0);
            const bool last = BWD ? (h == 1 && i == nk - 1) : (GU < 128 || h == 1);
            if (first && !warp_wait_uniform(bar_tempty + 8 * t.s, t.ph ^ 1u, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t d = tmem_base + static_cast<uint32_t>(t.s * tn);
#pragma unroll
            for (int k = 0; k < 4 / SUB; ++k) {
              const uint32_t kk = u * (4 / SUB) + k;
              if (issue) umma_f16(d, ad + kk * A_SLICE, bd + kk * B_SLICE, idesc, (first && k == 0) ? 0u : 1u);
            }
            if (u == SUB - 1 && issue) umma_commit(bar_empty + 8 * x.s);
            if (last) {
              if (issue) umma_commit(bar_tfull + 8 * t.s);
              t.next(2);
            }
          }
          if (!ok) break;
          x.next(NS);
        }
      }
      if (!ok) {  // MMAs may still be running: wait for them before tensor memory is released
        if (issue) umma_commit(bar_drain);
        mbar_wait_drain(bar_drain, 0);
      }
    }
  } else if (warp < 20) {
    // ---------------- unpack ----------------
    // Forward: grp 0 takes columns 0-63 of a chunk, 1 columns 64-127, a thread one row.  Gradient: grp 0
    // takes rows 0-63, 1 rows 64-127, two threads per row.  par: the even or the odd chunks.
    regs_dec<TC_REGS_UNPACK>();
    const int d = threadIdx.x & 127, grp = ((warp - 4) >> 2) & 1, par = (warp - 4) >> 3;
    const int r = BWD ? grp * 64 + (d >> 1) : d, h = BWD ? d & 1 : grp, r7 = r & 7;
    const uint32_t dst0 = a_base + (BWD ? h * (TC_STEP_A / 2) + (r & 63) * 128 : r * 128);
    constexpr int ZN = GU == 32 ? 2 : 1;  // groups of a half row
    float ns[ZN], nz[ZN];
    const int part = BWD ? exponent_part(go, mt, lane) : 0;
    auto load_sz = [&](int i) {
      const int c = ch0 + (BWD && i >= nch ? i - nch : i);
      const int gr = (BWD ? c : mt) * 128 + r;
      const bool in = gr < p.m;
      const size_t row = static_cast<size_t>(min(gr, p.m - 1)) * p.G;
#pragma unroll
      for (int j = 0; j < ZN; ++j) {
        const size_t at = row + group_of<GU>(p.gi, BWD ? mt : c, GU == 128 ? 0 : GU == 64 ? h : 2 * h + j);
        nz[j] = in ? __ldg(p.zeros + at) : 0.0f;
        if (BWD) ns[j] = in ? __ldg(p.scales + at) : 0.0f;  // rows past m: zero weights
      }
    };
    RingAt c;
    c.s = par;
    int as = 2 * par + grp;  // slot of this group's next step
    uint32_t aph = 0;
    // The words of the next chunk are taken before this chunk's stores are fenced, so that the stores
    // complete meanwhile.
    uint32_t w[2 * BITS];
    auto take = [&]() {
      if (!warp_wait_uniform(bar_cfull + 8 * c.s, c.ph, abort_flag)) return false;
      load_half_row<BITS>(smem + (c_base - sbase) + c.s * CODES, r, h, w);
      return true;
    };
    bool ok = nk > par;
    if (ok) {
      load_sz(par);
      ok = take();
    }
    const float up = BWD ? pow2(__reduce_min_sync(0xffffffffu, part)) : 1.0f;  // (its load waited for beside theirs)
    for (int i = par; i < nk && ok; i += 2) {
      float cs_[ZN], cz[ZN];
#pragma unroll
      for (int j = 0; j < ZN; ++j) {
        cz[j] = nz[j];
        cs_[j] = BWD ? ns[j] * up : 0.0f;
      }
      if (i + 2 < nk) load_sz(i + 2);
      if (!warp_wait_uniform(bar_empty + 8 * as, aph ^ 1u, abort_flag)) break;
      const uint32_t dst = dst0 + as * TC_STEP_A;
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        const int j = GU == 32 ? b >> 2 : 0;
        uint32_t v, v1, q[4];
        half_row_block<BITS>(w, b, v, v1);
        if (BWD) {
          dequant8<BITS>(v, v1, make_float2(-8388608.0f - cz[j], -8388608.0f - cz[j]), make_float2(cs_[j], cs_[j]), q);
          st_shared_v4(dst + ((b ^ r7) << 4), q[0], q[1], q[2], q[3]);
        } else {
          unpack8<BITS, BF>(v, v1, zero_term<BITS, BF>(cz[j]), q);
          // pairs (i, i + 4) -> columns in order
          st_shared_v4(dst + ((b ^ r7) << 4), __byte_perm(q[0], q[1], 0x5410), __byte_perm(q[2], q[3], 0x5410),
                       __byte_perm(q[0], q[1], 0x7632), __byte_perm(q[2], q[3], 0x7632));
        }
      }
      // (this chunk's words were used above, so its stage can go back)
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_cempty + 8 * c.s);
      c.next(SC);
      c.next(SC);
      if (i + 2 < nk) ok = take();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_full + 8 * as);
      as += 4;
      if (as >= NS) {
        as -= NS;
        aph ^= 1u;
      }
    }
  } else {
    // ---------------- drain ----------------
    regs_inc<TC_REGS_DRAIN>();
    const int qd = warp & 3, half = (warp - 20) >> 2;
    const int row = qd * 32 + lane, cols = tn / 2;  // tokens of this warp: 16, 32 or 64
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(qd * 32) << 16) + static_cast<uint32_t>(half * cols);
    float acc[64];
#pragma unroll
    for (int j = 0; j < 64; ++j) acc[j] = 0.0f;
    bool ok = true;
    RingAt t;
    const int units = BWD ? (nk > 0 ? 1 : 0) : nk * UNITS;
    const float* srow = p.scales + static_cast<size_t>(BWD ? 0 : min(mt * TC_BM + row, p.m - 1)) * p.G;
    float ns = !BWD && units > 0 ? __ldg(srow + group_of<GU>(p.gi, ch0, 0)) : 1.0f;
    for (int uc = 0; uc < units; ++uc) {
      const float sc = ns;
      if (!BWD && uc + 1 < units) ns = __ldg(srow + group_of<GU>(p.gi, ch0 + (uc + 1) / UNITS, (uc + 1) % UNITS));
      if (!warp_wait_uniform(bar_tfull + 8 * t.s, t.ph, abort_flag)) {
        ok = false;
        break;
      }
      tc_fence_after();
      // (two loads, then one wait: a load takes some 200 cycles while the MMAs run; four need registers)
#pragma unroll
      for (int c2 = 0; c2 < 4; c2 += 2) {
        uint32_t v[2][16];
#pragma unroll
        for (int cc = 0; cc < 2; ++cc)
          if ((c2 + cc) * 16 < cols) tmem_ld_32x32b_x16(lane_base + static_cast<uint32_t>(t.s * tn + (c2 + cc) * 16), v[cc]);
        tmem_ld_wait();
#pragma unroll
        for (int cc = 0; cc < 2; ++cc)
          if ((c2 + cc) * 16 < cols) {
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[(c2 + cc) * 16 + j] = fmaf(sc, __uint_as_float(v[cc][j]), acc[(c2 + cc) * 16 + j]);
          }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_tempty + 8 * t.s);
      t.next(2);
    }
    // sums as [token][row] over the operand ring (every MMA that read it has completed)
    if (ok) {
      float* sums = reinterpret_cast<float*>(smem);
#pragma unroll
      for (int j = 0; j < 64; ++j)
        if (j < cols) sums[(half * cols + j) * TC_BM + row] = acc[j];
    }
  }

  __syncthreads();
  if (cs > 1) cluster_sync();
  // tokens rank, rank + cs, ... of the tile: a warp takes a token, a lane four rows (columns of dX)
  if (!*abort_flag) {
    const float2 back = pow2_halves(BWD ? -column_exponent(go, mt, lane) : 0);
    for (int t = rank + cs * warp; t < tn; t += cs * (TC_THREADS / 32)) {
      const int tok = t0 + t, row = mt * TC_BM + 4 * lane;
      if (tok >= p.T || (!BWD && row >= p.m)) continue;
      const uint32_t at = sbase + static_cast<uint32_t>((t * TC_BM + 4 * lane) * 4);
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int o = 0; o < cs; ++o) {
        const float4 w = cs > 1 ? ld_dsmem_f4(mapa_shared(at, o)) : *reinterpret_cast<const float4*>(smem + (at - sbase));
        v.x += w.x;
        v.y += w.y;
        v.z += w.z;
        v.w += w.w;
      }
      if (BWD) {
        const Unscale s(go.token_scale ? go.token_scale[tok] : make_float2(1.0f, 1.0f), back);
        uint16_t* o = go.dX + static_cast<size_t>(tok) * go.lddx + row;
        const uint32_t lo = pack2<BF>(s(v.x), s(v.y)), hi = pack2<BF>(s(v.z), s(v.w));
        if (go.vec) {
          *reinterpret_cast<uint2*>(o) = make_uint2(lo, hi);
        } else {
          o[0] = static_cast<uint16_t>(lo);
          o[1] = static_cast<uint16_t>(lo >> 16);
          o[2] = static_cast<uint16_t>(hi);
          o[3] = static_cast<uint16_t>(hi >> 16);
        }
      } else {
        linear_epilogue4<BF>(p, tok, row, v);
      }
    }
  }
  if (cs > 1) cluster_sync();  // no block leaves while its sums may still be read
  if (threadIdx.x == 0 && *abort_flag) atomicOr(p.status, ST_TIMEOUT);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, tmem_cols);
  }
}

// ------------------------------------------------------------------------------------------
// launches, one translation unit per code width (packed_tc_inst.cuh)
// ------------------------------------------------------------------------------------------
struct TcLaunch {
  bool bf16;
  int unit;     // 32, 64 or 128
  int sms;
  int cluster;  // blocks that split k
  int device;
  cudaStream_t stream;
};

template <int BITS>
cudaError_t launch_packed_tc(const TcLaunch& l, bool backward, const CUtensorMap& codes, const CUtensorMap& x,
                             const CUtensorMap& xlo, const LinearTcArgs& a, const GradOut& go, int parts);

}  // namespace gptq
