// packed_tc.cuh — products of packed weights with many tokens on the sm_100a tensor cores
// (tcgen05): the linear layer (linear_tc_kernel) and its gradient (linear_bwd_tc_kernel).
//
// Forward, one block = 128 weight rows (the MMA's M) x TN tokens (its N) over a range of k:
//     y[t][r] = sum over groups G of  s[r][G] * ( sum over k in G of (u[r][k] - z[r][G]) x[t][k] )
// The A operand is the exact integer u - z; a unit of min(group, 128) columns is accumulated in one
// of two tensor-memory buffers and drained into fp32 registers with one fused multiply-add by the
// row's scale.  So weights are never rounded to 16 bits, and no sum on the tensor cores is longer
// than 128 terms (their accumulation truncates; the registers' additions round to nearest).
//   warp 0       TMA producer (one lane): packed codes (no swizzle) and activations (128-byte swizzle)
//   warp 1       tensor-memory allocation and MMA issue (one lane)
//   warps 2-9    unpack codes into the swizzled K-major operand tile (two threads per row)
//   warps 10-17  drain: lane = weight row, each warp half of the tokens
// Cost of a 128-column chunk at TN = 128: the MMAs take 512 cycles; unpacking issues about 16384 x 2
// / 128 = 256 cycles of the four schedulers, the drain 128 and its tensor-memory loads: all
// three overlap.  The blocks of a cluster split k when there are few tiles; their sums meet over
// distributed shared memory in a fixed order, in the epilogue that also adds the bias, applies the
// activation and adds the residual: one launch, no workspace, deterministic.
#pragma once

#include "packed_decode.cuh"

namespace gptq {

constexpr int TC_BM = 128;                    // weight rows of a block
constexpr int TC_BK = 128;                    // columns of a chunk (two 64-column swizzle atoms)
constexpr int TC_ATOM = TC_BM * 128;          // 16 KB: 128 rows x 64 sixteen-bit values
constexpr int TC_A_BYTES = 2 * TC_ATOM;
constexpr int TC_NA = 2;                      // unpacked tiles in flight
constexpr int TC_THREADS = 18 * 32;
constexpr int TC_SMEM_BUDGET = 224 * 1024;
constexpr int TC_MAX_TN = 128;

__host__ __device__ constexpr int tc_code_bytes(int bits) { return TC_BM * TC_BK * bits / 8; }
__host__ __device__ inline int tc_stage_bytes(int tn, int bits) { return tc_code_bytes(bits) + tn * 256; }
__host__ __device__ inline int tc_stages(int tn, int bits) {
  const int s = (TC_SMEM_BUDGET - 2048 - TC_NA * TC_A_BYTES) / tc_stage_bytes(tn, bits);
  return s > 8 ? 8 : s;
}
__host__ __device__ inline int tc_smem_bytes(int tn, int bits) {
  return 2048 + TC_NA * TC_A_BYTES + tc_stages(tn, bits) * tc_stage_bytes(tn, bits);
}

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

template <int BITS, bool BF, int GU>
__global__ void __launch_bounds__(TC_THREADS, 1)
    linear_tc_kernel(const __grid_constant__ CUtensorMap codes_map, const __grid_constant__ CUtensorMap x_map,
                     const LinearTcArgs p) {
  constexpr int UNITS = 128 / GU;
  extern __shared__ uint8_t tc_smem_raw[];
  const uint32_t raw_s = smem_u32(tc_smem_raw);
  uint8_t* smem = tc_smem_raw + (((raw_s + 1023u) & ~1023u) - raw_s);
  const uint32_t sbase = smem_u32(smem);
  const int tn = p.tn;
  const int stages = tc_stages(tn, BITS);
  const int stage_bytes = tc_stage_bytes(tn, BITS);
  const uint32_t a_base = sbase;
  const uint32_t st_base = sbase + TC_NA * TC_A_BYTES;  // stages: X atom 0 | X atom 1 | codes
  const uint32_t bar = st_base + stages * stage_bytes;
  const uint32_t bar_full = bar, bar_empty = bar + 64, bar_afull = bar + 128, bar_aempty = bar_afull + 8 * TC_NA,
                 bar_tfull = bar_aempty + 8 * TC_NA, bar_tempty = bar_tfull + 16, bar_drain = bar_tempty + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + (bar_drain + 8 - sbase));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cs = static_cast<int>(cluster_nctarank()), rank = static_cast<int>(cluster_ctarank());
  const int m0 = static_cast<int>(blockIdx.x) / cs * TC_BM;
  const int t0 = static_cast<int>(blockIdx.y) * tn;
  const int kt0 = p.chunks * rank / cs, nk = p.chunks * (rank + 1) / cs - kt0;
  const uint32_t tmem_cols = static_cast<uint32_t>(2 * tn);

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(bar_full + 8 * s, 1);
      mbar_init(bar_empty + 8 * s, 1);
    }
    for (int j = 0; j < TC_NA; ++j) {
      mbar_init(bar_afull + 8 * j, 8);
      mbar_init(bar_aempty + 8 * j, 1);
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

  if (warp == 0) {
    if (lane == 0) {
      const uint32_t tx = static_cast<uint32_t>(stage_bytes);
      int issued = 0;
      for (int i = 0; i < nk; ++i) {
        const int s = i % stages;
        if (!mbar_wait_bounded(bar_empty + 8 * s, (static_cast<uint32_t>(i / stages) & 1u) ^ 1u, abort_flag)) break;
        const uint32_t fb = bar_full + 8 * s, st = st_base + s * stage_bytes;
        mbar_arrive_expect_tx(fb, tx);
        const int kt = kt0 + i;
        tma_load_2d(st + tn * 256, &codes_map, fb, kt * (TC_BK * BITS / 32), m0);
        tma_load_2d(st, &x_map, fb, kt * TC_BK, t0);
        tma_load_2d(st + tn * 128, &x_map, fb, kt * TC_BK + 64, t0);
        issued = i + 1;
      }
      for (int i = max(0, issued - stages); i < issued; ++i)
        mbar_wait_drain(bar_full + 8 * (i % stages), static_cast<uint32_t>(i / stages) & 1u);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = idesc_make(BF ? 1u : 0u, BF ? 1u : 0u, 0u, 0u, TC_BM, static_cast<uint32_t>(tn));
      bool ok = true;
      for (int i = 0; i < nk && ok; ++i) {
        const int s = i % stages, j = i % TC_NA;
        if (!mbar_wait_bounded(bar_full + 8 * s, static_cast<uint32_t>(i / stages) & 1u, abort_flag) ||
            !mbar_wait_bounded(bar_afull + 8 * j, static_cast<uint32_t>(i / TC_NA) & 1u, abort_flag)) {
          ok = false;
          break;
        }
        const uint32_t a_t = a_base + j * TC_A_BYTES, x_t = st_base + s * stage_bytes;
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
          const int uc = i * UNITS + u, b = uc & 1;
          if (!mbar_wait_bounded(bar_tempty + 8 * b, (static_cast<uint32_t>(uc >> 1) & 1u) ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < GU / 16; ++k) {
            const int kk = u * (GU / 16) + k;  // 16-column step of the chunk: atom kk / 4
            const uint64_t ad = sdesc_sw128(a_t + (kk >> 2) * TC_ATOM + (kk & 3) * 32, 16, 1024);
            const uint64_t bd = sdesc_sw128(x_t + (kk >> 2) * (tn * 128) + (kk & 3) * 32, 16, 1024);
            umma_f16(tmem_base + static_cast<uint32_t>(b * tn), ad, bd, idesc, k > 0 ? 1u : 0u);
          }
          umma_commit(bar_tfull + 8 * b);
        }
        if (!ok) break;
        umma_commit(bar_empty + 8 * s);
        umma_commit(bar_aempty + 8 * j);
      }
      if (!ok) {  // MMAs may still be running: wait for them before tensor memory is released
        umma_commit(bar_drain);
        mbar_wait_drain(bar_drain, 0);
      }
    }
  } else if (warp < 10) {
    // ---------------- unpack: two threads per row ----------------
    const int d = threadIdx.x - 64, r = d >> 1, h = d & 1, r7 = r & 7;
    const int gr = m0 + r;
    constexpr int ZN = GU == 32 ? 2 : 1;  // zero-points of a half row
    const float* zrow = p.zeros + static_cast<size_t>(min(gr, p.m - 1)) * p.G;
    auto load_z = [&](int kt, float (&z)[ZN]) {
#pragma unroll
      for (int j = 0; j < ZN; ++j)
        z[j] = gr < p.m ? __ldg(zrow + group_of<GU>(p.gi, kt, GU == 128 ? 0 : GU == 64 ? h : 2 * h + j)) : 0.0f;
    };
    float nz[ZN];
    load_z(kt0, nz);
    for (int i = 0; i < nk; ++i) {
      ZeroTerm zt[ZN];
#pragma unroll
      for (int j = 0; j < ZN; ++j) zt[j] = zero_term<BITS, BF>(nz[j]);
      if (i + 1 < nk) load_z(kt0 + i + 1, nz);
      const int s = i % stages, j = i % TC_NA;
      if (!warp_wait(bar_full + 8 * s, static_cast<uint32_t>(i / stages) & 1u, abort_flag, lane) ||
          !warp_wait(bar_aempty + 8 * j, (static_cast<uint32_t>(i / TC_NA) & 1u) ^ 1u, abort_flag, lane))
        break;
      uint32_t w[2 * BITS];
      load_half_row<BITS>(smem + (st_base - sbase) + s * stage_bytes + tn * 256, r, h, w);
      const uint32_t dst = a_base + j * TC_A_BYTES + h * TC_ATOM + r * 128;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        uint32_t v, v1, q[4];
        half_row_block<BITS>(w, c, v, v1);
        unpack8<BITS, BF>(v, v1, zt[GU == 32 ? c >> 2 : 0], q);
        // pairs (i, i + 4) -> columns in order
        st_shared_v4(dst + ((c ^ r7) << 4), __byte_perm(q[0], q[1], 0x5410), __byte_perm(q[2], q[3], 0x5410),
                     __byte_perm(q[0], q[1], 0x7632), __byte_perm(q[2], q[3], 0x7632));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_afull + 8 * j);
    }
  } else {
    // ---------------- drain ----------------
    const int qd = warp & 3, half = (warp - 10) >> 2;
    const int row = qd * 32 + lane, gr = m0 + row;
    const int cols = tn / 2;  // tokens of this warp: 16, 32 or 64
    const float* srow = p.scales + static_cast<size_t>(min(gr, p.m - 1)) * p.G;
    float acc[64];
#pragma unroll
    for (int j = 0; j < 64; ++j) acc[j] = 0.0f;
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(qd * 32) << 16) + static_cast<uint32_t>(half * cols);
    float ns = nk > 0 ? __ldg(srow + group_of<GU>(p.gi, kt0, 0)) : 0.0f;
    bool ok = true;
    for (int uc = 0; uc < nk * UNITS; ++uc) {
      const float sc = ns;
      if (uc + 1 < nk * UNITS) ns = __ldg(srow + group_of<GU>(p.gi, kt0 + (uc + 1) / UNITS, (uc + 1) % UNITS));
      const int b = uc & 1;
      if (!warp_wait(bar_tfull + 8 * b, static_cast<uint32_t>(uc >> 1) & 1u, abort_flag, lane)) {
        ok = false;
        break;
      }
      tc_fence_after();
#pragma unroll
      for (int cc = 0; cc < 4; ++cc) {
        if (cc * 16 < cols) {
          uint32_t v[16];
          tmem_ld_32x32b_x16(lane_base + static_cast<uint32_t>(b * tn + cc * 16), v);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) acc[cc * 16 + j] = fmaf(sc, __uint_as_float(v[j]), acc[cc * 16 + j]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_tempty + 8 * b);
    }
    // sums as [token][row] over the operand tiles (every MMA that read them has completed)
    if (ok) {
      float* sums = reinterpret_cast<float*>(smem);
#pragma unroll
      for (int j = 0; j < 64; ++j)
        if (j < cols) sums[(half * cols + j) * TC_BM + row] = acc[j];
    }
  }

  __syncthreads();
  if (cs > 1) cluster_sync();
  // tokens rank, rank + cs, ... of the tile: a warp takes a token, a lane four rows
  if (!*abort_flag) {
    for (int t = rank + cs * warp; t < tn; t += cs * (TC_THREADS / 32)) {
      if (t0 + t >= p.T || m0 + 4 * lane >= p.m) continue;
      const uint32_t at = sbase + static_cast<uint32_t>((t * TC_BM + 4 * lane) * 4);
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int o = 0; o < cs; ++o) {
        const float4 w = cs > 1 ? ld_dsmem_f4(mapa_shared(at, o)) : *reinterpret_cast<const float4*>(smem + (at - sbase));
        v.x += w.x;
        v.y += w.y;
        v.z += w.z;
        v.w += w.w;
      }
      linear_epilogue4<BF>(p, t0 + t, m0 + 4 * lane, v);
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
// the gradient
// ------------------------------------------------------------------------------------------
//     dX[t][perm[k]] = scale_t * sum over rows r of W16[r][k] * dz[t][r],
//     W16 = fp16( fp32(u - z) * s ),   dz[t][r] = dY[t][r] act'(Z[t][r]) / scale_t  in fp16
// The sum runs over the rows, across which the scale varies, so the weights enter as their fp16
// values (the library's dequantized weight) and both operands are fp16 whatever the type of the
// activations: bf16 operands would lose three more bits of each.  scale_t is a power of two per
// token that puts the token's largest dY at 2^13 or above, so the range of bf16 gradients fits.
// With fp16 activations and a smooth act' the rounding of dz would be as large as that of dX
// itself: dz then comes as a sum of two fp16 values (parts = 2) and each chunk takes two MMAs.
//
// One block = 128 columns of W (the MMA's M; the operand is read transposed, MN-major, straight
// from the row-wise unpacked tile) x TN tokens, over a range of rows in chunks of 128.  Everything
// accumulates in one tensor-memory buffer.  Roles as in the forward kernel, without a drain loop.
constexpr int BW_THREADS = 10 * 32;
constexpr int BW_MAX_TN = 256;

__host__ __device__ inline int bw_stage_bytes(int tn, int bits, int parts) {
  return tc_code_bytes(bits) + parts * tn * 256;
}
__host__ __device__ inline int bw_stages(int tn, int bits, int parts) {
  const int s = (TC_SMEM_BUDGET - 2048 - TC_NA * TC_A_BYTES) / bw_stage_bytes(tn, bits, parts);
  return s > 8 ? 8 : s;
}
__host__ __device__ inline int bw_smem_bytes(int tn, int bits, int parts) {
  return 2048 + TC_NA * TC_A_BYTES + bw_stages(tn, bits, parts) * bw_stage_bytes(tn, bits, parts);
}

struct LinearBwdArgs {
  int T, m, n, G, tn, parts;
  int row_chunks;  // ceil(m / 128)
  GroupIndex gi;
  const float *scales, *zeros;
  const float* token_scale;  // [T] or null (1)
  uint16_t* dX;              // [T x n], sweep order
  int64_t lddx;
  int bf16_out;
  int vec;  // dX allows 8-byte accesses
  int* status;
};

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

template <int BITS, int GU>
__global__ void __launch_bounds__(BW_THREADS, 1)
    linear_bwd_tc_kernel(const __grid_constant__ CUtensorMap codes_map, const __grid_constant__ CUtensorMap dz_map,
                         const __grid_constant__ CUtensorMap dzlo_map, const LinearBwdArgs p) {
  extern __shared__ uint8_t tc_smem_raw[];
  const uint32_t raw_s = smem_u32(tc_smem_raw);
  uint8_t* smem = tc_smem_raw + (((raw_s + 1023u) & ~1023u) - raw_s);
  const uint32_t sbase = smem_u32(smem);
  const int tn = p.tn, parts = p.parts;
  const int stages = bw_stages(tn, BITS, parts);
  const int stage_bytes = bw_stage_bytes(tn, BITS, parts);
  const uint32_t a_base = sbase;
  const uint32_t st_base = sbase + TC_NA * TC_A_BYTES;  // stages: dz atoms | (low part's atoms) | codes
  const int code_off = parts * tn * 256;
  const uint32_t bar = st_base + stages * stage_bytes;
  const uint32_t bar_full = bar, bar_empty = bar + 64, bar_afull = bar + 128, bar_aempty = bar_afull + 8 * TC_NA,
                 bar_acc = bar_aempty + 8 * TC_NA, bar_drain = bar_acc + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + (bar_drain + 8 - sbase));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cs = static_cast<int>(cluster_nctarank()), rank = static_cast<int>(cluster_ctarank());
  const int kc = static_cast<int>(blockIdx.x) / cs;  // chunk of 128 columns
  const int t0 = static_cast<int>(blockIdx.y) * tn;
  const int rc0 = static_cast<int>(static_cast<int64_t>(p.row_chunks) * rank / cs);
  const int nk = static_cast<int>(static_cast<int64_t>(p.row_chunks) * (rank + 1) / cs) - rc0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(bar_full + 8 * s, 1);
      mbar_init(bar_empty + 8 * s, 1);
    }
    for (int j = 0; j < TC_NA; ++j) {
      mbar_init(bar_afull + 8 * j, 8);
      mbar_init(bar_aempty + 8 * j, 1);
    }
    mbar_init(bar_acc, 1);
    mbar_init(bar_drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), static_cast<uint32_t>(tn));
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&codes_map);
    tma_prefetch_desc(&dz_map);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  griddep_wait();
  griddep_launch_dependents();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) atomicExch(p.status, 0);

  if (warp == 0) {
    if (lane == 0) {
      int issued = 0;
      for (int i = 0; i < nk; ++i) {
        const int s = i % stages;
        if (!mbar_wait_bounded(bar_empty + 8 * s, (static_cast<uint32_t>(i / stages) & 1u) ^ 1u, abort_flag)) break;
        const uint32_t fb = bar_full + 8 * s, st = st_base + s * stage_bytes;
        mbar_arrive_expect_tx(fb, static_cast<uint32_t>(stage_bytes));
        const int r0 = (rc0 + i) * 128;
        tma_load_2d(st + code_off, &codes_map, fb, kc * (TC_BK * BITS / 32), r0);
        tma_load_2d(st, &dz_map, fb, r0, t0);
        tma_load_2d(st + tn * 128, &dz_map, fb, r0 + 64, t0);
        if (parts == 2) {
          tma_load_2d(st + tn * 256, &dzlo_map, fb, r0, t0);
          tma_load_2d(st + tn * 384, &dzlo_map, fb, r0 + 64, t0);
        }
        issued = i + 1;
      }
      for (int i = max(0, issued - stages); i < issued; ++i)
        mbar_wait_drain(bar_full + 8 * (i % stages), static_cast<uint32_t>(i / stages) & 1u);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = idesc_make(0u, 0u, 1u, 0u, TC_BM, static_cast<uint32_t>(tn));  // f16; A is MN-major
      bool ok = true;
      for (int i = 0; i < nk; ++i) {
        const int s = i % stages, j = i % TC_NA;
        if (!mbar_wait_bounded(bar_full + 8 * s, static_cast<uint32_t>(i / stages) & 1u, abort_flag) ||
            !mbar_wait_bounded(bar_afull + 8 * j, static_cast<uint32_t>(i / TC_NA) & 1u, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t a_t = a_base + j * TC_A_BYTES, x_t = st_base + s * stage_bytes;
        for (int part = 0; part < parts; ++part) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            // 16 rows = two 8-row swizzle atoms of 1024 bytes; the 64-column halves 16 KB apart
            const uint64_t ad = sdesc_sw128(a_t + kk * 2048, TC_ATOM, 1024);
            const uint64_t bd = sdesc_sw128(x_t + part * (tn * 256) + (kk >> 2) * (tn * 128) + (kk & 3) * 32, 16, 1024);
            umma_f16(tmem_base, ad, bd, idesc, (i > 0 || part > 0 || kk > 0) ? 1u : 0u);
          }
        }
        umma_commit(bar_empty + 8 * s);
        umma_commit(bar_aempty + 8 * j);
      }
      if (ok) {
        umma_commit(bar_acc);
      } else {
        umma_commit(bar_drain);
        mbar_wait_drain(bar_drain, 0);
      }
    }
  } else {
    // ---------------- unpack: two threads per row of W, 64 columns each ----------------
    const int d = threadIdx.x - 64, r = d >> 1, h = d & 1, r7 = r & 7;
    constexpr int ZN = GU == 32 ? 2 : 1;
    auto load_sz = [&](int rc, float (&s)[ZN], float (&z)[ZN]) {
      const int gr = rc * 128 + r;
#pragma unroll
      for (int j = 0; j < ZN; ++j) {
        const size_t at = static_cast<size_t>(min(gr, p.m - 1)) * p.G +
                          group_of<GU>(p.gi, kc, GU == 128 ? 0 : GU == 64 ? h : 2 * h + j);
        s[j] = gr < p.m ? __ldg(p.scales + at) : 0.0f;  // rows past m: zero weights
        z[j] = gr < p.m ? __ldg(p.zeros + at) : 0.0f;
      }
    };
    float ns[ZN], nz[ZN];
    if (nk > 0) load_sz(rc0, ns, nz);
    bool ok = true;
    for (int i = 0; i < nk; ++i) {
      float2 ss[ZN], nzm[ZN];
#pragma unroll
      for (int j = 0; j < ZN; ++j) {
        ss[j] = make_float2(ns[j], ns[j]);
        nzm[j] = make_float2(-8388608.0f - nz[j], -8388608.0f - nz[j]);
      }
      if (i + 1 < nk) load_sz(rc0 + i + 1, ns, nz);
      const int s = i % stages, j = i % TC_NA;
      if (!warp_wait(bar_full + 8 * s, static_cast<uint32_t>(i / stages) & 1u, abort_flag, lane) ||
          !warp_wait(bar_aempty + 8 * j, (static_cast<uint32_t>(i / TC_NA) & 1u) ^ 1u, abort_flag, lane)) {
        ok = false;
        break;
      }
      uint32_t w[2 * BITS];
      load_half_row<BITS>(smem + (st_base - sbase) + s * stage_bytes + code_off, r, h, w);
      const uint32_t dst = a_base + j * TC_A_BYTES + h * TC_ATOM + r * 128;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        uint32_t v, v1, q[4];
        half_row_block<BITS>(w, c, v, v1);
        dequant8<BITS>(v, v1, nzm[GU == 32 ? c >> 2 : 0], ss[GU == 32 ? c >> 2 : 0], q);
        st_shared_v4(dst + ((c ^ r7) << 4), q[0], q[1], q[2], q[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_afull + 8 * j);
    }
    // accumulator -> [token][column] sums over the operand tiles
    if (ok && nk > 0) ok = warp_wait(bar_acc, 0u, abort_flag, lane);
    if (ok) {
      tc_fence_after();
      const int qd = warp & 3, half = (warp - 2) >> 2, col = qd * 32 + lane;
      float* sums = reinterpret_cast<float*>(smem);
      for (int cc = half; cc < tn / 16; cc += 2) {
        uint32_t v[16];
        if (nk > 0) {
          tmem_ld_32x32b_x16(tmem_base + (static_cast<uint32_t>(qd * 32) << 16) + static_cast<uint32_t>(cc * 16), v);
          tmem_ld_wait();
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) sums[(cc * 16 + j) * TC_BM + col] = nk > 0 ? __uint_as_float(v[j]) : 0.0f;
      }
      tc_fence_before();
    }
  }

  __syncthreads();
  if (cs > 1) cluster_sync();
  if (!*abort_flag) {
    for (int t = rank + cs * warp; t < tn; t += cs * (BW_THREADS / 32)) {
      const int tok = t0 + t;
      if (tok >= p.T) continue;
      const uint32_t at = sbase + static_cast<uint32_t>((t * TC_BM + 4 * lane) * 4);
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int o = 0; o < cs; ++o) {
        const float4 w = cs > 1 ? ld_dsmem_f4(mapa_shared(at, o)) : *reinterpret_cast<const float4*>(smem + (at - sbase));
        v.x += w.x;
        v.y += w.y;
        v.z += w.z;
        v.w += w.w;
      }
      if (p.token_scale) {
        const float s = p.token_scale[tok];
        v.x *= s;
        v.y *= s;
        v.z *= s;
        v.w *= s;
      }
      uint16_t* d = p.dX + static_cast<size_t>(tok) * p.lddx + kc * 128 + 4 * lane;
      const uint32_t lo = p.bf16_out ? pack2<true>(v.x, v.y) : pack2<false>(v.x, v.y);
      const uint32_t hi = p.bf16_out ? pack2<true>(v.z, v.w) : pack2<false>(v.z, v.w);
      if (p.vec) {
        *reinterpret_cast<uint2*>(d) = make_uint2(lo, hi);
      } else {
        d[0] = static_cast<uint16_t>(lo);
        d[1] = static_cast<uint16_t>(lo >> 16);
        d[2] = static_cast<uint16_t>(hi);
        d[3] = static_cast<uint16_t>(hi >> 16);
      }
    }
  }
  if (cs > 1) cluster_sync();
  if (threadIdx.x == 0 && *abort_flag) atomicOr(p.status, ST_TIMEOUT);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, static_cast<uint32_t>(tn));
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
cudaError_t launch_linear_tc(const TcLaunch& l, const CUtensorMap& codes, const CUtensorMap& x, const LinearTcArgs& a);
template <int BITS>
cudaError_t launch_linear_bwd_tc(const TcLaunch& l, const CUtensorMap& codes, const CUtensorMap& dz,
                                 const CUtensorMap& dz_lo, const LinearBwdArgs& a);

}  // namespace gptq
