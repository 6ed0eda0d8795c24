// packed_pair.cuh — products of packed weights with more than 128 tokens: a persistent kernel on CTA
// pairs (tcgen05 cta_group::2), for the linear layer (BWD = false) and for its gradient (BWD = true;
// the mathematics of both stands in packed_tc.cuh).
//
// A cluster of two blocks owns a tile of 256 rows (forward) or 256 columns of W (gradient), 128 each,
// times 256 tokens.  Against one block with a 128 x 128 tile this reads half the activations from
// L2 and shared memory and unpacks each weight half as often: per 128-column chunk the MMAs take 1024
// cycles, in which a block unpacks 16384 weights (about 320 cycles of its integer pipes) and, in the
// forward kernel, drains 128 x 256 sums with one fused multiply-add each (256 cycles).
//   warp 0        activations by TMA (each block its 128 tokens; both halves of a stage complete on
//                 the even block's barrier)
//   warp 3        codes by TMA (each block its own)
//   warp 1        tensor-memory allocation; in the even block MMA issue for the pair
//   warps 4-7     unpack, one thread per weight row
//   warps 8-15    drain and epilogue: lane = tensor-memory lane, each warp 128 of the 256 tokens
// Tensor memory holds two accumulators of 256 columns.  Forward: they alternate by group unit, and
// the sums live in the drain warps' registers (128 each, hence the register split), whose epilogue
// overlaps the producers' next tile.  Gradient: they alternate by tile, so that a tile's epilogue
// overlaps the next tile's MMAs.
#pragma once

#include "packed_tc.cuh"

namespace gptq {

constexpr int PR_THREADS = 512;
constexpr int PR_TN = 256;                     // tokens of a tile
constexpr int PR_NA = 2;                       // unpacked operand tiles in flight
constexpr int PR_SX = 3;                       // activation stages
constexpr int PR_X_BYTES = 128 * 256;          // a block's half of a stage: 128 tokens x 128 values
constexpr int PR_EPI_BYTES = 8 * 2048;         // per drain warp: 16 tokens x 32 rows of sums
// Register split (setmaxnreg): 128 * (40 + 96 + 184 + 184) = 64512 of the 65536 that 512 threads of 128 start with.
constexpr int PR_REGS_MISC = 40, PR_REGS_UNPACK = 96, PR_REGS_DRAIN = 184;
static_assert(PR_REGS_MISC + PR_REGS_UNPACK + 2 * PR_REGS_DRAIN <= 4 * 128, "register split");

__host__ __device__ constexpr int pr_code_stages(int bits) { return bits == 8 ? 2 : 4; }
__host__ __device__ constexpr int pr_smem_bytes(int bits) {
  return 1024 + PR_NA * TC_A_BYTES + PR_SX * PR_X_BYTES + pr_code_stages(bits) * tc_code_bytes(bits) + PR_EPI_BYTES + 512;
}

struct PairArgs {
  int tiles_m, tiles_t;  // tiles of 256 rows (forward) or columns (gradient), and of 256 tokens
  int chunks, steps;     // 128-wide chunks of the reduction; steps = chunks, or 2 chunks with a low part
  LinearTcArgs lin;      // forward: everything; gradient: T, m, G, gi, scales, zeros, status
  const float* token_scale;  // gradient: [T] or null
  uint16_t* dX;
  int64_t lddx;
  int n, dx_vec;
};

template <int REGS>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}
template <int REGS>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
}
// Waits of a whole warp on a barrier that the peer block arrives on too.
__device__ __forceinline__ bool warp_wait_cl(uint32_t bar, uint32_t parity, volatile int* abort_flag, int lane) {
  int ok = 1;
  if (lane == 0) ok = mbar_wait_bounded_cl(bar, parity, abort_flag) ? 1 : 0;
  __syncwarp();
  return __shfl_sync(0xffffffffu, ok, 0) != 0;
}
// Position in a ring of N stages.
template <int N>
struct RingPos {
  int s = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next() {
    if (++s == N) {
      s = 0;
      ph ^= 1u;
    }
  }
};

template <int BITS, bool BF, int GU, bool BWD>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PR_THREADS, 1)
    packed_pair_kernel(const __grid_constant__ CUtensorMap codes_map, const __grid_constant__ CUtensorMap x_map,
                       const __grid_constant__ CUtensorMap xlo_map, const PairArgs p) {
  constexpr int UNITS = 128 / GU;
  constexpr int SC = pr_code_stages(BITS), CODES = tc_code_bytes(BITS);
  extern __shared__ uint8_t pr_smem_raw[];
  const uint32_t raw_s = smem_u32(pr_smem_raw);
  uint8_t* smem = pr_smem_raw + (((raw_s + 1023u) & ~1023u) - raw_s);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t a_base = sbase, x_base = a_base + PR_NA * TC_A_BYTES, c_base = x_base + PR_SX * PR_X_BYTES,
                 e_base = c_base + SC * CODES;
  const uint32_t bar_xfull = e_base + PR_EPI_BYTES, bar_xempty = bar_xfull + 8 * PR_SX, bar_cfull = bar_xempty + 8 * PR_SX,
                 bar_cempty = bar_cfull + 8 * SC, bar_afull = bar_cempty + 8 * SC, bar_aempty = bar_afull + 8 * PR_NA,
                 bar_tfull = bar_aempty + 8 * PR_NA, bar_tempty = bar_tfull + 16, bar_drain = bar_tempty + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + (bar_drain + 8 - sbase));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int cluster = static_cast<int>(blockIdx.x >> 1), clusters = static_cast<int>(gridDim.x >> 1);
  const int ntiles = p.tiles_m * p.tiles_t;

  if (threadIdx.x == 0) {
    for (int s = 0; s < PR_SX; ++s) {
      mbar_init(bar_xfull + 8 * s, 1);  // even block: one expect_tx arrival, the pair's bytes
      mbar_init(bar_xempty + 8 * s, 1);
    }
    for (int s = 0; s < SC; ++s) {
      mbar_init(bar_cfull + 8 * s, 1);
      mbar_init(bar_cempty + 8 * s, 4);
    }
    for (int j = 0; j < PR_NA; ++j) {
      mbar_init(bar_afull + 8 * j, 8);  // even block: the unpack warps of both
      mbar_init(bar_aempty + 8 * j, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar_tfull + 8 * b, 1);
      mbar_init(bar_tempty + 8 * b, 16);  // even block: the drain warps of both
    }
    mbar_init(bar_drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), 512);
    tmem_relinquish_pair();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&codes_map);
    tma_prefetch_desc(&x_map);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both blocks' barriers and tensor memory exist before either touches the other's
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  griddep_wait();
  griddep_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0) atomicExch(p.lin.status, 0);

  if (warp < 4) {
    regs_dec<PR_REGS_MISC>();
    if (warp == 0 && lane == 0) {
      // ---------------- activations ----------------
      const uint32_t lead_full = mapa_shared(bar_xfull, 0);
      RingPos<PR_SX> r;
      int issued = 0;
      bool ok = true;
      for (int tile = cluster; tile < ntiles && ok; tile += clusters) {
        const int t0 = tile / p.tiles_m * PR_TN + 128 * static_cast<int>(rank);
        for (int i = 0; i < p.steps; ++i) {
          if (!mbar_wait_bounded_cl(bar_xempty + 8 * r.s, r.ph ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          if (leader) mbar_arrive_expect_tx(bar_xfull + 8 * r.s, 2 * PR_X_BYTES);
          const uint32_t fb = lead_full + 8 * r.s, st = x_base + r.s * PR_X_BYTES;
          const CUtensorMap* map = (BWD && i >= p.chunks) ? &xlo_map : &x_map;
          const int k = ((BWD && i >= p.chunks) ? i - p.chunks : i) * 128;
          tma_load_2d_pair(st, map, fb, k, t0);
          tma_load_2d_pair(st + PR_X_BYTES / 2, map, fb, k + 64, t0);
          r.next();
          ++issued;
        }
      }
      // no copy of the pair may be in flight when either block leaves (the odd block is held by the
      // closing cluster barrier until the even one has seen its last stages complete)
      if (leader)
        for (int i = max(0, issued - PR_SX); i < issued; ++i)
          mbar_wait_drain(bar_xfull + 8 * (i % PR_SX), static_cast<uint32_t>(i / PR_SX) & 1u);
    } else if (warp == 3 && lane == 0) {
      // ---------------- codes ----------------
      RingPos<SC> r;
      int issued = 0;
      bool ok = true;
      for (int tile = cluster; tile < ntiles && ok; tile += clusters) {
        const int mt = tile % p.tiles_m * 2 + static_cast<int>(rank);  // 128 rows, or 128 columns
        for (int i = 0; i < p.steps; ++i) {
          if (!mbar_wait_bounded(bar_cempty + 8 * r.s, r.ph ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          const int c = (BWD && i >= p.chunks) ? i - p.chunks : i;
          mbar_arrive_expect_tx(bar_cfull + 8 * r.s, CODES);
          tma_load_2d(c_base + r.s * CODES, &codes_map, bar_cfull + 8 * r.s, (BWD ? mt : c) * (4 * BITS),
                      (BWD ? c : mt) * 128);
          r.next();
          ++issued;
        }
      }
      for (int i = max(0, issued - SC); i < issued; ++i)
        mbar_wait_drain(bar_cfull + 8 * (i % SC), static_cast<uint32_t>(i / SC) & 1u);
    } else if (warp == 1 && lane == 0 && leader) {
      // ---------------- MMA for the pair ----------------
      const uint32_t fmt = (BF && !BWD) ? 1u : 0u;
      const uint32_t idesc = idesc_make(fmt, fmt, BWD ? 1u : 0u, 0u, 256, PR_TN);
      RingPos<PR_SX> x;
      RingPos<PR_NA> a;
      RingPos<2> t;
      bool ok = true;
      for (int tile = cluster; tile < ntiles && ok; tile += clusters) {
        for (int i = 0; i < p.steps && ok; ++i) {
          if (!mbar_wait_bounded_cl(bar_xfull + 8 * x.s, x.ph, abort_flag) ||
              !mbar_wait_bounded_cl(bar_afull + 8 * a.s, a.ph, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t a_t = a_base + a.s * TC_A_BYTES, x_t = x_base + x.s * PR_X_BYTES;
#pragma unroll
          for (int u = 0; u < (BWD ? 1 : UNITS); ++u) {
            if (!BWD || i == 0) {
              if (!mbar_wait_bounded_cl(bar_tempty + 8 * t.s, t.ph ^ 1u, abort_flag)) {
                ok = false;
                break;
              }
            }
            tc_fence_after();
            const uint32_t d = tmem_base + static_cast<uint32_t>(t.s * PR_TN);
            constexpr int STEPS16 = BWD ? 8 : GU / 16;
#pragma unroll
            for (int k = 0; k < STEPS16; ++k) {
              const int kk = u * STEPS16 + k;
              // forward: K-major, atoms of 64 columns; gradient: MN-major, 16 rows = two 8-row atoms
              const uint64_t ad = BWD ? sdesc_sw128(a_t + kk * 2048, TC_ATOM, 1024)
                                      : sdesc_sw128(a_t + (kk >> 2) * TC_ATOM + (kk & 3) * 32, 16, 1024);
              const uint64_t bd = sdesc_sw128(x_t + (kk >> 2) * (PR_X_BYTES / 2) + (kk & 3) * 32, 16, 1024);
              umma_f16_pair(d, ad, bd, idesc, (BWD ? (i > 0 || k > 0) : k > 0) ? 1u : 0u);
            }
            if (BWD || u == UNITS - 1) {
              umma_commit_pair_mc(bar_xempty + 8 * x.s, 0x3);
              umma_commit_pair_mc(bar_aempty + 8 * a.s, 0x3);
            }
            if (!BWD || i == p.steps - 1) {
              umma_commit_pair_mc(bar_tfull + 8 * t.s, 0x3);
              t.next();
            }
          }
          x.next();
          a.next();
        }
      }
      if (!ok) {  // MMAs may still be running: wait for them before tensor memory is released
        umma_commit_pair(bar_drain);
        mbar_wait_drain(bar_drain, 0);
      }
    }
  } else if (warp < 8) {
    // ---------------- unpack: one thread per row of the tile ----------------
    regs_dec<PR_REGS_UNPACK>();
    const int r = threadIdx.x - 128, r7 = r & 7;
    const uint32_t lead_afull = mapa_shared(bar_afull, 0);
    RingPos<SC> c;
    RingPos<PR_NA> a;
    bool ok = true;
    for (int tile = cluster; tile < ntiles && ok; tile += clusters) {
      const int mt = tile % p.tiles_m * 2 + static_cast<int>(rank);
      // row of W and its groups: forward row mt * 128 + r in chunk i; gradient row i * 128 + r in chunk mt
      float ns[UNITS], nz[UNITS];
      auto load_sz = [&](int i) {
        const int gr = (BWD ? i : mt) * 128 + r;
        const bool in = gr < p.lin.m;
        const size_t row = static_cast<size_t>(min(gr, p.lin.m - 1)) * p.lin.G;
        const int kc = BWD ? min(mt, p.n / 128 - 1) : i;
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
          const size_t at = row + group_of<GU>(p.lin.gi, kc, u);
          nz[u] = in ? __ldg(p.lin.zeros + at) : 0.0f;
          if (BWD) ns[u] = in ? __ldg(p.lin.scales + at) : 0.0f;  // rows past m: zero weights
        }
      };
      load_sz(0);
      for (int i = 0; i < p.steps; ++i) {
        float cs[UNITS], cz[UNITS];
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
          cz[u] = nz[u];
          cs[u] = BWD ? ns[u] : 0.0f;
        }
        if (i + 1 < p.steps) load_sz((BWD && i + 1 >= p.chunks) ? i + 1 - p.chunks : i + 1);
        if (!warp_wait(bar_cfull + 8 * c.s, c.ph, abort_flag, lane) ||
            !warp_wait_cl(bar_aempty + 8 * a.s, a.ph ^ 1u, abort_flag, lane)) {
          ok = false;
          break;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t w[2 * BITS];
          load_half_row<BITS>(smem + (c_base - sbase) + c.s * CODES, r, h, w);
          const uint32_t dst = a_base + a.s * TC_A_BYTES + h * TC_ATOM + r * 128;
#pragma unroll
          for (int b = 0; b < 8; ++b) {
            const int u = GU == 128 ? 0 : GU == 64 ? h : 2 * h + (b >> 2);
            uint32_t v, v1, q[4];
            half_row_block<BITS>(w, b, v, v1);
            if (BWD) {
              dequant8<BITS>(v, v1, make_float2(-8388608.0f - cz[u], -8388608.0f - cz[u]), make_float2(cs[u], cs[u]), q);
              st_shared_v4(dst + ((b ^ r7) << 4), q[0], q[1], q[2], q[3]);
            } else {
              unpack8<BITS, BF>(v, v1, zero_term<BITS, BF>(cz[u]), q);
              // pairs (i, i + 4) -> columns in order
              st_shared_v4(dst + ((b ^ r7) << 4), __byte_perm(q[0], q[1], 0x5410), __byte_perm(q[2], q[3], 0x5410),
                           __byte_perm(q[0], q[1], 0x7632), __byte_perm(q[2], q[3], 0x7632));
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar_cempty + 8 * c.s);
          mbar_arrive_cluster(lead_afull + 8 * a.s);
        }
        c.next();
        a.next();
      }
    }
  } else {
    // ---------------- drain and epilogue ----------------
    regs_inc<PR_REGS_DRAIN>();
    const int qd = warp & 3, half = (warp - 8) >> 2;
    const uint32_t lead_tempty = mapa_shared(bar_tempty, 0);
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(qd * 32) << 16) + static_cast<uint32_t>(half * 128);
    float* stage = reinterpret_cast<float*>(smem + (e_base - sbase)) + (warp - 8) * 512;  // [16 tokens][32 rows]
    RingPos<2> t;
    bool ok = true;
    for (int tile = cluster; tile < ntiles && ok; tile += clusters) {
      const int mt = tile % p.tiles_m * 2 + static_cast<int>(rank);
      const int row0 = mt * 128 + qd * 32;                       // rows of Y, or columns of dX
      const int tok0 = tile / p.tiles_m * PR_TN + half * 128;
      // 16 tokens of the sums, from the staging buffer: lane = 4 rows of every fourth token
      auto write16 = [&](int j0) {
        __syncwarp();
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
          const int tl = k * 4 + (lane >> 3), tok = tok0 + j0 + tl, row = row0 + 4 * (lane & 7);
          const float4 v = *reinterpret_cast<const float4*>(stage + tl * 32 + 4 * (lane & 7));
          if (BWD) {
            if (tok < p.lin.T && row < p.n) {
              const float s = p.token_scale ? p.token_scale[tok] : 1.0f;
              uint16_t* d = p.dX + static_cast<size_t>(tok) * p.lddx + row;
              const uint32_t lo = pack2<BF>(v.x * s, v.y * s), hi = pack2<BF>(v.z * s, v.w * s);
              if (p.dx_vec) {
                *reinterpret_cast<uint2*>(d) = make_uint2(lo, hi);
              } else {
                d[0] = static_cast<uint16_t>(lo);
                d[1] = static_cast<uint16_t>(lo >> 16);
                d[2] = static_cast<uint16_t>(hi);
                d[3] = static_cast<uint16_t>(hi >> 16);
              }
            }
          } else if (tok < p.lin.T && row < p.lin.m) {
            linear_epilogue4<BF>(p.lin, tok, row, v);
          }
        }
        __syncwarp();
      };
      if (BWD) {
        if (!warp_wait_cl(bar_tfull + 8 * t.s, t.ph, abort_flag, lane)) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll 1
        for (int cc = 0; cc < 8; ++cc) {
          uint32_t v[16];
          tmem_ld_32x32b_x16(lane_base + static_cast<uint32_t>(t.s * PR_TN + cc * 16), v);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) stage[j * 32 + lane] = __uint_as_float(v[j]);
          write16(cc * 16);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(lead_tempty + 8 * t.s);
        t.next();
      } else {
        float acc[128];
#pragma unroll
        for (int j = 0; j < 128; ++j) acc[j] = 0.0f;
        const float* srow = p.lin.scales + static_cast<size_t>(min(row0 + lane, p.lin.m - 1)) * p.lin.G;
        float ns = __ldg(srow);
        for (int uc = 0; uc < p.chunks * UNITS; ++uc) {
          const float sc = ns;
          if (uc + 1 < p.chunks * UNITS) ns = __ldg(srow + group_of<GU>(p.lin.gi, (uc + 1) / UNITS, (uc + 1) % UNITS));
          if (!warp_wait_cl(bar_tfull + 8 * t.s, t.ph, abort_flag, lane)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t at = lane_base + static_cast<uint32_t>(t.s * PR_TN);
          uint32_t v[2][16];
          tmem_ld_32x32b_x16(at, v[0]);
#pragma unroll
          for (int cc = 0; cc < 8; ++cc) {
            tmem_ld_wait();
            if (cc + 1 < 8) tmem_ld_32x32b_x16(at + (cc + 1) * 16, v[(cc + 1) & 1]);
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[cc * 16 + j] = fmaf(sc, __uint_as_float(v[cc & 1][j]), acc[cc * 16 + j]);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(lead_tempty + 8 * t.s);
          t.next();
        }
        if (ok) {
#pragma unroll
          for (int cc = 0; cc < 8; ++cc) {
#pragma unroll
            for (int j = 0; j < 16; ++j) stage[j * 32 + lane] = acc[cc * 16 + j];
            write16(cc * 16);
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither block leaves while the other may still use its shared or tensor memory
  if (threadIdx.x == 0 && *abort_flag) atomicOr(p.lin.status, ST_TIMEOUT);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

template <int BITS>
cudaError_t launch_packed_pair(const TcLaunch& l, bool backward, const CUtensorMap& codes, const CUtensorMap& x,
                               const CUtensorMap& xlo, const PairArgs& a);

}  // namespace gptq
