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
//   warps 4-11    unpack: two groups of four warps, each its half of every chunk
//   warps 12-19   drain and epilogue: lane = tensor-memory lane, each warp 128 of the 256 tokens
// Operands move in steps of 64 along k.  Handing a step from the MMA back to the unpack warps and
// forward again takes about 2700 cycles (measured with empty unpack warps), against the 512 cycles
// of its MMAs: six steps of each operand are in flight (with two 128-wide ones the 70B-shaped layer
// took 3.7 ms).
// Tensor memory holds two accumulators of 256 columns.  Forward: they alternate by group unit, and
// the sums live in the drain warps' registers (128 each, hence the register split), whose epilogue
// overlaps the producers' next tile.  Gradient: they alternate by tile, so that a tile's epilogue
// overlaps the next tile's MMAs.
// Measured, 4 bits: 2048 tokens through 11008 x 4096 in 260 to 269 us (the slower 687 TFLOP/s, 0.42 of the
// library product's burst rate), 4096 through 8192 x 28672 in 1.7 ms cold and 2.0 ms in a row of them (1.1 and
// 0.96 PFLOP/s, 0.70 of its sustained rate), the gradient of 4096 through 11008 x 4096 in 345 to 361 us (1.02
// PFLOP/s).  The loss is in handing steps over
// and, where a tile has few chunks, in the epilogues, during which one of two accumulators is waited for.
#pragma once

#include "packed_tc.cuh"

namespace gptq {

constexpr int PR_THREADS = 640;
constexpr int PR_TN = 256;                     // tokens of a tile
constexpr int PR_A_BYTES = 128 * 128;          // an unpacked step: 128 x 64 values
constexpr int PR_X_BYTES = 128 * 128;          // a block's half of a step's activations: 128 tokens x 64 values
constexpr int PR_EPI_BYTES = 8 * 1024;         // per drain warp: 8 tokens x 32 rows of sums
// Register split (setmaxnreg): 128 * (32 + 2 * 48 + 2 * 176) = 61440, what 640 threads of 96 start with.
constexpr int PR_REGS_MISC = 32, PR_REGS_UNPACK = 48, PR_REGS_DRAIN = 176;
static_assert(PR_REGS_MISC + 2 * PR_REGS_UNPACK + 2 * PR_REGS_DRAIN <= 5 * 96, "register split");

__host__ __device__ constexpr int pr_steps(int bits) { return bits == 8 ? 4 : 6; }  // steps in flight (even)
__host__ __device__ constexpr int pr_code_chunks(int bits) { return bits == 8 ? 4 : 3; }  // code chunks in flight
__host__ __device__ constexpr int pr_smem_bytes(int bits) {
  return 1024 + pr_steps(bits) * (PR_A_BYTES + PR_X_BYTES) + pr_code_chunks(bits) * tc_code_bytes(bits) + PR_EPI_BYTES + 512 +
         256;
}
static_assert(pr_smem_bytes(4) <= 227 * 1024 && pr_smem_bytes(8) <= 227 * 1024, "shared memory");

struct PairArgs {
  int tiles_m, tiles_t;  // tiles of 256 rows (forward) or columns (gradient), and of 256 tokens
  int chunks, steps;     // 128-wide chunks of the reduction; steps = chunks, or 2 chunks with a low part
  LinearTcArgs lin;      // forward: everything; gradient: T, m, G, gi, scales, zeros, status
  GradOut go;            // gradient
};

// Arrival on a barrier of the pair's even block.  (A release at cluster scope would also wait for the
// warp's loads of the next step's parameters: with it the gradient's kernel ran 590 us, not 430.)
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
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
  constexpr int SC = pr_code_chunks(BITS), NS = pr_steps(BITS), CODES = tc_code_bytes(BITS);
  extern __shared__ uint8_t pr_smem_raw[];
  const uint32_t raw_s = smem_u32(pr_smem_raw);
  uint8_t* smem = pr_smem_raw + (((raw_s + 1023u) & ~1023u) - raw_s);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t a_base = sbase, x_base = a_base + NS * PR_A_BYTES, c_base = x_base + NS * PR_X_BYTES,
                 e_base = c_base + SC * CODES;
  const uint32_t bar_full = e_base + PR_EPI_BYTES, bar_empty = bar_full + 8 * NS, bar_cfull = bar_empty + 8 * NS,
                 bar_cempty = bar_cfull + 8 * SC, bar_tfull = bar_cempty + 8 * SC, bar_tempty = bar_tfull + 16,
                 bar_drain = bar_tempty + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + (bar_drain + 8 - sbase));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  // gradient: the weights' exponents of this block's columns, [tiles_m]
  int8_t* exponents = reinterpret_cast<int8_t*>(smem + (bar_full - sbase) + 512);

  // (a shuffled warp index is known to be uniform: operands of the MMAs stay in uniform registers)
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int cluster = static_cast<int>(blockIdx.x >> 1), clusters = static_cast<int>(gridDim.x >> 1);
  const int ntiles = p.tiles_m * p.tiles_t;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(bar_full + 8 * s, 9);  // even block: the pair's activations (one arrival and their bytes) and
      mbar_init(bar_empty + 8 * s, 1);  // a group of unpack warps of each block
    }
    for (int s = 0; s < SC; ++s) {
      mbar_init(bar_cfull + 8 * s, 1);
      mbar_init(bar_cempty + 8 * s, 8);
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
      const uint32_t lead_full = mapa_shared(bar_full, 0);
      RingPos<NS> r;
      int issued = 0;
      bool ok = true;
      for (int tile = cluster; tile < ntiles && ok; tile += clusters) {
        const int t0 = tile / p.tiles_m * PR_TN + 128 * static_cast<int>(rank);
        for (int i = 0; i < 2 * p.steps; ++i) {
          if (!mbar_wait_bounded_cl(bar_empty + 8 * r.s, r.ph ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          if (leader) mbar_arrive_expect_tx(bar_full + 8 * r.s, 2 * PR_X_BYTES);
          const bool low = BWD && i >= 2 * p.chunks;
          tma_load_2d_pair(x_base + r.s * PR_X_BYTES, low ? &xlo_map : &x_map, lead_full + 8 * r.s,
                           (low ? i - 2 * p.chunks : i) * 64, t0);
          r.next();
          ++issued;
        }
      }
      // no copy of the pair may be in flight when either block leaves (the odd block is held by the
      // closing cluster barrier until the even one has seen its last stages complete)
      if (leader)
        for (int i = max(0, issued - NS); i < issued; ++i)
          mbar_wait_drain(bar_full + 8 * (i % NS), static_cast<uint32_t>(i / NS) & 1u);
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
    } else if (warp == 1 && leader) {
      // ---------------- MMA for the pair: the whole warp runs the loop, one lane issues ----------------
      const bool issue = elect_one_sync();
      const uint32_t fmt = (BF && !BWD) ? 1u : 0u;
      const uint32_t idesc = idesc_make(fmt, fmt, BWD ? 1u : 0u, 0u, 256, PR_TN);
      // This warp shares its scheduler with unpack and drain warps, so its instructions are few:
      // descriptors are those of step 0 plus the slot's and the 16-wide slice's offsets.
      // Forward: K-major; gradient: MN-major, 16 rows = two 8-row atoms, 64-column halves 8 KB apart.
      const uint64_t ad0 = BWD ? sdesc_sw128(a_base, PR_A_BYTES / 2, 1024) : sdesc_sw128(a_base, 16, 1024);
      const uint64_t bd0 = sdesc_sw128(x_base, 16, 1024);
      constexpr uint32_t A_SLICE = (BWD ? 2048 : 32) >> 4, B_SLICE = 32 >> 4;
      constexpr int SUB = (!BWD && GU == 32) ? 2 : 1;  // accumulation units of a step
      RingPos<NS> x;
      RingPos<2> t;
      bool ok = true;
      for (int tile = cluster; tile < ntiles && ok; tile += clusters) {
        for (int i = 0; i < p.steps && ok; ++i) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!warp_wait_uniform_cl(bar_full + 8 * x.s, x.ph, abort_flag)) {
              ok = false;
              break;
            }
            const uint64_t ad = ad0 + static_cast<uint32_t>(x.s * (PR_A_BYTES >> 4)),
                           bd = bd0 + static_cast<uint32_t>(x.s * (PR_X_BYTES >> 4));
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
              // a unit starts and ends with this step's MMAs: gradient, the whole tile is one unit
              const bool first = BWD ? (h == 0 && i == 0) : (GU < 128 || h == 0);
              const bool last = BWD ? (h == 1 && i == p.steps - 1) : (GU < 128 || h == 1);
              if (first && !warp_wait_uniform_cl(bar_tempty + 8 * t.s, t.ph ^ 1u, abort_flag)) {
                ok = false;
                break;
              }
              tc_fence_after();
              const uint32_t d = tmem_base + static_cast<uint32_t>(t.s * PR_TN);
#pragma unroll
              for (int k = 0; k < 4 / SUB; ++k) {
                const uint32_t kk = u * (4 / SUB) + k;
                if (issue) umma_f16_pair(d, ad + kk * A_SLICE, bd + kk * B_SLICE, idesc, (first && k == 0) ? 0u : 1u);
              }
              if (u == SUB - 1 && issue) umma_commit_pair_mc(bar_empty + 8 * x.s, 0x3);
              if (last) {
                if (issue) umma_commit_pair_mc(bar_tfull + 8 * t.s, 0x3);
                t.next();
              }
            }
            if (!ok) break;
            x.next();
          }
        }
      }
      if (!ok) {  // MMAs may still be running: wait for them before tensor memory is released
        if (issue) umma_commit_pair(bar_drain);
        mbar_wait_drain(bar_drain, 0);
      }
    }
  } else if (warp < 12) {
    // ---------------- unpack ----------------
    // Forward: group 0 takes columns 0-63 of every chunk, group 1 columns 64-127, a thread one row.
    // Gradient: group 0 takes rows 0-63 of every chunk, group 1 rows 64-127, two threads per row.
    regs_dec<PR_REGS_UNPACK>();
    const int d = threadIdx.x & 127, grp = (warp - 4) >> 2;
    const int r = BWD ? grp * 64 + (d >> 1) : d, h = BWD ? d & 1 : grp, r7 = r & 7;
    const uint32_t lead_full = mapa_shared(bar_full, 0);
    const uint32_t dst0 = a_base + (BWD ? h * (PR_A_BYTES / 2) + (r & 63) * 128 : r * 128);
    constexpr int ZN = GU == 32 ? 2 : 1;  // groups of a half row
    uint32_t w[2 * BITS];
    RingPos<SC> c;
    auto take = [&]() {  // the next chunk's words
      if (!warp_wait_uniform(bar_cfull + 8 * c.s, c.ph, abort_flag)) return false;
      load_half_row<BITS>(smem + (c_base - sbase) + c.s * CODES, r, h, w);
      return true;
    };
    int as = grp;  // slot of this group's next step
    uint32_t aph = 0;
    if (BWD) {
      for (int i0 = warp - 4; i0 < p.tiles_m; i0 += 32) {
        int part[4];  // (four loads in flight)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          part[k] = exponent_part(p.go, min(2 * (i0 + 8 * k) + static_cast<int>(rank), p.go.n / 128 - 1), lane);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          part[k] = __reduce_min_sync(0xffffffffu, part[k]);
          if (lane == 0 && i0 + 8 * k < p.tiles_m) exponents[i0 + 8 * k] = static_cast<int8_t>(part[k]);
        }
      }
      asm volatile("bar.sync 1, 512;" ::: "memory");  // unpack and drain warps
    }
    bool ok = cluster < ntiles && take();
    for (int tile = cluster; tile < ntiles && ok; tile += clusters) {
      const int mt = tile % p.tiles_m * 2 + static_cast<int>(rank);
      // row of W and its groups: forward row mt * 128 + r in chunk i; gradient row i * 128 + r in chunk mt
      const float up = BWD ? pow2(exponents[tile % p.tiles_m]) : 1.0f;
      float ns[ZN], nz[ZN];
      auto load_sz = [&](int i) {
        const int gr = (BWD ? i : mt) * 128 + r;
        const bool in = gr < p.lin.m;
        const size_t row = static_cast<size_t>(min(gr, p.lin.m - 1)) * p.lin.G;
        const int kc = BWD ? min(mt, p.go.n / 128 - 1) : i;
#pragma unroll
        for (int j = 0; j < ZN; ++j) {
          const size_t at = row + group_of<GU>(p.lin.gi, kc, GU == 128 ? 0 : GU == 64 ? h : 2 * h + j);
          nz[j] = in ? __ldg(p.lin.zeros + at) : 0.0f;
          if (BWD) ns[j] = in ? __ldg(p.lin.scales + at) : 0.0f;  // rows past m: zero weights
        }
      };
      load_sz(0);
      for (int i = 0; i < p.steps && ok; ++i) {
        float cs[ZN], cz[ZN];
#pragma unroll
        for (int j = 0; j < ZN; ++j) {
          cz[j] = nz[j];
          cs[j] = BWD ? ns[j] * up : 0.0f;
        }
        if (i + 1 < p.steps) load_sz((BWD && i + 1 >= p.chunks) ? i + 1 - p.chunks : i + 1);
        if (!warp_wait_uniform_cl(bar_empty + 8 * as, aph ^ 1u, abort_flag)) {
          ok = false;
          break;
        }
        const uint32_t dst = dst0 + as * PR_A_BYTES;
#pragma unroll
        for (int b = 0; b < 8; ++b) {
          const int j = GU == 32 ? b >> 2 : 0;
          uint32_t v, v1, q[4];
          half_row_block<BITS>(w, b, v, v1);
          if (BWD) {
            dequant8<BITS>(v, v1, make_float2(-8388608.0f - cz[j], -8388608.0f - cz[j]), make_float2(cs[j], cs[j]), q);
            st_shared_v4(dst + ((b ^ r7) << 4), q[0], q[1], q[2], q[3]);
          } else {
            unpack8<BITS, BF>(v, v1, zero_term<BITS, BF>(cz[j]), q);
            // pairs (i, i + 4) -> columns in order
            st_shared_v4(dst + ((b ^ r7) << 4), __byte_perm(q[0], q[1], 0x5410), __byte_perm(q[2], q[3], 0x5410),
                         __byte_perm(q[0], q[1], 0x7632), __byte_perm(q[2], q[3], 0x7632));
          }
        }
        // (the words were used above, so their stage can go back; the next chunk's are taken before this
        // chunk's stores are fenced, which complete meanwhile)
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_cempty + 8 * c.s);
        c.next();
        if (i + 1 < p.steps || tile + clusters < ntiles) ok = take();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(lead_full + 8 * as);
        as += 2;
        if (as >= NS) {
          as = grp;
          aph ^= 1u;
        }
      }
    }
  } else {
    // ---------------- drain and epilogue ----------------
    regs_inc<PR_REGS_DRAIN>();
    const int qd = warp & 3, half = (warp - 12) >> 2;
    const uint32_t lead_tempty = mapa_shared(bar_tempty, 0);
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(qd * 32) << 16) + static_cast<uint32_t>(half * 128);
    float* stage = reinterpret_cast<float*>(smem + (e_base - sbase)) + (warp - 12) * 256;  // [8 tokens][32 rows]
    if (BWD) asm volatile("bar.sync 1, 512;" ::: "memory");  // the exponents are there
    RingPos<2> t;
    bool ok = true;
    for (int tile = cluster; tile < ntiles && ok; tile += clusters) {
      const int mt = tile % p.tiles_m * 2 + static_cast<int>(rank);
      const int row0 = mt * 128 + qd * 32;                       // rows of Y, or columns of dX
      const int tok0 = tile / p.tiles_m * PR_TN + half * 128;
      // Eight tokens from the staging buffer to rows of `out` (f32: fp32, else 16 bits), + res: a lane
      // writes four rows of two tokens.  Little code: the callers unroll it over the registers.
      const int row = row0 + 4 * (lane & 7), tl = lane >> 3, rows = BWD ? p.go.n : p.lin.m;
      const bool whole = (BWD ? p.go.vec : p.lin.vec) && row + 4 <= rows;
      auto put8 = [&](int j0, void* out, int64_t ld, bool f32, const uint16_t* res) {
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int t = tok0 + j0 + 4 * k + tl;
          if (t < p.lin.T && row < rows) {
            const float4 v = *reinterpret_cast<const float4*>(stage + (4 * k + tl) * 32 + 4 * (lane & 7));
            float z[4] = {v.x, v.y, v.z, v.w};
            const size_t at = static_cast<size_t>(t) * ld + row;
            if (whole) {
              if (res) {
                const ushort4 r = *reinterpret_cast<const ushort4*>(res + static_cast<size_t>(t) * p.lin.ld_res + row);
                z[0] += h2f<BF>(r.x);
                z[1] += h2f<BF>(r.y);
                z[2] += h2f<BF>(r.z);
                z[3] += h2f<BF>(r.w);
              }
              if (f32)
                *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = make_float4(z[0], z[1], z[2], z[3]);
              else
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) =
                    make_uint2(pack2<BF>(z[0], z[1]), pack2<BF>(z[2], z[3]));
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                if (row + j < rows) {
                  if (res) z[j] += h2f<BF>(res[static_cast<size_t>(t) * p.lin.ld_res + row + j]);
                  if (f32)
                    static_cast<float*>(out)[at + j] = z[j];
                  else
                    static_cast<uint16_t*>(out)[at + j] = f2h<BF>(z[j]);
                }
              }
            }
          }
        }
        __syncwarp();
      };
      if (BWD) {
        const float2 back = pow2_halves(-exponents[tile % p.tiles_m]);
        if (!warp_wait_uniform_cl(bar_tfull + 8 * t.s, t.ph, abort_flag)) {
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
          for (int g = 0; g < 2; ++g) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int t = tok0 + cc * 16 + 8 * g + j;
              const Unscale s(p.go.token_scale && t < p.lin.T ? __ldg(p.go.token_scale + t) : make_float2(1.0f, 1.0f), back);
              stage[j * 32 + lane] = s(__uint_as_float(v[8 * g + j]));
            }
            put8(cc * 16 + 8 * g, p.go.dX, p.go.lddx, false, nullptr);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(lead_tempty + 8 * t.s);
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
          if (!warp_wait_uniform_cl(bar_tfull + 8 * t.s, t.ph, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t at = lane_base + static_cast<uint32_t>(t.s * PR_TN);
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) {
            uint32_t v[32];
            tmem_ld_32x32b_x32(at + cc * 32, v);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) acc[cc * 32 + j] = fmaf(sc, __uint_as_float(v[j]), acc[cc * 32 + j]);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(lead_tempty + 8 * t.s);
          t.next();
        }
        if (ok) {
          if (p.lin.bias) {
            const float bias = h2f<BF>(p.lin.bias[min(row0 + lane, p.lin.m - 1)]);
#pragma unroll
            for (int j = 0; j < 128; ++j) acc[j] += bias;
          }
          if (p.lin.preact) {
#pragma unroll
            for (int cc = 0; cc < 16; ++cc) {
#pragma unroll
              for (int j = 0; j < 8; ++j) stage[j * 32 + lane] = acc[cc * 8 + j];
              put8(cc * 8, p.lin.preact, p.lin.m, false, nullptr);
            }
          }
          if (p.lin.act == ACT_RELU) {
#pragma unroll
            for (int j = 0; j < 128; ++j) acc[j] = acc[j] > 0.0f ? acc[j] : 0.0f;
          } else if (p.lin.act == ACT_SILU) {
#pragma unroll
            for (int j = 0; j < 128; ++j) acc[j] = silu(acc[j]);
          } else if (p.lin.act == ACT_GELU) {
#pragma unroll
            for (int j = 0; j < 128; ++j) acc[j] = gelu(acc[j]);
          }
#pragma unroll
          for (int cc = 0; cc < 16; ++cc) {
#pragma unroll
            for (int j = 0; j < 8; ++j) stage[j * 32 + lane] = acc[cc * 8 + j];
            put8(cc * 8, p.lin.Y, p.lin.ldy, p.lin.y_fp32 != 0, p.lin.residual);
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
