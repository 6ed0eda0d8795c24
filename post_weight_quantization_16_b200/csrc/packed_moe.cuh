// packed_moe.cuh — routing of the mixture-of-experts layer: router product, softmax, top-k and the
// lists of tokens per expert, in one launch of one cluster; and the gathers of activations into
// sweep order.
#pragma once

#include "packed_decode.cuh"

namespace gptq {

// out[t][k] = X[t][perm[k]] in rows of n: rows pass through shared memory, so that global reads and
// writes are whole lines, the gather itself is from shared memory and a block reads the order once.
// PAIR: two rows at a time, interleaved as 32-bit words there, so that one 32-bit gather (conflicts
// of random banks are its cost) serves both: 4096 x 28672 values in 108 us (4.4 TB/s).  Grid (tokens /
// rows rounded up), dynamic shared memory rows * n * 2 bytes, rows even with PAIR.
template <bool PAIR>
__global__ void __launch_bounds__(512) gather_x_kernel(const uint16_t* __restrict__ X, int64_t ldx, int T, int n,
                                                       const int32_t* __restrict__ perm, int rows,
                                                       uint16_t* __restrict__ out) {
  extern __shared__ __align__(16) uint16_t gather_rows[];
  griddep_wait();
  griddep_launch_dependents();
  const int t0 = blockIdx.x * rows, cnt = min(rows, T - t0);
  constexpr int STEP = PAIR ? 2 : 1;
  for (int r = 0; r < cnt; r += STEP) {
    const uint4* a = reinterpret_cast<const uint4*>(X + static_cast<size_t>(t0 + r) * ldx);
    uint4* dst = reinterpret_cast<uint4*>(gather_rows + static_cast<size_t>(r) * n);
    if (PAIR) {
      // (an odd last row is paired with itself)
      const uint4* b = reinterpret_cast<const uint4*>(X + static_cast<size_t>(t0 + min(r + 1, cnt - 1)) * ldx);
      for (int k = threadIdx.x; k < n / 8; k += 512) {
        const uint4 u = a[k], v = b[k];
        dst[2 * k] = make_uint4(__byte_perm(u.x, v.x, 0x5410), __byte_perm(u.x, v.x, 0x7632),
                                __byte_perm(u.y, v.y, 0x5410), __byte_perm(u.y, v.y, 0x7632));
        dst[2 * k + 1] = make_uint4(__byte_perm(u.z, v.z, 0x5410), __byte_perm(u.z, v.z, 0x7632),
                                    __byte_perm(u.w, v.w, 0x5410), __byte_perm(u.w, v.w, 0x7632));
      }
    } else {
      for (int k = threadIdx.x; k < n / 8; k += 512) dst[k] = a[k];
    }
  }
  __syncthreads();
  for (int k = threadIdx.x * 4; k < n; k += 2048) {
    const int4 i = *reinterpret_cast<const int4*>(perm + k);
    for (int r = 0; r < cnt; r += STEP) {
      uint16_t* o = out + static_cast<size_t>(t0 + r) * n + k;
      if (PAIR) {
        const uint32_t* row = reinterpret_cast<const uint32_t*>(gather_rows + static_cast<size_t>(r) * n);
        const uint32_t w0 = row[i.x], w1 = row[i.y], w2 = row[i.z], w3 = row[i.w];
        *reinterpret_cast<uint2*>(o) = make_uint2(__byte_perm(w0, w1, 0x5410), __byte_perm(w2, w3, 0x5410));
        if (r + 1 < cnt)
          *reinterpret_cast<uint2*>(o + n) = make_uint2(__byte_perm(w0, w1, 0x7632), __byte_perm(w2, w3, 0x7632));
      } else {
        const uint16_t* row = gather_rows + static_cast<size_t>(r) * n;
        *reinterpret_cast<ushort4*>(o) = make_ushort4(row[i.x], row[i.y], row[i.z], row[i.w]);
      }
    }
  }
}

// Few tokens in fragment order, [chunk][tiles][FRAG_BYTES], for units of gu columns.  Grid (chunks,
// tiles), 128 threads, one 16-byte piece each; tokens past T repeat the last one.
__global__ void __launch_bounds__(128) fragment_kernel(const uint16_t* __restrict__ X, int64_t ldx, int T, int gu,
                                                       const int32_t* __restrict__ perm, uint4* __restrict__ out,
                                                       int* __restrict__ status) {
  griddep_wait();
  griddep_launch_dependents();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *status = 0;
  const int kb = threadIdx.x >> 5, n = (threadIdx.x >> 2) & 7, q = threadIdx.x & 3;
  const int t = min(static_cast<int>(blockIdx.y) * 8 + n, T - 1);
  out[(static_cast<size_t>(blockIdx.x) * gridDim.y + blockIdx.y) * (FRAG_BYTES / 16) + threadIdx.x] =
      frag_gather(X + t * ldx, perm, static_cast<int>(blockIdx.x) * 128 + frag_column(gu, kb, q));
}

// The experts' tokens in fragment order and their expert's sweep order.  Grid (chunks, tiles at most).
__global__ void __launch_bounds__(128) moe_fragment_kernel(const uint16_t* __restrict__ X, int64_t ldx, int H, int gu,
                                                           const int32_t* __restrict__ perm, MoePlan plan, int top_k,
                                                           uint4* __restrict__ out) {
  griddep_wait();
  griddep_launch_dependents();
  const int tile = static_cast<int>(blockIdx.y);
  if (tile >= *plan.tiles) return;
  const int seg = plan.tile_seg[tile], tile0 = plan.tile0[seg], count = plan.count[seg];
  const int kb = threadIdx.x >> 5, n = (threadIdx.x >> 2) & 7, q = threadIdx.x & 3;
  const int i = min((tile - tile0) * 8 + n, count - 1), tiles = (count + 7) / 8;
  const int t = plan.pair[plan.begin[seg] + i] / top_k;
  const size_t at = (static_cast<size_t>(tile0) * gridDim.x + static_cast<size_t>(blockIdx.x) * tiles + (tile - tile0)) *
                        (FRAG_BYTES / 16) +
                    threadIdx.x;
  out[at] = frag_gather(X + t * ldx, perm ? perm + static_cast<size_t>(plan.expert[seg]) * H : nullptr,
                        static_cast<int>(blockIdx.x) * 128 + frag_column(gu, kb, q));
}

// ------------------------------------------------------------------------------------------
// router
// ------------------------------------------------------------------------------------------
constexpr int ROUTER_CLUSTER = 8;
constexpr int ROUTER_WARPS = 16;

struct RouterArgs {
  const uint16_t* X;
  int64_t ldx;
  const uint16_t* R;  // [E x H]
  int T, E, H, top_k, renorm;
  int seg_pairs;       // pairs of a segment at most
  double* logits;      // [T x E] (workspace)
  float* bounds;       // [T x E] of their errors (workspace)
  int32_t* ids;        // [T x top_k] (workspace)
  float* weights;      // [T x top_k] (workspace)
  int32_t* ids_out;    // the caller's copies, or null
  float* weights_out;
  MoePlan plan;
  int* tickets;        // of the down product, set to zero here
  int ntickets;
  int* status;
};

// Bound of a logit's error by the sum S of its products' magnitudes: an MMA adds 16 products, exact in
// fp32, to its addend with at least single precision, at most 16 roundings or truncations of 2^-23 of the
// partial sum, and eight follow one another before fp64 takes over: 2^-16 S; 1.01 for S's own rounding.
// (The largest seen is 2^-20.5 S, of tokens with outliers and of logits whose products are all positive.)
constexpr float ROUTER_ERROR = 1.01f / 65536.0f;

// The logit of one expert in fp64, by a warp: products, exact in fp32, are added in 64 bits in a fixed order.
template <bool BF>
__device__ __noinline__ double exact_logit(const uint16_t* __restrict__ x, const uint16_t* __restrict__ r, int H,
                                           int lane) {
  double sum[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll 4
  for (int c = lane * 8; c < H; c += 256) {
    const uint4 a = *reinterpret_cast<const uint4*>(x + c), b = *reinterpret_cast<const uint4*>(r + c);
    const uint32_t u[4] = {a.x, a.y, a.z, a.w}, v[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      sum[j] += static_cast<double>(h2f<BF>(u[j] & 0xFFFFu) * h2f<BF>(v[j] & 0xFFFFu));
      sum[j] += static_cast<double>(h2f<BF>(u[j] >> 16) * h2f<BF>(v[j] >> 16));
    }
  }
  double s = (sum[0] + sum[1]) + (sum[2] + sum[3]);
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// One cluster.  (1) Logits: tiles of 16 experts x 8 tokens go round the blocks, as many at a time as a
// round of all needs; a tile's warps split H; products of 16-bit values are exact in fp32, 128 columns
// are summed on the tensor cores and the partial sums of those in fp64; the same MMAs on the magnitudes
// bound the error.  (2) Softmax and top-k: a warp per token, in fp64; equal values go to the lower expert;
// a NaN logit is chosen last (its weights are NaN).  Where two of the largest top_k + 1 logits stand so
// close that their errors could swap them, all logits at stake are formed again in fp64: the choices are
// those of the 64-bit logits.  (3) The lists, in block 0: a thread per choice, whose place is what its expert
// has before its group of 32 choices and its rank inside it, so positions are deterministic.
// By its own clock: 7 us for two tokens over 32 experts (2048 wide), 18 for 33 over 64, of which 9 are the
// logits (eight SMs fetch R and X, four trips to memory each), 5 the softmax and the choices, 4 the
// lists and barriers (lists by a warp per expert took 7 more); 1 for the errors' bounds and, where a
// token's choices are formed again (9 of 198 tokens in six such calls), 4.
template <bool BF>
__global__ void __launch_bounds__(ROUTER_WARPS * 32) moe_router_kernel(const RouterArgs p) {
  constexpr int CHOICES = MOE_MAX_T * MOE_MAX_TOPK, MINE = CHOICES / (ROUTER_WARPS * 32);
  __shared__ union {
    struct {
      double red[ROUTER_WARPS][128];
      float mag[ROUTER_WARPS][128];
    } l;                                        // (1)
    uint16_t before[CHOICES / 32 * MOE_MAX_E];  // (3) [group of choices][expert]
  } sh;
  __shared__ int counts[MOE_MAX_E];
  __shared__ int begins[MOE_MAX_E];
  __shared__ int slots[MOE_MAX_E];
  __shared__ int tiles[MOE_MAX_E];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int rank = static_cast<int>(cluster_ctarank());
  if (rank == 0 && threadIdx.x == 0) *p.status = 0;
  for (int i = rank * ROUTER_WARPS * 32 + threadIdx.x; i < p.ntickets; i += ROUTER_CLUSTER * ROUTER_WARPS * 32) p.tickets[i] = 0;
  const int et = (p.E + 15) / 16, tt = (p.T + 7) / 8, blocks = p.H / 32;
  const int ntiles = et * tt;
  int at_once = 1;  // tiles of a block
  while (at_once < ROUTER_WARPS && at_once * ROUTER_CLUSTER < ntiles) at_once *= 2;
  const int KW = ROUTER_WARPS / at_once, slot = warp / KW, kw = warp % KW;  // warps of a tile
  for (int first = rank * at_once; first < ntiles; first += ROUTER_CLUSTER * at_once) {
    const int tile = min(first + slot, ntiles - 1);  // (past the last: computed again, alike)
    const int e0 = (tile % et) * 16, t0 = (tile / et) * 8;
    const uint16_t* ra = p.R + static_cast<size_t>(min(e0 + g, p.E - 1)) * p.H + q * 8;
    const uint16_t* rb = p.R + static_cast<size_t>(min(e0 + g + 8, p.E - 1)) * p.H + q * 8;
    const uint16_t* x = p.X + static_cast<size_t>(min(t0 + g, p.T - 1)) * p.ldx + q * 8;
    double acc[4] = {0.0, 0.0, 0.0, 0.0};
    float mag[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const int b0 = blocks * kw / KW, b1 = blocks * (kw + 1) / KW;
    uint4 na[4], nb[4], nx[4];
    auto load = [&](int b) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int at = min(b + j, b1 - 1) * 32;
        na[j] = *reinterpret_cast<const uint4*>(ra + at);
        nb[j] = *reinterpret_cast<const uint4*>(rb + at);
        nx[j] = *reinterpret_cast<const uint4*>(x + at);
      }
    };
    if (b0 < b1) load(b0);
    for (int b = b0; b < b1; b += 4) {
      uint4 va[4], vb[4], vx[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        va[j] = na[j];
        vb[j] = nb[j];
        vx[j] = nx[j];
      }
      if (b + 4 < b1) load(b + 4);
      float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (b + j < b1) {
          mma_16816<BF>(d, va[j].x, vb[j].x, va[j].y, vb[j].y, vx[j].x, vx[j].y);
          mma_16816<BF>(d, va[j].z, vb[j].z, va[j].w, vb[j].w, vx[j].z, vx[j].w);
          constexpr uint32_t M = 0x7FFF7FFFu;
          mma_16816<BF>(mag, va[j].x & M, vb[j].x & M, va[j].y & M, vb[j].y & M, vx[j].x & M, vx[j].y & M);
          mma_16816<BF>(mag, va[j].z & M, vb[j].z & M, va[j].w & M, vb[j].w & M, vx[j].z & M, vx[j].w & M);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] += static_cast<double>(d[j]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      sh.l.red[warp][lane * 4 + j] = acc[j];
      sh.l.mag[warp][lane * 4 + j] = mag[j];
    }
    __syncthreads();
    for (int k = threadIdx.x; k < at_once * 128; k += ROUTER_WARPS * 32) {
      const int mine = first + (k >> 7), i = k & 127;
      double v = 0.0;
      float s = 0.0f;
      for (int w = 0; w < KW; ++w) {
        v += sh.l.red[(k >> 7) * KW + w][i];
        s += sh.l.mag[(k >> 7) * KW + w][i];
      }
      const int l = i >> 2, j = i & 3;
      const int e = (mine % et) * 16 + (l >> 2) + 8 * (j >> 1), t = (mine / et) * 8 + 2 * (l & 3) + (j & 1);
      if (mine < ntiles && e < p.E && t < p.T) {
        p.logits[static_cast<size_t>(t) * p.E + e] = v;
        p.bounds[static_cast<size_t>(t) * p.E + e] = ROUTER_ERROR * s;
      }
    }
    __syncthreads();
  }
  cluster_sync();  // the logits are written

  constexpr int PER = MOE_MAX_E / 32;
  const int per = (p.E + 31) / 32;
  for (int t = rank * ROUTER_WARPS + warp; t < p.T; t += ROUTER_CLUSTER * ROUTER_WARPS) {
    double v[PER], best = -INFINITY;
    float bound = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      v[i] = 0.0;
      if (i < per && lane + 32 * i < p.E) {
        v[i] = __ldcg(p.logits + static_cast<size_t>(t) * p.E + lane + 32 * i);
        const float b = __ldcg(p.bounds + static_cast<size_t>(t) * p.E + lane + 32 * i);
        bound = fmaxf(bound, b < INFINITY ? b : 0.0f);  // (such a logit is not finite either)
        best = fmax(best, v[i]);
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      best = fmax(best, __shfl_xor_sync(0xffffffffu, best, o));
      bound = fmaxf(bound, __shfl_xor_sync(0xffffffffu, bound, o));
    }
    auto value = [](unsigned long long key) {
      const unsigned long long u = (key >> 63) ? key & 0x7FFFFFFFFFFFFFFFull : ~key;
      return __longlong_as_double(key == 1ull ? 0x7FF8000000000000ll : static_cast<long long>(u));
    };
    int my_id = 0;
    unsigned long long my_key = 0;
    const double apart = 2.0 * bound;
    for (bool again = false;; again = true) {
      // The largest logits in order, the k-th left to lane k.  As keys whose unsigned order is theirs: a
      // NaN comes after every number, a place past E is never taken (key 0)
      unsigned long long key[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(v[i] + 0.0));
        key[i] = i < per && lane + 32 * i < p.E
                     ? (v[i] != v[i] ? 1ull : ((u >> 63) ? ~u : (u | 0x8000000000000000ull)))
                     : 0ull;
      }
      const int rounds = again ? p.top_k : min(p.top_k + 1, p.E);
      for (int k = 0; k < rounds; ++k) {
        unsigned long long bk = 0;
        unsigned bi = 0xffffffffu;
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (i < per && key[i] > bk) {  // (equal keys: the lower expert stands first)
            bk = key[i];
            bi = lane + 32 * i;
          }
        const unsigned hi = __reduce_max_sync(0xffffffffu, static_cast<unsigned>(bk >> 32));
        const bool top = static_cast<unsigned>(bk >> 32) == hi;
        const unsigned lo = __reduce_max_sync(0xffffffffu, top ? static_cast<unsigned>(bk) : 0u);
        const unsigned id = __reduce_min_sync(0xffffffffu, top && static_cast<unsigned>(bk) == lo ? bi : 0xffffffffu);
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (static_cast<unsigned>(lane + 32 * i) == id) key[i] = 0;
        if (lane == k) {
          my_id = static_cast<int>(id);
          my_key = (static_cast<unsigned long long>(hi) << 32) | lo;
        }
      }
      if (again) break;
      // bit k: the next one is less than `apart` below the k-th (a NaN is not)
      const double mine = value(my_key), next = __shfl_down_sync(0xffffffffu, mine, 1);
      const unsigned close = __ballot_sync(0xffffffffu, lane + 1 < rounds && mine - next < apart);
      if (close == 0) break;
      const uint16_t* x = p.X + static_cast<size_t>(t) * p.ldx;
      const double least = __shfl_sync(0xffffffffu, mine, p.top_k - 1) - apart;
      const bool border = (close >> (p.top_k - 1)) & 1u;
      // These are formed again; and where the border of the choices is one of them, so is every other expert
      // less than `apart` below the last choice (one further below is below all true choices).
      unsigned picks = close | (close << 1);
      for (int i = -1; i < (border ? per : 0); ++i) {
        unsigned at = picks;
        if (i >= 0) {
          bool mine_too = false;
#pragma unroll
          for (int j = 0; j < PER; ++j) mine_too |= j == i && key[j] != 0 && v[j] >= least;
          at = __ballot_sync(0xffffffffu, mine_too);
        }
        for (; at; at &= at - 1) {
          const int l = __ffs(at) - 1, e = i < 0 ? __shfl_sync(0xffffffffu, my_id, l) : l + 32 * i;
          const double d = exact_logit<BF>(x, p.R + static_cast<size_t>(e) * p.H, p.H, lane);
#pragma unroll
          for (int j = 0; j < PER; ++j)
            if (lane + 32 * j == e) v[j] = d;
        }
      }
    }
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i < per && lane + 32 * i < p.E) sum += exp(v[i] - best);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    // (top_k <= E: every round finds an expert)
    double mine = 0.0;
    if (lane < p.top_k) {
      mine = exp(value(my_key) - best);
    }
    if (p.renorm) {
      sum = mine;
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    if (lane < p.top_k) {
      const size_t o = static_cast<size_t>(t) * p.top_k + lane;
      const float w = static_cast<float>(mine / sum);
      p.ids[o] = my_id;
      p.weights[o] = w;
      if (p.ids_out) p.ids_out[o] = my_id;
      if (p.weights_out) p.weights_out[o] = w;
    }
  }
  cluster_sync();  // the choices are written
  if (rank != 0) return;

  const int pairs = p.T * p.top_k, groups = (pairs + 31) / 32;
  int id[MINE], place[MINE];
  float weight[MINE];
#pragma unroll
  for (int j = 0; j < MINE; ++j) {
    const int i = threadIdx.x + j * ROUTER_WARPS * 32;
    id[j] = -1;
    if (i < pairs) {
      id[j] = __ldcg(p.ids + i);
      weight[j] = __ldcg(p.weights + i);
    }
  }
  for (int k = threadIdx.x; k < groups * p.E; k += ROUTER_WARPS * 32) sh.before[k] = 0;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < MINE; ++j) {
    if (j * ROUTER_WARPS * 32 < pairs) {
      const unsigned same = __match_any_sync(0xffffffffu, id[j]);
      place[j] = __popc(same & ((1u << lane) - 1u));
      if (id[j] >= 0 && place[j] == 0)
        sh.before[(warp + j * ROUTER_WARPS) * p.E + id[j]] = static_cast<uint16_t>(__popc(same));
    }
  }
  __syncthreads();
  if (threadIdx.x < p.E) {
    int n = 0;
    for (int k = 0; k < groups; ++k) {
      uint16_t& at = sh.before[k * p.E + threadIdx.x];
      const int here = at;
      at = static_cast<uint16_t>(n);
      n += here;
    }
    counts[threadIdx.x] = n;
  }
  __syncthreads();
  if (warp == 0) {
    // exclusive sums over the experts of pairs, segments and tiles
    int base = 0, seg = 0, tile = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      const int n = e < p.E ? counts[e] : 0;
      const int ns = (n + p.seg_pairs - 1) / p.seg_pairs, nt = (n + 7) / 8;
      int in = n, is = ns, it = nt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int un = __shfl_up_sync(0xffffffffu, in, o), us = __shfl_up_sync(0xffffffffu, is, o),
                  ut = __shfl_up_sync(0xffffffffu, it, o);
        if (lane >= o) {
          in += un;
          is += us;
          it += ut;
        }
      }
      if (e < p.E) {
        begins[e] = base + in - n;
        slots[e] = seg + is - ns;
        tiles[e] = tile + it - nt;
      }
      base += __shfl_sync(0xffffffffu, in, 31);
      seg += __shfl_sync(0xffffffffu, is, 31);
      tile += __shfl_sync(0xffffffffu, it, 31);
    }
    if (lane == 0) {
      *p.plan.segments = seg;
      *p.plan.tiles = tile;
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < MINE; ++j) {
    if (id[j] >= 0) {
      const int o = begins[id[j]] + sh.before[(warp + j * ROUTER_WARPS) * p.E + id[j]] + place[j];
      p.plan.pair[o] = threadIdx.x + j * ROUTER_WARPS * 32;
      p.plan.weight[o] = weight[j];
    }
  }
  for (int e = warp; e < p.E; e += ROUTER_WARPS) {
    const int n = counts[e];
    const int per = p.seg_pairs;  // a multiple of 8
    for (int k = lane; k * per < n; k += 32) {
      const int s = slots[e] + k;
      p.plan.expert[s] = e;
      p.plan.begin[s] = begins[e] + k * per;
      p.plan.count[s] = min(per, n - k * per);
      p.plan.tile0[s] = tiles[e] + k * (per / 8);
      p.plan.high[s] = 0;
    }
    for (int k = lane; k * 8 < n; k += 32) p.plan.tile_seg[tiles[e] + k] = slots[e] + k * 8 / per;
  }
}

}  // namespace gptq
