// packed_api.cu — the C ABI of the products on packed layers (include/gptq.h: gptq_dequant_linear,
// gptq_dequant_linear_backward, gptq_dequant_moe): argument checks, workspace layout and launches.
#include <algorithm>
#include <utility>

#include "api_common.cuh"
#include "packed_decode.cuh"
#include "packed_grad.cuh"
#include "packed_moe.cuh"
#include "packed_pair.cuh"
#include "packed_tc.cuh"

using namespace gptq;

namespace {

constexpr int64_t kPackedMaxN = 65536;
constexpr int64_t kPackedMaxM = int64_t(1) << 24;
constexpr int64_t kPackedMaxT = int64_t(1) << 22;
constexpr int kSms = 148;

size_t up256(size_t x) { return (x + 255) / 256 * 256; }
bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }
bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool valid_width(int64_t n) { return n >= 128 && n <= kPackedMaxN && n % 128 == 0; }

bool valid_packed(const gptq_packed& w) {
  gptq_qparams qp = w.qp;
  qp.sym = 0;  // not read
  return w.codes && w.scales && w.zeros && valid_width(w.n) && w.m >= 1 && w.m <= kPackedMaxM &&
         valid_qparams(qp, w.n) && aligned16(w.codes) && aligned_to(w.scales, 4) && aligned_to(w.zeros, 4) &&
         (!w.perm || aligned16(w.perm));
}

// Whether `rows` rows of wa and wb bytes at strides lda and ldb share memory.  Column slices of one
// buffer (equal strides) may lie between each other.
bool overlap(const void* a, int64_t lda, int64_t wa, const void* b, int64_t ldb, int64_t wb, int64_t rows) {
  if (!a || !b) return false;
  uint64_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
  if (pa > pb) {
    std::swap(pa, pb);
    std::swap(lda, ldb);
    std::swap(wa, wb);
  }
  if (pa + static_cast<uint64_t>((rows - 1) * lda + wa) <= pb) return false;
  if (rows == 1 || lda != ldb) return true;
  const int64_t off = static_cast<int64_t>((pb - pa) % static_cast<uint64_t>(lda));
  return off < wa || off + wb > lda;
}

int group_width(const gptq_packed& w) { return w.qp.group_size == -1 ? static_cast<int>(w.n) : w.qp.group_size; }

// Values of a scale or zero-point row that one aligned load takes.
int param_vec(const gptq_packed& w) {
  const int64_t G = w.n / group_width(w);
  if (G % 4 == 0 && aligned16(w.scales) && aligned16(w.zeros)) return 4;
  return G % 2 == 0 && aligned_to(w.scales, 8) && aligned_to(w.zeros, 8) ? 2 : 1;
}

GroupIndex group_index(int g) {
  GroupIndex gi;
  gi.div = g >= 128 ? g / 128 : 1;
  gi.magic = gi.div > 1 ? static_cast<uint32_t>(((uint64_t(1) << 32) + gi.div - 1) / gi.div) : 0u;
  return gi;
}

gptq_status check_device(int device) {
  static std::atomic<int> known{0};  // devices; does not change during the process
  int ndev = known.load(std::memory_order_relaxed);
  if (ndev == 0) {
    if (cudaGetDeviceCount(&ndev) != cudaSuccess) {
      cudaGetLastError();
      return GPTQ_ERR_CUDA;
    }
    known.store(ndev, std::memory_order_relaxed);
  }
  return device >= 0 && device < ndev ? GPTQ_OK : GPTQ_ERR_CUDA;
}

template <typename F>
cudaError_t by_bits(int bits, F&& f) {
  switch (bits) {
    case 2: return f(std::integral_constant<int, 2>());
    case 3: return f(std::integral_constant<int, 3>());
    case 4: return f(std::integral_constant<int, 4>());
    default: return f(std::integral_constant<int, 8>());
  }
}

template <typename F>
cudaError_t by_act(int act, F&& f) {
  switch (act) {
    case GPTQ_ACT_RELU: return f(std::integral_constant<int, ACT_RELU>());
    case GPTQ_ACT_GELU: return f(std::integral_constant<int, ACT_GELU>());
    case GPTQ_ACT_SILU: return f(std::integral_constant<int, ACT_SILU>());
    default: return f(std::integral_constant<int, ACT_NONE>());
  }
}

// Blocks of a cluster that split k: as many as two blocks per SM allow for `tiles` row tiles, each
// with at least two chunks.
int k_split(int64_t tiles, int chunks) {
  int cs = 1;
  while (cs < 8 && tiles * (cs + 1) <= 2 * kSms && chunks >= 2 * (cs + 1)) ++cs;
  return cs;
}

// Tokens up to which the warp-level kernel runs; beyond, tcgen05.
constexpr int kDecodeTokens = 16;
// Tokens up to which one block's 128-row tile runs; beyond, CTA pairs with 256-token tiles.
constexpr int kSingleTokens = 128;

// Whether the decode kernels lay out the tokens themselves, each block its chunk range, instead of a
// launch before them: every block of 128 rows repeats the layout.  Measured with 4-bit layers: a
// 4096 x 4096 one (4 chunks a block) takes 8.4 us with four tokens against 13.7 with the launch and
// 9.1 / 13.6 with eight, an 11008 x 4096 one (11 chunks) 15.5 / 15.2 and 20.9 / 15.1; gathered through
// an order, 10.5 / 13.9 and 16.1 / 13.9, and 17.2 / 15.2 already with two tokens.
bool lay_out_locally(int64_t T, bool perm, int chunks_per_block) {
  return T <= 8 && T * chunks_per_block <= (perm ? 16 : 44) && T * chunks_per_block * 256 <= DEC_LOCAL_BYTES;
}

// The gather of X takes two rows at a time where they fit.  Against one, 16-bit, measured: 4096 x 28672
// values 108 / 131 us, 8192 x 8192 49 / 71, 300 x 4096 4.6 / 6.3, 77 x 4096 4.2 / 4.1.
constexpr int kGatherPairBytes = 224 * 1024;

size_t linear_workspace(int64_t T, int64_t n, int act_order) {
  const size_t rows = T <= kDecodeTokens ? static_cast<size_t>((T + 7) / 8 * 8) : act_order ? static_cast<size_t>(T) : 0;
  return 256 + up256(rows * n * 2);
}

// Row-major 2-D tensor map: `cols` x `rows` elements of a type, boxes of box_cols x box_rows.
gptq_status encode_map(CUtensorMap* map, CUtensorMapDataType type, int elem, const void* base, int64_t cols,
                       int64_t rows, int64_t ld, int box_cols, int box_rows, CUtensorMapSwizzle swizzle) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = get_encode();
  if (!encode) return GPTQ_ERR_CUDA;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * elem};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  return encode(map, type, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? GPTQ_OK
             : GPTQ_ERR_CUDA;
}

// The codes of `layers` stacked matrices, boxes of one 128-column chunk of box_rows rows.
gptq_status encode_codes(CUtensorMap* map, const gptq_packed& w, int box_rows, int64_t layers = 1) {
  const int64_t words = w.n * w.qp.bits / 32;
  return encode_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, w.codes, words, w.m * layers, words, 4 * w.qp.bits, box_rows,
                    CU_TENSOR_MAP_SWIZZLE_NONE);
}
gptq_status encode_act(CUtensorMap* map, int dtype, const void* base, int64_t cols, int64_t rows, int64_t ld,
                       int box_rows) {
  return encode_map(map, dtype == GPTQ_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                    base, cols, rows, ld, 64, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Blocks of a cluster that split a reduction of `chunks` chunks when `tiles` tiles leave SMs idle.
int tc_cluster(int64_t tiles, int chunks) {
  int cs = 1;
  while (cs < 8 && tiles * (cs + 1) <= kSms && chunks >= 2 * (cs + 1)) ++cs;
  return cs;
}
// Whether CTA pairs (one 256 x 256 tile per two SMs) serve a product of `rows` x T outputs: they need
// tiles for most SM pairs.
bool use_pairs(int64_t rows, int64_t T) {
  return T > kSingleTokens && ((rows + 255) / 256) * ((T + PR_TN - 1) / PR_TN) >= kSms / 4;
}

// The linear layer on tcgen05: X in sweep order.
gptq_status linear_many_tokens(const gptq_linear_args& a, const uint16_t* X, int64_t ldx, int device,
                               cudaStream_t st) {
  const int m = static_cast<int>(a.W.m), n = static_cast<int>(a.W.n), T = static_cast<int>(a.T);
  const int g = group_width(a.W);
  LinearTcArgs d;
  d.T = T;
  d.m = m;
  d.chunks = n / 128;
  d.G = n / g;
  d.gi = group_index(g);
  d.tn = T <= 32 ? 32 : T <= 64 ? 64 : TC_MAX_TN;
  d.scales = a.W.scales;
  d.zeros = a.W.zeros;
  d.bias = static_cast<const uint16_t*>(a.bias);
  d.residual = static_cast<const uint16_t*>(a.residual);
  d.ld_res = a.ld_res;
  d.ldy = a.ld_y;
  d.Y = a.Y;
  d.preact = static_cast<uint16_t*>(a.preact);
  d.act = a.act;
  d.y_fp32 = a.y_fp32;
  d.vec = a.ld_y % 4 == 0 && aligned_to(a.Y, a.y_fp32 ? 16 : 8) &&
          (!a.residual || (a.ld_res % 4 == 0 && aligned_to(a.residual, 8))) &&
          (!a.preact || (m % 4 == 0 && aligned_to(a.preact, 8)));
  d.status = static_cast<int*>(a.workspace);
  CUtensorMap cmap, xmap;
  gptq_status s = encode_codes(&cmap, a.W, TC_BM);
  if (s == GPTQ_OK) s = encode_act(&xmap, a.dtype, X, n, T, ldx, d.tn);
  if (s != GPTQ_OK) return s;
  TcLaunch l;
  l.bf16 = a.dtype == GPTQ_BF16;
  l.unit = std::min(g, 128);
  l.sms = kSms;
  l.device = device;
  l.stream = st;
  if (use_pairs(m, T)) {
    PairArgs p = {};
    p.tiles_m = (m + 255) / 256;
    p.tiles_t = (T + PR_TN - 1) / PR_TN;
    p.chunks = p.steps = d.chunks;
    p.lin = d;
    CK(by_bits(a.W.qp.bits,
               [&](auto b) { return launch_packed_pair<decltype(b)::value>(l, false, cmap, xmap, xmap, p); }));
    return GPTQ_OK;
  }
  l.cluster = tc_cluster(static_cast<int64_t>((m + TC_BM - 1) / TC_BM) * ((T + d.tn - 1) / d.tn), d.chunks);
  CK(by_bits(a.W.qp.bits, [&](auto b) {
    return launch_packed_tc<decltype(b)::value>(l, false, cmap, xmap, xmap, d, GradOut{}, 1);
  }));
  return GPTQ_OK;
}

// Slabs of rows whose scales a block each looks at, eight a thread, at most.
constexpr int kSlabs = 256;
// What the gradient's product needs in the workspace.
struct GradLayout {
  int parts;       // 0: dY itself is the operand, else fp16 values of dz (1, or 2: high and low)
  int64_t ldz;
  size_t scale, exponent, hi, lo, dx, total;
};
bool grad_layout(int64_t T, int64_t m, int64_t n, int act_order, int dtype, int act, bool direct, GradLayout* l) {
  if (T < 0 || T > kPackedMaxT || m < 1 || m > kPackedMaxM || !valid_width(n) ||
      (dtype != GPTQ_FP16 && dtype != GPTQ_BF16) || act < GPTQ_ACT_NONE || act > GPTQ_ACT_SILU)
    return false;
  const bool smooth = act == GPTQ_ACT_GELU || act == GPTQ_ACT_SILU;
  l->parts = direct && dtype == GPTQ_FP16 && act == GPTQ_ACT_NONE ? 0 : dtype == GPTQ_FP16 && smooth ? 2 : 1;
  l->ldz = (m + 7) / 8 * 8;
  size_t off = 256;  // status word
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += up256(bytes);
    return at;
  };
  const size_t dz = static_cast<size_t>(T) * l->ldz * 2;
  l->scale = take(static_cast<size_t>(T) * 8);
  l->exponent = take(static_cast<size_t>(n / 128) * kSlabs * 4);
  l->hi = take(l->parts >= 1 ? dz : 0);
  l->lo = take(l->parts == 2 ? dz : 0);
  l->dx = take(act_order ? static_cast<size_t>(T) * n * 2 : 0);
  l->total = off;
  return true;
}

// Tiles of eight tokens in a segment; an expert with more tokens takes a second segment, which reads and
// unpacks its weights again.  (An expert gets a token at most once.)  Measured, 2 tiles against 4: 24
// tokens an expert 98 / 123 us (16 experts of 2048 x 1408), 12 tokens 259 / 306 (8 of 4096 x 11008), 32
// tokens 723 / 586 there; fewer registers and smaller stages let three blocks share an SM.
int moe_nt(int64_t T, int64_t E, int64_t top_k) { return T <= 8 ? 1 : T * top_k <= 28 * E ? 2 : 4; }
// Their ring: three blocks per SM by shared memory where registers allow it, and the next launch's blocks
// find room early (33 tokens over 64 experts: 123 us against 140 with two), else the deepest that two
// hold (one token over 32 experts: 25.3 us against 26.0).
int moe_ring(int64_t T, int nt) { return T <= 8 || nt == 4 ? DEC_SMEM : 66 * 1024; }
// Blocks of the down product: clusters of `cluster` over the list of (segment, chunk), `splits` of them.
struct DownSplit {
  int cluster, splits;
};
DownSplit down_split(int64_t H, int64_t I, int64_t experts) {
  DownSplit d;
  const int tiles = static_cast<int>(H / DEC_ROWS), chunks = static_cast<int>(experts * (I / 128));
  d.cluster = k_split(tiles, chunks);
  d.splits = std::max(1, std::min(2 * kSms / (tiles * d.cluster), chunks / (4 * d.cluster)));
  return d;
}

struct MoeLayout {
  int max_segments, max_tiles;
  DownSplit down;
  size_t logits, bounds, ids, weights, segments, tiles, expert, begin, count, tile0, high, tile_seg, pair, pweight, x, h, h_high,
      partial, tickets, total;
};
bool moe_layout(int64_t T, int64_t E, int64_t top_k, int64_t H, int64_t I, MoeLayout* l) {
  if (T < 0 || T > MOE_MAX_T || E < 1 || E > MOE_MAX_E || top_k < 1 || top_k > E || top_k > MOE_MAX_TOPK ||
      !valid_width(H) || !valid_width(I))
    return false;
  size_t off = 256;  // status word
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += up256(bytes);
    return at;
  };
  const int64_t pairs = T * top_k;
  // experts with a token, and what more than one segment (tile) of an expert adds
  l->max_segments = static_cast<int>(std::min(pairs, std::min(E, pairs) + pairs / (8 * moe_nt(T, E, top_k))));
  l->max_tiles = static_cast<int>(std::min(pairs, std::min(E, pairs) + pairs / 8));
  l->logits = take(static_cast<size_t>(T) * E * 8);
  l->bounds = take(static_cast<size_t>(T) * E * 4);
  l->ids = take(pairs * 4);
  l->weights = take(pairs * 4);
  l->segments = take(4);
  l->tiles = take(4);
  l->expert = take(l->max_segments * 4);
  l->begin = take(l->max_segments * 4);
  l->count = take(l->max_segments * 4);
  l->tile0 = take(l->max_segments * 4);
  l->high = take(l->max_segments * 4);
  l->tile_seg = take(l->max_tiles * 4);
  l->pair = take(pairs * 4);
  l->pweight = take(pairs * 4);
  l->x = take(static_cast<size_t>(l->max_tiles) * (H / 128) * FRAG_BYTES);
  l->h = take(static_cast<size_t>(l->max_tiles) * (I / 128) * FRAG_BYTES);
  l->h_high = take(static_cast<size_t>(l->max_tiles) * (I / 128) * FRAG_BYTES);
  l->down = down_split(H, I, std::max<int64_t>(1, std::min(E, pairs)));
  l->partial = take(l->down.splits > 1 ? static_cast<size_t>(l->down.splits) * T * H * 4 : 0);
  l->tickets = take(l->down.splits > 1 ? static_cast<size_t>(H / DEC_ROWS) * l->down.cluster * 4 : 0);
  l->total = off;
  return true;
}

}  // namespace

extern "C" size_t gptq_dequant_linear_workspace_bytes(int64_t T, int64_t n, int act_order) {
  if (T < 0 || T > kPackedMaxT || !valid_width(n)) return 0;
  return linear_workspace(T, n, act_order);
}

extern "C" gptq_status gptq_dequant_linear(const gptq_linear_args* args, int device, void* cuda_stream) {
  if (!args) return GPTQ_ERR_ARG;
  const gptq_linear_args& a = *args;
  if (a.T < 0 || a.T > kPackedMaxT || !valid_packed(a.W)) return GPTQ_ERR_ARG;
  if (a.dtype != GPTQ_FP16 && a.dtype != GPTQ_BF16) return GPTQ_ERR_ARG;
  if (a.act < GPTQ_ACT_NONE || a.act > GPTQ_ACT_SILU || (a.y_fp32 != 0 && a.y_fp32 != 1)) return GPTQ_ERR_ARG;
  if (a.T == 0) return GPTQ_OK;
  if (!a.X || !a.Y || !a.workspace) return GPTQ_ERR_ARG;
  if (!aligned16(a.X) || a.ld_x < a.W.n || a.ld_x % 8 || !aligned256(a.workspace)) return GPTQ_ERR_ARG;
  if (a.ld_y < a.W.m || !aligned_to(a.Y, a.y_fp32 ? 4 : 2) || !aligned_to(a.bias, 2) || !aligned_to(a.preact, 2))
    return GPTQ_ERR_ARG;
  if (a.residual && (a.ld_res < a.W.m || !aligned_to(a.residual, 2))) return GPTQ_ERR_ARG;
  if (a.workspace_bytes < linear_workspace(a.T, a.W.n, a.W.perm ? 1 : 0)) return GPTQ_ERR_ARG;
  {
    // outputs against inputs and each other; Y may take the residual's place
    const int64_t ys = a.y_fp32 ? 4 : 2, yw = a.W.m * ys, w = a.W.m * 2;
    const bool in_place = a.residual == a.Y && !a.y_fp32 && (a.ld_res == a.ld_y || a.T == 1);
    if (overlap(a.X, a.ld_x * 2, a.W.n * 2, a.Y, a.ld_y * ys, yw, a.T) ||
        overlap(a.X, a.ld_x * 2, a.W.n * 2, a.preact, w, w, a.T) ||
        overlap(a.preact, w, w, a.Y, a.ld_y * ys, yw, a.T) ||
        overlap(a.preact, w, w, a.residual, a.ld_res * 2, w, a.T) ||
        (!in_place && overlap(a.residual, a.ld_res * 2, w, a.Y, a.ld_y * ys, yw, a.T)))
      return GPTQ_ERR_ARG;
  }
  const gptq_status ds = check_device(device);
  if (ds != GPTQ_OK) return ds;
  DeviceGuard dg(device);
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  const int n = static_cast<int>(a.W.n), T = static_cast<int>(a.T), m = static_cast<int>(a.W.m);
  const int g = group_width(a.W);
  const uint16_t* X = static_cast<const uint16_t*>(a.X);
  int64_t ldx = a.ld_x;
  if (T > kDecodeTokens) {
    if (a.W.perm) {
      uint16_t* xs = reinterpret_cast<uint16_t*>(ws + 256);
      const bool pair = n * 4 <= kGatherPairBytes;
      static std::atomic<uint64_t> done[2];
      const auto kernel = pair ? gather_x_kernel<true> : gather_x_kernel<false>;
      CK(raise_smem_limit(done[pair], device, kernel, pair ? kGatherPairBytes : static_cast<int>(kPackedMaxN) * 2));
      // rows of a block: as many as 64 KB hold, while the blocks still fill the GPU
      int rows = std::max(1, std::min(32768 / n, T / (4 * kSms)));
      if (pair) rows = std::max(2, rows / 2 * 2);
      CK(launch_pdl(kernel, dim3((T + rows - 1) / rows), dim3(512), static_cast<size_t>(rows) * n * 2, 1, st, X, ldx, T, n,
                    a.W.perm, rows, xs));
      X = xs;
      ldx = n;
    }
    return linear_many_tokens(a, X, ldx, device, st);
  }
  LinearDecodeArgs d;
  d.T = T;
  d.tiles = (T + 7) / 8;
  d.m = m;
  d.chunks = n / 128;
  d.G = n / g;
  d.vec = param_vec(a.W);
  d.gi = group_index(g);
  d.scales = a.W.scales;
  d.zeros = a.W.zeros;
  d.bias = static_cast<const uint16_t*>(a.bias);
  d.residual = static_cast<const uint16_t*>(a.residual);
  d.ld_res = a.ld_res;
  d.ldy = a.ld_y;
  d.Y = a.Y;
  d.preact = static_cast<uint16_t*>(a.preact);
  d.act = a.act;
  d.y_fp32 = a.y_fp32;
  d.status = reinterpret_cast<int*>(ws);
  d.x = ws + 256;
  DecodeLaunch l;
  l.bf16 = a.dtype == GPTQ_BF16;
  l.unit = std::min(g, 128);
  l.nt = d.tiles;
  l.ring = DEC_SMEM;
  l.cluster = k_split((m + DEC_ROWS - 1) / DEC_ROWS, d.chunks);
  l.device = device;
  l.stream = st;
  l.chunks = (d.chunks + l.cluster - 1) / l.cluster;
  l.local = lay_out_locally(T, a.W.perm != nullptr, l.chunks) ? T : 0;
  d.X = X;
  d.ldx = ldx;
  d.perm = a.W.perm;
  CUtensorMap cmap;
  const gptq_status s = encode_codes(&cmap, a.W, 64);
  if (s != GPTQ_OK) return s;
  if (!l.local)
    CK(launch_pdl(fragment_kernel, dim3(d.chunks, d.tiles), dim3(128), 0, 1, st, X, ldx, T, l.unit, a.W.perm,
                reinterpret_cast<uint4*>(ws + 256), d.status));
  CK(by_bits(a.W.qp.bits, [&](auto b) { return launch_linear_decode<decltype(b)::value>(l, cmap, d); }));
  return GPTQ_OK;
}

extern "C" size_t gptq_dequant_linear_backward_workspace_bytes(int64_t T, int64_t m, int64_t n, int act_order,
                                                               int dtype, int act) {
  GradLayout l;
  return grad_layout(T, m, n, act_order, dtype, act, false, &l) ? l.total : 0;
}

extern "C" gptq_status gptq_dequant_linear_backward(const gptq_linear_grad_args* args, int device,
                                                    void* cuda_stream) {
  if (!args) return GPTQ_ERR_ARG;
  const gptq_linear_grad_args& a = *args;
  GradLayout need, lay;
  if (!valid_packed(a.W) || !grad_layout(a.T, a.W.m, a.W.n, a.W.perm ? 1 : 0, a.dtype, a.act, false, &need))
    return GPTQ_ERR_ARG;
  if (a.T > 0 && !a.dX && !a.dbias) return GPTQ_ERR_ARG;  // (an empty dX may have no address)
  if (!aligned_to(a.dbias, 4) || (a.T > 0 && a.ld_dy < a.W.m) || (a.T > 0 && a.dX && a.ld_dx < a.W.n) ||
      !aligned_to(a.dX, 2))
    return GPTQ_ERR_ARG;
  if (a.T > 0 && (!a.dY || !aligned_to(a.dY, 2) || !a.workspace || !aligned256(a.workspace) ||
                  a.workspace_bytes < need.total))
    return GPTQ_ERR_ARG;
  if (a.T > 0 && a.act != GPTQ_ACT_NONE && (!a.preact || !aligned_to(a.preact, 2))) return GPTQ_ERR_ARG;
  if (a.T > 0 && (overlap(a.dY, a.ld_dy * 2, a.W.m * 2, a.dX, a.ld_dx * 2, a.W.n * 2, a.T) ||
                  (a.act != GPTQ_ACT_NONE &&
                   overlap(a.preact, a.W.m * 2, a.W.m * 2, a.dX, a.ld_dx * 2, a.W.n * 2, a.T))))
    return GPTQ_ERR_ARG;
  if (a.T == 0 && !a.dbias) return GPTQ_OK;
  const gptq_status ds = check_device(device);
  if (ds != GPTQ_OK) return ds;
  DeviceGuard dg(device);
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if (a.T == 0) {
    CK(cudaMemsetAsync(a.dbias, 0, static_cast<size_t>(a.W.m) * 4, st));
    return GPTQ_OK;
  }
  const bool bf = a.dtype == GPTQ_BF16;
  const int T = static_cast<int>(a.T), m = static_cast<int>(a.W.m), n = static_cast<int>(a.W.n);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  const uint16_t* dY = static_cast<const uint16_t*>(a.dY);
  const uint16_t* Z = a.act == GPTQ_ACT_NONE ? nullptr : static_cast<const uint16_t*>(a.preact);
  const int vec = a.ld_dy % 8 == 0 && aligned16(dY) && (!Z || (m % 8 == 0 && aligned16(Z)));
  // dY is the operand itself when it is fp16, nothing is to be multiplied and TMA can read it
  const bool direct = aligned16(dY) && a.ld_dy % 8 == 0;
  grad_layout(a.T, m, n, a.W.perm ? 1 : 0, a.dtype, a.act, direct, &lay);
  if (a.dbias)
    CK(by_act(a.act, [&](auto k) {
      constexpr int A = decltype(k)::value;
      return launch_pdl(bf ? dbias_kernel<true, A> : dbias_kernel<false, A>,
                        dim3((m + DBIAS_COLS - 1) / DBIAS_COLS * DBIAS_CLUSTER), dim3(DBIAS_WARPS * 32), 0, DBIAS_CLUSTER,
                        st, dY, a.ld_dy, Z, T, m, vec, a.dbias,
                        reinterpret_cast<int*>(ws));
    }));
  if (!a.dX) return GPTQ_OK;
  const int g = group_width(a.W);
  const uint16_t *hi = dY, *lo = dY;
  int64_t ldz = a.ld_dy;
  SlabArgs w;
  w.scales = a.W.scales;
  w.G = n / g;
  w.per = g >= 128 ? 1 : 128 / g;
  w.bits = a.W.qp.bits;
  w.chunks = n / 128;
  w.slabs = static_cast<int>(std::min<int64_t>({kSlabs, m, (a.W.m * w.G + 4095) / 4096}));
  w.gi = group_index(g);
  w.exponent = reinterpret_cast<int*>(ws + lay.exponent);
  {
    uint16_t* h = lay.parts >= 1 ? reinterpret_cast<uint16_t*>(ws + lay.hi) : nullptr;
    uint16_t* o = lay.parts == 2 ? reinterpret_cast<uint16_t*>(ws + lay.lo) : nullptr;
    CK(by_act(a.act, [&](auto k) {
      constexpr int A = decltype(k)::value;
      const auto kernel = bf ? (m <= 4096 ? act_grad_kernel<true, A, 1> : act_grad_kernel<true, A, 3>)
                             : (m <= 4096 ? act_grad_kernel<false, A, 1> : act_grad_kernel<false, A, 3>);
      return launch_pdl(kernel, dim3(w.slabs + (h ? T : 0)), dim3(512), 0, 1, st, dY, a.ld_dy, Z, m, vec, h, o,
                        lay.ldz, reinterpret_cast<float2*>(ws + lay.scale), w);
    }));
    if (h) {
      ldz = lay.ldz;
      hi = h;
      lo = o ? o : h;
    }
  }
  LinearTcArgs d = {};
  d.T = T;
  d.m = m;
  d.chunks = (m + 127) / 128;
  d.G = n / g;
  d.gi = group_index(g);
  d.tn = T <= 32 ? 32 : T <= 64 ? 64 : TC_MAX_TN;
  d.scales = a.W.scales;
  d.zeros = a.W.zeros;
  d.status = reinterpret_cast<int*>(ws);
  GradOut go;
  go.token_scale = lay.parts >= 1 ? reinterpret_cast<const float2*>(ws + lay.scale) : nullptr;
  go.exponent = reinterpret_cast<const int*>(ws + lay.exponent);
  go.dX = a.W.perm ? reinterpret_cast<uint16_t*>(ws + lay.dx) : static_cast<uint16_t*>(a.dX);
  go.lddx = a.W.perm ? n : a.ld_dx;
  go.n = n;
  go.vec = go.lddx % 4 == 0 && aligned_to(go.dX, 8);
  go.slabs = w.slabs;
  const int parts = std::max(1, lay.parts);
  CUtensorMap cmap, hmap, lmap;
  gptq_status s = encode_codes(&cmap, a.W, TC_BM);
  if (s == GPTQ_OK) s = encode_act(&hmap, GPTQ_FP16, hi, m, T, ldz, d.tn);
  if (s == GPTQ_OK) s = encode_act(&lmap, GPTQ_FP16, lo, m, T, ldz, d.tn);
  if (s != GPTQ_OK) return s;
  TcLaunch l;
  l.bf16 = bf;
  l.unit = std::min(g, 128);
  l.sms = kSms;
  l.device = device;
  l.stream = st;
  if (use_pairs(n, T)) {
    PairArgs p = {};
    p.tiles_m = (n + 255) / 256;
    p.tiles_t = (T + PR_TN - 1) / PR_TN;
    p.chunks = d.chunks;
    p.steps = parts * d.chunks;
    p.lin = d;
    p.go = go;
    CK(by_bits(a.W.qp.bits,
               [&](auto b) { return launch_packed_pair<decltype(b)::value>(l, true, cmap, hmap, lmap, p); }));
  } else {
    l.cluster = tc_cluster(static_cast<int64_t>(n / 128) * ((T + d.tn - 1) / d.tn), d.chunks);
    CK(by_bits(a.W.qp.bits,
               [&](auto b) { return launch_packed_tc<decltype(b)::value>(l, true, cmap, hmap, lmap, d, go, parts); }));
  }
  if (a.W.perm) {
    static std::atomic<uint64_t> done{0};
    CK(raise_smem_limit(done, device, unpermute_kernel, static_cast<int>(kPackedMaxN) * 2));
    CK(launch_pdl(unpermute_kernel, dim3(T), dim3(256), static_cast<size_t>(n) * 2, 1, st,
                  static_cast<const uint16_t*>(go.dX), n, a.W.perm, static_cast<uint16_t*>(a.dX), a.ld_dx));
  }
  return GPTQ_OK;
}

extern "C" size_t gptq_dequant_moe_workspace_bytes(int64_t T, int64_t E, int top_k, int64_t H, int64_t I) {
  MoeLayout l;
  return moe_layout(T, E, top_k, H, I, &l) ? l.total : 0;
}

extern "C" gptq_status gptq_dequant_moe(const gptq_moe_args* args, int device, void* cuda_stream) {
  if (!args) return GPTQ_ERR_ARG;
  const gptq_moe_args& a = *args;
  const int64_t H = a.gate_up.n, I = a.down.n;
  MoeLayout lay;
  if (!valid_packed(a.gate_up) || !valid_packed(a.down) || a.gate_up.m != 2 * I || a.down.m != H || a.down.perm ||
      a.gate_up.qp.bits != a.down.qp.bits)
    return GPTQ_ERR_ARG;
  if (!moe_layout(a.T, a.E, a.top_k, H, I, &lay) || 2 * I * a.E > INT32_MAX || H * a.E > INT32_MAX) return GPTQ_ERR_ARG;
  if ((a.dtype != GPTQ_FP16 && a.dtype != GPTQ_BF16) || (a.renormalize != 0 && a.renormalize != 1) ||
      a.act < GPTQ_ACT_NONE || a.act > GPTQ_ACT_SILU)
    return GPTQ_ERR_ARG;
  if (a.T == 0) return GPTQ_OK;
  if (!a.X || !a.router || !a.Y || !a.workspace) return GPTQ_ERR_ARG;
  if (!aligned16(a.X) || a.ld_x < H || a.ld_x % 8 || !aligned16(a.router) || !aligned256(a.workspace))
    return GPTQ_ERR_ARG;
  if (a.ld_y < H || !aligned_to(a.Y, 2) || (a.residual && (a.ld_res < H || !aligned_to(a.residual, 2))) ||
      !aligned_to(a.ids_out, 4) || !aligned_to(a.weights_out, 4))
    return GPTQ_ERR_ARG;
  if (a.workspace_bytes < lay.total) return GPTQ_ERR_ARG;
  // (X is read before the last launch writes Y; the residual beside it)
  if (!(a.residual == a.Y && (a.ld_res == a.ld_y || a.T == 1)) &&
      overlap(a.residual, a.ld_res * 2, H * 2, a.Y, a.ld_y * 2, H * 2, a.T))
    return GPTQ_ERR_ARG;
  const gptq_status ds = check_device(device);
  if (ds != GPTQ_OK) return ds;
  DeviceGuard dg(device);
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  const bool bf = a.dtype == GPTQ_BF16;
  const int pairs = static_cast<int>(a.T) * a.top_k;

  RouterArgs r;
  r.X = static_cast<const uint16_t*>(a.X);
  r.ldx = a.ld_x;
  r.R = static_cast<const uint16_t*>(a.router);
  r.T = static_cast<int>(a.T);
  r.E = static_cast<int>(a.E);
  r.H = static_cast<int>(H);
  r.top_k = a.top_k;
  r.renorm = a.renormalize;
  r.seg_pairs = 8 * moe_nt(a.T, a.E, a.top_k);
  r.logits = reinterpret_cast<double*>(ws + lay.logits);
  r.bounds = reinterpret_cast<float*>(ws + lay.bounds);
  r.ids = reinterpret_cast<int32_t*>(ws + lay.ids);
  r.weights = reinterpret_cast<float*>(ws + lay.weights);
  r.ids_out = a.ids_out;
  r.weights_out = a.weights_out;
  r.plan.segments = reinterpret_cast<int*>(ws + lay.segments);
  r.plan.tiles = reinterpret_cast<int*>(ws + lay.tiles);
  r.plan.expert = reinterpret_cast<int*>(ws + lay.expert);
  r.plan.begin = reinterpret_cast<int*>(ws + lay.begin);
  r.plan.count = reinterpret_cast<int*>(ws + lay.count);
  r.plan.tile0 = reinterpret_cast<int*>(ws + lay.tile0);
  r.plan.high = reinterpret_cast<int*>(ws + lay.high);
  r.plan.tile_seg = reinterpret_cast<int*>(ws + lay.tile_seg);
  r.plan.pair = reinterpret_cast<int*>(ws + lay.pair);
  r.plan.weight = reinterpret_cast<float*>(ws + lay.pweight);
  r.tickets = reinterpret_cast<int*>(ws + lay.tickets);
  r.ntickets = lay.down.splits > 1 ? static_cast<int>(H / DEC_ROWS) * lay.down.cluster : 0;
  r.status = reinterpret_cast<int*>(ws);
  CUtensorMap gmap, dmap;
  gptq_status s = encode_codes(&gmap, a.gate_up, 64, a.E);
  if (s == GPTQ_OK) s = encode_codes(&dmap, a.down, 64, a.E);
  if (s != GPTQ_OK) return s;
  CK(launch_pdl(bf ? moe_router_kernel<true> : moe_router_kernel<false>, dim3(ROUTER_CLUSTER), dim3(ROUTER_WARPS * 32), 0,
                ROUTER_CLUSTER, st, r));

  const int gg = group_width(a.gate_up), gd = group_width(a.down);
  DecodeLaunch l;
  l.bf16 = bf;
  l.nt = moe_nt(a.T, a.E, a.top_k);
  l.ring = moe_ring(a.T, l.nt);
  l.device = device;
  l.stream = st;
  l.unit = std::min(gg, 128);
  l.cluster = k_split(I / 64 * std::min<int64_t>(a.E, pairs), r.H / 128);
  l.chunks = (r.H / 128 + l.cluster - 1) / l.cluster;
  l.local = lay_out_locally(a.T, a.gate_up.perm != nullptr, l.chunks) ? r.T : 0;
  if (!l.local)
    CK(launch_pdl(moe_fragment_kernel, dim3(static_cast<unsigned>(H / 128), lay.max_tiles), dim3(128), 0, 1, st, r.X,
                  a.ld_x, r.H, std::min(gg, 128), a.gate_up.perm, r.plan, a.top_k,
                  reinterpret_cast<uint4*>(ws + lay.x)));

  MoeArgs m;
  m.x = ws + lay.x;
  m.X = r.X;
  m.ldx = a.ld_x;
  m.perm = a.gate_up.perm;
  m.plan = r.plan;
  m.T = r.T;
  m.E = r.E;
  m.top_k = a.top_k;
  m.H = r.H;
  m.I = static_cast<int>(I);
  m.gu_scales = a.gate_up.scales;
  m.gu_zeros = a.gate_up.zeros;
  m.dn_scales = a.down.scales;
  m.dn_zeros = a.down.zeros;
  m.gu_G = m.H / gg;
  m.dn_G = m.I / gd;
  m.gu_vec = param_vec(a.gate_up);
  m.dn_vec = param_vec(a.down);
  m.gu_gi = group_index(gg);
  m.dn_gi = group_index(gd);
  m.act = a.act;
  m.dn_unit = std::min(gd, 128);
  m.h = ws + lay.h;
  m.h_high = ws + lay.h_high;
  m.status = r.status;
  m.splits = lay.down.splits;
  m.partial = reinterpret_cast<float*>(ws + lay.partial);
  m.tickets = r.tickets;
  m.residual = static_cast<const uint16_t*>(a.residual);
  m.ld_res = a.ld_res;
  m.ldy = a.ld_y;
  m.Y = static_cast<uint16_t*>(a.Y);
  CK(by_bits(a.gate_up.qp.bits,
             [&](auto b) { return launch_moe_gate_up<decltype(b)::value>(l, gmap, m, lay.max_segments); }));
  l.unit = m.dn_unit;
  l.local = 0;
  l.cluster = lay.down.cluster;
  CK(by_bits(a.down.qp.bits, [&](auto b) { return launch_moe_down<decltype(b)::value>(l, dmap, m); }));
  return GPTQ_OK;
}
