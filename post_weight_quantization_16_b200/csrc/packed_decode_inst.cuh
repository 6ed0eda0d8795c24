// packed_decode_inst.cuh — the decode kernels of one code width (PACKED_BITS).  Each width is a
// translation unit of its own so that they compile side by side.
#include "packed_decode.cuh"

namespace gptq {

namespace {
template <bool BF, int GU, int NT, bool XL>
struct Of {
  static constexpr int TILES = XL ? 0 : NT;  // of a stage
  static int smem(const DecodeLaunch& l) {
    return dec_ring_bytes(PACKED_BITS, TILES, l.ring) + (XL ? l.local * l.chunks * 256 : 0);
  }
  static constexpr int smem_limit = dec_ring_bytes(PACKED_BITS, TILES, DEC_SMEM) + (XL ? DEC_LOCAL_BYTES : 0);
  static cudaError_t linear(const DecodeLaunch& l, const CUtensorMap& codes, LinearDecodeArgs& a) {
    static std::atomic<uint64_t> done{0};
    const auto kernel = linear_decode_kernel<PACKED_BITS, BF, GU, NT, XL>;
    const cudaError_t e = raise_smem_limit(done, l.device, kernel, smem_limit);
    if (e != cudaSuccess) return e;
    a.stages = dec_stages(PACKED_BITS, TILES, l.ring);
    const dim3 grid(static_cast<unsigned>((a.m + DEC_ROWS - 1) / DEC_ROWS * l.cluster));
    return launch_pdl(kernel, grid, dim3(DEC_THREADS), smem(l), l.cluster, l.stream, codes, a);
  }
  static cudaError_t gate_up(const DecodeLaunch& l, const CUtensorMap& codes, MoeArgs& a, int segments) {
    static std::atomic<uint64_t> done{0};
    const auto kernel = moe_gate_up_kernel<PACKED_BITS, BF, GU, NT, XL>;
    const cudaError_t e = raise_smem_limit(done, l.device, kernel, smem_limit);
    if (e != cudaSuccess) return e;
    a.stages = dec_stages(PACKED_BITS, TILES, l.ring);
    const dim3 grid(static_cast<unsigned>(a.I / 64 * l.cluster), static_cast<unsigned>(segments));
    return launch_pdl(kernel, grid, dim3(DEC_THREADS), smem(l), l.cluster, l.stream, codes, a);
  }
  static cudaError_t down(const DecodeLaunch& l, const CUtensorMap& codes, MoeArgs& a) {
    static std::atomic<uint64_t> done{0};
    const auto kernel = moe_down_kernel<PACKED_BITS, BF, GU, NT>;
    const cudaError_t e = raise_smem_limit(done, l.device, kernel, smem_limit + MOE_MAX_T * DEC_ROWS * 4);
    if (e != cudaSuccess) return e;
    a.stages = dec_stages(PACKED_BITS, NT, l.ring);
    const dim3 grid(static_cast<unsigned>(a.H / DEC_ROWS * l.cluster), static_cast<unsigned>(a.splits));
    return launch_pdl(kernel, grid, dim3(DEC_THREADS), static_cast<size_t>(smem(l)) + static_cast<size_t>(a.T) * DEC_ROWS * 4,
                      l.cluster, l.stream, codes, a);
  }
};

enum Op { LINEAR, GATE_UP, DOWN };
template <Op OP, bool BF, int GU, typename F>
cudaError_t by_tiles(const DecodeLaunch& l, F&& f) {
  if constexpr (OP != DOWN)
    if (l.local) return f(Of<BF, GU, 1, true>());
  if constexpr (OP != LINEAR)  // (a segment of an expert has up to 32 tokens, the linear decode kernel 16)
    if (l.nt == 4) return f(Of<BF, GU, 4, false>());
  if (l.nt == 1) return f(Of<BF, GU, 1, false>());
  return f(Of<BF, GU, 2, false>());
}
template <Op OP, bool BF, typename F>
cudaError_t by_unit(const DecodeLaunch& l, F&& f) {
  if (l.unit == 32) return by_tiles<OP, BF, 32>(l, f);
  if (l.unit == 64) return by_tiles<OP, BF, 64>(l, f);
  return by_tiles<OP, BF, 128>(l, f);
}
template <Op OP, typename F>
cudaError_t by_type(const DecodeLaunch& l, F&& f) {
  return l.bf16 ? by_unit<OP, true>(l, f) : by_unit<OP, false>(l, f);
}
}  // namespace

template <>
cudaError_t launch_linear_decode<PACKED_BITS>(const DecodeLaunch& l, const CUtensorMap& codes, LinearDecodeArgs& a) {
  return by_type<LINEAR>(l, [&](auto of) { return decltype(of)::linear(l, codes, a); });
}
template <>
cudaError_t launch_moe_gate_up<PACKED_BITS>(const DecodeLaunch& l, const CUtensorMap& codes, MoeArgs& a, int segments) {
  return by_type<GATE_UP>(l, [&](auto of) { return decltype(of)::gate_up(l, codes, a, segments); });
}
template <>
cudaError_t launch_moe_down<PACKED_BITS>(const DecodeLaunch& l, const CUtensorMap& codes, MoeArgs& a) {
  return by_type<DOWN>(l, [&](auto of) { return decltype(of)::down(l, codes, a); });
}

}  // namespace gptq
