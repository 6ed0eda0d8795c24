// packed_decode_inst.cuh — the decode kernels of one code width (PACKED_BITS).  Each width is a
// translation unit of its own so that they compile side by side.
#include "packed_decode.cuh"

namespace gptq {

namespace {
template <bool BF, int GU, int NT, bool XL>
struct Of {
  static int smem(const DecodeLaunch& l) {
    return XL ? dec_ring_bytes(PACKED_BITS, 0) + l.local * l.chunks * 256 : dec_ring_bytes(PACKED_BITS, NT);
  }
  static constexpr int smem_limit = XL ? dec_ring_bytes(PACKED_BITS, 0) + DEC_LOCAL_BYTES : dec_ring_bytes(PACKED_BITS, NT);
  static cudaError_t linear(const DecodeLaunch& l, const CUtensorMap& codes, const LinearDecodeArgs& a) {
    static std::atomic<uint64_t> done{0};
    const auto kernel = linear_decode_kernel<PACKED_BITS, BF, GU, NT, XL>;
    const cudaError_t e = raise_smem_limit(done, l.device, kernel, smem_limit);
    if (e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>((a.m + DEC_ROWS - 1) / DEC_ROWS * l.cluster));
    return launch_pdl(kernel, grid, dim3(DEC_THREADS), smem(l), l.cluster, l.stream, codes, a);
  }
  static cudaError_t gate_up(const DecodeLaunch& l, const CUtensorMap& codes, const MoeArgs& a, int segments) {
    static std::atomic<uint64_t> done{0};
    const auto kernel = moe_gate_up_kernel<PACKED_BITS, BF, GU, NT, XL>;
    const cudaError_t e = raise_smem_limit(done, l.device, kernel, smem_limit);
    if (e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>(a.I / 64 * l.cluster), static_cast<unsigned>(segments));
    return launch_pdl(kernel, grid, dim3(DEC_THREADS), smem(l), l.cluster, l.stream, codes, a);
  }
  static cudaError_t down(const DecodeLaunch& l, const CUtensorMap& codes, const MoeArgs& a) {
    static std::atomic<uint64_t> done{0};
    const auto kernel = moe_down_kernel<PACKED_BITS, BF, GU, NT>;
    const int ring = dec_ring_bytes(PACKED_BITS, NT);
    const cudaError_t e = raise_smem_limit(done, l.device, kernel, ring + MOE_MAX_T * DEC_ROWS * 4);
    if (e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>(a.H / DEC_ROWS * l.cluster));
    return launch_pdl(kernel, grid, dim3(DEC_THREADS), static_cast<size_t>(ring) + static_cast<size_t>(a.T) * DEC_ROWS * 4,
                      l.cluster, l.stream, codes, a);
  }
};

template <bool MOE, bool BF, int GU, typename F>
cudaError_t by_tiles(const DecodeLaunch& l, F&& f) {
  if (l.local) return f(Of<BF, GU, 1, true>());
  if (l.nt == 1) return f(Of<BF, GU, 1, false>());
  if constexpr (MOE)  // (a segment of an expert has up to 32 tokens, the linear decode kernel 16)
    if (l.nt == 4) return f(Of<BF, GU, 4, false>());
  return f(Of<BF, GU, 2, false>());
}
template <bool MOE, bool BF, typename F>
cudaError_t by_unit(const DecodeLaunch& l, F&& f) {
  if (l.unit == 32) return by_tiles<MOE, BF, 32>(l, f);
  if (l.unit == 64) return by_tiles<MOE, BF, 64>(l, f);
  return by_tiles<MOE, BF, 128>(l, f);
}
template <bool MOE, typename F>
cudaError_t by_type(const DecodeLaunch& l, F&& f) {
  return l.bf16 ? by_unit<MOE, true>(l, f) : by_unit<MOE, false>(l, f);
}
}  // namespace

template <>
cudaError_t launch_linear_decode<PACKED_BITS>(const DecodeLaunch& l, const CUtensorMap& codes,
                                              const LinearDecodeArgs& a) {
  return by_type<false>(l, [&](auto of) { return decltype(of)::linear(l, codes, a); });
}
template <>
cudaError_t launch_moe_gate_up<PACKED_BITS>(const DecodeLaunch& l, const CUtensorMap& codes, const MoeArgs& a,
                                            int segments) {
  return by_type<true>(l, [&](auto of) { return decltype(of)::gate_up(l, codes, a, segments); });
}
template <>
cudaError_t launch_moe_down<PACKED_BITS>(const DecodeLaunch& l, const CUtensorMap& codes, const MoeArgs& a) {
  return by_type<true>(l, [&](auto of) { return decltype(of)::down(l, codes, a); });
}

}  // namespace gptq
