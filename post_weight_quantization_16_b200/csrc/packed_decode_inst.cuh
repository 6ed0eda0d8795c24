// packed_decode_inst.cuh — the decode kernels of one code width (PACKED_BITS).  Each width is a
// translation unit of its own so that they compile side by side.
#include "packed_decode.cuh"

namespace gptq {

namespace {
template <bool BF, int GU, int NT, int RT>
cudaError_t linear_of(const DecodeLaunch& l, const LinearDecodeArgs& a) {
  const dim3 grid(static_cast<unsigned>((a.m + 16 * RT - 1) / (16 * RT) * l.cluster),
                  static_cast<unsigned>((a.T + 8 * NT - 1) / (8 * NT)));
  return launch_pdl(linear_decode_kernel<PACKED_BITS, BF, GU, NT, RT>, grid, dim3(DEC_WARPS * 32), 0, l.cluster,
                    l.stream, a);
}
template <bool BF, int GU, int NT, int RT>
cudaError_t gate_up_of(const DecodeLaunch& l, const MoeArgs& a, int slots) {
  const dim3 grid(static_cast<unsigned>(a.I / (8 * RT)), static_cast<unsigned>(slots));
  return launch_pdl(moe_gate_up_kernel<PACKED_BITS, BF, GU, NT, RT>, grid, dim3(DEC_WARPS * 32), 0, 1, l.stream, a);
}
template <bool BF, int GU, int NT, int RT>
cudaError_t down_of(const DecodeLaunch& l, const MoeArgs& a) {
  static std::atomic<uint64_t> done{0};
  const auto kernel = moe_down_kernel<PACKED_BITS, BF, GU, NT, RT>;
  const cudaError_t e = raise_smem_limit(done, l.device, kernel, DEC_WARPS * MOE_MAX_T * 16 * RT * 4);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>((a.H + 16 * RT - 1) / (16 * RT) * l.cluster));
  return launch_pdl(kernel, grid, dim3(DEC_WARPS * 32), static_cast<size_t>(DEC_WARPS) * a.T * 16 * RT * 4, l.cluster,
                    l.stream, a);
}

template <bool BF, int GU, typename F>
cudaError_t by_tile(const DecodeLaunch& l, F&& f) {
  if (l.nt == 1) return f(std::integral_constant<bool, BF>(), std::integral_constant<int, GU>(),
                          std::integral_constant<int, 1>(), std::integral_constant<int, 1>());
  return f(std::integral_constant<bool, BF>(), std::integral_constant<int, GU>(), std::integral_constant<int, 2>(),
           std::integral_constant<int, 1>());
}
template <bool BF, typename F>
cudaError_t by_unit(const DecodeLaunch& l, F&& f) {
  if (l.unit == 32) return by_tile<BF, 32>(l, f);
  if (l.unit == 64) return by_tile<BF, 64>(l, f);
  return by_tile<BF, 128>(l, f);
}
template <typename F>
cudaError_t by_type(const DecodeLaunch& l, F&& f) {
  return l.bf16 ? by_unit<true>(l, f) : by_unit<false>(l, f);
}
}  // namespace

template <>
cudaError_t launch_linear_decode<PACKED_BITS>(const DecodeLaunch& l, const LinearDecodeArgs& a) {
  return by_type(l, [&](auto bf, auto gu, auto nt, auto rt) {
    return linear_of<decltype(bf)::value, decltype(gu)::value, decltype(nt)::value, decltype(rt)::value>(l, a);
  });
}
template <>
cudaError_t launch_moe_gate_up<PACKED_BITS>(const DecodeLaunch& l, const MoeArgs& a, int slots) {
  return by_type(l, [&](auto bf, auto gu, auto nt, auto rt) {
    return gate_up_of<decltype(bf)::value, decltype(gu)::value, decltype(nt)::value, decltype(rt)::value>(l, a, slots);
  });
}
template <>
cudaError_t launch_moe_down<PACKED_BITS>(const DecodeLaunch& l, const MoeArgs& a) {
  return by_type(l, [&](auto bf, auto gu, auto nt, auto rt) {
    return down_of<decltype(bf)::value, decltype(gu)::value, decltype(nt)::value, decltype(rt)::value>(l, a);
  });
}

}  // namespace gptq
