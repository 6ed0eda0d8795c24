// packed_pair_inst.cuh — the CTA-pair kernels of one code width (PACKED_BITS).
#include "packed_pair.cuh"

namespace gptq {

namespace {
template <bool BF, int GU, bool BWD>
cudaError_t pair_of(const TcLaunch& l, const CUtensorMap& codes, const CUtensorMap& x, const CUtensorMap& xlo,
                    const PairArgs& a) {
  static std::atomic<uint64_t> done{0};
  const auto kernel = packed_pair_kernel<PACKED_BITS, BF, GU, BWD>;
  const cudaError_t e = raise_smem_limit(done, l.device, kernel, pr_smem_bytes(PACKED_BITS));
  if (e != cudaSuccess) return e;
  // the clusters take tiles in turn; as many as the SM pairs, spread evenly over the rounds
  const int tiles = a.tiles_m * a.tiles_t, pairs = l.sms / 2, rounds = (tiles + pairs - 1) / pairs;
  const dim3 grid(static_cast<unsigned>(2 * ((tiles + rounds - 1) / rounds)));
  return launch_pdl(kernel, grid, dim3(PR_THREADS), pr_smem_bytes(PACKED_BITS), 1, l.stream, codes, x, xlo, a);
}
template <bool BF, bool BWD>
cudaError_t by_unit(const TcLaunch& l, const CUtensorMap& codes, const CUtensorMap& x, const CUtensorMap& xlo,
                    const PairArgs& a) {
  if (l.unit == 32) return pair_of<BF, 32, BWD>(l, codes, x, xlo, a);
  if (l.unit == 64) return pair_of<BF, 64, BWD>(l, codes, x, xlo, a);
  return pair_of<BF, 128, BWD>(l, codes, x, xlo, a);
}
}  // namespace

template <>
cudaError_t launch_packed_pair<PACKED_BITS>(const TcLaunch& l, bool backward, const CUtensorMap& codes,
                                            const CUtensorMap& x, const CUtensorMap& xlo, const PairArgs& a) {
  if (backward)
    return l.bf16 ? by_unit<true, true>(l, codes, x, xlo, a) : by_unit<false, true>(l, codes, x, xlo, a);
  return l.bf16 ? by_unit<true, false>(l, codes, x, xlo, a) : by_unit<false, false>(l, codes, x, xlo, a);
}

}  // namespace gptq
