// packed_tc_inst.cuh — the tensor-core kernels of one code width (PACKED_BITS).
#include "packed_tc.cuh"

namespace gptq {

namespace {
template <bool BF, int GU, bool BWD>
cudaError_t tc_of(const TcLaunch& l, const CUtensorMap& codes, const CUtensorMap& x, const CUtensorMap& xlo,
                  const LinearTcArgs& a, const GradOut& go, int parts) {
  static std::atomic<uint64_t> done{0};
  const auto kernel = packed_tc_kernel<PACKED_BITS, BF, GU, BWD>;
  const cudaError_t e = raise_smem_limit(done, l.device, kernel, 227 * 1024);
  if (e != cudaSuccess) return e;
  const int tiles = BWD ? go.n / 128 : (a.m + TC_BM - 1) / TC_BM;
  const dim3 grid(static_cast<unsigned>(tiles * l.cluster), static_cast<unsigned>((a.T + a.tn - 1) / a.tn));
  return launch_pdl(kernel, grid, dim3(TC_THREADS), tc_smem_bytes(a.tn, PACKED_BITS), l.cluster, l.stream, codes, x, xlo,
                    a, go, parts);
}
template <bool BF, bool BWD>
cudaError_t by_unit(const TcLaunch& l, const CUtensorMap& codes, const CUtensorMap& x, const CUtensorMap& xlo,
                    const LinearTcArgs& a, const GradOut& go, int parts) {
  if (l.unit == 32) return tc_of<BF, 32, BWD>(l, codes, x, xlo, a, go, parts);
  if (l.unit == 64) return tc_of<BF, 64, BWD>(l, codes, x, xlo, a, go, parts);
  return tc_of<BF, 128, BWD>(l, codes, x, xlo, a, go, parts);
}
}  // namespace

template <>
cudaError_t launch_packed_tc<PACKED_BITS>(const TcLaunch& l, bool backward, const CUtensorMap& codes,
                                          const CUtensorMap& x, const CUtensorMap& xlo, const LinearTcArgs& a,
                                          const GradOut& go, int parts) {
  if (backward)
    return l.bf16 ? by_unit<true, true>(l, codes, x, xlo, a, go, parts)
                  : by_unit<false, true>(l, codes, x, xlo, a, go, parts);
  return l.bf16 ? by_unit<true, false>(l, codes, x, xlo, a, go, parts)
                : by_unit<false, false>(l, codes, x, xlo, a, go, parts);
}

}  // namespace gptq
