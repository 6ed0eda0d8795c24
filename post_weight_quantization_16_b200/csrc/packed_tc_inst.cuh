// packed_tc_inst.cuh — the tensor-core kernels of one code width (PACKED_BITS).
#include "packed_tc.cuh"

namespace gptq {

namespace {
template <bool BF, int GU>
cudaError_t linear_tc_of(const TcLaunch& l, const CUtensorMap& codes, const CUtensorMap& x, const LinearTcArgs& a) {
  static std::atomic<uint64_t> done{0};
  const auto kernel = linear_tc_kernel<PACKED_BITS, BF, GU>;
  const cudaError_t e = raise_smem_limit(done, l.device, kernel, TC_SMEM_BUDGET);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>((a.m + TC_BM - 1) / TC_BM * l.cluster),
                  static_cast<unsigned>((a.T + a.tn - 1) / a.tn));
  return launch_pdl(kernel, grid, dim3(TC_THREADS), tc_smem_bytes(a.tn, PACKED_BITS), l.cluster, l.stream, codes, x, a);
}
template <int GU>
cudaError_t linear_bwd_of(const TcLaunch& l, const CUtensorMap& codes, const CUtensorMap& dz, const CUtensorMap& dz_lo,
                          const LinearBwdArgs& a) {
  static std::atomic<uint64_t> done{0};
  const auto kernel = linear_bwd_tc_kernel<PACKED_BITS, GU>;
  const cudaError_t e = raise_smem_limit(done, l.device, kernel, TC_SMEM_BUDGET);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(a.n / 128 * l.cluster), static_cast<unsigned>((a.T + a.tn - 1) / a.tn));
  return launch_pdl(kernel, grid, dim3(BW_THREADS), bw_smem_bytes(a.tn, PACKED_BITS, a.parts), l.cluster, l.stream,
                    codes, dz, dz_lo, a);
}
}  // namespace

template <>
cudaError_t launch_linear_tc<PACKED_BITS>(const TcLaunch& l, const CUtensorMap& codes, const CUtensorMap& x,
                                          const LinearTcArgs& a) {
  if (l.bf16) {
    if (l.unit == 32) return linear_tc_of<true, 32>(l, codes, x, a);
    if (l.unit == 64) return linear_tc_of<true, 64>(l, codes, x, a);
    return linear_tc_of<true, 128>(l, codes, x, a);
  }
  if (l.unit == 32) return linear_tc_of<false, 32>(l, codes, x, a);
  if (l.unit == 64) return linear_tc_of<false, 64>(l, codes, x, a);
  return linear_tc_of<false, 128>(l, codes, x, a);
}

template <>
cudaError_t launch_linear_bwd_tc<PACKED_BITS>(const TcLaunch& l, const CUtensorMap& codes, const CUtensorMap& dz,
                                              const CUtensorMap& dz_lo, const LinearBwdArgs& a) {
  if (l.unit == 32) return linear_bwd_of<32>(l, codes, dz, dz_lo, a);
  if (l.unit == 64) return linear_bwd_of<64>(l, codes, dz, dz_lo, a);
  return linear_bwd_of<128>(l, codes, dz, dz_lo, a);
}

}  // namespace gptq
