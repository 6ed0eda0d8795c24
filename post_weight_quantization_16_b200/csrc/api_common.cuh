// api_common.cuh — helpers shared by the translation units that implement the C ABI: error
// mapping, the device guard, argument checks and the tensor-map encoder.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <mutex>

#include "../../include/gptq.h"

namespace gptq {

inline gptq_status cuda_fail(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return GPTQ_OK;
  if (std::getenv("GPTQ_VERBOSE")) std::fprintf(stderr, "gptq: %s: %s\n", what, cudaGetErrorString(e));
  return GPTQ_ERR_CUDA;
}
#define CK(call)                                         \
  do {                                                   \
    gptq_status _s = cuda_fail((call), #call);           \
    if (_s != GPTQ_OK) return _s;                        \
  } while (0)
#define CKL(what) CK(cudaGetLastError())

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Makes `dev` the calling thread's device until the end of the scope.  The device is set also where it
// is the current one already: on a host thread that has not used CUDA yet it is that call that binds
// the device's context, and encoding a tensor map, the first thing some entry points do, needs one.
class DeviceGuard {
 public:
  explicit DeviceGuard(int dev) : dev_(dev) {
    cudaGetDevice(&prev_);
    cudaSetDevice(dev_);
  }
  ~DeviceGuard() {
    if (prev_ != dev_) cudaSetDevice(prev_);
  }

 private:
  int dev_, prev_ = 0;
};

inline int64_t env_int(const char* name, int64_t dflt) {
  const char* v = std::getenv(name);
  if (!v || !*v) return dflt;
  return std::strtoll(v, nullptr, 10);
}

inline PFN_cuTensorMapEncodeTiled_v12000 get_encode() {
  static PFN_cuTensorMapEncodeTiled_v12000 cached = nullptr;
  static std::mutex mu;
  std::lock_guard<std::mutex> lk(mu);
  if (cached) return cached;
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess)
    return nullptr;
  cached = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  return cached;
}

inline bool valid_qparams(const gptq_qparams& qp, int64_t n) {
  if (!(qp.bits == 2 || qp.bits == 3 || qp.bits == 4 || qp.bits == 8)) return false;
  if (!(qp.sym == 0 || qp.sym == 1)) return false;
  const int64_t g = (qp.group_size == -1) ? n : qp.group_size;
  if (g < 32 || g > n || n % g) return false;
  if (!(g % 128 == 0 || 128 % g == 0)) return false;
  return true;
}

}  // namespace gptq
