// host.h -- host-side helpers shared by the C ABI's translation units: the last error's
// message, error returns, and the driver's tensor-map encoder.
#pragma once
#include <cudaTypedefs.h>

#include <string>

#include "tfl.h"

namespace tfl {

inline thread_local std::string g_err;

inline int fail(int code, const std::string& msg) {
  g_err = msg;
  return code;
}

inline int cuda_fail(cudaError_t e, const char* what) {
  return fail(TFL_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

#define TFL_CUDA(call, what)                         \
  do {                                               \
    cudaError_t e_ = (call);                         \
    if (e_ != cudaSuccess) return cuda_fail(e_, what); \
  } while (0)

inline PFN_cuTensorMapEncodeTiled_v12000 get_encode() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }
  return fn;
}

}  // namespace tfl
