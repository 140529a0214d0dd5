// Host side of the calls around a layer: enqueueing, and what the runtime says of it.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/kdn.h"

namespace kdn {

// The status of a runtime call that enqueues.  It is the call's own result:
// cudaGetLastError would also give an error that some earlier call left behind,
// for work that was enqueued all the same.  (An error of this call is cleared, so
// that it is not found behind a later one.)
inline kdn_status enqueued(cudaError_t result) {
  if (result == cudaSuccess) return KDN_OK;
  cudaGetLastError();
  return KDN_ERR_CUDA;
}
template <typename... P, typename... A>
inline kdn_status launch(void (*kernel)(P...), int64_t blocks, int threads, size_t smem,
                         cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  return enqueued(cudaLaunchKernelEx(&cfg, kernel, P(args)...));
}

}  // namespace kdn
