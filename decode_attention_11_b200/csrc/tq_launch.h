// Host helpers of the paged kernels' launches.
#pragma once

#include <cuda_runtime.h>

#include "tq_internal.h"

namespace tq {

// SMs of the current device.
inline int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      n <= 0) {
    cudaGetLastError();
    return 148;
  }
  return n;
}

// Launch a kernel; `dependent`: as a programmatic dependent of the stream's last one.
template <typename... K, typename... A>
tq_status launch(void (*kernel)(K...), int64_t grid, int threads, size_t smem, cudaStream_t s, bool dependent, const char* name,
                 const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = dependent ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e != cudaSuccess) return fail(TQ_ERR_CUDA, "%s launch: %s", name, cudaGetErrorString(e));
  return TQ_OK;
}

}  // namespace tq
