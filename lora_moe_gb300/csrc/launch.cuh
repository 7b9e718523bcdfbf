// launch.cuh -- how the 8-bit operators' kernels are launched.
#pragma once

#include <cuda_runtime.h>

#include "moe_lora.h"

namespace moe_lora {

// A launch of `grid` CTAs in clusters of `cluster`.  The kernel may start while
// the one before it on the stream is finishing (programmatic dependent launch):
// each waits for it, with wait_for_prior_grid(), before it touches memory.
template <typename... Params, typename... Args>
int launch_dependent(void (*kernel)(Params...), unsigned grid, int threads, int cluster, int smem_bytes,
                     cudaStream_t stream, const Args &...args) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(grid, 1, 1);
  lc.blockDim = dim3((unsigned)threads, 1, 1);
  lc.dynamicSmemBytes = (size_t)smem_bytes;
  lc.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&lc, kernel, args...) == cudaSuccess ? 0 : MOE_LORA_ERR_LAUNCH;
}

}  // namespace moe_lora
