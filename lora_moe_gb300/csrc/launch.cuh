// launch.cuh -- how the kernels of the serving operators are launched.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "internal.h"
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

// Clusters of this shape that are resident at once; asked once for each shape.
template <typename Kernel>
int resident_clusters(Kernel kernel, int cluster, int smem_bytes, int threads, const DeviceInfo &dev) {
  if (cluster == 1) return dev.sm_count;
  struct Entry {
    const void *kernel;
    int device, cluster, smem, clusters;
  };
  static std::mutex mu;
  static Entry known[256];
  static int n = 0;
  std::lock_guard<std::mutex> lock(mu);
  for (int i = 0; i < n; ++i)
    if (known[i].kernel == (const void *)kernel && known[i].device == dev.device && known[i].cluster == cluster &&
        known[i].smem == smem_bytes)
      return known[i].clusters;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)cluster, 1, 1);
  lc.blockDim = dim3(threads, 1, 1);
  lc.dynamicSmemBytes = smem_bytes;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  int clusters = 0;
  if (cudaOccupancyMaxActiveClusters(&clusters, (const void *)kernel, &lc) != cudaSuccess) {
    cudaGetLastError();   // a failed query leaves no sticky error
    clusters = 0;
  }
  if (clusters < 1) clusters = std::max(1, dev.sm_count / cluster / 2);
  if (n < 256) known[n++] = {(const void *)kernel, dev.device, cluster, smem_bytes, clusters};
  return clusters;
}

}  // namespace moe_lora
