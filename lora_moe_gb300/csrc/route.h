// route.h -- argument block and launcher of the router, shared between its
// C-ABI layer (api_route.cu) and kernel.  Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"

namespace moe_lora {

constexpr int kRouteMaxTopk = 32, kRouteMaxGroups = 32;

struct RouteArgs {
  const void *logits;      // bf16 or fp32 [M, ld]
  const float *bias;       // fp32 [E], or null
  int32_t *ids;            // [M, topk]
  float *weights;          // [M, topk]
  long long ld;
  int logits_f32, sigmoid, renormalize;
  int M, E, topk;
  int groups, topk_groups, best;   // groups == topk_groups: no choice among groups
  float scale;
};
int launch_route(const RouteArgs &a, const DeviceInfo &dev, cudaStream_t stream);

}  // namespace moe_lora
