// api_route.cu -- the C ABI of the router (declared in include/moe_lora.h):
// argument validation, on the host before anything is enqueued.
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_lora.h"
#include "route.h"

using namespace moe_lora;

static_assert(kRouteMaxTopk == MOE_ROUTE_MAX_TOPK && kRouteMaxGroups == MOE_ROUTE_MAX_GROUPS, "the header's limits");

extern "C" int moe_route(const void *logits, int logits_f32, long long ld_logits, const float *bias, int scoring,
                         int renormalize, float scale, int num_groups, int topk_groups, int group_best,
                         int32_t *topk_ids, float *topk_weights, int M, int num_experts, int topk, void *stream) {
  if (M < 0 || num_experts < 1 || topk < 1 || num_groups < 1 || topk_groups < 1) return MOE_LORA_ERR_INVALID_ARG;
  if (scoring != MOE_ROUTE_SOFTMAX && scoring != MOE_ROUTE_SIGMOID) return MOE_LORA_ERR_INVALID_ARG;
  if (group_best != 1 && group_best != 2) return MOE_LORA_ERR_INVALID_ARG;
  if (num_experts > 1024 || topk > kRouteMaxTopk || num_groups > kRouteMaxGroups) return MOE_LORA_ERR_UNSUPPORTED;
  if (num_experts % num_groups != 0 || topk_groups > num_groups || topk > topk_groups * (num_experts / num_groups))
    return MOE_LORA_ERR_INVALID_ARG;
  if (ld_logits < num_experts || ld_logits >= (1ll << 39)) return MOE_LORA_ERR_INVALID_ARG;
  if (M == 0) return MOE_LORA_OK;
  if (!logits || !topk_ids || !topk_weights) return MOE_LORA_ERR_INVALID_ARG;
  auto on = [](const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; };
  if (!on(logits, logits_f32 ? 4 : 2) || !on(bias, 4) || !on(topk_ids, 4) || !on(topk_weights, 4))
    return MOE_LORA_ERR_MISALIGNED;
  DeviceInfo dev;
  if (int st = current_device_info(&dev)) return st;
  RouteArgs a = {};
  a.logits = logits;
  a.bias = bias;
  a.ids = topk_ids;
  a.weights = topk_weights;
  a.ld = ld_logits;
  a.logits_f32 = logits_f32 ? 1 : 0;
  a.sigmoid = scoring == MOE_ROUTE_SIGMOID;
  a.renormalize = renormalize ? 1 : 0;
  a.M = M;
  a.E = num_experts;
  a.topk = topk;
  a.groups = num_groups;
  a.topk_groups = topk_groups;
  a.best = group_best;
  a.scale = scale;
  return launch_route(a, dev, static_cast<cudaStream_t>(stream));
}
