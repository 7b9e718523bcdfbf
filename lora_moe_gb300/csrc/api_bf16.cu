// api_bf16.cu -- the C ABI of the bf16 products (declared in
// include/moe_lora.h): argument validation.  Every check runs on the host
// before anything is enqueued.
#include <cuda_runtime.h>
#include <stdint.h>

#include "bf16.h"
#include "moe_lora.h"

using namespace moe_lora;

namespace {

constexpr int kMaxExperts = 1024;
constexpr long long kMaxLd = 1ll << 39;   // leading dimensions whose byte offsets stay far from 64 bits

bool on(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool ld_ok(long long ld, long long columns) { return ld >= columns && ld < kMaxLd; }

// What the products share.  *empty is set when there is nothing to do.
int check_product(const Bf16Args &a, bool *empty) {
  if (a.K < 1 || a.N < 1 || a.act < MOE_ACT_NONE || a.act > MOE_ACT_GELU_TANH) return MOE_LORA_ERR_INVALID_ARG;
  if (!ld_ok(a.ldx, a.K) || !ld_ok(a.ldw, a.K) || !ld_ok(a.ldy, a.N) || (a.residual && !ld_ok(a.ldr, a.N)))
    return MOE_LORA_ERR_INVALID_ARG;
  if (a.K > INT32_MAX / 2 - 128 || a.N > INT32_MAX - 256) return MOE_LORA_ERR_UNSUPPORTED;
  if (a.ldx % 8 != 0 || a.ldw % 8 != 0) return MOE_LORA_ERR_MISALIGNED;
  if ((long long)a.N * a.ldw >= kMaxLd) return MOE_LORA_ERR_UNSUPPORTED;   // (a tensor map's stride)
  *empty = a.pairs == 0;
  if (*empty) return 0;
  if (!a.x || !a.w || !a.y) return MOE_LORA_ERR_INVALID_ARG;
  const size_t y = a.y_f32 ? 4 : 2;
  if (!on(a.x, 16) || !on(a.w, 16) || !on(a.y, y) || !on(a.residual, y) || !on(a.bias, a.bias_f32 ? 4 : 2) ||
      !on(a.topk_weights, 4) || !on(a.err, 4))
    return MOE_LORA_ERR_MISALIGNED;
  return 0;
}

int grouped(Bf16Args a, ProductMode mode, int M, void *workspace, size_t workspace_bytes, void *stream) {
  if (M < 0 || a.topk < 1 || a.E < 1) return MOE_LORA_ERR_INVALID_ARG;
  if (a.E > kMaxExperts || a.topk > a.E) return MOE_LORA_ERR_UNSUPPORTED;
  const long long pairs = (long long)M * a.topk;
  if (pairs > INT32_MAX / 2) return MOE_LORA_ERR_UNSUPPORTED;
  a.pairs = (int)pairs;
  a.rows = a.x_per_pair ? a.pairs : M;
  bool empty = false;
  if (int st = check_product(a, &empty)) return st;
  if (empty) return MOE_LORA_OK;
  a.KB = (a.K + kBf16Group - 1) / kBf16Group;
  const void *ids[4] = {a.sorted_token_ids, a.expert_ids, a.num_tokens_post_padded, a.topk_ids};
  for (int i = 0; i < 4; ++i) {
    if (!ids[i] && (i == 3) == (mode == kNaive)) return MOE_LORA_ERR_INVALID_ARG;
    if (!on(ids[i], 4)) return MOE_LORA_ERR_MISALIGNED;
  }
  if (!bf16_items_fit(a, mode)) return MOE_LORA_ERR_UNSUPPORTED;
  if (mode == kSorted) {
    const size_t need = bf16_sorted_workspace(a);
    if (need && (!workspace || workspace_bytes < need)) return MOE_LORA_ERR_WORKSPACE;
    if (need && !on(workspace, 16)) return MOE_LORA_ERR_MISALIGNED;
  }
  DeviceInfo dev;
  if (int st = current_device_info(&dev)) return st;
  return launch_bf16_matmul(a, mode, workspace, dev, static_cast<cudaStream_t>(stream));
}

bool valid_block(int bs) { return bs == 16 || bs == 32 || bs == 64 || bs == 128; }

}  // namespace

extern "C" {

int moe_bf16_matmul(const moe_lora_bf16 *x, long long ldx, const moe_lora_bf16 *w, long long ldw, const void *bias,
                    int bias_f32, const void *residual, long long ld_residual, void *y, long long ldy, int y_f32,
                    int activation, int M, int N, int K, int32_t *err_flag, void *stream) {
  if (M < 0) return MOE_LORA_ERR_INVALID_ARG;
  if (M > INT32_MAX / 2) return MOE_LORA_ERR_UNSUPPORTED;
  Bf16Args a = {};
  a.x = x;
  a.ldx = ldx;
  a.w = w;
  a.ldw = ldw;
  a.bias = bias;
  a.bias_f32 = bias_f32 ? 1 : 0;
  a.residual = residual;
  a.ldr = residual ? ld_residual : 0;
  a.y = y;
  a.ldy = ldy;
  a.y_f32 = y_f32 ? 1 : 0;
  a.act = activation;
  a.err = err_flag;
  a.rows = a.pairs = M;
  a.topk = 1;
  a.E = 1;
  a.K = K;
  a.N = N;
  a.x_per_pair = 1;
  bool empty = false;
  if (int st = check_product(a, &empty)) return st;
  if (empty) return MOE_LORA_OK;
  a.KB = (K + kBf16Group - 1) / kBf16Group;
  if (!bf16_items_fit(a, kDense)) return MOE_LORA_ERR_UNSUPPORTED;
  DeviceInfo dev;
  if (int st = current_device_info(&dev)) return st;
  return launch_bf16_matmul(a, kDense, nullptr, dev, static_cast<cudaStream_t>(stream));
}

size_t moe_bf16_grouped_workspace_bytes(int M, int topk, int num_experts, int K, int N, int block_size) {
  if (M < 0 || topk < 1 || num_experts < 1 || num_experts > kMaxExperts || topk > num_experts || K < 1 ||
      K > INT32_MAX / 2 - 128 || N < 1 || N > INT32_MAX - 256 || !valid_block(block_size))
    return 0;
  const long long cap = (long long)M * topk + (long long)num_experts * (block_size - 1);
  if (cap > INT32_MAX / 2) return 0;
  Bf16Args a = {};
  a.pairs = M * topk;
  a.E = num_experts;
  a.K = K;
  a.N = N;
  a.block = block_size;
  a.max_blocks = (int)(cap / block_size);
  return a.pairs == 0 ? 0 : bf16_sorted_workspace(a);
}

int moe_bf16_grouped_matmul(const moe_lora_bf16 *x, int x_per_pair, long long ldx, const moe_lora_bf16 *w,
                            long long ldw, const void *bias, int bias_f32, moe_lora_bf16 *y, long long ldy,
                            int activation, const float *topk_weights, const int32_t *sorted_token_ids,
                            const int32_t *expert_ids, const int32_t *num_tokens_post_padded, int M, int topk,
                            int num_experts, int K, int N, int block_size, int max_num_tokens_padded,
                            int max_num_m_blocks, void *workspace, size_t workspace_bytes, int32_t *err_flag,
                            void *stream) {
  if (M < 0 || topk < 1 || num_experts < 1) return MOE_LORA_ERR_INVALID_ARG;
  if (!valid_block(block_size)) return MOE_LORA_ERR_UNSUPPORTED;
  const long long cap = (long long)M * topk + (long long)num_experts * (block_size - 1);
  if (cap > INT32_MAX / 2) return MOE_LORA_ERR_UNSUPPORTED;
  if (max_num_tokens_padded < cap || (long long)max_num_m_blocks * block_size < cap) return MOE_LORA_ERR_INVALID_ARG;
  Bf16Args a = {};
  a.x = x;
  a.x_per_pair = x_per_pair ? 1 : 0;
  a.ldx = ldx;
  a.w = w;
  a.ldw = ldw;
  a.bias = bias;
  a.bias_f32 = bias_f32 ? 1 : 0;
  a.y = y;
  a.ldy = ldy;
  a.act = activation;
  a.topk_weights = topk_weights;
  a.sorted_token_ids = sorted_token_ids;
  a.expert_ids = expert_ids;
  a.num_tokens_post_padded = num_tokens_post_padded;
  a.topk = topk;
  a.E = num_experts;
  a.K = K;
  a.N = N;
  a.block = block_size;
  a.max_blocks = (int)(cap / block_size);   // an align's blocks are whole ones
  a.err = err_flag;
  return grouped(a, kSorted, M, workspace, workspace_bytes, stream);
}

int moe_bf16_grouped_matmul_naive(const moe_lora_bf16 *x, int x_per_pair, long long ldx, const moe_lora_bf16 *w,
                                  long long ldw, const void *bias, int bias_f32, moe_lora_bf16 *y, long long ldy,
                                  int activation, const float *topk_weights, const int32_t *topk_ids, int M, int topk,
                                  int num_experts, int K, int N, int32_t *err_flag, void *stream) {
  Bf16Args a = {};
  a.x = x;
  a.x_per_pair = x_per_pair ? 1 : 0;
  a.ldx = ldx;
  a.w = w;
  a.ldw = ldw;
  a.bias = bias;
  a.bias_f32 = bias_f32 ? 1 : 0;
  a.y = y;
  a.ldy = ldy;
  a.act = activation;
  a.topk_weights = topk_weights;
  a.topk_ids = topk_ids;
  a.topk = topk;
  a.E = num_experts;
  a.K = K;
  a.N = N;
  a.block = 16;
  a.err = err_flag;
  return grouped(a, kNaive, M, nullptr, 0, stream);
}

}  // extern "C"
