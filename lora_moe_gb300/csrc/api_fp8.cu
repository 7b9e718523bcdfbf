// api_fp8.cu -- the C ABI of the 8-bit serving operators (declared in
// include/moe_lora.h): argument validation.  Every check runs on the host
// before anything is enqueued.
#include <cuda_runtime.h>
#include <stdint.h>

#include "fp8.h"
#include "moe_lora.h"

using namespace moe_lora;

namespace {

constexpr int kMaxExperts = 1024;
constexpr long long kMaxLd = 1ll << 40;   // leading dimensions whose byte offsets stay far from 64 bits

bool on(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool ld_ok(long long ld, long long columns) { return ld >= columns && ld < kMaxLd; }

// What the three products share.  *empty is set when there is nothing to do.
int check_product(const Fp8Args &a, bool *empty) {
  if (a.K < 1 || a.N < 1) return MOE_LORA_ERR_INVALID_ARG;
  if (!ld_ok(a.ldx, a.K) || !ld_ok(a.ldw, a.K) || !ld_ok(a.ldy, a.N)) return MOE_LORA_ERR_INVALID_ARG;
  if (a.K > INT32_MAX - 128 || a.N > INT32_MAX - 256) return MOE_LORA_ERR_UNSUPPORTED;
  if (a.ldx % 16 != 0 || a.ldw % 16 != 0) return MOE_LORA_ERR_MISALIGNED;
  if ((long long)a.N * a.ldw >= kMaxLd) return MOE_LORA_ERR_UNSUPPORTED;   // (a tensor map's stride)
  *empty = a.pairs == 0;
  if (*empty) return 0;
  if (!a.x || !a.x_scales || !a.w || !a.w_scales || !a.y) return MOE_LORA_ERR_INVALID_ARG;
  if (!on(a.x, 16) || !on(a.w, 16) || !on(a.x_scales, 4) || !on(a.w_scales, 4) || !on(a.y, 2) ||
      !on(a.topk_weights, 4) || !on(a.err, 4))
    return MOE_LORA_ERR_MISALIGNED;
  return 0;
}

int grouped(Fp8Args a, ProductMode mode, int M, void *workspace, size_t workspace_bytes, void *stream) {
  if (M < 0 || a.topk < 1 || a.E < 1) return MOE_LORA_ERR_INVALID_ARG;
  if (a.E > kMaxExperts || a.topk > a.E) return MOE_LORA_ERR_UNSUPPORTED;
  const long long pairs = (long long)M * a.topk;
  if (pairs > INT32_MAX / 2) return MOE_LORA_ERR_UNSUPPORTED;
  a.pairs = (int)pairs;
  a.rows = a.x_per_pair ? a.pairs : M;
  a.KB = fp8_groups(a.K);
  a.NB = fp8_groups(a.N);
  bool empty = false;
  if (int st = check_product(a, &empty)) return st;
  if (empty) return MOE_LORA_OK;
  const void *ids[4] = {a.sorted_token_ids, a.expert_ids, a.num_tokens_post_padded, a.topk_ids};
  for (int i = 0; i < 4; ++i) {
    if (!ids[i] && (i == 3) == (mode == kNaive)) return MOE_LORA_ERR_INVALID_ARG;
    if (!on(ids[i], 4)) return MOE_LORA_ERR_MISALIGNED;
  }
  if (!fp8_items_fit(a, mode)) return MOE_LORA_ERR_UNSUPPORTED;
  if (mode == kSorted) {
    const size_t need = fp8_sorted_workspace(a);
    if (need && (!workspace || workspace_bytes < need)) return MOE_LORA_ERR_WORKSPACE;
    if (need && !on(workspace, 16)) return MOE_LORA_ERR_MISALIGNED;
  }
  DeviceInfo dev;
  if (int st = current_device_info(&dev)) return st;
  return launch_fp8_matmul(a, mode, workspace, dev, static_cast<cudaStream_t>(stream));
}

bool valid_block(int bs) { return bs == 16 || bs == 32 || bs == 64 || bs == 128; }

}  // namespace

extern "C" {

int moe_add_rms_norm_fp8(const moe_lora_bf16 *x, long long ldx, long long ld_part, int parts,
                         const moe_lora_bf16 *residual, long long ld_residual, const moe_lora_bf16 *weight, float eps,
                         moe_lora_bf16 *residual_out, long long ld_residual_out, moe_lora_bf16 *normed,
                         long long ld_normed, moe_lora_fp8 *q, long long ldq, float *scales, int M, int H,
                         void *stream) {
  if (M < 0 || H < 1 || parts < 1 || !(eps >= 0.f)) return MOE_LORA_ERR_INVALID_ARG;
  if (H > MOE_FP8_MAX_NORM_COLUMNS) return MOE_LORA_ERR_UNSUPPORTED;
  if (!ld_ok(ldx, H) || (parts > 1 && !ld_ok(ld_part, H)) || !ld_ok(ldq, H) || (residual && !ld_ok(ld_residual, H)) ||
      (residual_out && !ld_ok(ld_residual_out, H)) || (normed && !ld_ok(ld_normed, H)))
    return MOE_LORA_ERR_INVALID_ARG;
  if (M == 0) return MOE_LORA_OK;
  if (!x || !weight || !q || !scales) return MOE_LORA_ERR_INVALID_ARG;
  if (!on(x, 2) || !on(residual, 2) || !on(weight, 2) || !on(residual_out, 2) || !on(normed, 2) || !on(scales, 4))
    return MOE_LORA_ERR_MISALIGNED;
  DeviceInfo dev;
  if (int st = current_device_info(&dev)) return st;
  NormArgs a = {};
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.residual_out = residual_out;
  a.normed = normed;
  a.q = q;
  a.scales = scales;
  a.ldx = ldx;
  a.ld_part = parts > 1 ? ld_part : 0;
  a.ld_res = ld_residual;
  a.ld_res_out = ld_residual_out;
  a.ld_normed = ld_normed;
  a.ldq = ldq;
  a.M = M;
  a.parts = parts;
  a.H = H;
  a.eps = eps;
  return launch_norm_fp8(a, dev, static_cast<cudaStream_t>(stream));
}

int moe_silu_mul_fp8(const moe_lora_bf16 *x, long long ldx, moe_lora_bf16 *act, long long ld_act, moe_lora_fp8 *q,
                     long long ldq, float *scales, int rows, int I, void *stream) {
  if (rows < 0 || I < 1) return MOE_LORA_ERR_INVALID_ARG;
  if (!ld_ok(ldx, 2ll * I) || !ld_ok(ldq, I) || (act && !ld_ok(ld_act, I))) return MOE_LORA_ERR_INVALID_ARG;
  if (I > INT32_MAX - 256) return MOE_LORA_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_LORA_OK;
  if (!x || !q || !scales) return MOE_LORA_ERR_INVALID_ARG;
  if (!on(x, 2) || !on(act, 2) || !on(scales, 4)) return MOE_LORA_ERR_MISALIGNED;
  DeviceInfo dev;
  if (int st = current_device_info(&dev)) return st;
  ActArgs a = {};
  a.x = x;
  a.act = act;
  a.ld_act = act ? ld_act : 0;
  a.q = q;
  a.scales = scales;
  a.ldx = ldx;
  a.ldq = ldq;
  a.rows = rows;
  a.I = I;
  return launch_act_fp8(a, dev, static_cast<cudaStream_t>(stream));
}

int moe_fp8_matmul(const moe_lora_fp8 *x, long long ldx, const float *x_scales, const moe_lora_fp8 *w, long long ldw,
                   const float *w_scales, moe_lora_bf16 *y, long long ldy, int M, int N, int K, int32_t *err_flag,
                   void *stream) {
  if (M < 0) return MOE_LORA_ERR_INVALID_ARG;
  if (M > INT32_MAX / 2) return MOE_LORA_ERR_UNSUPPORTED;
  Fp8Args a = {};
  a.x = x;
  a.x_scales = x_scales;
  a.w = w;
  a.w_scales = w_scales;
  a.y = y;
  a.err = err_flag;
  a.ldx = ldx;
  a.ldw = ldw;
  a.ldy = ldy;
  a.rows = a.pairs = M;
  a.topk = 1;
  a.E = 1;
  a.K = K;
  a.N = N;
  a.x_per_pair = 1;
  bool empty = false;
  if (int st = check_product(a, &empty)) return st;
  if (empty) return MOE_LORA_OK;
  a.KB = fp8_groups(K);
  a.NB = fp8_groups(N);
  if (!fp8_items_fit(a, kDense)) return MOE_LORA_ERR_UNSUPPORTED;
  DeviceInfo dev;
  if (int st = current_device_info(&dev)) return st;
  return launch_fp8_matmul(a, kDense, nullptr, dev, static_cast<cudaStream_t>(stream));
}

size_t moe_fp8_grouped_workspace_bytes(int M, int topk, int num_experts, int K, int N, int block_size) {
  if (M < 0 || topk < 1 || num_experts < 1 || num_experts > kMaxExperts || topk > num_experts || K < 1 ||
      K > INT32_MAX - 128 || N < 1 || N > INT32_MAX - 256 || !valid_block(block_size))
    return 0;
  const long long cap = (long long)M * topk + (long long)num_experts * (block_size - 1);
  if (cap > INT32_MAX / 2) return 0;
  Fp8Args a = {};
  a.pairs = M * topk;
  a.E = num_experts;
  a.K = K;
  a.N = N;
  a.block = block_size;
  a.max_blocks = (int)(cap / block_size);
  return a.pairs == 0 ? 0 : fp8_sorted_workspace(a);
}

int moe_fp8_grouped_matmul(const moe_lora_fp8 *x, int x_per_pair, long long ldx, const float *x_scales,
                           const moe_lora_fp8 *w, long long ldw, const float *w_scales, moe_lora_bf16 *y,
                           long long ldy, const float *topk_weights, const int32_t *sorted_token_ids,
                           const int32_t *expert_ids, const int32_t *num_tokens_post_padded, int M, int topk,
                           int num_experts, int K, int N, int block_size, int max_num_tokens_padded,
                           int max_num_m_blocks, void *workspace, size_t workspace_bytes, int32_t *err_flag,
                           void *stream) {
  if (M < 0 || topk < 1 || num_experts < 1) return MOE_LORA_ERR_INVALID_ARG;
  if (!valid_block(block_size)) return MOE_LORA_ERR_UNSUPPORTED;
  const long long cap = (long long)M * topk + (long long)num_experts * (block_size - 1);
  if (cap > INT32_MAX / 2) return MOE_LORA_ERR_UNSUPPORTED;
  if (max_num_tokens_padded < cap || (long long)max_num_m_blocks * block_size < cap) return MOE_LORA_ERR_INVALID_ARG;
  Fp8Args a = {};
  a.x = x;
  a.x_per_pair = x_per_pair ? 1 : 0;
  a.ldx = ldx;
  a.x_scales = x_scales;
  a.w = w;
  a.ldw = ldw;
  a.w_scales = w_scales;
  a.y = y;
  a.ldy = ldy;
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

int moe_fp8_grouped_matmul_naive(const moe_lora_fp8 *x, int x_per_pair, long long ldx, const float *x_scales,
                                 const moe_lora_fp8 *w, long long ldw, const float *w_scales, moe_lora_bf16 *y,
                                 long long ldy, const float *topk_weights, const int32_t *topk_ids, int M, int topk,
                                 int num_experts, int K, int N, int32_t *err_flag, void *stream) {
  Fp8Args a = {};
  a.x = x;
  a.x_per_pair = x_per_pair ? 1 : 0;
  a.ldx = ldx;
  a.x_scales = x_scales;
  a.w = w;
  a.ldw = ldw;
  a.w_scales = w_scales;
  a.y = y;
  a.ldy = ldy;
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
