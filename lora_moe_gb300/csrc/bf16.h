// bf16.h -- argument block and launchers of the bf16 products, shared between
// their C-ABI layer (api_bf16.cu) and kernels.  Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "blocks.cuh"
#include "internal.h"

namespace moe_lora {

constexpr int kBf16Group = 64;   // columns of a tile: one swizzle row of 128 bytes

// y[f][n] = weight[f] * act(sum_k x[r][k] * w[e][n][k] + bias[e][n]) + residual[f][n]
struct Bf16Args : PairBlocks {
  const uint16_t *x;          // bf16 [rows, ldx]
  const uint16_t *w;          // bf16 [E, N, ldw]
  void *y;                    // bf16 or fp32 [pairs, ldy]
  const void *bias;           // bf16 or fp32 [E, N], or null
  const void *residual;       // y's type [pairs, ldr], or null; may be y
  long long ldx, ldw, ldy, ldr;
  int rows, K, N, KB;         // KB: groups of K
  int act;                    // MOE_ACT_*
  int bias_f32, y_f32;
};

// Single pairs, and dense calls of at most 16 rows, whose weights are small.
int launch_bf16_stream(const Bf16Args &a, ProductMode mode, const DeviceInfo &dev, cudaStream_t stream);
// Sorted calls with many pairs an expert gather x into the workspace (the
// bytes it needs; 0: none).
size_t bf16_sorted_workspace(const Bf16Args &a);
// Whether the kernels' work items of a call can be counted in an int; asked
// before anything is enqueued.
bool bf16_items_fit(const Bf16Args &a, ProductMode mode);
int launch_bf16_matmul(const Bf16Args &a, ProductMode mode, void *workspace, const DeviceInfo &dev, cudaStream_t stream);

}  // namespace moe_lora
