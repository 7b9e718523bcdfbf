// fp8.h -- argument blocks and launchers of the 8-bit serving operators,
// shared between their C-ABI layer (api_fp8.cu) and kernels.  Not part of the
// public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "blocks.cuh"
#include "internal.h"

namespace moe_lora {

constexpr int kFp8Group = 128;   // columns that share a scale

inline __host__ __device__ int fp8_groups(int n) { return (n + kFp8Group - 1) / kFp8Group; }

// Residual addition, root-mean-square norm, 8-bit output.  As validated by the C-ABI layer.
struct NormArgs {
  const uint16_t *x;          // bf16 [M, parts, ldx]
  const uint16_t *residual;   // bf16 [M, ld_res] or null
  const uint16_t *weight;     // bf16 [H]
  uint16_t *residual_out;     // bf16 [M, ld_res_out] or null
  uint16_t *normed;           // bf16 [M, ld_normed] or null
  uint8_t *q;                 // e4m3 [M, ldq]
  float *scales;              // fp32 [M, groups]
  long long ldx, ld_part, ld_res, ld_res_out, ld_normed, ldq;   // ldx: from token to token, ld_part: from part to part
  int M, parts, H;
  float eps;
};
int launch_norm_fp8(const NormArgs &a, const DeviceInfo &dev, cudaStream_t stream);
constexpr int kNormMaxH = 16384;

// silu(gate) * up, 8-bit output.
struct ActArgs {
  const uint16_t *x;   // bf16 [rows, ldx]: gate in columns [0, I), up in [I, 2I)
  uint16_t *act;       // bf16 [rows, ld_act] or null
  uint8_t *q;          // e4m3 [rows, ldq]
  float *scales;       // fp32 [rows, groups]
  long long ldx, ld_act, ldq;
  int rows, I;
};
int launch_act_fp8(const ActArgs &a, const DeviceInfo &dev, cudaStream_t stream);

// 8-bit products.
struct Fp8Args : PairBlocks {
  const uint8_t *x;           // e4m3 [rows, ldx]
  const float *x_scales;      // fp32 [rows, KB]
  const uint8_t *w;           // e4m3 [E, N, ldw]
  const float *w_scales;      // fp32 [E, NB, KB]
  uint16_t *y;                // bf16 [pairs, ldy]
  long long ldx, ldw, ldy;
  int rows, K, N, KB, NB;
};
// Naive calls, and dense ones of at most 16 rows, whose weights are small.
int launch_fp8_stream(const Fp8Args &a, ProductMode mode, const DeviceInfo &dev, cudaStream_t stream);
// Sorted calls with many pairs an expert gather x into the workspace (the
// bytes it needs; 0: none).
size_t fp8_sorted_workspace(const Fp8Args &a);
// Whether the kernels' work items of a call can be counted in an int; asked
// before anything is enqueued.
bool fp8_items_fit(const Fp8Args &a, ProductMode mode);
int launch_fp8_matmul(const Fp8Args &a, ProductMode mode, void *workspace, const DeviceInfo &dev, cudaStream_t stream);

}  // namespace moe_lora
