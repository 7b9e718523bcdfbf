// bf16_epilogue.cuh -- what becomes of a bf16 product's fp32 sums:
//
//   y[f][n] = weight[f] * act(sum + bias[e][n]) + residual[f][n]
//
// in fp32, rounded once to y's type.  Exponentials are CUDA's expf (its fast
// form is 2^-21 off, 8 fp32 roundings; the sums cost more than either).
#pragma once

#include "bf16.h"
#include "blocks.cuh"
#include "device_utils.cuh"
#include "moe_lora.h"

namespace moe_lora {

// v / (1 + exp(-z)), from exp(-|z|), which cannot overflow.
__device__ __forceinline__ float times_sigmoid(float v, float z) {
  const float e = expf(-fabsf(z));
  return v * (z < 0.f ? e : 1.f) / (1.f + e);
}

template <int W>
__device__ __forceinline__ void activate(float (&v)[W], int act) {
  if (act == MOE_ACT_NONE) return;
  if (act == MOE_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = v[i] < 0.f ? 0.f : v[i];   // (keeps NaN)
  } else if (act == MOE_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = times_sigmoid(v[i], v[i]);
  } else if (act == MOE_ACT_GELU) {
    // v * Phi(v): erfc keeps the bits that 1 + erf(v) loses for v < 0
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = 0.5f * v[i] * erfcf(-0.70710678118654752f * v[i]);
  } else {
    // 0.5 v (1 + tanh(u)) = v * sigmoid(2u), u = sqrt(2 / pi) (v + 0.044715 v^3)
#pragma unroll
    for (int i = 0; i < W; ++i)
      v[i] = times_sigmoid(v[i], 1.5957691216057308f * (v[i] + 0.044715f * v[i] * v[i] * v[i]));
  }
}

__device__ __forceinline__ float load_as_f32(const void *p, long long i, int f32) {
  return f32 ? load_global(static_cast<const float *>(p) + i)
             : bf16_bits_to_float(load_global(static_cast<const uint16_t *>(p) + i));
}

__device__ __forceinline__ float bias_of(const Bf16Args &p, int e, int n) {
  return p.bias && n < p.N ? load_as_f32(p.bias, (long long)e * p.N + n, p.bias_f32) : 0.f;
}

__device__ __forceinline__ void store_one(const Bf16Args &p, int f, int n, float v) {
  if (p.y_f32) static_cast<float *>(p.y)[f * p.ldy + n] = v;
  else static_cast<uint16_t *>(p.y)[f * p.ldy + n] = float_to_bf16_bits(v);
}

// Column n of the pairs f (negative: none), whose sums v are.  All loads come
// before the first store: residual may be y.
template <int MODE, int W>
__device__ __forceinline__ void finish_column(const Bf16Args &p, const int (&f)[W], int n, float bias, const float (&v)[W]) {
  if (n >= p.N) return;
  float w[W], r[W], o[W];
#pragma unroll
  for (int i = 0; i < W; ++i) {
    w[i] = f[i] >= 0 ? pair_weight<MODE>(p, f[i]) : 0.f;
    r[i] = f[i] >= 0 && p.residual ? load_as_f32(p.residual, f[i] * p.ldr + n, p.y_f32) : 0.f;
    o[i] = v[i] + bias;
  }
  activate(o, p.act);
#pragma unroll
  for (int i = 0; i < W; ++i)
    if (f[i] >= 0) store_one(p, f[i], n, o[i] * w[i] + r[i]);
}

// The same for a warp whose lanes hold neighbouring columns n, and the pairs f:
// pair j is lane j's.
template <int MODE>
__device__ __forceinline__ void finish_part(const Bf16Args &p, int f, int n, float bias, float (&v)[32]) {
  const float w = f < 0 ? 0.f : pair_weight<MODE>(p, f);
  const bool weighted = MODE != kDense && p.topk_weights;
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] += bias;
  activate(v, p.act);
  if (weighted) {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] *= __shfl_sync(0xFFFFFFFFu, w, j);
  }
  if (MODE == kDense && p.residual) {
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const int fj = __shfl_sync(0xFFFFFFFFu, f, j);
      if (fj >= 0 && n < p.N) v[j] += load_as_f32(p.residual, fj * p.ldr + n, p.y_f32);
    }
  }
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const int fj = __shfl_sync(0xFFFFFFFFu, f, j);
    if (fj >= 0 && n < p.N) store_one(p, fj, n, v[j]);
  }
}

}  // namespace moe_lora
