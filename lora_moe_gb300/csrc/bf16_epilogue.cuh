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

__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {
    case MOE_ACT_RELU: return v > 0.f ? v : (v == v ? 0.f : v);   // (keeps NaN)
    case MOE_ACT_SILU: return times_sigmoid(v, v);
    // v * Phi(v): erfc keeps the bits that 1 + erf(v) loses for v < 0
    case MOE_ACT_GELU: return 0.5f * v * erfcf(-0.70710678118654752f * v);
    // 0.5 v (1 + tanh(u)) = v * sigmoid(2u), u = sqrt(2 / pi) (v + 0.044715 v^3)
    case MOE_ACT_GELU_TANH: return times_sigmoid(v, 1.5957691216057308f * (v + 0.044715f * v * v * v));
    default: return v;
  }
}

__device__ __forceinline__ float load_as_f32(const void *p, long long i, int f32) {
  return f32 ? load_global(static_cast<const float *>(p) + i)
             : bf16_bits_to_float(load_global(static_cast<const uint16_t *>(p) + i));
}

__device__ __forceinline__ float bias_of(const Bf16Args &p, int e, int n) {
  return p.bias && n < p.N ? load_as_f32(p.bias, (long long)e * p.N + n, p.bias_f32) : 0.f;
}

// Column n of the pairs f (negative: none), whose sums v are.  All loads come
// before the first store: residual may be y.
template <int MODE, int W>
__device__ __forceinline__ void finish_column(const Bf16Args &p, const int (&f)[W], int n, float bias, const float (&v)[W]) {
  if (n >= p.N) return;
  float w[W], r[W];
#pragma unroll
  for (int i = 0; i < W; ++i) {
    w[i] = f[i] >= 0 ? pair_weight<MODE>(p, f[i]) : 0.f;
    r[i] = f[i] >= 0 && p.residual ? load_as_f32(p.residual, f[i] * p.ldr + n, p.y_f32) : 0.f;
  }
#pragma unroll
  for (int i = 0; i < W; ++i) {
    if (f[i] < 0) continue;
    const float o = activate(v[i] + bias, p.act) * w[i] + r[i];
    if (p.y_f32) static_cast<float *>(p.y)[f[i] * p.ldy + n] = o;
    else static_cast<uint16_t *>(p.y)[f[i] * p.ldy + n] = float_to_bf16_bits(o);
  }
}

}  // namespace moe_lora
