// bf16_epilogue.cuh -- what becomes of a bf16 product's fp32 sums:
//
//   y[f][n] = weight[f] * act(sum + bias[e][n]) + residual[f][n]
//
// in fp32, rounded once to y's type.  For a bf16 y the activations use the
// approximate units (a few instructions a value: with CUDA's own expf and its
// division a decode batch's epilogue took four times the product, 48 x 176 with
// silu 15.6 us); for an fp32 one, CUDA's functions.  The tensor-core kernels bring
// the sums to shared memory, where a loop of few instructions takes them four
// columns a thread: a tile's epilogue runs a few times a launch, and code that is unrolled
// over the sums in registers costs more to fetch than to run (64 x 2880, K of
// 256: 7700 clk of 12900).
#pragma once

#include "bf16.h"
#include "blocks.cuh"
#include "device_utils.cuh"
#include "moe_lora.h"

namespace moe_lora {

// v / (1 + exp(-z)), from exp(-|z|), which cannot overflow.  FAST: 2^x and 1 / x of
// the approximate units, within 2^-21 + |z| 2^-23 of the value.
template <bool FAST>
__device__ __forceinline__ float times_sigmoid(float v, float z) {
  if constexpr (FAST) {
    const float e = exp2_unit(-1.44269504f * fabsf(z)), r = v * rcp_unit(1.f + e);
    return z < 0.f ? r * e : r;
  } else {
    const float e = expf(-fabsf(z));
    return v * (z < 0.f ? e : 1.f) / (1.f + e);
  }
}

// v * Phi(v), Phi(v) = erfc(-v / sqrt(2)) / 2: erfc keeps the bits that 1 + erf(v)
// loses for v < 0.  FAST: erfc(x) = (a1 t + .. + a7 t^7) exp(-x^2), t = 1 / (1 + 0.51 x),
// the polynomial fitted to erfc(x) exp(x^2) in relation to its value: within 2^-20 of
// it for 0 <= x <= 10, so that the tail of v < 0 keeps its bits too (an error in
// relation to one leaves gelu(-8) 1e-2 off, past half a step of bf16).  The argument of exp
// is rounded: 2^-16 of the value at x = 9.
template <bool FAST>
__device__ __forceinline__ float gelu(float v) {
  if constexpr (FAST) {
    const float x = 0.70710678f * fabsf(v), t = rcp_unit(1.f + 0.51f * x);
    float q = 0.0945045054f * t - 0.35915038f;
    q = q * t + 0.358466744f;
    q = q * t + 0.0550384037f;
    q = q * t + 0.279071361f;
    q = q * t + 0.284151375f;
    q = (q * t + 0.287917554f) * t * exp2_unit(-0.72134752f * v * v);   // erfc(x); x^2 log2(e) = v^2 log2(e) / 2
    return v * (v < 0.f ? 0.5f * q : 1.f - 0.5f * q);
  } else {
    return 0.5f * v * erfcf(-0.70710678118654752f * v);
  }
}

template <bool FAST, int W>
__device__ __forceinline__ void activate(float (&v)[W], int act) {
  if (act == MOE_ACT_NONE) return;
  if (act == MOE_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = v[i] < 0.f ? 0.f : v[i];   // (keeps NaN)
  } else if (act == MOE_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = times_sigmoid<FAST>(v[i], v[i]);
  } else if (act == MOE_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = gelu<FAST>(v[i]);
  } else {
    // 0.5 v (1 + tanh(u)) = v * sigmoid(2u), u = sqrt(2 / pi) (v + 0.044715 v^3)
#pragma unroll
    for (int i = 0; i < W; ++i)
      v[i] = times_sigmoid<FAST>(v[i], 1.5957691216057308f * (v[i] + 0.044715f * v[i] * v[i] * v[i]));
  }
}

__device__ __forceinline__ float load_as_f32(const void *p, long long i, int f32) {
  return f32 ? load_global(static_cast<const float *>(p) + i)
             : bf16_bits_to_float(load_global(static_cast<const uint16_t *>(p) + i));
}

__device__ __forceinline__ float bias_of(const Bf16Args &p, int e, int n) {
  return p.bias && n < p.N ? load_as_f32(p.bias, (long long)e * p.N + n, p.bias_f32) : 0.f;
}

__device__ __forceinline__ void store_one(const Bf16Args &p, long long at, float v) {
  if (p.y_f32) static_cast<float *>(p.y)[at] = v;
  else static_cast<uint16_t *>(p.y)[at] = float_to_bf16_bits(v);
}

// One sum: column n of pair f (negative: none).
template <int MODE>
__device__ __forceinline__ void finish_one(const Bf16Args &p, int f, int e, int n, float v) {
  if (f < 0 || n >= p.N) return;
  const float w = pair_weight<MODE>(p, f);
  const float r = p.residual ? load_as_f32(p.residual, f * p.ldr + n, p.y_f32) : 0.f;
  float o[1] = {v + bias_of(p, e, n)};
  if (p.y_f32) activate<false>(o, p.act);
  else activate<true>(o, p.act);
  store_one(p, f * p.ldy + n, o[0] * w + r);
}

// Rows of p, ld elements apart, whose elements can be read and written four at
// a time, from a multiple of four on.
__device__ __forceinline__ bool in_fours(const void *p, long long ld, int f32) {
  return (ld & 3) == 0 && (reinterpret_cast<uintptr_t>(p) & (f32 ? 15 : 7)) == 0;
}

// The sums' way out, four columns of a row of the output a thread, neighbours
// where the rows allow that they are written at once.  That is looked at once, so that
// the loops run through.
enum { kOutSingly, kOutBf16, kOutF32 };
__device__ __forceinline__ int out_kind(const Bf16Args &p) {
  if (p.N % 4 != 0 || !in_fours(p.y, p.ldy, p.y_f32) || (p.residual && !in_fours(p.residual, p.ldr, p.y_f32)))
    return kOutSingly;
  return p.y_f32 ? kOutF32 : kOutBf16;
}

// Four columns, n + i * step, of the pairs f (negative: none), whose sums v are,
// times w (dense: not used); step is 1 and n a multiple of four below N but for
// kOutSingly.  All loads come before the first store: residual may be y.
template <int MODE, int KIND, int B>
__device__ __forceinline__ void finish_fours(const Bf16Args &p, const int (&f)[B], const float (&w)[B], int n, int step,
                                             const float (&bias)[4], float (&v)[4 * B]) {
#pragma unroll
  for (int i = 0; i < 4 * B; ++i) v[i] += bias[i & 3];
  if (p.act != MOE_ACT_NONE) {
    if (KIND == kOutF32 || (KIND == kOutSingly && p.y_f32)) activate<false>(v, p.act);
    else activate<true>(v, p.act);
  }
  if (MODE != kDense) {
#pragma unroll
    for (int i = 0; i < 4 * B; ++i) v[i] *= w[i >> 2];
  }
  if (p.residual) {
    if constexpr (KIND == kOutSingly) {
      float r[4 * B];
#pragma unroll
      for (int i = 0; i < 4 * B; ++i)
        r[i] = f[i >> 2] >= 0 && n + (i & 3) * step < p.N
                   ? load_as_f32(p.residual, f[i >> 2] * p.ldr + n + (i & 3) * step, p.y_f32) : 0.f;
#pragma unroll
      for (int i = 0; i < 4 * B; ++i) v[i] += r[i];
    } else if constexpr (KIND == kOutF32) {
      float4 r[B];
#pragma unroll
      for (int b = 0; b < B; ++b)   // (for no pair: another's, not used)
        r[b] = load_global(reinterpret_cast<const float4 *>(static_cast<const float *>(p.residual) + max(f[b], 0) * p.ldr + min(n, p.N - 4)));
#pragma unroll
      for (int b = 0; b < B; ++b) v[4 * b] += r[b].x, v[4 * b + 1] += r[b].y, v[4 * b + 2] += r[b].z, v[4 * b + 3] += r[b].w;
    } else {
      uint2 r[B];
#pragma unroll
      for (int b = 0; b < B; ++b)
        r[b] = load_global(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p.residual) + max(f[b], 0) * p.ldr + min(n, p.N - 4)));
#pragma unroll
      for (int b = 0; b < B; ++b) {
        v[4 * b] += __uint_as_float(r[b].x << 16), v[4 * b + 1] += __uint_as_float(r[b].x & 0xFFFF0000u);
        v[4 * b + 2] += __uint_as_float(r[b].y << 16), v[4 * b + 3] += __uint_as_float(r[b].y & 0xFFFF0000u);
      }
    }
  }
#pragma unroll
  for (int b = 0; b < B; ++b) {
    if constexpr (KIND == kOutSingly) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (f[b] >= 0 && n + i * step < p.N) store_one(p, f[b] * p.ldy + n + i * step, v[4 * b + i]);
    } else if constexpr (KIND == kOutF32) {
      if (f[b] >= 0)
        *reinterpret_cast<float4 *>(static_cast<float *>(p.y) + f[b] * p.ldy + n) =
            make_float4(v[4 * b], v[4 * b + 1], v[4 * b + 2], v[4 * b + 3]);
    } else {
      uint2 u;
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u.x) : "f"(v[4 * b + 1]), "f"(v[4 * b]));
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u.y) : "f"(v[4 * b + 3]), "f"(v[4 * b + 2]));
      if (f[b] >= 0) *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.y) + f[b] * p.ldy + n) = u;
    }
  }
}

// Fetches the residual's line at column n of row f into L2, while the sums are on their way.
__device__ __forceinline__ void fetch_residual(const Bf16Args &p, int f, int n) {
  const char *at = static_cast<const char *>(p.residual) + (f * p.ldr + n) * (p.y_f32 ? 4 : 2);
  asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
}

}  // namespace moe_lora
