// fp8_rows.cu -- the row operators of the 8-bit path: residual addition with
// root-mean-square norm, and the gated activation, both with an 8-bit output
// that has one fp32 scale for each 128 columns.
//
//   norm:  h = residual + sum_p x[p]        (fp32, p ascending)
//          n = h / sqrt(mean(h^2) + eps) * weight
//   act:   n = gate / (1 + exp(-gate)) * up
//   both:  s = max(amax(|n| over the group) / 448, 2^-126),  q = e4m3(n / s)
//
// Both are bound by HBM: a few operations for each byte.  A thread takes 8
// columns at a time (16 bytes of bf16), 16 neighbouring threads a group of 128,
// whose amax is four shuffles away.
#include <cuda_runtime.h>

#include "device_utils.cuh"
#include "fp8.h"

namespace moe_lora {

namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kMinScale = 1.17549435e-38f;   // 2^-126: a zero group has a normal scale, whose reciprocal is finite

// 8 bf16 columns as fp32; the scalar form takes any alignment and stops at n.
template <bool VEC>
__device__ __forceinline__ void load8(const uint16_t *p, int n, float (&v)[8]) {
  if constexpr (VEC) {
    if (n > 0) {
      const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p));
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? bf16_bits_to_float(__ldg(p + i)) : 0.f;
  }
}

template <bool VEC>
__device__ __forceinline__ void store8(uint16_t *p, int n, const float (&v)[8]) {
  if constexpr (VEC) {
    if (n > 0) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
      *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = float_to_bf16_bits(v[i]);
  }
}

// Quantise a group of 128 columns held by 16 neighbouring lanes, 8 columns
// each, n of which exist in this lane's 8.  The amax is taken over the bit
// patterns of |v|, which order like the values and put NaN above infinity: a
// NaN makes the scale, and so the group, NaN.  n / s is computed as n * (1/s):
// one rounding more than a division, at most one unit of fp32 before the
// rounding to 3 bits.
template <bool VEC>
__device__ __forceinline__ void quantize8(const float (&v)[8], int n, uint8_t *q, float *scale, bool leader) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
#pragma unroll
  for (int d = 8; d; d >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
  const float t = __uint_as_float(m) / kE4m3Max;
  const float s = t < kMinScale ? kMinScale : t;   // (keeps NaN)
  const float inv = 1.f / s;
  if (leader) *scale = s;
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(v[4 * i + 1] * inv), "f"(v[4 * i] * inv));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(v[4 * i + 3] * inv), "f"(v[4 * i + 2] * inv));
    w[i] = lo | (uint32_t(hi) << 16);
  }
  if constexpr (VEC) {
    if (n > 0) *reinterpret_cast<uint2 *>(q) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) q[i] = uint8_t(w[i >> 2] >> (8 * (i & 3)));
  }
}

// One CTA per row; the row stays in registers (NV vectors of 8 columns a
// thread) between the sum of squares and the output.
template <int NV, bool VEC>
__global__ void __launch_bounds__(512) norm_fp8_kernel(const NormArgs p) {
  __shared__ float warp_sum[16];
  const int tid = threadIdx.x, threads = blockDim.x;
  const size_t m = blockIdx.x;
  const int G = fp8_groups(p.H);
  float h[NV][8];
  float sum = 0.f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * threads + tid) * 8, n = p.H - c;
    if (p.residual) load8<VEC>(p.residual + m * p.ld_res + c, n, h[v]);
    else load8<VEC>(p.x, 0, h[v]);
  }
  for (int k = 0; k < p.parts; ++k) {
    const uint16_t *row = p.x + m * p.ldx + k * p.ld_part;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * threads + tid) * 8;
      float a[8];
      load8<VEC>(row + c, p.H - c, a);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[v][i] += a[i];
    }
  }
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * threads + tid) * 8;
    if (p.residual_out) store8<VEC>(p.residual_out + m * p.ld_res_out + c, p.H - c, h[v]);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += h[v][i] * h[v][i];
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
  if ((tid & 31) == 0) warp_sum[tid >> 5] = sum;
  __syncthreads();
  sum = 0.f;
  for (int w = 0; w < threads / 32; ++w) sum += warp_sum[w];
  const float r = rsqrtf(sum / (float)p.H + p.eps);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * threads + tid) * 8, n = p.H - c;
    float w[8];
    load8<VEC>(p.weight + c, n, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[v][i] = h[v][i] * r * w[i];
    if (p.normed) store8<VEC>(p.normed + m * p.ld_normed + c, n, h[v]);
    const int g = c / kFp8Group;
    quantize8<VEC>(h[v], n, p.q + m * p.ldq + c, p.scales + m * G + g, (tid & 15) == 0 && g < G);
  }
}

template <bool VEC>
__global__ void __launch_bounds__(256) act_fp8_kernel(const ActArgs p, long long items, int G) {
  const int lane16 = threadIdx.x & 15;
  const long long first = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 4;
  // whole warps leave together: the shuffles need both groups of a warp
  const long long step = (long long)gridDim.x * blockDim.x >> 4;
  for (long long it = first; (it & ~1ll) < items; it += step) {
    const bool live = it < items;
    const long long row = live ? it / G : 0;
    const int g = live ? (int)(it - row * G) : 0;
    const int c = g * kFp8Group + lane16 * 8, n = live ? p.I - c : 0;
    const uint16_t *src = p.x + row * p.ldx + c;
    float a[8], b[8];
    load8<VEC>(src, n, a);
    load8<VEC>(src + p.I, n, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = a[i] / (1.f + __expf(-a[i])) * b[i];
    quantize8<VEC>(a, n, p.q + row * p.ldq + c, p.scales + row * G + g, live && lane16 == 0);
  }
}

template <typename... Params, typename... Args>
int launch(void (*kernel)(Params...), unsigned grid, unsigned threads, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(grid, 1, 1);
  lc.blockDim = dim3(threads, 1, 1);
  lc.stream = stream;
  return cudaLaunchKernelEx(&lc, kernel, args...) == cudaSuccess ? 0 : MOE_LORA_ERR_LAUNCH;
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

template <bool VEC>
int launch_norm(const NormArgs &a, cudaStream_t s) {
  // threads: a multiple of 32 that covers the row once, up to 512; then more vectors a thread
  const int vecs = (a.H + 7) / 8;
  const int nv = vecs <= 512 ? 1 : (vecs <= 1024 ? 2 : 4);
  const int threads = ((vecs + nv - 1) / nv + 31) / 32 * 32;
  if (nv == 1) return launch(norm_fp8_kernel<1, VEC>, a.M, threads, s, a);
  if (nv == 2) return launch(norm_fp8_kernel<2, VEC>, a.M, threads, s, a);
  return launch(norm_fp8_kernel<4, VEC>, a.M, threads, s, a);
}

}  // namespace

// The 16-byte forms need whole vectors in every row: H a multiple of 8, rows
// and pointers on 16 bytes (8 for the 8-bit output).  Other layouts take the
// scalar form.
int launch_norm_fp8(const NormArgs &a, const DeviceInfo &, cudaStream_t s) {
  auto ok = [](const void *p, long long ld) { return p == nullptr || (aligned(p, 16) && ld % 8 == 0); };
  const bool vec = a.H % 8 == 0 && ok(a.x, a.ldx) && a.ld_part % 8 == 0 && ok(a.residual, a.ld_res) &&
                   ok(a.residual_out, a.ld_res_out) && ok(a.normed, a.ld_normed) && aligned(a.weight, 16) &&
                   aligned(a.q, 8) && a.ldq % 8 == 0;
  return vec ? launch_norm<true>(a, s) : launch_norm<false>(a, s);
}

int launch_act_fp8(const ActArgs &a, const DeviceInfo &dev, cudaStream_t s) {
  const bool vec = a.I % 8 == 0 && aligned(a.x, 16) && a.ldx % 8 == 0 && aligned(a.q, 8) && a.ldq % 8 == 0;
  const int G = fp8_groups(a.I);
  const long long items = (long long)a.rows * G;
  long long grid = (items + 15) / 16;
  const long long most = (long long)dev.sm_count * 64;
  if (grid > most) grid = most;
  return launch(vec ? act_fp8_kernel<true> : act_fp8_kernel<false>, (unsigned)grid, 256, s, a, items, G);
}

}  // namespace moe_lora
