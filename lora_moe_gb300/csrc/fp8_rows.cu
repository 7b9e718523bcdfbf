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
// whose amax is four shuffles away.  Measured: norm of 8192 x 4096 with two
// parts (370 MB) 54 to 57 us, 6.5 to 6.8 TB/s; activation of 16384 x 14336
// (1.18 GB) 178 to 180 us, 6.6 TB/s; a decode batch of either 1.3 to 2 us,
// launch to launch.
#include <cuda_runtime.h>

#include <algorithm>

#include "device_utils.cuh"
#include "fp8.h"
#include "launch.cuh"

namespace moe_lora {

namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kMinScale = 1.17549435e-38f;   // 2^-126: a zero group has a normal scale, whose reciprocal is finite

// 8 bf16 columns, n of which exist; the scalar form takes any alignment.
template <bool VEC>
__device__ __forceinline__ uint4 load8(const uint16_t *p, int n) {
  uint32_t w[4] = {0, 0, 0, 0};
  if constexpr (VEC) {
    if (n > 0) return load_global(reinterpret_cast<const uint4 *>(p));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) w[i >> 1] |= (uint32_t)load_global(p + i) << (16 * (i & 1));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void widen8(const uint4 u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
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

// max(|a|, |b|, |c|), NaN if one of them is.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Quantise a group of 128 columns held by 16 neighbouring lanes, 8 columns
// each, n of which exist in this lane's 8.  A NaN makes the scale, and so the
// group, NaN.  n / s is computed as n * (1/s): one rounding more than a
// division, at most one unit of fp32 before the rounding to 3 bits.
template <bool VEC>
__device__ __forceinline__ void quantize8(const float (&v)[8], int n, uint8_t *q, float *scale, bool leader) {
  float m = max3_abs(max3_abs(v[0], v[1], v[2]), max3_abs(v[3], v[4], v[5]), max3_abs(v[6], v[7], 0.f));
#pragma unroll
  for (int d = 8; d; d >>= 1) m = max3_abs(m, __shfl_xor_sync(0xFFFFFFFFu, m, d), 0.f);
  const float t = m * (1.f / kE4m3Max);   // (within a unit of m / 448)
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
// thread) between the sum of squares and the output.  PB parts are loaded
// before the first of them is added.
template <int NV, int PB, bool VEC>
__global__ void __launch_bounds__(512) norm_fp8_kernel(const NormArgs p) {
  __shared__ float warp_sum[16];
  const int tid = threadIdx.x, threads = blockDim.x;
  const size_t m = blockIdx.x;
  const int G = fp8_groups(p.H);
  wait_for_prior_grid();
  float h[NV][8];
  uint4 raw[PB][NV], res[NV];
  auto load_parts = [&](int k0) {
#pragma unroll
    for (int k = 0; k < PB; ++k)
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = (v * threads + tid) * 8;
        raw[k][v] = load8<VEC>(p.x + m * p.ldx + (k0 + k) * p.ld_part + c, k0 + k < p.parts ? p.H - c : 0);
      }
  };
  load_parts(0);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * threads + tid) * 8;
    res[v] = load8<VEC>(p.residual + m * p.ld_res + c, p.residual ? p.H - c : 0);
  }
#pragma unroll
  for (int v = 0; v < NV; ++v) widen8(res[v], h[v]);
  for (int k0 = 0; k0 < p.parts; k0 += PB) {
    if (k0) load_parts(k0);
#pragma unroll
    for (int k = 0; k < PB; ++k)
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float a[8];
        widen8(raw[k][v], a);   // (zeros past the last part: adding them changes no value)
#pragma unroll
        for (int i = 0; i < 8; ++i) h[v][i] += a[i];
      }
  }
  float sum = 0.f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * threads + tid) * 8;
    if (p.residual_out) store8<VEC>(p.residual_out + m * p.ld_res_out + c, p.H - c, h[v]);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += h[v][i] * h[v][i];
    raw[0][v] = load8<VEC>(p.weight + c, p.H - c);
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
    widen8(raw[0][v], w);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[v][i] = h[v][i] * r * w[i];
    if (p.normed) store8<VEC>(p.normed + m * p.ld_normed + c, n, h[v]);
    const int g = c / kFp8Group;
    quantize8<VEC>(h[v], n, p.q + m * p.ldq + c, p.scales + m * G + g, (tid & 15) == 0 && g < G);
  }
}

// Exact quotients of 31-bit numbers by a divisor, with one multiplication
// (Granlund and Montgomery, "Division by invariant integers using
// multiplication", 1994).
struct FastDiv {
  uint32_t d, mul, shift;
  explicit FastDiv(uint32_t div) : d(div), shift(0) {
    while ((1ull << shift) < d) ++shift;
    mul = (uint32_t)(((1ull << 32) * ((1ull << shift) - d)) / d + 1);
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(n, mul) + n) >> shift; }
};

// silu(a) = a / (1 + exp(-a)), from exp(-|a|), which cannot overflow.
__device__ __forceinline__ float silu(float a) {
  const float e = __expf(-fabsf(a));
  const float r = __fdividef(a, 1.f + e);
  return a < 0.f ? r * e : r;
}

// 16 threads a group; UNROLL groups a thread at a time, so that enough loads
// are in flight.
constexpr int kActThreads = 256;
template <int UNROLL, bool VEC>
__global__ void __launch_bounds__(kActThreads, 8) act_fp8_kernel(const ActArgs p, uint32_t items, const FastDiv G) {
  const uint32_t lane16 = threadIdx.x & 15;
  const uint32_t per_cta = kActThreads / 16 * UNROLL;
  wait_for_prior_grid();
  uint4 gate[UNROLL], up[UNROLL];
  uint32_t row[UNROLL], grp[UNROLL];
  int n[UNROLL];
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const uint32_t it = blockIdx.x * per_cta + u * (kActThreads / 16) + (threadIdx.x >> 4);
    row[u] = G.div(it);
    grp[u] = it - row[u] * G.d;
    const uint32_t c = grp[u] * kFp8Group + lane16 * 8;
    n[u] = it < items ? p.I - (int)c : 0;
    const uint16_t *src = p.x + row[u] * p.ldx + c;
    gate[u] = load8<VEC>(src, n[u]);
    up[u] = load8<VEC>(src + p.I, n[u]);
    if (it >= items) row[u] = 0xFFFFFFFFu;
  }
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    float a[8], b[8];
    widen8(gate[u], a);
    widen8(up[u], b);
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = silu(a[i]) * b[i];
    const bool live = row[u] != 0xFFFFFFFFu;
    if (p.act) store8<VEC>(p.act + (long long)row[u] * p.ld_act + grp[u] * kFp8Group + lane16 * 8, n[u], a);
    quantize8<VEC>(a, n[u], p.q + (long long)row[u] * p.ldq + grp[u] * kFp8Group + lane16 * 8,
                   p.scales + (size_t)row[u] * G.d + grp[u], live && lane16 == 0);
  }
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

template <bool VEC>
int launch_norm(const NormArgs &a, const DeviceInfo &dev, cudaStream_t s) {
  const int vecs = (a.H + 7) / 8;
  // Few rows: a vector a thread and four parts in flight (latency).  Many: two
  // vectors a thread, so that more, smaller CTAs overlap their phases.
  const bool few = a.M <= 2 * dev.sm_count;
  const int nv = vecs > 1024 ? 4 : (vecs > 512 || (!few && vecs >= 128) ? 2 : 1);
  const int threads = ((vecs + nv - 1) / nv + 31) / 32 * 32;
  if (nv == 1)
    return a.parts > 2 ? launch_dependent(norm_fp8_kernel<1, 4, VEC>, a.M, threads, 1, 0, s, a)
                       : launch_dependent(norm_fp8_kernel<1, 2, VEC>, a.M, threads, 1, 0, s, a);
  if (nv == 2) return launch_dependent(norm_fp8_kernel<2, 2, VEC>, a.M, threads, 1, 0, s, a);
  return launch_dependent(norm_fp8_kernel<4, 1, VEC>, a.M, threads, 1, 0, s, a);
}

}  // namespace

// The 16-byte forms need whole vectors in every row: H a multiple of 8, rows
// and pointers on 16 bytes (8 for the 8-bit output).  Other layouts take the
// scalar form.
int launch_norm_fp8(const NormArgs &a, const DeviceInfo &dev, cudaStream_t s) {
  auto ok = [](const void *p, long long ld) { return p == nullptr || (aligned(p, 16) && ld % 8 == 0); };
  const bool vec = a.H % 8 == 0 && ok(a.x, a.ldx) && a.ld_part % 8 == 0 && ok(a.residual, a.ld_res) &&
                   ok(a.residual_out, a.ld_res_out) && ok(a.normed, a.ld_normed) && aligned(a.weight, 16) &&
                   aligned(a.q, 8) && a.ldq % 8 == 0;
  return vec ? launch_norm<true>(a, dev, s) : launch_norm<false>(a, dev, s);
}

int launch_act_fp8(const ActArgs &all, const DeviceInfo &dev, cudaStream_t s) {
  const bool vec = all.I % 8 == 0 && aligned(all.x, 16) && all.ldx % 8 == 0 && aligned(all.q, 8) && all.ldq % 8 == 0 &&
                   aligned(all.act, 16) && all.ld_act % 8 == 0;
  const int G = fp8_groups(all.I);
  const FastDiv div(G);
  // 31 bits of groups a launch
  const int most = (int)std::min<long long>(all.rows, ((1ll << 31) - 4096) / G);
  for (long long r0 = 0; r0 < all.rows; r0 += most) {
    ActArgs a = all;
    a.rows = (int)std::min<long long>(most, all.rows - r0);
    a.x += r0 * a.ldx;
    if (a.act) a.act += r0 * a.ld_act;
    a.q += r0 * a.ldq;
    a.scales += r0 * G;
    const uint32_t items = (uint32_t)a.rows * G;
    // two groups a thread once that leaves every SM's eight CTAs work, else one (latency)
    const bool many = items >= (uint32_t)dev.sm_count * 8 * 32;
    const uint32_t per_cta = kActThreads / 16 * (many ? 2 : 1), grid = (items + per_cta - 1) / per_cta;
    const auto kernel = many ? (vec ? act_fp8_kernel<2, true> : act_fp8_kernel<2, false>)
                             : (vec ? act_fp8_kernel<1, true> : act_fp8_kernel<1, false>);
    if (int st = launch_dependent(kernel, grid, kActThreads, 1, 0, s, a, items, div)) return st;
  }
  return 0;
}

}  // namespace moe_lora
