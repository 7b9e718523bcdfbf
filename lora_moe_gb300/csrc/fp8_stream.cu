// fp8_stream.cu -- the 8-bit products of a few rows: at most 16 pairs share a
// weight, which is read once from HBM straight into registers.
//
//   y[f][n] = bf16( weight[f] * sum_g sx[r][g] * sw[e][n/128][g] * sum_{k in group g} x[r][k] * w[e][n][k] )
//
// Bound by the weight's bytes, and for small weights by latency: there is no
// operand ring, tensor memory or cluster to set up.  A warp multiplies 16
// weight rows by 8 or 16 pairs with warp-level MMAs (m16n8k32, fp32 sums) over
// its share of K; the CTA's warps split K or take further rows, and their
// sums meet in shared memory in a fixed order.  Measured: one row by 2048 x
// 2048 2.5 us (4.9 on tcgen05), by 4096 x 7168 7.7 us (10.0), 3.8 TB/s; eight
// pairs of 2048 x 1536 7.0 us (8.5).  Past 32 MB of weights the tcgen05 kernel's
// ring keeps more bytes in flight and wins.
//
// The tensor core sees the columns of a group in an order of its own: lane
// (r, t) holds bytes [16t, 16t + 16) and [64 + 16t, 64 + 16t + 16) of its row,
// four 16-byte pieces of each 64 bytes by four neighbouring lanes, and feeds 4
// of them to each half of a step.  Weight and pairs use the same order.
#include <cuda_runtime.h>

#include <algorithm>

#include "device_utils.cuh"
#include "fp8.h"
#include "fp8_blocks.cuh"
#include "launch.cuh"

namespace moe_lora {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;

__device__ __forceinline__ uint4 load_weight(const uint8_t *p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

// 16 bytes of a row from column k on, zeros past the row's K columns; nothing
// past them is read.
__device__ __forceinline__ uint4 load_tail(const uint8_t *row, int k, int K) {
  if (k + 16 <= K) return load_global(reinterpret_cast<const uint4 *>(row + k));
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (k + i < K) w[i >> 2] |= (uint32_t)load_global(row + k + i) << (8 * (i & 3));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// RG groups of 16 weight rows a CTA, K split over its other warps; NT tiles of 8 pairs.
constexpr int ctas_per_sm(int mode) { return mode == kFp8Naive ? 3 : 2; }
// Two groups of K in flight a warp, and registers for two CTAs an SM (three for
// single pairs, whose items are many), measured best of 2 to 4 groups and 1 to
// 3 CTAs.
template <int NT, int RG, int MODE>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(MODE)) fp8_stream_kernel(const Fp8Args p, int tiles) {
  constexpr int KS = kWarps / RG, kRowsCta = 16 * RG;
  constexpr int U = 2;
  __shared__ float red[kWarps][8 * NT][16 + 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rg = warp % RG, ks = warp / RG;
  const int g = lane >> 2, t = lane & 3;
  wait_for_prior_grid();
  constexpr int kUnit = 8 * NT;   // positions of a unit
  const long long items = (long long)num_units<MODE>(p, kUnit) * tiles;
  const int kb0 = p.KB * ks / KS, kb1 = p.KB * (ks + 1) / KS;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int b = (int)(it / tiles), tile = (int)(it - (long long)b * tiles);
    const int e = block_expert<MODE>(p, b, kUnit);
    if (tile == 0 && warp == 0) flag_unit<MODE>(p, b, kUnit, e, lane);
    if (e < 0) continue;
    // this lane's pairs: of the operand (g), and of the sums (2t, 2t + 1); row offsets, or -1
    int row[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int f = block_pair<MODE>(p, b, j * 8 + g, kUnit);
      row[j] = f < 0 ? -1 : pair_row<MODE>(p, f);
    }
    const int n0 = tile * kRowsCta + rg * 16;
    // rows past N are read from the last one and not stored
    const uint8_t *w0 = p.w + ((size_t)e * p.N + min(n0 + g, p.N - 1)) * p.ldw;
    const uint8_t *w1 = p.w + ((size_t)e * p.N + min(n0 + g + 8, p.N - 1)) * p.ldw;
    const float *sw = p.w_scales + ((size_t)e * p.NB + min(n0, p.N - 1) / kFp8Group) * p.KB;
    float acc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;

    for (int kb = kb0; kb < kb1; kb += U) {
      uint4 a[U][4];
      float s[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (kb + u >= kb1) continue;
        const int k = (kb + u) * kFp8Group + 16 * t;
        s[u] = load_global(sw + kb + u);
        if (k - 16 * t + kFp8Group <= p.K) {
          a[u][0] = load_weight(w0 + k);
          a[u][1] = load_weight(w0 + k + 64);
          a[u][2] = load_weight(w1 + k);
          a[u][3] = load_weight(w1 + k + 64);
        } else {
          a[u][0] = load_tail(w0, k, p.K);
          a[u][1] = load_tail(w0, k + 64, p.K);
          a[u][2] = load_tail(w1, k, p.K);
          a[u][3] = load_tail(w1, k + 64, p.K);
        }
      }
      uint4 x[NT][U][2];
      float sx[NT][U][2];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int r0 = __shfl_sync(0xFFFFFFFFu, row[j], 8 * t), r1 = __shfl_sync(0xFFFFFFFFu, row[j], 8 * t + 4);
        const uint8_t *xr = p.x + (size_t)max(row[j], 0) * p.ldx;
        const float *s0 = p.x_scales + (size_t)max(r0, 0) * p.KB, *s1 = p.x_scales + (size_t)max(r1, 0) * p.KB;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          x[j][u][0] = x[j][u][1] = make_uint4(0, 0, 0, 0);
          sx[j][u][0] = sx[j][u][1] = 0.f;
          if (kb + u >= kb1) continue;
          const int k = (kb + u) * kFp8Group + 16 * t;
          if (row[j] >= 0) {
            if (k - 16 * t + kFp8Group <= p.K) {
              x[j][u][0] = load_global(reinterpret_cast<const uint4 *>(xr + k));
              x[j][u][1] = load_global(reinterpret_cast<const uint4 *>(xr + k + 64));
            } else {
              x[j][u][0] = load_tail(xr, k, p.K);
              x[j][u][1] = load_tail(xr, k + 64, p.K);
            }
          }
          if (r0 >= 0) sx[j][u][0] = load_global(s0 + kb + u);
          if (r1 >= 0) sx[j][u][1] = load_global(s1 + kb + u);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (kb + u >= kb1) continue;
        const uint32_t a0[8] = {a[u][0].x, a[u][0].y, a[u][0].z, a[u][0].w, a[u][1].x, a[u][1].y, a[u][1].z, a[u][1].w};
        const uint32_t a1[8] = {a[u][2].x, a[u][2].y, a[u][2].z, a[u][2].w, a[u][3].x, a[u][3].y, a[u][3].z, a[u][3].w};
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const uint4 b0 = x[j][u][0], b1 = x[j][u][1];
          const uint32_t bb[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
          float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_e4m3(c, a0[2 * k], a1[2 * k], a0[2 * k + 1], a1[2 * k + 1], bb[2 * k], bb[2 * k + 1]);
          const float sc0 = sx[j][u][0] * s[u], sc1 = sx[j][u][1] * s[u];
          acc[j][0] += c[0] * sc0;
          acc[j][1] += c[1] * sc1;
          acc[j][2] += c[2] * sc0;
          acc[j][3] += c[3] * sc1;
        }
      }
    }
    // sums of this warp: rows g and g + 8, pairs 2t and 2t + 1
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[warp][j * 8 + 2 * t + (i & 1)][g + (i >> 1) * 8] = acc[j][i];
    __syncthreads();
    constexpr int kLive = MODE == kFp8Naive ? 1 : kUnit;
    for (int o = tid; o < kRowsCta * kLive; o += kThreads) {
      const int r = o % kRowsCta, c = o / kRowsCta, n = tile * kRowsCta + r;
      float v = 0.f;
#pragma unroll
      for (int q = 0; q < KS; ++q) v += red[q * RG + (r >> 4)][c][r & 15];
      const int f = block_pair<MODE>(p, b, c, kUnit);
      if (f >= 0 && n < p.N) p.y[(size_t)f * p.ldy + n] = float_to_bf16_bits(v * pair_weight<MODE>(p, f));
    }
    __syncthreads();
  }
}

template <int NT, int RG, int MODE>
int launch_rg(const Fp8Args &a, long long units, cudaStream_t stream) {
  const int tiles = (a.N + 16 * RG - 1) / (16 * RG);
  return launch_dependent(fp8_stream_kernel<NT, RG, MODE>, (unsigned)std::min<long long>(units * tiles, 1ll << 30), kThreads,
                          1, 0, stream, a, tiles);
}

// CTAs of 16, 32 or 64 rows, their eight warps splitting K in eight, four or
// two: the fewest rows whose CTAs are all resident at once, as a second wave
// costs more than a longer share of K (8 pairs of 2048 x 1536: 6.8 us with 384
// CTAs of 32 rows, 7.9 with 768 of 16).  A short K is not split further than
// it has groups for.
template <int NT, int MODE>
int launch_nt(const Fp8Args &a, long long units, const DeviceInfo &dev, cudaStream_t stream) {
  auto fits = [&](int rg) { return units * ((a.N + 16 * rg - 1) / (16 * rg)) <= ctas_per_sm(MODE) * dev.sm_count; };
  if (fits(1) && a.KB > 4) return launch_rg<NT, 1, MODE>(a, units, stream);
  if (fits(2) && a.KB > 2) return launch_rg<NT, 2, MODE>(a, units, stream);
  return launch_rg<NT, 4, MODE>(a, units, stream);
}

}  // namespace

int launch_fp8_stream(const Fp8Args &a, Fp8Mode mode, const DeviceInfo &dev, cudaStream_t stream) {
  if (mode == kFp8Naive) return launch_nt<1, kFp8Naive>(a, a.pairs, dev, stream);
  return a.pairs <= 8 ? launch_nt<1, kFp8Dense>(a, 1, dev, stream) : launch_nt<2, kFp8Dense>(a, 1, dev, stream);
}

}  // namespace moe_lora
