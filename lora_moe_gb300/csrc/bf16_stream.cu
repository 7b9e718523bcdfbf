// bf16_stream.cu -- the bf16 products of a few rows: at most 16 pairs share a
// weight, which is read once from HBM straight into registers.
//
//   y[f][n] = weight[f] * act(sum_k x[r][k] * w[e][n][k] + bias[e][n]) + residual[f][n]
//
// Bound by the weight's bytes, and for small weights by latency: there is no
// operand ring, tensor memory or cluster to set up.  A warp multiplies 16
// weight rows by 8 or 16 pairs with warp-level MMAs (m16n8k16, fp32 sums of 64
// columns, added in fp32) over its share of K; the CTA's warps split K or take
// further rows, and their sums meet in shared memory in a fixed order.  Measured:
// one row by 128 x 2048 2.4 us, by 4096 x 4096 7.3; one token's eight experts of
// 1536 x 2048 (50 MB) 9.6 us, 5.2 TB/s (12.3 on tcgen05); one row by 14336 x 8192
// (235 MB) 38.0 us, 6.2 TB/s.
//
// The tensor core sees the columns of a group of 64 in an order of its own:
// lane (r, t) holds bytes [16t, 16t + 16) and [64 + 16t, 64 + 16t + 16) of its
// row, four 16-byte pieces of each 64 bytes by four neighbouring lanes, and
// feeds 4 of them to each half of a step.  Weight and pairs use the same order.
#include <cuda_runtime.h>

#include <algorithm>

#include "bf16.h"
#include "bf16_epilogue.cuh"
#include "blocks.cuh"
#include "device_utils.cuh"
#include "launch.cuh"

namespace moe_lora {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kGroupBytes = kBf16Group * 2;

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// RG groups of 16 weight rows a CTA, K split over its other warps; NT tiles of 8 pairs.
// Groups of K in flight a warp, and registers for two CTAs an SM (three for
// single pairs, whose items are many), measured best of 2 to 4 groups and 2 or 3
// CTAs (1 x 4096 x 4096 7.3 us with four groups, 7.5 with two; 16 rows 14.4 and
// 9.3; single pairs 10.8 and 9.7).
constexpr int ctas_per_sm(int mode) { return mode == kNaive ? 3 : 2; }
constexpr int unroll(int mode, int nt) { return mode == kNaive || nt > 1 ? 2 : 4; }
template <int NT, int RG, int MODE>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(MODE)) bf16_stream_kernel(const Bf16Args p, int tiles) {
  constexpr int KS = kWarps / RG, kRowsCta = 16 * RG, U = unroll(MODE, NT);
  __shared__ float red[kWarps][8 * NT][16 + 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rg = warp % RG, ks = warp / RG;
  const int g = lane >> 2, t = lane & 3;
  wait_for_prior_grid();
  constexpr int kUnit = 8 * NT;   // positions of a unit
  const long long items = (long long)num_units<MODE>(p, kUnit) * tiles;
  const int kb0 = (int)((long long)p.KB * ks / KS), kb1 = (int)((long long)p.KB * (ks + 1) / KS);
  const int row_bytes = 2 * p.K;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int b = (int)(it / tiles), tile = (int)(it - (long long)b * tiles);
    const int e = block_expert<MODE>(p, b, kUnit);
    if (tile == 0 && warp == 0) flag_unit<MODE>(p, b, kUnit, e, lane);
    if (e < 0) continue;
    // this lane's pair of each tile; row offset, or -1
    int row[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int f = block_pair<MODE>(p, b, j * 8 + g, kUnit);
      row[j] = f < 0 ? -1 : pair_row<MODE>(p, f);
    }
    const int n0 = tile * kRowsCta + rg * 16;
    // rows past N are read from the last one and not stored
    const uint8_t *w0 = reinterpret_cast<const uint8_t *>(p.w + ((size_t)e * p.N + min(n0 + g, p.N - 1)) * p.ldw);
    const uint8_t *w1 = reinterpret_cast<const uint8_t *>(p.w + ((size_t)e * p.N + min(n0 + g + 8, p.N - 1)) * p.ldw);
    float acc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;

    for (int kb = kb0; kb < kb1; kb += U) {
      uint4 a[U][4], x[NT][U][2];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (kb + u >= kb1) continue;
        const int k = (kb + u) * kGroupBytes + 16 * t;
        if (k - 16 * t + kGroupBytes <= row_bytes) {
          a[u][0] = load_streamed(w0 + k);
          a[u][1] = load_streamed(w0 + k + 64);
          a[u][2] = load_streamed(w1 + k);
          a[u][3] = load_streamed(w1 + k + 64);
        } else {
          a[u][0] = load_tail(w0, k, row_bytes);
          a[u][1] = load_tail(w0, k + 64, row_bytes);
          a[u][2] = load_tail(w1, k, row_bytes);
          a[u][3] = load_tail(w1, k + 64, row_bytes);
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const uint8_t *xr = reinterpret_cast<const uint8_t *>(p.x + (size_t)max(row[j], 0) * p.ldx);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          x[j][u][0] = x[j][u][1] = make_uint4(0, 0, 0, 0);
          if (kb + u >= kb1 || row[j] < 0) continue;
          const int k = (kb + u) * kGroupBytes + 16 * t;
          if (k - 16 * t + kGroupBytes <= row_bytes) {
            x[j][u][0] = load_global(reinterpret_cast<const uint4 *>(xr + k));
            x[j][u][1] = load_global(reinterpret_cast<const uint4 *>(xr + k + 64));
          } else {
            x[j][u][0] = load_tail(xr, k, row_bytes);
            x[j][u][1] = load_tail(xr, k + 64, row_bytes);
          }
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
            mma_bf16(c, a0[2 * k], a1[2 * k], a0[2 * k + 1], a1[2 * k + 1], bb[2 * k], bb[2 * k + 1]);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[j][i] += c[i];
        }
      }
    }
    // sums of this warp: rows g and g + 8, pairs 2t and 2t + 1
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[warp][j * 8 + 2 * t + (i & 1)][g + (i >> 1) * 8] = acc[j][i];
    __syncthreads();
    constexpr int kLive = MODE == kNaive ? 1 : kUnit;
    for (int o = tid; o < kRowsCta * kLive; o += kThreads) {
      const int r = o % kRowsCta, c = o / kRowsCta, n = tile * kRowsCta + r;
      float v = 0.f;
#pragma unroll
      for (int q = 0; q < KS; ++q) v += red[q * RG + (r >> 4)][c][r & 15];
      finish_one<MODE>(p, block_pair<MODE>(p, b, c, kUnit), e, n, v);
    }
    __syncthreads();
  }
}

template <int NT, int RG, int MODE>
int launch_rg(const Bf16Args &a, long long units, cudaStream_t stream) {
  const int tiles = (a.N + 16 * RG - 1) / (16 * RG);
  return launch_dependent(bf16_stream_kernel<NT, RG, MODE>, (unsigned)std::min<long long>(units * tiles, 1ll << 30),
                          kThreads, 1, 0, stream, a, tiles);
}

// CTAs of 16, 32 or 64 rows, their eight warps splitting K in eight, four or
// two: the fewest rows whose CTAs are all resident at once, as a second wave
// costs more than a longer share of K.  A short K is not split further than it
// has groups for.
template <int NT, int MODE>
int launch_nt(const Bf16Args &a, long long units, const DeviceInfo &dev, cudaStream_t stream) {
  auto fits = [&](int rg) { return units * ((a.N + 16 * rg - 1) / (16 * rg)) <= ctas_per_sm(MODE) * dev.sm_count; };
  if (fits(1) && a.KB > 4) return launch_rg<NT, 1, MODE>(a, units, stream);
  if (fits(2) && a.KB > 2) return launch_rg<NT, 2, MODE>(a, units, stream);
  return launch_rg<NT, 4, MODE>(a, units, stream);
}

}  // namespace

int launch_bf16_stream(const Bf16Args &a, ProductMode mode, const DeviceInfo &dev, cudaStream_t stream) {
  if (mode == kNaive) return launch_nt<1, kNaive>(a, a.pairs, dev, stream);
  return a.pairs <= 8 ? launch_nt<1, kDense>(a, 1, dev, stream) : launch_nt<2, kDense>(a, 1, dev, stream);
}

}  // namespace moe_lora
