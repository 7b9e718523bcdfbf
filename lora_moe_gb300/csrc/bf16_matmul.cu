// bf16_matmul.cu -- bf16 matrix products, dense and over a MoE layer's experts,
// on the 5th-generation tensor cores, with bias, activation, the router's
// weight and a residual in the epilogue (bf16_epilogue.cuh):
//
//   y[f][n] = weight[f] * act(sum_k x[r][k] * w[e][n][k] + bias[e][n]) + residual[f][n]
//
// with r the row of x that pair f reads and e its expert.
//
// Two kernels, both persistent, with a warp that loads (TMA), one that issues
// the MMAs and epilogue warps:
//   narrow  the weight on the 128 rows of the MMA, 16 to 64 pairs on its
//           columns: few pairs for each weight (decode), bound by the weight's
//           bytes.  Where there are few items, clusters of CTAs split K, their
//           partial sums exchanged through distributed shared memory and added
//           in a fixed order.  gpt-oss-shaped w2 decode (1.8 GB of weights): 264
//           us, 6.9 TB/s; 64 x 2880 x 4096 with a residual 9.2 us, of which the
//           bytes take 3.7, set-up and first loads 3.5, the exchange and the way
//           out 2.5.
//   wide    pairs of CTAs (cta_group::2), 256 of the weight's rows by up to 256
//           pairs, on rows gathered into the blocks' order: bound by the tensor
//           cores, and over seconds by power.  Dense 8192 x 4096 x 14336: 488 us
//           (1.97 PFLOP/s), 570 in calls that go on for seconds; Mixtral-shaped
//           w13 prefill 2.28 ms (1.69 PFLOP/s) and 2.49.  Experts of few rows are
//           bound by the weight's bytes: 1024 tokens, 8 of 128 experts of 2048 x
//           1536, 148 us, 123 of them at the copy rate.  In chunks, K split over
//           two pairs: 4096 x 256, K of 7168, to fp32 20.4 us.
// Products of few rows are bf16_stream.cu's.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "bf16.h"
#include "bf16_epilogue.cuh"
#include "blocks.cuh"
#include "device_utils.cuh"
#include "gather.h"
#include "launch.cuh"
#include "narrow.cuh"
#include "stream_pipeline.cuh"

namespace moe_lora {

namespace {

constexpr int kGroupBytes = kBf16Group * 2;       // of a row
constexpr int kTileBytes = kRows * kGroupBytes;   // 128 rows of one group: 16 KB

struct Bf16Maps {
  CUtensorMap w;      // [E][N][K] in bytes, box 1 x 128 x 128
  CUtensorMap x[4];   // [rows][K], box BT x 128 (dense), 1 x 128 (gathered by row); wide: 128, 64, 32 and 16 x 128
};

// Launch shape of a call.
struct Bf16Cfg {
  int stages;      // operand ring
  int nt;          // output tiles along N
  int cluster;     // CTAs of a cluster, which splits K
  int tile_rows;   // pairs of a tile (wide, dense)
  int chunk;       // groups of K that the tensor cores add up (wide, chunked)
  int stage_bytes; // (wide)
  int off_red, off_tile, off_list, off_ctrl;
  int list;        // units that the list of live ones holds (0: none is made)
  int smem_bytes;
};

// ------------------------------------------------------------------ narrow

constexpr int kMaxRing = 5;    // stages: 5 gave 264 us, 4 265, 3 272 and 6 272 (64 tokens, 4 of 128 experts of 2880 x 2880)
constexpr int kMaxSmem = 227 * 1024;
// Groups of K whose products the tensor cores add up.  Their additions truncate,
// so a long sum drifts (K of 7168, products of one sign: 2.4e-5 of the sum); the
// epilogue adds the chunks in fp32, rounding to nearest.  The wide kernel's chunks
// are longer where y is bf16, 2^-17 of the sum at most: us with 4 / 8 / 16 groups and with all of
// K, 8192 x 4096 x 14336 565 / 531 / 491 / 489, sorted 4096 tokens, 8 of 64 experts
// of 2048 x 2048 261 / 236 / 222 / 221.
constexpr int kChunk = 4, kLongChunk = 16;

template <int BT>
struct Narrow {
  static constexpr int kGroup = kTileBytes + BT * kGroupBytes;
  static constexpr int kStage = 2 * kGroup;           // two groups a stage, requested together
  static constexpr int kBufs = 4;                     // accumulators in tensor memory
  static constexpr int kCols = kBufs * BT;            // power of two, >= 32
};

struct NarrowCtrl {
  uint64_t full[kMaxRing], empty[kMaxRing];
  uint64_t tfull[4], tempty[4];
  uint64_t red_full;
  uint64_t done;                             // every MMA of this CTA
  uint32_t tmem;
  int abort;
  int live;                                  // units in the list
  int warp_live[kNarrowThreads / 32];
};

template <int BT, int MODE>
__global__ void __launch_bounds__(kNarrowThreads, 1)
    bf16_narrow_kernel(const __grid_constant__ Bf16Maps maps, const Bf16Args p, const Bf16Cfg cfg) {
  using C = Narrow<BT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  NarrowCtrl &ctl = *reinterpret_cast<NarrowCtrl *>(smem + cfg.off_ctrl);
  volatile int *abort = &ctl.abort;
  const int cs = cfg.cluster;

  if (warp == 0) {
    if (lane < cfg.stages) {
      mbar_init(&ctl.full[lane], 1);
      mbar_init(&ctl.empty[lane], 1);
    }
    if (lane < C::kBufs) {
      mbar_init(&ctl.tfull[lane], 1);
      mbar_init(&ctl.tempty[lane], 4);
    }
    if (lane == 0) {
      mbar_init(&ctl.red_full, 1);
      mbar_init(&ctl.done, 1);
      ctl.abort = 0;
      prefetch_tensor_map(&maps.w);
      prefetch_tensor_map(&maps.x[0]);
    }
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&ctl.tmem, C::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (cs > 1) cluster_arrive_release();   // this CTA's barriers are initialised; waited for before anything is sent
  wait_for_prior_grid();
  let_next_grid_start();
  const uint32_t tmem = ctl.tmem;
  const int all_units = num_units<MODE>(p, BT);
  int units = all_units;
  const int *list = nullptr;
  if (MODE == kSorted && cfg.list && units <= cfg.list) {
    int *l = reinterpret_cast<int *>(smem + cfg.off_list);
    list_units<BT>(p, units, l, ctl.warp_live, &ctl.live, tid);
    list = l;
    units = ctl.live;
  }
  const int items = units * cfg.nt;
  auto unit = [&](int i) { return list ? list[i] : i; };
  NarrowWork wk(items, p.KB, cs);
  bool waited = false;   // for the cluster's barriers

  if (warp == 0) {
    // ---------------- operands: the weight's tile, and the pairs' rows
    int s = 0;
    uint32_t ph = 0, fills = 0;
    bool go = true;   // falls with a wait that gave up: nothing more is requested
    while (go && wk.advance()) {
      const int ui = wk.it / cfg.nt, nt = wk.it - ui * cfg.nt, b = unit(ui), e = block_expert<MODE>(p, b, BT);
      if (e < 0) continue;
      int row[4];
      bool mine = false;   // lane i gathers rows 4i .. 4i+3; groups without a pair are left as they are
      if (MODE != kDense && lane < BT / 4) {
        int some = -1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int f = block_pair<MODE>(p, b, lane * 4 + i, BT);
          row[i] = f < 0 ? -1 : pair_row<MODE>(p, f);
          if (row[i] >= 0) some = row[i];
        }
        mine = some >= 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (row[i] < 0) row[i] = some;
      }
      const int groups = MODE == kDense ? BT / 4 : __popc(__ballot_sync(0xFFFFFFFFu, mine));
      for (int kb = wk.kb0; kb < wk.kb1; kb += 2) {
        go = __all_sync(0xFFFFFFFFu, mbar_wait(&ctl.empty[s], ph ^ 1, abort, p.err));
        if (!go) break;
        ++fills;
        uint8_t *st = smem + (size_t)s * C::kStage;
        const int n = min(2, wk.kb1 - kb);
        if (elect_one()) {
          mbar_arrive_expect_tx(&ctl.full[s], n * (kTileBytes + groups * 4 * kGroupBytes));
          for (int i = 0; i < n; ++i)
            tma_load_3d(st + i * C::kGroup, &maps.w, (kb + i) * kGroupBytes, nt * kRows, e, &ctl.full[s]);
          if (MODE == kDense)
            for (int i = 0; i < n; ++i)
              tma_load_2d(st + i * C::kGroup + kTileBytes, &maps.x[0], (kb + i) * kGroupBytes, b * BT, &ctl.full[s]);
        }
        __syncwarp();
        if (MODE != kDense && mine)
          for (int i = 0; i < n; ++i)
            tma_gather4(st + i * C::kGroup + kTileBytes + lane * 4 * kGroupBytes, &maps.x[0], (kb + i) * kGroupBytes, row,
                        &ctl.full[s]);
        if (++s == cfg.stages) { s = 0; ph ^= 1; }
      }
    }
    // the copies have landed, the stages' hand-backs arrived and the MMAs completed before this CTA exits
    __syncwarp();
    drain_ring_warp(ctl.full, cfg.stages, fills, lane);
    drain_ring_warp(ctl.empty, cfg.stages, fills, lane);
    drain_wait(&ctl.done, 0);
    __syncwarp();
  } else if (warp == 1) {
    // ---------------- MMA: each chunk of K into an accumulator of its own
    constexpr uint32_t idesc = make_idesc_bf16(kRows, BT);
    const uint64_t desc0 = make_sdesc_sw128(smem_addr(smem));   // (addresses in units of 16 bytes)
    int s = 0, a = 0;
    uint32_t ph = 0, aph = 0;
    while (wk.advance()) {
      if (block_expert<MODE>(p, unit(wk.it / cfg.nt), BT) < 0) continue;
      for (int kb = wk.kb0; kb < wk.kb1; ++kb) {
        const int at = (kb - wk.kb0) % kChunk, i = at & 1;
        const bool last = i == 1 || kb + 1 == wk.kb1;                    // of the stage
        const bool last_of_chunk = at == kChunk - 1 || kb + 1 == wk.kb1;
        if (at == 0) mbar_wait(&ctl.tempty[a], aph ^ 1, abort, p.err);
        if (i == 0) mbar_wait(&ctl.full[s], ph, abort, p.err);
        tc_fence_after();
        const uint64_t dw = desc0 + (s * C::kStage + i * C::kGroup) / 16, dx = dw + kTileBytes / 16;
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kBf16Group / 16; ++k)
            tc_mma_bf16(tmem + a * BT, dw + k * 2, dx + k * 2, idesc, at > 0 || k > 0);
          if (last) tc_commit(&ctl.empty[s]);
          if (last_of_chunk) tc_commit(&ctl.tfull[a]);
        }
        __syncwarp();
        if (last && ++s == cfg.stages) { s = 0; ph ^= 1; }
        if (last_of_chunk && ++a == C::kBufs) { a = 0; aph ^= 1; }
      }
    }
    if (elect_one()) tc_commit(&ctl.done);
    __syncwarp();
  } else if (warp == 2) {
    // (clusters have an item each for all blocks that an align writes)
    if (cs > 1 && blockIdx.x == 0 && lane == 0 && items > (int)gridDim.x / cs) flag_error(p.err, MOE_LORA_DEVERR_CAPACITY);
  } else if (warp == 3) {
    // ---------------- what is out of range, each unit once
    if (MODE != kDense)
      for (int b = blockIdx.x; b < all_units; b += gridDim.x)
        flag_unit<MODE>(p, b, BT, block_expert<MODE>(p, b, BT), lane);
  } else {
    // ---------------- epilogue: this thread's weight row, BT pairs; then four rows, a pair a warp
    const int row = (warp - 4) * 32 + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)(warp - 4) << 21);   // lane offset 32 * quarter in bits 16..31
    float *sums = reinterpret_cast<float *>(smem + cfg.off_tile);     // [this CTA's positions][kRows]
    const int out = out_kind(p);
    int a = 0;
    uint32_t aph = 0;
    while (wk.advance()) {
      const int ui = wk.it / cfg.nt, nt = wk.it - ui * cfg.nt, b = unit(ui), e = block_expert<MODE>(p, b, BT);
      if (e < 0) continue;
      // the pair of position `lane` (dense: not used), and biases of the four rows
      const int step = out == kOutSingly ? 32 : 1, col = out == kOutSingly ? lane : lane * 4, n = nt * kRows + col;
      int pair = -1;
      float weight = 0.f, bias[4];
      if (MODE != kDense) {
        static_assert(MODE == kDense || BT <= 32, "a lane for each position");
        pair = lane < BT ? block_pair<MODE>(p, b, lane, BT) : -1;
        weight = pair < 0 ? 0.f : pair_weight<MODE>(p, pair);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) bias[i] = bias_of(p, e, n + i * step);
      if (MODE == kDense && p.residual) {   // this warp's rows of it, 64 bytes a lane
        const int from = cs == 1 ? 0 : join_first(BT, cs, wk.rank), to = cs == 1 ? BT : join_first(BT, cs, wk.rank + 1);
        const int at = nt * kRows + (lane & 7) * (p.y_f32 ? 16 : 32);
        for (int t = from + (warp - 4) * 4 + (lane >> 3); t < to; t += 16)
          if (at < min(p.N, (nt + 1) * kRows) && b * BT + t < p.pairs) fetch_residual(p, b * BT + t, at);
      }
      float acc[BT];
#pragma unroll
      for (int c = 0; c < BT; ++c) acc[c] = 0.f;
      for (int kb = wk.kb0; kb < wk.kb1; kb += kChunk) {
        mbar_wait(&ctl.tfull[a], aph, abort, p.err);
        tc_fence_after();
#pragma unroll
        for (int c0 = 0; c0 < BT; c0 += 16) {
          uint32_t v[16];
          tmem_ld16(lane_addr + a * BT + c0, v);
          tc_wait_ld();
          tc_pin(v);
#pragma unroll
          for (int c = 0; c < 16; ++c) acc[c0 + c] += __uint_as_float(v[c]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.tempty[a]);
        if (++a == C::kBufs) { a = 0; aph ^= 1; }
      }
      constexpr int kLive = MODE == kNaive ? 1 : BT;   // positions that can hold a pair
      int first = 0, last = kLive;
      if (cs == 1) {
        named_barrier(1, 128);   // the last item's sums are out
#pragma unroll
        for (int c = 0; c < kLive; ++c) sums[c * kRows + row] = acc[c];
      } else {
        first = BT, last = 0;
        join_ranks<BT, MODE == kNaive>(acc, cs, wk.rank, row, smem + cfg.off_red, &ctl.red_full, abort, p.err,
                                       [&](int t, const auto &v) {
                                         constexpr int W = sizeof(v) / sizeof(float);
                                         first = min(first, t);
                                         last = t + W;
#pragma unroll
                                         for (int i = 0; i < W; ++i) sums[(t - first + i) * kRows + row] = v[i];
                                       });
        waited = true;
      }
      named_barrier(1, 128);
      auto put_out = [&](auto kind) {
#pragma unroll 1
        for (int c = first + warp - 4; c < last; c += 16) {
          int f[4];
          float w[4], v[16];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int t = c + 4 * i;
            if (MODE == kDense) {
              f[i] = b * BT + t < p.pairs ? b * BT + t : -1;
            } else {
              f[i] = __shfl_sync(0xFFFFFFFFu, pair, t & 31);
              w[i] = __shfl_sync(0xFFFFFFFFu, weight, t & 31);
            }
            if (t >= last || n >= p.N) f[i] = -1;
            const float *from = sums + (min(t, last - 1) - first) * kRows + col;
            if constexpr (decltype(kind)::value == kOutSingly) {
#pragma unroll
              for (int k = 0; k < 4; ++k) v[4 * i + k] = from[k * step];
            } else {
              const float4 u = *reinterpret_cast<const float4 *>(from);
              v[4 * i] = u.x, v[4 * i + 1] = u.y, v[4 * i + 2] = u.z, v[4 * i + 3] = u.w;
            }
          }
          finish_fours<MODE, decltype(kind)::value, 4>(p, f, w, n, step, bias, v);
        }
      };
      if (out == kOutBf16) put_out(std::integral_constant<int, kOutBf16>());
      else if (out == kOutF32) put_out(std::integral_constant<int, kOutF32>());
      else put_out(std::integral_constant<int, kOutSingly>());
    }
  }
  if (cs > 1 && !waited) cluster_wait();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
}

// ------------------------------------------------------------------ wide

// Pairs of CTAs (cta_group::2): 256 of the weight's rows on the rows of the MMA,
// up to 256 pairs on its columns (as many as the tile has, in steps of 32: MMAs
// of a partly filled tile take less).  Each CTA holds 128 of the weight's rows
// and half of the pairs', at most 32 KB a group, and 128 x 256 of an
// accumulator in tensor memory, twice.
//
// CHUNKED = false: an accumulator takes all of K, at most kLongChunk groups; one is read
// while the next item's is added up.  CHUNKED: an accumulator takes a chunk of K, and the
// epilogue adds the chunks in registers.  (A K of one chunk by the second: 8192 x 512
// x 8192 59 -> 68 us, 2048 x 1024 x 8192 25.7 -> 27.5.)  A cluster
// of several pairs splits K where there are few items: each pair's sums go to
// the pair that owns the columns, in the operand ring's memory.
constexpr int kWideThreads = 384;
constexpr int kWideN = 256;
constexpr int kWideRing = 12;                    // stages at most; each 128 of the weight's rows, and half of a tile's pairs'
constexpr int kPartBytes = 32 * 32 * 4;          // 32 pairs' sums of 32 rows, on their way out, for each epilogue warp
constexpr int kPart = 32;                        // columns of an accumulator that a warp takes at a time
constexpr int kParts = kTileRows / kPart / 2;    // of one of the two warps of a lane quarter
// Tiles that are neighbours in the order of the items: the pairs' rows of so many
// stay in L2 while the weight goes by (Mixtral-shaped w13 prefill reads 134 MB of
// rows 112 times otherwise).  In calls that go on for seconds: dense 8192 x 4096 x
// 14336 580 us with 16, 591 with 8 and 606 with 4 or 32; that prefill 2.61 ms with 16,
// 2.57 with 8, 2.69 with 32.
constexpr int raster(int mode) { return mode == kDense ? 16 : 8; }
// Registers a thread where chunks are added: loading and MMA warps, epilogue warps.
constexpr int kWideRegsIssue = 56, kWideRegsEpilogue = 216;

struct WideCtrl {
  uint64_t full[kWideRing], empty[kWideRing];
  uint64_t tfull[2], tempty[2];
  uint64_t done;       // every MMA of the pair
  uint64_t red_full;   // the other pairs' sums
  uint32_t tmem;
  int abort;
};

// The items of a pair: tiles of rows in groups of RASTER, within a group the
// weight's tiles one after the other.
template <int RASTER>
struct WideWork {
  int ntiles, nt_all, it, step, items;
  int t, nt;   // of the item
  __device__ __forceinline__ WideWork(int tiles, int nts, int first, int stride)
      : ntiles(tiles), nt_all(nts), it(first - stride), step(stride), items(tiles * nts) {}
  __device__ __forceinline__ bool advance() {
    it += step;
    if (it >= items) return false;
    const int g = it / (RASTER * nt_all), r = it - g * RASTER * nt_all, size = min(RASTER, ntiles - g * RASTER);
    nt = r / size;
    t = g * RASTER + r - nt * size;
    return true;
  }
};

__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

template <int MODE, bool CHUNKED>
__global__ void __launch_bounds__(kWideThreads, 1)
    bf16_wide_kernel(const __grid_constant__ Bf16Maps maps, const Bf16Args p, const WideTile *tiles, const Bf16Cfg cfg) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  WideCtrl &ctl = *reinterpret_cast<WideCtrl *>(smem + cfg.off_ctrl);
  volatile int *abort = &ctl.abort;
  const int rank = blockIdx.x & 1;   // rank 0 issues the pair's MMAs
  // the pair in its cluster, and its share of K
  constexpr bool kSplit = CHUNKED && MODE == kDense;
  const int pairs = kSplit ? cfg.cluster >> 1 : 1, q = kSplit ? (blockIdx.x >> 1) % pairs : 0;
  const int kb0 = (int)((long long)p.KB * q / pairs), kb1 = (int)((long long)p.KB * (q + 1) / pairs);
  const int leader = q * 2;          // the pair's rank 0 in the cluster

  const int stages = cfg.stages, stage_bytes = cfg.stage_bytes;
  if (warp == 0) {
    if (lane < stages) {
      mbar_init(&ctl.full[lane], 1);
      mbar_init(&ctl.empty[lane], 1);
    }
    if (lane < 2) {
      mbar_init(&ctl.tfull[lane], 1);
      mbar_init(&ctl.tempty[lane], 16);   // the epilogue warps of both CTAs
    }
    if (lane == 0) {
      mbar_init(&ctl.done, 1);
      mbar_init(&ctl.red_full, 1);
      ctl.abort = 0;
    }
    if (lane < 5) prefetch_tensor_map(lane < 4 ? &maps.x[lane] : &maps.w);
    fence_barrier_init();
  }
  __syncthreads();
  cluster_arrive_release();   // the barriers are initialised
  if (warp == 1) tmem_alloc_pair(&ctl.tmem, 512);
  tc_fence_before();
  cluster_wait();
  __syncthreads();
  tc_fence_after();
  wait_for_prior_grid();
  let_next_grid_start();
  const uint32_t tmem = ctl.tmem;
  const int height = cfg.tile_rows;   // of a dense call's tiles
  const int ntiles = MODE == kDense ? (p.pairs + height - 1) / height : load_global(&tiles[0].row0);
  WideWork<raster(MODE)> wk(ntiles, cfg.nt, blockIdx.x / (2 * pairs), gridDim.x / (2 * pairs));
  auto tile = [&](int t) {
    if (MODE == kDense) return WideTile{t * height, min(height, p.pairs - t * height), 0, 0};
    const int4 v = load_global(reinterpret_cast<const int4 *>(tiles) + 1 + t);
    return WideTile{v.x, v.y, v.z, 0};
  };
  auto columns = [](int rows) { return (rows + kPart - 1) / kPart * kPart; };   // of the MMA

  if (warp < 4) {
    if (CHUNKED) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kWideRegsIssue));
    if (warp == 0) {
      // ---------------- operands: this CTA's half of the weight's rows, and of the pairs'
      const uint32_t full0 = cluster_map(smem_addr(&ctl.full[0]), leader);
      int s = 0;
      uint32_t ph = 0, fills = 0;
      bool go = true;   // falls with a wait that gave up: nothing more is requested
      while (go && wk.advance()) {
        const WideTile t = tile(wk.t);
        const int half = columns(t.rows) / 2, row0 = t.row0 + rank * half;
        const uint32_t bytes = 2 * kTileBytes + 2 * half * kGroupBytes;
        // two groups at a time: 256 consecutive bytes of each row
        for (int kb = kb0; kb < kb1; kb += 2) {
          const int n = min(2, kb1 - kb);
          const int s1 = s + 1 == stages ? 0 : s + 1;
          const uint32_t ph1 = s + 1 == stages ? ph ^ 1 : ph;
          bool ok = mbar_wait(&ctl.empty[s], ph ^ 1, abort, p.err);
          if (n > 1) ok = mbar_wait(&ctl.empty[s1], ph1 ^ 1, abort, p.err) && ok;
          go = __all_sync(0xFFFFFFFFu, ok);
          if (!go) break;
          fills += n;
          if (elect_one()) {
            for (int i = 0; i < n; ++i) {
              const int at = i ? s1 : s;
              if (rank == 0) mbar_arrive_expect_tx(&ctl.full[at], bytes);
              tma_load_3d_pair(smem + (size_t)at * stage_bytes, &maps.w, (kb + i) * kGroupBytes,
                               wk.nt * kWideN + rank * kRows, t.expert, full0 + at * 8);
            }
            for (int i = 0; i < n; ++i) {
              const int at = i ? s1 : s;
              uint8_t *st = smem + (size_t)at * stage_bytes + kTileBytes;
              // half is a multiple of 16, at most 128: a box for each of its bits
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int box = kRows >> j;
                if (half & box) {
                  const int r = half & ~(2 * box - 1);
                  tma_load_2d_pair(st + r * kGroupBytes, &maps.x[j], (kb + i) * kGroupBytes, row0 + r, full0 + at * 8);
                }
              }
            }
          }
          __syncwarp();
          s = n > 1 ? s1 : s;
          ph = n > 1 ? ph1 : ph;
          if (++s == stages) { s = 0; ph ^= 1; }
        }
      }
      // The pair's copies have landed (rank 0's barriers count both CTAs'), the
      // hand-backs of the last stages have arrived here and the MMAs have
      // completed before the pair exits: the epilogue waits for neither.
      __syncwarp();
      if (rank == 0) drain_ring_warp(ctl.full, stages, fills, lane);
      drain_ring_warp(ctl.empty, stages, fills, lane);
      drain_wait(&ctl.done, 0);
    } else if (warp == 1 && rank == 0) {
      // ---------------- MMA, for both CTAs
      const uint64_t desc0 = make_sdesc_sw128(smem_addr(smem));   // (addresses in units of 16 bytes)
      const uint16_t both = (uint16_t)(3u << leader);
      int s = 0, a = 0;
      uint32_t ph = 0, aph = 0;
      bool more = wk.advance();
      int rows = more ? tile(wk.t).rows : 0;
      while (more) {
        const uint32_t idesc = make_idesc_bf16(2 * kRows, columns(rows));
        more = wk.advance();
        rows = more ? tile(wk.t).rows : 0;   // the next item's, on its way meanwhile
        for (int kb = kb0, at = 0; kb < kb1; ++kb) {   // at: group of the accumulator
          const bool last = kb + 1 == kb1 || (CHUNKED && at + 1 == cfg.chunk);
          if (at == 0) mbar_wait(&ctl.tempty[a], aph ^ 1, abort, p.err);
          mbar_wait(&ctl.full[s], ph, abort, p.err);
          tc_fence_after();
          const uint64_t dw = desc0 + s * (stage_bytes >> 4), dx = dw + (kTileBytes >> 4);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kBf16Group / 16; ++k)
              tc_mma_bf16_pair(tmem + a * kTileRows, dw + k * 2, dx + k * 2, idesc, at > 0 || k > 0);
            tc_commit_pair(&ctl.empty[s], both);
            if (last) tc_commit_pair(&ctl.tfull[a], both);
          }
          __syncwarp();
          if (++s == stages) { s = 0; ph ^= 1; }
          ++at;
          if (last) {
            at = 0;
            a ^= 1;
            if (a == 0) aph ^= 1;
          }
        }
      }
      if (elect_one()) tc_commit_pair(&ctl.done, both);
    }
    __syncwarp();
    if (kSplit && pairs > 1) {   // the ring is free for other pairs' sums
      cluster_arrive_release();
      cluster_wait();
    }
  } else {
    if (CHUNKED) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kWideRegsEpilogue));
    // ---------------- epilogue: this thread's weight row; 32 pairs at a time, every other 32 of the tile's
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const uint32_t lane_addr = tmem + ((uint32_t)quarter << 21);
    const uint32_t tempty0 = cluster_map(smem_addr(&ctl.tempty[0]), leader);
    float *stage = reinterpret_cast<float *>(smem + cfg.off_tile + (warp - 4) * kPartBytes);   // [pair][row]
    int a = 0;
    uint32_t aph = 0;
    const int out = out_kind(p);
    bool met = false;   // the cluster's pairs, at the barrier that frees the ring
    while (wk.advance()) {
      const WideTile t = tile(wk.t);
      const int cols = columns(t.rows);
      // four of the 32 rows, for the way out
      const int step = out == kOutSingly ? 8 : 1, col = (lane & 7) * (out == kOutSingly ? 1 : 4);
      const int n = wk.nt * kWideN + rank * kRows + quarter * 32 + col;
      float bias[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) bias[i] = bias_of(p, t.expert, n + i * step);
      auto hand_back = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote_relaxed(tempty0 + a * 8);   // (only tensor memory is handed back)
        a ^= 1;
        if (a == 0) aph ^= 1;
      };
      // The sums of `count` pairs (a multiple of 8) that the warp has put into
      // `stage`: pair k is number off + k % width of part i + k / width.
      auto put_out = [&](int i, int off, int width, int count) {
        const uint32_t inv = (65535u + width) / width;   // k / width is k * inv >> 16 for k below 32
        auto row = [&](int k) {                          // of the tile
          const int part = k * inv >> 16;
          return (2 * (i + part) + half) * kPart + off + k - part * width;
        };
        int f = -1;
        float weight = 0.f;
        if (MODE != kDense) {
          const int r = row(lane);
          if (lane < count && r < t.rows) f = load_global(p.sorted_token_ids + t.row0 + r);
          if ((unsigned)f >= (unsigned)p.pairs) f = -1;
          if (f >= 0) weight = pair_weight<MODE>(p, f);
        }
        __syncwarp();
        auto rows = [&](auto kind) {
#pragma unroll 1
          for (int j0 = 0; j0 < count; j0 += 16) {
            int fj[4];
            float w[4], v[16];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int j = j0 + 4 * k + (lane >> 3);
              if (MODE == kDense) {
                fj[k] = row(j) < t.rows ? t.row0 + row(j) : -1;
              } else {
                fj[k] = __shfl_sync(0xFFFFFFFFu, f, j);
                w[k] = __shfl_sync(0xFFFFFFFFu, weight, j);
              }
              if (n >= p.N || j >= count) fj[k] = -1;
              const float *from = stage + j * 32 + col;
              if constexpr (decltype(kind)::value == kOutSingly) {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[4 * k + i] = from[i * step];
              } else {
                const float4 u = *reinterpret_cast<const float4 *>(from);
                v[4 * k] = u.x, v[4 * k + 1] = u.y, v[4 * k + 2] = u.z, v[4 * k + 3] = u.w;
              }
            }
            finish_fours<MODE, decltype(kind)::value, 4>(p, fj, w, n, step, bias, v);
          }
        };
        // (an fp32 y is added up in chunks, and dense)
        if (out == kOutBf16) rows(std::integral_constant<int, kOutBf16>());
        else if (kSplit && out == kOutF32) rows(std::integral_constant<int, kOutF32>());
        else rows(std::integral_constant<int, kOutSingly>());
        __syncwarp();
      };
      if (MODE == kDense && p.residual) {
        const int at = wk.nt * kWideN + rank * kRows + quarter * 32;
        for (int r = half * kPart + lane; r < t.rows; r += 2 * kPart)
          if (at < p.N) fetch_residual(p, t.row0 + r, at);
      }
      if constexpr (!CHUNKED) {
        mbar_wait(&ctl.tfull[a], aph, abort, p.err);
        tc_fence_after();
#pragma unroll 1
        for (int i = 0; i < kParts; ++i) {
          const int c0 = (2 * i + half) * kPart;
          if (c0 >= cols) break;
          uint32_t raw[kPart];
          tmem_ld32(lane_addr + a * kTileRows + c0, raw);
          tc_wait_ld();
          tc_pin(raw);
#pragma unroll
          for (int j = 0; j < kPart; ++j) stage[j * 32 + lane] = __uint_as_float(raw[j]);
          put_out(i, 0, kPart, kPart);
        }
        hand_back();
      } else {
        f32x2 acc[kParts][kPart / 2];
#pragma unroll
        for (int i = 0; i < kParts; ++i)
#pragma unroll
          for (int j = 0; j < kPart / 2; ++j) acc[i][j] = 0;
#pragma unroll 1
        for (int kb = kb0; kb < kb1; kb += cfg.chunk) {
          mbar_wait_lean(smem_addr(&ctl.tfull[0]) + a * 8, aph, abort, p.err);
          tc_fence_after();
#pragma unroll
          for (int i = 0; i < kParts; ++i) {
            if ((2 * i + half) * kPart < cols) {
              uint32_t raw[kPart];
              tmem_ld32(lane_addr + a * kTileRows + (2 * i + half) * kPart, raw);
              tc_wait_ld();
              tc_pin(raw);
#pragma unroll
              for (int j = 0; j < kPart / 2; ++j)
                acc[i][j] = add2(acc[i][j], f2_pack(__uint_as_float(raw[2 * j]), __uint_as_float(raw[2 * j + 1])));
            }
          }
          hand_back();
        }
        if (kSplit && pairs > 1) {
          // Pair q has its share of every part's columns: `own` quads from `first` on.  A sum's place: [quad of the
          // owner's][source][this thread].  One item a cluster, so that the memory is used once; what is sent to a CTA
          // is waited for there.
          const uint32_t inv = (65535u + pairs) / pairs;   // (x / pairs is x * inv >> 16 here)
          auto start = [&](int of) { return (int)(kPart / 4 * of * inv >> 16); };
          const int first = start(q), own = start(q + 1) - first;
          const int live = max(0, (cols / kPart - half + 1) / 2);   // parts of this warp
          if (tid == kWideThreads - 1)
            mbar_arrive_expect_tx(&ctl.red_full, cols / kPart * own * (pairs - 1) * 128 * 16);
          cluster_arrive_release();
          cluster_wait();
          met = true;
          uint8_t *here = smem + (tid - 128) * 16;
          const uint32_t base = smem_addr(here), bar = smem_addr(&ctl.red_full);
#pragma unroll 1   // (code that runs once a launch is fetched as it runs)
          for (int part = 0; part < live; ++part) {
            float4 *mine = reinterpret_cast<float4 *>(stage) + lane;   // [quad][this thread]
#pragma unroll
            for (int i = 0; i < kParts; ++i) {
              if (i != part) continue;
#pragma unroll
              for (int j = 0; j < kPart / 4; ++j) {
                float4 u;
                f2_unpack(acc[i][2 * j], u.x, u.y);
                f2_unpack(acc[i][2 * j + 1], u.z, u.w);
                mine[j * 32] = u;
              }
            }
#pragma unroll 2
            for (int j = 0; j < kPart / 4; ++j) {
              const int to = ((j + 1) * pairs - 1) / (kPart / 4), s0 = start(to);
              const int at = ((part * (start(to + 1) - s0) + j - s0) * pairs + q) * 4096;
              const float4 u = mine[j * 32];
              if (to == q) *reinterpret_cast<float4 *>(here + at) = u;
              else st_async_v4(cluster_map(base + at, to * 2 + rank), u, cluster_map(bar, to * 2 + rank));
            }
          }
          __syncwarp();
          mbar_wait_cluster(&ctl.red_full, 0, abort, p.err);
          const int some = kPart / (own * 4);   // parts at a time, as `stage` holds
#pragma unroll 1
          for (int i = 0; i < live; i += some) {
            const int quads = min(some, live - i) * own;
#pragma unroll 1
            for (int j = 0; j < quads; ++j) {
              float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
              for (int src = 0; src < 4; ++src) {
                if (src >= pairs) break;
                const float4 u = *reinterpret_cast<const float4 *>(here + ((i * own + j) * pairs + src) * 4096);
                v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
              }
              float *to = stage + j * 4 * 32 + lane;
              to[0] = v.x, to[32] = v.y, to[64] = v.z, to[96] = v.w;
            }
            put_out(i, first * 4, own * 4, quads * 4);
          }
        } else {
#pragma unroll 1
          for (int part = 0; part < kParts; ++part) {
            if ((2 * part + half) * kPart >= cols) break;
#pragma unroll
            for (int i = 0; i < kParts; ++i) {
              if (i != part) continue;
#pragma unroll
              for (int j = 0; j < kPart / 2; ++j) {
                float lo, hi;
                f2_unpack(acc[i][j], lo, hi);
                stage[(2 * j) * 32 + lane] = lo;
                stage[(2 * j + 1) * 32 + lane] = hi;
              }
            }
            put_out(part, 0, kPart, kPart);
          }
        }
      }
    }
    if (kSplit && pairs > 1 && !met) {
      cluster_arrive_release();
      cluster_wait();
    }
  }
  tc_fence_before();
  __syncthreads();
  // The pair's accumulators are read, and nothing is on its way to any CTA's shared memory: copies, commits and the
  // other pairs' sums were waited for above, and the release orders the epilogue's remote arrivals.
  cluster_arrive_release();
  cluster_wait();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ------------------------------------------------------------------ launch

// (in bytes: tiles of 128 bytes a row whatever the type)
int make_maps(const Bf16Args &a, const void *x, long long rows, long long ld_bytes, int x_box_rows, int x_maps,
              Bf16Maps *maps) {
  if (int st = stream::encode_u8(&maps->w, a.w, 3, 2ull * a.K, a.N, a.E, 2ull * a.ldw, 2ull * a.ldw * a.N, kRows)) return st;
  for (int i = 0; i < x_maps; ++i)
    if (int st = stream::encode_u8(&maps->x[i], x, 2, 2ull * a.K, rows, 1, ld_bytes, 0, x_box_rows >> i)) return st;
  return 0;
}

template <int BT, int MODE>
int launch_narrow(const Bf16Args &a, const DeviceInfo &dev, cudaStream_t stream) {
  using C = Narrow<BT>;
  Bf16Cfg cfg = {};
  cfg.nt = (a.N + kRows - 1) / kRows;
  const long long items = unit_bound(a, (ProductMode)MODE, BT) * cfg.nt;
  if (items <= 0) return 0;
  if (int st = allow_dynamic_smem((const void *)bf16_narrow_kernel<BT, MODE>)) return st;
  if (MODE == kSorted && a.block > BT) cfg.list = kListUnits;
  // Clusters that split K: while there are too few items for the SMs, as large
  // as leaves each CTA a chunk and every item a cluster of its own.  A ring no
  // longer than a CTA's share lets more clusters fit.
  auto shape = [&](int cs) {
    cfg.cluster = cs;
    const int red = cs > 1 ? join_bytes(BT, cs, MODE == kNaive) : 0;
    const int tile = cs > 1 ? red / cs : (MODE == kNaive ? 1 : BT) * kRows * 4;
    const int fixed = red + tile + cfg.list * 4 + (int)sizeof(NarrowCtrl);
    const int share = items * cs <= dev.sm_count ? ((a.KB + cs - 1) / cs + 1) / 2 : kMaxRing;
    cfg.stages = std::max(2, std::min(share, std::min(kMaxRing, (kMaxSmem - fixed) / C::kStage)));
    cfg.off_red = cfg.stages * C::kStage;
    cfg.off_tile = cfg.off_red + red;
    cfg.off_list = cfg.off_tile + tile;
    cfg.off_ctrl = cfg.off_list + cfg.list * 4;
    cfg.smem_bytes = cfg.off_ctrl + (int)sizeof(NarrowCtrl);
    return resident_clusters(bf16_narrow_kernel<BT, MODE>, cs, cfg.smem_bytes, kNarrowThreads, dev);
  };
  int cs = (int)std::max<long long>(1, std::min<long long>(std::min<long long>(8, dev.sm_count / items), a.KB / kChunk));
  int fit = shape(cs);
  while (cs > 1 && fit < items) fit = shape(--cs);
  const unsigned clusters = (unsigned)std::min<long long>(items, std::min(fit, dev.sm_count / cs));
  Bf16Maps maps;
  if (int st = make_maps(a, a.x, a.rows, 2 * a.ldx, MODE == kDense ? BT : 1, 1, &maps)) return st;
  return launch_dependent(bf16_narrow_kernel<BT, MODE>, clusters * cs, kNarrowThreads, cs, cfg.smem_bytes, stream, maps, a,
                          cfg);
}

// The chunked kernel's warps trade registers after the launch: the shares must
// fit what the block was launched with, or the trade would wait forever.
template <typename Kernel>
bool register_shares_fit(Kernel kernel) {
  cudaFuncAttributes attr;
  if (cudaFuncGetAttributes(&attr, (const void *)kernel) != cudaSuccess) return false;
  return attr.numRegs * kWideThreads >= 128 * kWideRegsIssue + 256 * kWideRegsEpilogue;
}

// Dense calls in chunks of kChunk groups: fp32 outputs, and those whose tiles leave
// pairs of CTAs to split K.
bool in_short_chunks(const Bf16Args &a, const DeviceInfo &dev) {
  return a.y_f32 || tile_bound(a, false, kTileRows) * ((a.N + kWideN - 1) / kWideN) * 4 <= dev.sm_count;
}

// Height of a dense call's tiles, and the pairs of CTAs that split K: the
// cheapest by a count of clocks, whose constants were measured.  A group of 64
// columns takes a pair 2 clk for each of the tile's rows in the tensor cores,
// and its operands come at 58 bytes a clk into each SM, all of them at 3100 a
// clk from HBM; joining shares of K, 75 for each row that is sent (4096 x 256, K of
// 7168: 22.0 us in 128 rows by two pairs, 23.6 in 192 by three).  Several rounds
// of items, or a share below two chunks, are not split.
template <typename Kernel>
void wide_shape(const Bf16Args &a, Kernel kernel, bool split, const DeviceInfo &dev, Bf16Cfg *cfg, long long *items) {
  double best = 0;
  for (int pairs = 1; pairs <= (split ? 4 : 1); ++pairs) {
    if (pairs > 1 && a.KB < pairs * 2 * kChunk) break;
    const int fit = std::min(resident_clusters(kernel, 2 * pairs, cfg->smem_bytes, kWideThreads, dev), dev.sm_count / (2 * pairs));
    for (int rows = kTileRows; rows >= 64; rows -= 32) {
      const long long n = ((long long)a.pairs + rows - 1) / rows * cfg->nt, rounds = (n + fit - 1) / fit;
      if (pairs > 1 && rounds > 1) continue;
      const double group = std::max(2.0 * rows, (kTileBytes + rows / 2 * kGroupBytes) / 58.0);
      const double run = std::max(rounds * ((double)a.KB / pairs) * group, 2.0 * a.K * ((double)a.pairs + a.N) / 3100);
      const double cost = run + 75.0 * rows * (pairs - 1) / pairs;
      if (best == 0 || cost < best) {
        best = cost;
        cfg->cluster = 2 * pairs;
        cfg->tile_rows = rows;
        *items = n;
      }
    }
  }
}

// Height of a sorted call's tiles: of lower ones the ring holds more.  128 experts
// of 2048 x 1536, us with 128 / 256 rows: 64 pairs an expert 147 / 151, 96 156 / 160,
// 128 166 / 172; above, most experts would have more tiles than they need.
int sorted_height(const Bf16Args &a) { return a.pairs <= 128ll * a.E ? 128 : kTileRows; }

template <int MODE, bool CHUNKED>
int launch_wide(const Bf16Args &a, void *workspace, const DeviceInfo &dev, cudaStream_t stream) {
  const auto kernel = bf16_wide_kernel<MODE, CHUNKED>;
  Bf16Cfg cfg = {};
  cfg.nt = (a.N + kWideN - 1) / kWideN;
  const int height = MODE == kSorted ? sorted_height(a) : kTileRows;
  const long long tiles = tile_bound(a, MODE == kSorted, height);
  if (tiles <= 0) return 0;
  // a ring as long as fits, of stages for the highest tile
  auto ring = [&](int rows) {
    cfg.tile_rows = rows;
    cfg.stage_bytes = kTileBytes + rows / 2 * kGroupBytes;
    cfg.stages = std::min(kWideRing, (kMaxSmem - 8 * kPartBytes - (int)sizeof(WideCtrl)) / cfg.stage_bytes);
    cfg.off_tile = cfg.stages * cfg.stage_bytes;
    cfg.off_ctrl = cfg.off_tile + 8 * kPartBytes;
    cfg.smem_bytes = cfg.off_ctrl + (int)sizeof(WideCtrl);
  };
  ring(height);
  const bool fine = MODE == kDense && in_short_chunks(a, dev);
  cfg.chunk = fine ? kChunk : kLongChunk;
  if (CHUNKED) {
    static const bool fits = register_shares_fit(kernel);
    if (!fits) return MOE_LORA_ERR_LAUNCH;
  }
  if (int st = allow_dynamic_smem((const void *)kernel)) return st;
  Bf16Maps maps;
  const WideTile *list = nullptr;
  if (MODE == kDense) {
    if (int st = make_maps(a, a.x, a.rows, 2 * a.ldx, kRows, 4, &maps)) return st;
  } else {
    const long long rows = (long long)a.max_blocks * a.block;
    const GatherSpace w = gather_space(rows, 2ll * a.K);
    uint8_t *base = static_cast<uint8_t *>(workspace);
    list = reinterpret_cast<const WideTile *>(base);
    if (int st = make_maps(a, base + w.x, rows, w.ld, kRows, 4, &maps)) return st;
    if (int st = launch_gather(a, a.x, 2 * a.ldx, 2ll * a.K, height, workspace, dev, stream)) return st;
  }
  cfg.cluster = 2;
  long long items = tiles * cfg.nt;   // (the sorted arrays' own tiles are no more, but for entries that no align writes)
  if (MODE == kDense) {
    wide_shape(a, kernel, fine, dev, &cfg, &items);
    ring(cfg.tile_rows);
  }
  const long long clusters = std::min<long long>(items, dev.sm_count / cfg.cluster);
  return launch_dependent(kernel, (unsigned)(clusters * cfg.cluster), kWideThreads, cfg.cluster, cfg.smem_bytes, stream,
                          maps, a, list, cfg);
}

// Sorted calls run the wide kernel from 12 pairs an expert on (on average), the
// narrow one, in units of 16, below: an expert's units read its weight again.  128
// experts of 2048 x 1536, us narrow / wide: 4 pairs an expert 119 / 120, 8 123 / 126,
// 16 129 / 130 (with a skewed router 146 / 128), 24 169 / 132, 64 377 / 147; 8
// experts of 4096 x 14336 and 12 pairs 147 / 140.  The narrow one also while a round of its
// items covers the output.  A round is a GB300's 152 SMs, not the current device's: the
// workspace's size is asked for on hosts without one.
constexpr long long kRoundItems = 152;
bool sorted_is_wide(const Bf16Args &a) {
  const long long units = a.pairs / 16 + std::min(a.E, a.pairs);
  return a.pairs >= 12ll * a.E && units * ((a.N + kRows - 1) / kRows) > kRoundItems;
}

// Up to this many bytes of weights, calls of single pairs or of at most 16 rows
// run the kernel that streams the weight through registers: it starts sooner.  us,
// streaming / narrow: one token's eight experts of 1536 x 2048 (50 MB) 9.7 / 12.3,
// one row by 4096 x 4096 7.5 / 10.0, 16 rows by 8192 x 4096 (67 MB) 14.5 / 15.1.  Around the
// limit: single pairs, 201 MB 32.4 / 37.5, 268 MB 51 / 42, 537 MB 85 / 81; one row, 134 MB
// 22.8 / 23.0, 235 MB 38.0 / 38.7, 268 MB 43.0 / 42.8, 470 MB 73.0 / 73.8; 8 rows, 134 MB 23.5 /
// 23.2, 235 MB 39.3 / 38.8.  (9 to 16 rows would gain from a lower one: 134 MB 24.9 / 23.5,
// 235 MB 44.4 / 39.1.)
constexpr double kStreamBytes = 256e6;

}  // namespace

size_t bf16_sorted_workspace(const Bf16Args &a) {
  return sorted_is_wide(a) ? gather_space((long long)a.max_blocks * a.block, 2ll * a.K).bytes : 0;
}

bool bf16_items_fit(const Bf16Args &a, ProductMode mode) {
  if (mode == kDense ? a.pairs > 64 : mode == kSorted && sorted_is_wide(a))
    return tile_bound(a, mode == kSorted, mode == kSorted ? sorted_height(a) : 64) * ((a.N + kWideN - 1) / kWideN) <= kMostItems / 16;
  // every unit that the sorted arrays can hold, whatever they hold
  const long long units = mode == kSorted ? (long long)a.max_blocks * (a.block / 16) : unit_bound(a, mode, 16);
  return units * ((a.N + kRows - 1) / kRows) <= kMostItems;
}

int launch_bf16_matmul(const Bf16Args &a, ProductMode mode, void *workspace, const DeviceInfo &dev, cudaStream_t s) {
  const bool small = (mode == kNaive ? (double)a.pairs : 1.0) * a.N * a.K * 2 <= kStreamBytes;
  if (mode == kNaive) return small ? launch_bf16_stream(a, mode, dev, s) : launch_narrow<16, kNaive>(a, dev, s);
  if (mode == kSorted) {
    if (sorted_is_wide(a))
      return a.KB > kLongChunk ? launch_wide<kSorted, true>(a, workspace, dev, s)
                               : launch_wide<kSorted, false>(a, workspace, dev, s);
    return launch_narrow<16, kSorted>(a, dev, s);
  }
  if (small && a.pairs <= 16) return launch_bf16_stream(a, mode, dev, s);
  // Up to 64 rows, one unit of the narrow kernel.  us, narrow / wide: 32 x 4096 x 4096 9.2 / 11.5;
  // 64 rows 10.3 / 12.1, by 28672 x 8192 77.6 / 83.0; in two units and more, which read the weight again, 65 x 4096 x
  // 4096 12.8 / 12.5, 128 rows 13.0 / 12.8, 256 16.6 / 14.8, 512 29 / 17; 128 x 4096 x 2880 12.8 / 11.8, 128 x 8192
  // x 28672 142 / 89.  (Small weights would gain: 128 x 2048 x 1536 6.2 / 7.7, by 128 columns 5.0 / 6.5.)
  if (a.pairs <= 16) return launch_narrow<16, kDense>(a, dev, s);
  if (a.pairs <= 32) return launch_narrow<32, kDense>(a, dev, s);
  if (a.pairs <= 64) return launch_narrow<64, kDense>(a, dev, s);
  if (a.KB > kLongChunk || in_short_chunks(a, dev)) return launch_wide<kDense, true>(a, nullptr, dev, s);
  return launch_wide<kDense, false>(a, nullptr, dev, s);
}

}  // namespace moe_lora
