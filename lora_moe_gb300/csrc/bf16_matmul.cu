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
//   narrow  the weight on the 128 rows of the MMA, 16 to 128 pairs on its
//           columns: few pairs for each weight (decode), bound by the weight's
//           bytes.  Where there are few items, clusters of CTAs split K, their
//           partial sums exchanged through distributed shared memory and added
//           in a fixed order.
//   wide    pairs of CTAs (cta_group::2), 256 pairs by 256 output columns, on
//           rows gathered into the blocks' order: bound by the tensor cores.
// Products of few rows and small weights are bf16_stream.cu's.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>

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
  CUtensorMap w;   // [E][N][K] in bytes, box 1 x 128 x 128
  CUtensorMap x;   // [rows][K], box BT x 128 (dense), 1 x 128 (gathered by row) or 128 x 128 (wide)
};

// Launch shape of a call.
struct Bf16Cfg {
  int stages;      // operand ring
  int nt;          // output tiles along N
  int cluster;     // CTAs that split K (narrow)
  int off_red, off_list, off_ctrl;
  int list;        // units that the list of live ones holds (0: none is made)
  int smem_bytes;
};

// ------------------------------------------------------------------ narrow

constexpr int kMaxRing = 12;
// Groups of K whose products the tensor cores add up.  Their additions truncate,
// so a long sum drifts; the epilogue adds the chunks in fp32, rounding to nearest.
constexpr int kChunk = 4;

template <int BT>
struct Narrow {
  static constexpr int kGroup = kTileBytes + BT * kGroupBytes;
  static constexpr int kStage = 2 * kGroup;           // two groups a stage, requested together
  static constexpr int kBufs = BT == 128 ? 2 : 4;     // accumulators in tensor memory
  static constexpr int kCols = kBufs * BT;            // power of two, >= 32
  static constexpr int kRedBytes = BT * kRows * 4;    // every rank's partial sums of this CTA's columns
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

  if (tid == 0) {
    for (int s = 0; s < cfg.stages; ++s) {
      mbar_init(&ctl.full[s], 1);
      mbar_init(&ctl.empty[s], 1);
    }
    for (int s = 0; s < C::kBufs; ++s) {
      mbar_init(&ctl.tfull[s], 1);
      mbar_init(&ctl.tempty[s], 4);
    }
    mbar_init(&ctl.red_full, 1);
    mbar_init(&ctl.done, 1);
    ctl.abort = 0;
    fence_barrier_init();
    prefetch_tensor_map(&maps.w);
    prefetch_tensor_map(&maps.x);
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
              tma_load_2d(st + i * C::kGroup + kTileBytes, &maps.x, (kb + i) * kGroupBytes, b * BT, &ctl.full[s]);
        }
        __syncwarp();
        if (MODE != kDense && mine)
          for (int i = 0; i < n; ++i)
            tma_gather4(st + i * C::kGroup + kTileBytes + lane * 4 * kGroupBytes, &maps.x, (kb + i) * kGroupBytes, row,
                        &ctl.full[s]);
        if (++s == cfg.stages) { s = 0; ph ^= 1; }
      }
    }
    // the copies have landed, the stages' hand-backs arrived and the MMAs completed before this CTA exits
    __syncwarp();
    if (lane == 0) {
      drain_ring(ctl.full, cfg.stages, fills);
      drain_ring(ctl.empty, cfg.stages, fills);
      drain_wait(&ctl.done, 0);
    }
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
    // ---------------- epilogue: this thread's weight row, BT pairs
    const int row = (warp - 4) * 32 + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)(warp - 4) << 21);   // lane offset 32 * quarter in bits 16..31
    int a = 0;
    uint32_t aph = 0;
    while (wk.advance()) {
      const int ui = wk.it / cfg.nt, nt = wk.it - ui * cfg.nt, b = unit(ui), e = block_expert<MODE>(p, b, BT);
      if (e < 0) continue;
      const int n = nt * kRows + row;
      const float bias = bias_of(p, e, n);
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
      auto store = [&](int t, const auto &v) {
        constexpr int W = sizeof(v) / sizeof(float);
        int f[W];
#pragma unroll
        for (int i = 0; i < W; ++i) f[i] = block_pair<MODE>(p, b, t + i, BT);
        finish_column<MODE, W>(p, f, n, bias, v);
      };
      if (cs == 1) {
        constexpr int W = MODE == kNaive ? 1 : 16;   // positions at a time; the naive form has one pair
#pragma unroll
        for (int c = 0; c < (MODE == kNaive ? 1 : BT); c += W) {
          float v[W];
#pragma unroll
          for (int i = 0; i < W; ++i) v[i] = acc[c + i];
          store(c, v);
        }
        continue;
      }
      join_ranks<BT, MODE == kNaive>(acc, cs, wk.rank, row, smem + cfg.off_red, &ctl.red_full, abort, p.err, store);
      waited = true;
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

// Pairs of CTAs (cta_group::2), 256 rows by 256 output columns.  Each CTA holds
// 128 of the rows and 128 of the weight's in shared memory, 32 KB a group, and
// 128 x 256 of an accumulator in tensor memory, twice: one is read while the
// next item's is added up.
constexpr int kWideThreads = 384;
constexpr int kWideN = 256;
constexpr int kHalf = kWideN / 2;
constexpr int kWideStage = 2 * kTileBytes;       // 128 rows, and 128 of the weight
constexpr int kWideStages = 6;
constexpr int kWideOut = 32 * 128;               // an epilogue warp's sums on their way out: 32 rows of 32 fp32

struct WideCtrl {
  uint64_t full[kWideStages], empty[kWideStages];
  uint64_t tfull[2], tempty[2];
  uint64_t done;   // every MMA of the pair
  uint32_t tmem;
  int abort;
};

// 8 columns of a row of y (or of the residual, which is alike) from n on, `cols`
// of which exist.
__device__ __forceinline__ void load_columns(const void *p, long long at, int f32, bool whole, int cols, float (&v)[8]) {
  if (whole && f32) {
    const float4 *s = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at);
    const float4 lo = load_global(s), hi = load_global(s + 1);
    v[0] = lo.x, v[1] = lo.y, v[2] = lo.z, v[3] = lo.w, v[4] = hi.x, v[5] = hi.y, v[6] = hi.z, v[7] = hi.w;
  } else if (whole) {
    const uint4 u = load_global(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + at));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < cols ? load_as_f32(p, at + i, f32) : 0.f;
  }
}
__device__ __forceinline__ void store_columns(void *p, long long at, int f32, bool whole, int cols, const float (&v)[8]) {
  if (whole && f32) {
    float4 *d = reinterpret_cast<float4 *>(static_cast<float *>(p) + at);
    d[0] = make_float4(v[0], v[1], v[2], v[3]);
    d[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else if (whole) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + at) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < cols) {
        if (f32) static_cast<float *>(p)[at + i] = v[i];
        else static_cast<uint16_t *>(p)[at + i] = float_to_bf16_bits(v[i]);
      }
  }
}
// Whether rows of p, ld elements apart, start on 16 bytes.
__device__ __forceinline__ bool rows_on_16(const void *p, long long ld, int f32) {
  return (ld & (f32 ? 3 : 7)) == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0;
}

template <int MODE>
__global__ void __launch_bounds__(kWideThreads, 1)
    bf16_wide_kernel(const __grid_constant__ Bf16Maps maps, const Bf16Args p, const WideTile *tiles, const Bf16Cfg cfg) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  WideCtrl &ctl = *reinterpret_cast<WideCtrl *>(smem + cfg.off_ctrl);
  volatile int *abort = &ctl.abort;
  const int rank = blockIdx.x & 1;   // rank 0 issues the pair's MMAs

  if (tid == 0) {
    for (int s = 0; s < kWideStages; ++s) {
      mbar_init(&ctl.full[s], 1);
      mbar_init(&ctl.empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ctl.tfull[s], 1);
      mbar_init(&ctl.tempty[s], 16);   // the epilogue warps of both CTAs
    }
    mbar_init(&ctl.done, 1);
    ctl.abort = 0;
    fence_barrier_init();
    prefetch_tensor_map(&maps.w);
    prefetch_tensor_map(&maps.x);
  }
  if (warp == 1) tmem_alloc_pair(&ctl.tmem, 512);
  tc_fence_before();
  __syncthreads();
  cluster_arrive_release();
  cluster_wait();
  tc_fence_after();
  wait_for_prior_grid();
  const uint32_t tmem = ctl.tmem;
  const int ntiles = MODE == kDense ? (p.pairs + kTileRows - 1) / kTileRows : load_global(&tiles[0].row0);
  const int items = ntiles * cfg.nt;   // rows fastest: pairs at work share the weight's columns
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;
  auto tile = [&](int t) {
    if (MODE == kDense) return WideTile{t * kTileRows, min(kTileRows, p.pairs - t * kTileRows), 0, 0};
    const int4 v = load_global(reinterpret_cast<const int4 *>(tiles) + 1 + t);
    return WideTile{v.x, v.y, v.z, 0};
  };

  if (warp == 0) {
    // ---------------- operands: this CTA's half of the rows, and of the weight's
    const uint32_t full0 = cluster_map(smem_addr(&ctl.full[0]), 0);   // rank 0's
    int s = 0;
    uint32_t ph = 0, fills = 0;
    bool go = true;   // falls with a wait that gave up: nothing more is requested
    for (int it = first; go && it < items; it += step) {
      const int nt = it / ntiles;
      const WideTile t = tile(it - nt * ntiles);
      const bool have = t.rows > rank * kRows;
      const uint32_t bytes = 2 * kTileBytes + (t.rows > kRows ? 2 : 1) * kTileBytes;
      for (int kb = 0; kb < p.KB; ++kb) {
        go = __all_sync(0xFFFFFFFFu, mbar_wait(&ctl.empty[s], ph ^ 1, abort, p.err));
        if (!go) break;
        ++fills;
        uint8_t *st = smem + (size_t)s * kWideStage;
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(&ctl.full[s], bytes);
          if (have) tma_load_2d_pair(st, &maps.x, kb * kGroupBytes, t.row0 + rank * kRows, full0 + s * 8);
          tma_load_3d_pair(st + kTileBytes, &maps.w, kb * kGroupBytes, nt * kWideN + rank * kHalf, t.expert, full0 + s * 8);
        }
        __syncwarp();
        if (++s == kWideStages) { s = 0; ph ^= 1; }
      }
    }
    // The pair's copies have landed (rank 0's barriers count both CTAs'), the
    // hand-backs of the last stages have arrived here and the MMAs have
    // completed before the pair exits: the epilogue waits for neither.
    __syncwarp();
    if (lane == 0) {
      if (rank == 0) drain_ring(ctl.full, kWideStages, fills);
      drain_ring(ctl.empty, kWideStages, fills);
      drain_wait(&ctl.done, 0);
    }
    __syncwarp();
  } else if (warp == 1 && rank == 0) {
    // ---------------- MMA, for both CTAs
    constexpr uint32_t idesc = make_idesc_bf16(2 * kRows, kWideN);
    const uint64_t desc0 = make_sdesc_sw128(smem_addr(smem));   // (addresses in units of 16 bytes)
    int s = 0, a = 0;
    uint32_t ph = 0, aph = 0;
    for (int it = first; it < items; it += step) {
      mbar_wait(&ctl.tempty[a], aph ^ 1, abort, p.err);
      for (int kb = 0; kb < p.KB; ++kb) {
        mbar_wait(&ctl.full[s], ph, abort, p.err);
        tc_fence_after();
        const uint64_t dx = desc0 + s * (kWideStage >> 4), dw = dx + (kTileBytes >> 4);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kBf16Group / 16; ++k)
            tc_mma_bf16_pair(tmem + a * kWideN, dx + k * 2, dw + k * 2, idesc, kb > 0 || k > 0);
          tc_commit_pair(&ctl.empty[s]);
          if (kb + 1 == p.KB) tc_commit_pair(&ctl.tfull[a]);
        }
        __syncwarp();
        if (++s == kWideStages) { s = 0; ph ^= 1; }
      }
      a ^= 1;
      if (a == 0) aph ^= 1;
    }
    if (elect_one()) tc_commit_pair(&ctl.done);
    __syncwarp();
  } else if (warp >= 4) {
    // ---------------- epilogue: 32 rows, and 128 of the output columns, a warp
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const uint32_t lane_addr = tmem + ((uint32_t)quarter << 21) + half * kHalf;
    const uint32_t tempty0 = cluster_map(smem_addr(&ctl.tempty[0]), 0);   // rank 0's
    uint8_t *out = smem + kWideStages * kWideStage + (warp - 4) * kWideOut;
    const bool y16 = rows_on_16(p.y, p.ldy, p.y_f32), r16 = rows_on_16(p.residual, p.ldr, p.y_f32);
    int a = 0;
    uint32_t aph = 0;
    for (int it = first; it < items; it += step) {
      const int nt = it / ntiles;
      const WideTile t = tile(it - nt * ntiles);
      const int r = rank * kRows + quarter * 32 + lane;   // row of the tile
      int f = -1;
      if (r < t.rows) f = MODE == kDense ? t.row0 + r : load_global(p.sorted_token_ids + t.row0 + r);
      if ((unsigned)f >= (unsigned)p.pairs) f = -1;
      const float weight = f < 0 ? 0.f : pair_weight<MODE>(p, f);
      mbar_wait(&ctl.tfull[a], aph, abort, p.err);
      tc_fence_after();
      // 32 columns at a time, through shared memory, so that 4 lanes write
      // neighbouring columns of one row
#pragma unroll 1
      for (int part = 0; part < 4; ++part) {
        uint32_t v[32];
        tmem_ld32(lane_addr + a * kWideN + part * 32, v);
        tc_wait_ld();
        tc_pin(v);
        if (part == 3) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote_relaxed(tempty0 + a * 8);   // (only tensor memory is handed back)
        }
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *reinterpret_cast<uint4 *>(out + lane * 128 + ((c ^ (lane & 7)) << 4)) =
              make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
        __syncwarp();
        const int chunk = lane & 3, n = nt * kWideN + half * kHalf + part * 32 + chunk * 8, cols = p.N - n;
        const bool whole = cols >= 8;
        float bias[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) bias[j] = bias_of(p, t.expert, n + j);
        int fr[4];
        float res[4][8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          fr[i] = __shfl_sync(0xFFFFFFFFu, f, i * 8 + (lane >> 2));
          if (p.residual && fr[i] >= 0) load_columns(p.residual, fr[i] * p.ldr + n, p.y_f32, whole && r16, cols, res[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int rr = i * 8 + (lane >> 2);
          const float w = __shfl_sync(0xFFFFFFFFu, weight, rr);
          const float4 lo = *reinterpret_cast<const float4 *>(out + rr * 128 + (((2 * chunk) ^ (rr & 7)) << 4));
          const float4 hi = *reinterpret_cast<const float4 *>(out + rr * 128 + (((2 * chunk + 1) ^ (rr & 7)) << 4));
          float o[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
          if (fr[i] < 0) continue;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            o[j] = activate(o[j] + bias[j], p.act) * w;
            if (p.residual) o[j] += res[i][j];
          }
          store_columns(p.y, fr[i] * p.ldy + n, p.y_f32, whole && y16, cols, o);
        }
      }
      a ^= 1;
      if (a == 0) aph ^= 1;
    }
  }
  tc_fence_before();
  __syncthreads();
  // The pair's accumulators are read, and nothing is on its way to either CTA's shared memory: copies and commits were
  // waited for above, and the release orders the epilogue's remote arrivals.
  cluster_arrive_release();
  cluster_wait();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ------------------------------------------------------------------ launch

// (in bytes: tiles of 128 bytes a row whatever the type)
int make_maps(const Bf16Args &a, const void *x, long long rows, long long ld_bytes, int x_box_rows, Bf16Maps *maps) {
  if (int st = stream::encode_u8(&maps->w, a.w, 3, 2ull * a.K, a.N, a.E, 2ull * a.ldw, 2ull * a.ldw * a.N, kRows)) return st;
  return stream::encode_u8(&maps->x, x, 2, 2ull * a.K, rows, 1, ld_bytes, 0, x_box_rows);
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
    const int list_bytes = cfg.list * 4;
    const int fixed = (cs > 1 ? C::kRedBytes : 0) + list_bytes + (int)sizeof(NarrowCtrl) + 128;
    const int share = items * cs <= dev.sm_count ? ((a.KB + cs - 1) / cs + 1) / 2 : kMaxRing;
    cfg.stages = std::max(2, std::min(share, std::min(kMaxRing, (224 * 1024 - fixed) / C::kStage)));
    cfg.off_red = cfg.stages * C::kStage;
    cfg.off_list = cfg.off_red + (cs > 1 ? C::kRedBytes : 0);
    cfg.off_ctrl = cfg.off_list + list_bytes;
    cfg.smem_bytes = cfg.off_ctrl + (int)sizeof(NarrowCtrl);
    return resident_clusters(bf16_narrow_kernel<BT, MODE>, cs, cfg.smem_bytes, kNarrowThreads, dev);
  };
  int cs = 1;
  while (cs < 8 && items * cs * 2 <= dev.sm_count && a.KB >= cs * 2 * kChunk) cs *= 2;
  int fit = shape(cs);
  while (cs > 1 && fit < items) fit = shape(cs /= 2);
  const unsigned clusters = (unsigned)std::min<long long>(items, std::min(fit, dev.sm_count / cs));
  Bf16Maps maps;
  if (int st = make_maps(a, a.x, a.rows, 2 * a.ldx, MODE == kDense ? BT : 1, &maps)) return st;
  return launch_dependent(bf16_narrow_kernel<BT, MODE>, clusters * cs, kNarrowThreads, cs, cfg.smem_bytes, stream, maps, a,
                          cfg);
}

template <int MODE>
int launch_wide(const Bf16Args &a, void *workspace, const DeviceInfo &dev, cudaStream_t stream) {
  Bf16Cfg cfg = {};
  cfg.nt = (a.N + kWideN - 1) / kWideN;
  const long long tiles = tile_bound(a, MODE == kSorted);
  if (tiles <= 0) return 0;
  cfg.off_ctrl = kWideStages * kWideStage + 8 * kWideOut;
  cfg.smem_bytes = cfg.off_ctrl + (int)sizeof(WideCtrl);
  if (int st = allow_dynamic_smem((const void *)bf16_wide_kernel<MODE>)) return st;
  Bf16Maps maps;
  const WideTile *list = nullptr;
  if (MODE == kDense) {
    if (int st = make_maps(a, a.x, a.rows, 2 * a.ldx, kRows, &maps)) return st;
  } else {
    const long long rows = (long long)a.max_blocks * a.block;
    const GatherSpace w = gather_space(rows, 2ll * a.K);
    uint8_t *base = static_cast<uint8_t *>(workspace);
    list = reinterpret_cast<const WideTile *>(base);
    if (int st = make_maps(a, base + w.x, rows, w.ld, kRows, &maps)) return st;
    if (int st = launch_gather(a, a.x, 2 * a.ldx, 2ll * a.K, workspace, dev, stream)) return st;
  }
  const long long items = tiles * cfg.nt;   // (the sorted arrays' own tiles are no more, but for entries that no align writes)
  const unsigned grid = 2 * (unsigned)std::min<long long>(items, dev.sm_count / 2);
  return launch_dependent(bf16_wide_kernel<MODE>, grid, kWideThreads, 2, cfg.smem_bytes, stream, maps, a, list, cfg);
}

// The narrow kernel while one round of its 128 x 128 items covers the output,
// else the wide one.  The narrow one for fp32 outputs of any size: all of K
// added up by the tensor cores is 2.4e-5 off for 7168 products of one sign.
bool dense_is_wide(const Bf16Args &a, int sms) {
  if (a.y_f32) return false;
  const long long items = ((a.pairs + 127ll) / 128) * ((a.N + kRows - 1) / kRows);
  return a.pairs > 128 && items > sms;
}

// A round is a GB300's 152 SMs, not the current device's: the workspace's size
// is asked for on hosts without one.
constexpr long long kRoundItems = 152;
bool sorted_is_wide(const Bf16Args &a) {
  const long long units = a.pairs / 16 + std::min(a.E, a.pairs);
  return a.pairs >= 20ll * a.E && units * ((a.N + kRows - 1) / kRows) > kRoundItems;
}

// Up to this many bytes of weights, calls of single pairs or of at most 16 rows
// run the kernel that streams the weight through registers.
constexpr double kStreamBytes = 32e6;

}  // namespace

size_t bf16_sorted_workspace(const Bf16Args &a) {
  return sorted_is_wide(a) ? gather_space((long long)a.max_blocks * a.block, 2ll * a.K).bytes : 0;
}

bool bf16_items_fit(const Bf16Args &a, ProductMode mode) {
  if (mode == kDense ? dense_is_wide(a, 0) : mode == kSorted && sorted_is_wide(a))
    return tile_bound(a, mode == kSorted) * ((a.N + kWideN - 1) / kWideN) <= INT32_MAX / 16;
  // every unit that the sorted arrays can hold, whatever they hold
  const long long units = mode == kSorted ? (long long)a.max_blocks * (a.block / 16) : unit_bound(a, mode, 16);
  return units * ((a.N + kRows - 1) / kRows) <= INT32_MAX;
}

int launch_bf16_matmul(const Bf16Args &a, ProductMode mode, void *workspace, const DeviceInfo &dev, cudaStream_t s) {
  const bool small = (mode == kNaive ? (double)a.pairs : 1.0) * a.N * a.K * 2 <= kStreamBytes;
  if (mode == kNaive) return small ? launch_bf16_stream(a, mode, dev, s) : launch_narrow<16, kNaive>(a, dev, s);
  if (mode == kSorted) {
    if (sorted_is_wide(a)) return launch_wide<kSorted>(a, workspace, dev, s);
    return launch_narrow<16, kSorted>(a, dev, s);
  }
  if (small && a.pairs <= 16) return launch_bf16_stream(a, mode, dev, s);
  if (a.pairs <= 16) return launch_narrow<16, kDense>(a, dev, s);
  if (a.pairs <= 32) return launch_narrow<32, kDense>(a, dev, s);
  if (a.pairs <= 64) return launch_narrow<64, kDense>(a, dev, s);
  return dense_is_wide(a, dev.sm_count) ? launch_wide<kDense>(a, nullptr, dev, s) : launch_narrow<128, kDense>(a, dev, s);
}

}  // namespace moe_lora
