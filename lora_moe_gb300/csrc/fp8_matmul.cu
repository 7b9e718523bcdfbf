// fp8_matmul.cu -- 8-bit matrix products with a scale for each block of 128,
// dense and over a MoE layer's experts, on the 5th-generation tensor cores.
//
//   y[f][n] = bf16( weight[f] * sum_g sx[r][g] * sw[e][n/128][g] * sum_{k in group g} x[r][k] * w[e][n][k] )
//
// with r the row of x that pair f reads and e its expert.  The scales change
// with every group g of 128 columns, so each group's product is its own
// accumulation in tensor memory; the epilogue warps scale it into fp32
// registers while the next groups are multiplied.
//
// Two kernels, both persistent, with warps that load (TMA), warps that issue
// the MMAs and epilogue warps:
//   narrow  the weight on the 128 rows of the MMA, 16 pairs (dense: to 64) on
//           its columns: few pairs for each weight (decode), bound by the weight's
//           bytes.  Where there are few items, clusters of CTAs split K, their
//           partial sums exchanged through distributed shared memory and added
//           in a fixed order.  gpt-oss-shaped w2 decode (0.88 GB of weights):
//           135 to 140 us, 6.3 to 6.6 TB/s.
//   wide    pairs of CTAs (cta_group::2), 256 pairs by 256 output columns, on
//           rows gathered into the blocks' order: bound by the tensor cores,
//           the hand-shake with the epilogue and, over seconds, by power.
//           8192 x 4096 x 4096 dense: 111 us (2.5 PFLOP/s) in calls that go on
//           for seconds, with the power limit reached, 97 us in short runs;
//           Mixtral-shaped w13 prefill: 1.79 ms (2.15 PFLOP/s), and 1.5.
// Products of few rows and small weights are fp8_stream.cu's.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "device_utils.cuh"
#include "fp8.h"
#include "fp8_blocks.cuh"
#include "launch.cuh"
#include "stream_pipeline.cuh"

namespace moe_lora {

namespace {

constexpr int kRows = 128;                     // rows of an accumulator: lanes of tensor memory
constexpr int kTileBytes = kRows * kFp8Group;  // 128 rows of one group: 16 KB, one swizzle row of 128 bytes each

struct Fp8Maps {
  CUtensorMap w;   // [E][N][K], box 1 x 128 (narrow) or 64 (wide) x 128
  CUtensorMap x;   // [rows][K], box BT x 128 (dense), 1 x 128 (gathered by row) or 128 x 128 (wide)
};

// Launch shape of a call.
struct Fp8Cfg {
  int stages;      // operand ring
  int nt;          // output tiles along N
  int cluster;     // CTAs that split K (narrow)
  int off_scale, off_red, off_list, off_ctrl;
  int list;        // units that the list of live ones holds (0: none is made)
  int smem_bytes;
};

// ------------------------------------------------------------------ narrow

constexpr int kNarrowThreads = 256;
constexpr int kMaxRing = 12;
constexpr int kScaleSlots = 16;   // ring of scale rows, one group each
constexpr int kListUnits = 2048;

template <int BT>
struct Narrow {
  static constexpr int kGroup = kTileBytes + BT * kFp8Group;
  // Two groups a stage, requested together: 256 consecutive bytes of each of
  // the weight's rows (gpt-oss-shaped w2 decode 140 us, against 145 with one).
  static constexpr int kStage = 2 * kGroup;
  static constexpr int kScaleRow = BT + 4;    // BT row scales and the weight's, padded to 16 bytes
  static constexpr int kBufs = 4;             // accumulators in tensor memory
  static constexpr int kCols = kBufs * BT;    // power of two, >= 32
  static constexpr int kRedBytes = BT * kRows * 4;   // every rank's partial sums of this CTA's columns
};

struct NarrowCtrl {
  uint64_t full[kMaxRing], empty[kMaxRing];
  uint64_t sfull[kScaleSlots], sempty[kScaleSlots];
  uint64_t tfull[4], tempty[4];
  uint64_t red_full;
  uint64_t done;                             // every MMA of this CTA
  uint32_t tmem;
  int abort;
  int live;                                  // units in the list
  int warp_live[kNarrowThreads / 32];
};

// The units of a sorted call that hold pairs, in order: where a block is
// several units, most of a decode batch's hold none, and every CTA would look
// each of them up for every tile of N (256 tokens, blocks of 64: 97 us against
// 76 in blocks of 16, which need no list).  By the whole CTA.
template <int BT>
__device__ __forceinline__ void list_units(const Fp8Args &p, int units, int *list, NarrowCtrl &ctl, int tid) {
  const int lane = tid & 31, warp = tid >> 5;
  int n = 0;   // (the same in every thread)
  for (int base = 0; base < units; base += kNarrowThreads) {
    const int b = base + tid;
    const int e = b < units ? block_expert<kFp8Sorted>(p, b, BT) : kNoPairs;
    const uint32_t live = __ballot_sync(0xFFFFFFFFu, e >= 0);
    if (lane == 0) ctl.warp_live[warp] = __popc(live);
    __syncthreads();
    int at = n;
    for (int w = 0; w < kNarrowThreads / 32; ++w) {
      if (w < warp) at += ctl.warp_live[w];
      n += ctl.warp_live[w];
    }
    if (e >= 0) list[at + __popc(live & ((1u << lane) - 1))] = b;
    __syncthreads();
  }
  if (tid == 0) ctl.live = n;
  __syncthreads();
}

// The items of a CTA, in the order of its warps' loops: all of K, or (a cluster
// of cs > 1 CTAs, which has one item at most) this CTA's share of it.
struct NarrowWork {
  int items, next, step, it, kb0, kb1, rank;
  __device__ __forceinline__ NarrowWork(int n, int KB, int cs) : items(n) {
    rank = blockIdx.x % cs;   // (a cluster is cs consecutive CTAs)
    next = blockIdx.x / cs;
    step = cs > 1 ? items : gridDim.x;
    kb0 = (int)((long long)KB * rank / cs);
    kb1 = (int)((long long)KB * (rank + 1) / cs);
  }
  __device__ __forceinline__ bool advance() {
    if (next >= items) return false;
    it = next;
    next += step;   // (cs > 1: past the last)
    return true;
  }
};

// The sums of one CTA's positions over CS ranks, in rank order; Q of 4
// positions (or 2) at a time.
template <int CS, int W>
__device__ __forceinline__ void sum_ranks(const float *buf, int per_rank, int at, int row, float (&v)[W]) {
#pragma unroll
  for (int i = 0; i < W; ++i) v[i] = 0.f;
#pragma unroll
  for (int q = 0; q < CS; ++q) {
    const float *src = buf + ((q * per_rank + at) * kRows + row) * W;
    if constexpr (W == 4) {
      const float4 u = *reinterpret_cast<const float4 *>(src);
      v[0] += u.x;
      v[1] += u.y;
      v[2] += u.z;
      v[3] += u.w;
    } else if constexpr (W == 2) {
      const float2 u = *reinterpret_cast<const float2 *>(src);
      v[0] += u.x;
      v[1] += u.y;
    } else {
      v[0] += *src;
    }
  }
}

template <int BT, int MODE>
__global__ void __launch_bounds__(kNarrowThreads, 1)
    fp8_narrow_kernel(const __grid_constant__ Fp8Maps maps, const Fp8Args p, const Fp8Cfg cfg) {
  using C = Narrow<BT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  NarrowCtrl &ctl = *reinterpret_cast<NarrowCtrl *>(smem + cfg.off_ctrl);
  float *scales = reinterpret_cast<float *>(smem + cfg.off_scale);
  volatile int *abort = &ctl.abort;
  const int cs = cfg.cluster;

  if (tid == 0) {
    for (int s = 0; s < cfg.stages; ++s) {
      mbar_init(&ctl.full[s], 1);
      mbar_init(&ctl.empty[s], 1);
    }
    for (int s = 0; s < kScaleSlots; ++s) {
      mbar_init(&ctl.sfull[s], 32);
      mbar_init(&ctl.sempty[s], 4);
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
  if (MODE == kFp8Sorted && cfg.list && units <= cfg.list) {
    int *l = reinterpret_cast<int *>(smem + cfg.off_list);
    list_units<BT>(p, units, l, ctl, tid);
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
      if (MODE != kFp8Dense && lane < BT / 4) {
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
      const int groups = MODE == kFp8Dense ? BT / 4 : __popc(__ballot_sync(0xFFFFFFFFu, mine));
      for (int kb = wk.kb0; kb < wk.kb1; kb += 2) {
        go = __all_sync(0xFFFFFFFFu, mbar_wait(&ctl.empty[s], ph ^ 1, abort, p.err));
        if (!go) break;
        ++fills;
        uint8_t *st = smem + (size_t)s * C::kStage;
        const int n = min(2, wk.kb1 - kb);
        if (elect_one()) {
          mbar_arrive_expect_tx(&ctl.full[s], n * (kTileBytes + groups * 4 * kFp8Group));
          for (int i = 0; i < n; ++i)
            tma_load_3d(st + i * C::kGroup, &maps.w, (kb + i) * kFp8Group, nt * kRows, e, &ctl.full[s]);
          if (MODE == kFp8Dense)
            for (int i = 0; i < n; ++i)
              tma_load_2d(st + i * C::kGroup + kTileBytes, &maps.x, (kb + i) * kFp8Group, b * BT, &ctl.full[s]);
        }
        __syncwarp();
        if (MODE != kFp8Dense && mine)
          for (int i = 0; i < n; ++i)
            tma_gather4(st + i * C::kGroup + kTileBytes + lane * 4 * kFp8Group, &maps.x, (kb + i) * kFp8Group, row,
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
    // ---------------- MMA: each group of 128 columns into an accumulator of its own
    constexpr uint32_t idesc = make_idesc_e4m3(kRows, BT);
    const uint64_t desc0 = make_sdesc_sw128(smem_addr(smem));   // (addresses in units of 16 bytes)
    int s = 0, a = 0;
    uint32_t ph = 0, aph = 0;
    while (wk.advance()) {
      if (block_expert<MODE>(p, unit(wk.it / cfg.nt), BT) < 0) continue;
      for (int kb = wk.kb0; kb < wk.kb1; ++kb) {
        mbar_wait(&ctl.tempty[a], aph ^ 1, abort, p.err);
        const int i = (kb - wk.kb0) & 1;
        const bool last = i == 1 || kb + 1 == wk.kb1;   // of the stage
        if (i == 0) mbar_wait(&ctl.full[s], ph, abort, p.err);
        tc_fence_after();
        const uint64_t dw = desc0 + (s * C::kStage + i * C::kGroup) / 16, dx = dw + kTileBytes / 16;
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kFp8Group / 32; ++k) tc_mma_f8(tmem + a * BT, dw + k * 2, dx + k * 2, idesc, k > 0);
          if (last) tc_commit(&ctl.empty[s]);
          tc_commit(&ctl.tfull[a]);
        }
        __syncwarp();
        if (last && ++s == cfg.stages) { s = 0; ph ^= 1; }
        if (++a == C::kBufs) { a = 0; aph ^= 1; }
      }
    }
    if (elect_one()) tc_commit(&ctl.done);
    __syncwarp();
  } else if (warp == 2) {
    // ---------------- scales: a row of BT + 1 for each group
    // (clusters have an item each for all blocks that an align writes)
    if (cs > 1 && blockIdx.x == 0 && lane == 0 && items > (int)gridDim.x / cs) flag_error(p.err, MOE_LORA_DEVERR_CAPACITY);
    int s = 0;
    uint32_t ph = 0;
    while (wk.advance()) {
      const int ui = wk.it / cfg.nt, nt = wk.it - ui * cfg.nt, b = unit(ui), e = block_expert<MODE>(p, b, BT);
      if (e < 0) continue;
      constexpr int kPer = (BT + 31) / 32;
      const float *src[kPer];
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int t = j * 32 + lane;
        int f = -1;
        if (t < BT) f = block_pair<MODE>(p, b, t, BT);
        src[j] = f < 0 ? nullptr : p.x_scales + (size_t)pair_row<MODE>(p, f) * p.KB;
      }
      const float *sw = p.w_scales + ((size_t)e * p.NB + nt) * p.KB;
      for (int kb = wk.kb0; kb < wk.kb1; ++kb) {
        mbar_wait(&ctl.sempty[s], ph ^ 1, abort, p.err);
        float *dst = scales + s * C::kScaleRow;
#pragma unroll
        for (int j = 0; j < kPer; ++j)
          if (j * 32 + lane < BT) cp_async_4(dst + j * 32 + lane, src[j] ? src[j] + kb : p.x_scales, src[j] ? 4 : 0);
        if (lane == 0) cp_async_4(dst + BT, sw + kb, 4);
        cp_async_mbar_arrive_noinc(&ctl.sfull[s]);
        if (++s == kScaleSlots) { s = 0; ph ^= 1; }
      }
    }
    cp_async_wait_all();
  } else if (warp == 3) {
    // ---------------- what is out of range, each unit once
    if (MODE != kFp8Dense)
      for (int b = blockIdx.x; b < all_units; b += gridDim.x)
        flag_unit<MODE>(p, b, BT, block_expert<MODE>(p, b, BT), lane);
  } else if (warp >= 4) {
    // ---------------- epilogue: this thread's weight row, BT pairs
    const int row = (warp - 4) * 32 + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)(warp - 4) << 21);   // lane offset 32 * quarter in bits 16..31
    int s = 0, a = 0;
    uint32_t sph = 0, aph = 0;
    while (wk.advance()) {
      const int ui = wk.it / cfg.nt, nt = wk.it - ui * cfg.nt, b = unit(ui);
      if (block_expert<MODE>(p, b, BT) < 0) continue;
      float acc[BT];
#pragma unroll
      for (int c = 0; c < BT; ++c) acc[c] = 0.f;
      for (int kb = wk.kb0; kb < wk.kb1; ++kb) {
        mbar_wait(&ctl.sfull[s], sph, abort, p.err);
        mbar_wait(&ctl.tfull[a], aph, abort, p.err);
        tc_fence_after();
        const float *sc = scales + s * C::kScaleRow;
        const float sw = sc[BT];
#pragma unroll
        for (int c0 = 0; c0 < BT; c0 += 16) {
          uint32_t v[16];
          tmem_ld16(lane_addr + a * BT + c0, v);
          tc_wait_ld();
          tc_pin(v);
#pragma unroll
          for (int c = 0; c < 16; c += 4) {
            const float4 q = *reinterpret_cast<const float4 *>(sc + c0 + c);
            acc[c0 + c] += __uint_as_float(v[c]) * (q.x * sw);
            acc[c0 + c + 1] += __uint_as_float(v[c + 1]) * (q.y * sw);
            acc[c0 + c + 2] += __uint_as_float(v[c + 2]) * (q.z * sw);
            acc[c0 + c + 3] += __uint_as_float(v[c + 3]) * (q.w * sw);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&ctl.tempty[a]);
          mbar_arrive(&ctl.sempty[s]);
        }
        if (++s == kScaleSlots) { s = 0; sph ^= 1; }
        if (++a == C::kBufs) { a = 0; aph ^= 1; }
      }
      const int n = nt * kRows + row;
      auto store = [&](int f, float v) {
        if (f >= 0 && n < p.N) p.y[(size_t)f * p.ldy + n] = float_to_bf16_bits(v * pair_weight<MODE>(p, f));
      };
      constexpr int kLive = MODE == kFp8Naive ? 1 : BT;   // positions that can hold a pair
      if (cs == 1) {
#pragma unroll
        for (int c = 0; c < kLive; ++c) store(block_pair<MODE>(p, b, c, BT), acc[c]);
        continue;
      }
      // Rank q sums the positions [q * tc, (q + 1) * tc) of every rank's
      // partial sums, in rank order (one position: rank 0 does).  There is one
      // item at most, so that the buffer is used once, and every CTA waits for
      // all that is sent to it: nothing reaches a CTA that has left.
      const int tc = MODE == kFp8Naive ? 1 : BT / cs, lg = __ffs(tc) - 1;
      const uint32_t red_base = smem_addr(smem + cfg.off_red), red_bar = smem_addr(&ctl.red_full);
      const bool receives = MODE != kFp8Naive || wk.rank == 0;
      if (row == 0 && receives) mbar_arrive_expect_tx(&ctl.red_full, (MODE == kFp8Naive ? cs : BT) * kRows * 4);
      cluster_wait();
      waited = true;
      if constexpr (MODE == kFp8Naive) {
        st_async_f1(cluster_map(red_base + (wk.rank * kRows + row) * 4, 0), acc[0], cluster_map(red_bar, 0));
      } else if (tc >= 4) {
#pragma unroll
        for (int c = 0; c < BT; c += 4) {
          const int q = c >> lg, quad = (c - (q << lg)) >> 2;
          st_async_v4(cluster_map(red_base + (((wk.rank * tc) >> 2) + quad) * kRows * 16 + row * 16, q),
                      make_float4(acc[c], acc[c + 1], acc[c + 2], acc[c + 3]), cluster_map(red_bar, q));
        }
      } else {   // two positions a rank
#pragma unroll
        for (int c = 0; c < BT; c += 2)
          st_async_f2(cluster_map(red_base + (wk.rank * kRows + row) * 8, c >> 1), acc[c], acc[c + 1],
                      cluster_map(red_bar, c >> 1));
      }
      if (!receives) continue;
      mbar_wait_cluster(&ctl.red_full, 0, abort, p.err);
      const float *buf = reinterpret_cast<const float *>(smem + cfg.off_red);
      auto finish = [&](auto ranks) {
        constexpr int CS = decltype(ranks)::value;
        if constexpr (MODE == kFp8Naive) {
          float v[1];
          sum_ranks<CS>(buf, 1, 0, row, v);
          store(b, v[0]);
        } else if constexpr (BT / CS >= 4) {
#pragma unroll 4
          for (int quad = 0; quad < BT / CS / 4; ++quad) {
            float v[4];
            sum_ranks<CS>(buf, BT / CS / 4, quad, row, v);
#pragma unroll
            for (int i = 0; i < 4; ++i) store(block_pair<MODE>(p, b, wk.rank * (BT / CS) + quad * 4 + i, BT), v[i]);
          }
        } else {
          float v[2];
          sum_ranks<CS>(buf, 1, 0, row, v);
#pragma unroll
          for (int i = 0; i < 2; ++i) store(block_pair<MODE>(p, b, wk.rank * 2 + i, BT), v[i]);
        }
      };
      if (cs == 2) finish(std::integral_constant<int, 2>());
      else if (cs == 4) finish(std::integral_constant<int, 4>());
      else finish(std::integral_constant<int, 8>());
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

// The rows of the sorted pairs, gathered once into the order of
// sorted_token_ids: the wide kernel reads each of them N / 256 times, and TMA
// fetches gathered rows four at a time at 80 clk each, cp.async by the
// kernel's own warps at 40 % of the tensor cores' time.  CTA 0 also lists the
// tiles of at most 256 rows of one expert.
struct WideTile {
  int row0, rows, expert, pad;
};
constexpr int kGatherThreads = 256;
constexpr int kTileRows = 256;

struct WideSpace {   // offsets into the workspace
  size_t tiles, x, bytes;
  long long rows, ld;   // capacity of the sorted arrays in whole blocks; bytes from row to row
};
WideSpace wide_space(long long rows, int K) {
  WideSpace w;
  w.rows = rows;
  w.ld = (long long)fp8_groups(K) * kFp8Group;
  w.tiles = 0;
  // at most a tile for each of the sorted arrays' smallest blocks, and the count
  w.x = ((size_t)(rows / 16 + 1) * sizeof(WideTile) + sizeof(WideTile) + 127) / 128 * 128;
  w.bytes = w.x + (size_t)rows * w.ld;
  return w;
}

__global__ void __launch_bounds__(kGatherThreads)
    fp8_gather_kernel(const Fp8Args p, WideTile *tiles, uint8_t *xg, long long ld) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bs = p.block;
  wait_for_prior_grid();
  const int nb = num_blocks(p);
  if (blockIdx.x == 0) {
    // Tile list.  Blocks of one expert are neighbours: a run.  A block heads a
    // tile when the blocks before it in its run are a multiple of 256 rows; the
    // last block of a tile writes it down.
    __shared__ int warp_last[kGatherThreads / 32], warp_heads[kGatherThreads / 32], carry_first, carry_heads;
    if (tid == 0) carry_first = carry_heads = 0;
    __syncthreads();
    const int per_tile = kTileRows / bs;
    for (int base = 0; base < nb; base += kGatherThreads) {
      const int b = base + tid;
      const int e = b < nb ? load_global(p.expert_ids + b) : -1;
      const int before_e = b > 0 && b < nb ? load_global(p.expert_ids + b - 1) : e, after_e = b + 1 < nb ? load_global(p.expert_ids + b + 1) : e;
      int run = b < nb && (b == 0 || before_e != e) ? b : -1;   // first block of b's run: the last such at or before b
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, run, d);
        if (lane >= d) run = max(run, o);
      }
      if (lane == 31) warp_last[warp] = run;
      __syncthreads();
      int before = carry_first;
      for (int w = 0; w < warp; ++w) before = max(before, warp_last[w]);
      run = max(run, before);
      const bool good = (unsigned)e < (unsigned)p.E;
      if (b < nb && !good) flag_error(p.err, MOE_LORA_DEVERR_EXPERT_ID);
      const int at = (b - run) % per_tile;   // place in the tile
      const uint32_t heads = __ballot_sync(0xFFFFFFFFu, b < nb && good && at == 0);
      if (lane == 31) warp_heads[warp] = __popc(heads);
      __syncthreads();
      int index = carry_heads + __popc(heads & (0xFFFFFFFFu >> (31 - lane)));   // heads up to b, b among them
      for (int w = 0; w < warp; ++w) index += warp_heads[w];
      // (tiles[0] is the count: tile i is tiles[1 + i])
      if (b < nb && good && (at == per_tile - 1 || b + 1 == nb || after_e != e))
        tiles[index] = {(b - at) * bs, (at + 1) * bs, e, 0};
      __syncthreads();
      if (tid == 0) {
        for (int w = 0; w < kGatherThreads / 32; ++w) {
          carry_first = max(carry_first, warp_last[w]);
          carry_heads += warp_heads[w];
        }
      }
      __syncthreads();
    }
    if (tid == 0) tiles[0] = {carry_heads, 0, 0, 0};
  }
  // one warp a row
  const long long warps = (long long)gridDim.x * (kGatherThreads / 32);
  for (long long r = (long long)blockIdx.x * (kGatherThreads / 32) + warp; r < (long long)nb * bs; r += warps) {
    const int f = load_global(p.sorted_token_ids + r);
    if ((unsigned)f >= (unsigned)p.pairs) {
      if (f != p.pairs && lane == 0) flag_error(p.err, MOE_LORA_DEVERR_PAIR_ID);
      continue;
    }
    const int xr = pair_row<kFp8Sorted>(p, f);
    const uint8_t *src = p.x + (size_t)xr * p.ldx;
    uint8_t *dst = xg + (size_t)r * ld;
    const int whole = p.K / 16;
    for (int c = lane; c < whole; c += 32)
      *reinterpret_cast<uint4 *>(dst + c * 16) = load_global(reinterpret_cast<const uint4 *>(src + c * 16));
    for (int c = whole * 16 + lane; c < p.K; c += 32) dst[c] = load_global(src + c);
  }
}

// The wide kernel: pairs of CTAs (cta_group::2), 256 rows by 256 output
// columns.  Each CTA holds 128 of the rows and half of the weight's columns in
// shared memory, 32 KB a group, and 128 x 256 of the accumulators in tensor
// memory: four accumulators of 128 columns, two groups of two halves.
// A group takes the tensor cores 512 clk, and about 750 in all (8192 x 4096 x
// 4096 dense): the epilogue's reads and FMAs of an accumulator take 550 of the
// 768 that pass before it is due again, the hand-shake over two CTAs the rest.
// A single CTA with 128 x 256 tiles and two accumulators took 108 us, accumulators
// handed back before their FMAs 104, sixteen epilogue warps 115, MMAs of 256
// columns 99, against 97.
constexpr int kWideThreads = 384;
constexpr int kWideN = 256;
constexpr int kHalf = kWideN / 2;
constexpr int kWideStage = 2 * kTileBytes;       // 128 rows, and 128 columns of the weight
constexpr int kWideStages = 6;
constexpr int kWideOut = 32 * 128;               // an epilogue warp's rows on their way out: 32 rows of 64 bf16
// Registers a thread: loading and MMA warps, epilogue warps.  A split by which
// the compiler spills nothing: with 48 and 224, or 64 and 208, it spills 80 to
// 136 bytes in the epilogue's loop (97 -> 145 us).
constexpr int kWideRegsIssue = 56, kWideRegsEpilogue = 216;

struct WideCtrl {
  uint64_t full[kWideStages], empty[kWideStages];
  uint64_t tfull[4], tempty[4];
  uint64_t done;   // every MMA of the pair
  uint32_t tmem;
  int abort;
};

struct WideArgs {
  const WideTile *tiles;   // sorted: count, then the tiles
};

template <int MODE>
__global__ void __launch_bounds__(kWideThreads, 1)
    fp8_wide_kernel(const __grid_constant__ Fp8Maps maps, const Fp8Args p, const WideArgs g, const Fp8Cfg cfg) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  WideCtrl &ctl = *reinterpret_cast<WideCtrl *>(smem + cfg.off_ctrl);
  volatile int *abort = &ctl.abort;
  const int rank = blockIdx.x & 1;   // rank 0 issues the pair's MMAs

  if (tid == 0) {
    for (int s = 0; s < kWideStages; ++s) {
      mbar_init(&ctl.full[s], 1);
      mbar_init(&ctl.empty[s], 2);   // a commit for each half of the columns
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&ctl.tfull[s], 1);
      mbar_init(&ctl.tempty[s], 8);   // four epilogue warps of each CTA
    }
    mbar_init(&ctl.done, 2);          // a commit of each MMA warp
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
  const int ntiles = MODE == kFp8Dense ? (p.pairs + kTileRows - 1) / kTileRows : load_global(&g.tiles[0].row0);
  const int items = ntiles * cfg.nt;   // rows fastest: pairs at work share the weight's columns
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;
  auto tile = [&](int t) {
    if (MODE == kFp8Dense) return WideTile{t * kTileRows, min(kTileRows, p.pairs - t * kTileRows), 0, 0};
    const int4 v = load_global(reinterpret_cast<const int4 *>(g.tiles) + 1 + t);
    return WideTile{v.x, v.y, v.z, 0};
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kWideRegsIssue));
    if (warp == 0) {
      // ---------------- operands: this CTA's rows, and its 64 of each 128 columns
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
            if (have) tma_load_2d_pair(st, &maps.x, kb * kFp8Group, t.row0 + rank * kRows, full0 + s * 8);
#pragma unroll
            for (int h = 0; h < 2; ++h)
              tma_load_3d_pair(st + kTileBytes + h * (kTileBytes / 2), &maps.w, kb * kFp8Group,
                               nt * kWideN + h * kHalf + rank * (kHalf / 2), t.expert, full0 + s * 8);
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
    } else if (warp <= 2 && rank == 0) {
      // ---------------- MMA, for both CTAs: a warp for each half of the
      // columns, with accumulators of its own.  (An MMA takes 51 to 64 clk to
      // issue, and 64 to run.)
      constexpr uint32_t idesc = make_idesc_e4m3(2 * kRows, kHalf);
      const int h = warp - 1;
      const uint64_t desc0 = make_sdesc_sw128(smem_addr(smem));   // (addresses in units of 16 bytes)
      int s = 0, a = 0;
      uint32_t ph = 0, aph = 0;
      for (int it = first; it < items; it += step) {
        for (int kb = 0; kb < p.KB; ++kb) {
          mbar_wait(&ctl.tempty[a + h], aph ^ 1, abort, p.err);
          mbar_wait(&ctl.full[s], ph, abort, p.err);
          tc_fence_after();
          const uint64_t dx = desc0 + s * (kWideStage >> 4), dw = dx + (kTileBytes >> 4) + h * (kTileBytes >> 5);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kFp8Group / 32; ++k)
              tc_mma_f8_pair(tmem + (a + h) * kHalf, dx + k * 2, dw + k * 2, idesc, k > 0);
            tc_commit_pair(&ctl.tfull[a + h]);
            tc_commit_pair(&ctl.empty[s]);
          }
          __syncwarp();
          if (++s == kWideStages) { s = 0; ph ^= 1; }
          a ^= 2;
          if (a == 0) aph ^= 1;
        }
      }
      if (elect_one()) tc_commit_pair(&ctl.done);
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kWideRegsEpilogue));
    // ---------------- epilogue: this thread's row, one half (128 columns: one scale) of the output tile
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const uint32_t lane_addr = tmem + ((uint32_t)quarter << 21) + half * kHalf;
    const uint32_t tempty0 = cluster_map(smem_addr(&ctl.tempty[half]), 0);   // rank 0's
    const uint32_t tfull0 = smem_addr(&ctl.tfull[half]);
    int a = 0;
    uint32_t aph = 0;
    for (int it = first; it < items; it += step) {
      const int nt = it / ntiles;
      const WideTile t = tile(it - nt * ntiles);
      const int r = rank * kRows + quarter * 32 + lane;   // row of the tile
      int f = -1;
      if (r < t.rows) f = MODE == kFp8Dense ? t.row0 + r : load_global(p.sorted_token_ids + t.row0 + r);
      if ((unsigned)f >= (unsigned)p.pairs) f = -1;
      const int nblk = nt * 2 + half;
      const float *sx = f < 0 ? nullptr : p.x_scales + (size_t)pair_row<MODE>(p, f) * p.KB;
      const float *sw = nblk < p.NB ? p.w_scales + ((size_t)t.expert * p.NB + nblk) * p.KB : nullptr;
      f32x2 acc[64];
#pragma unroll
      for (int c = 0; c < 64; ++c) acc[c] = 0;
      // the scales of the next two groups are on their way
      auto load = [](const float *s, int kb, int n) { return s && kb < n ? load_global(s + kb) : 0.f; };
      float sc0 = load(sx, 0, p.KB) * load(sw, 0, p.KB), sx1 = load(sx, 1, p.KB), sw1 = load(sw, 1, p.KB);
#pragma unroll 1
      for (int kb = 0; kb < p.KB; ++kb) {
        const f32x2 sc2 = f2_pack(sc0, sc0);
        const float sx2 = load(sx, kb + 2, p.KB), sw2 = load(sw, kb + 2, p.KB);
        mbar_wait_lean(tfull0 + a * 8, aph, abort, p.err);
        tc_fence_after();
        const uint32_t src = lane_addr + a * kHalf;
        // the next 32 columns are on their way while these are added
        uint32_t v[2][32];
        tmem_ld32(src, v[0]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          tc_wait_ld();
          tc_pin(v[q & 1]);
          if (q < 3) {
            tmem_ld32(src + (q + 1) * 32, v[(q + 1) & 1]);
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote_relaxed(tempty0 + a * 8);   // (only tensor memory is handed back)
          }
#pragma unroll
          for (int c = 0; c < 16; ++c)
            acc[q * 16 + c] = ffma2(f2_pack(__uint_as_float(v[q & 1][2 * c]), __uint_as_float(v[q & 1][2 * c + 1])), sc2,
                                    acc[q * 16 + c]);
        }
        sc0 = sx1 * sw1;
        sx1 = sx2;
        sw1 = sw2;
        a ^= 2;
        if (a == 0) aph ^= 1;
      }
      // Out through shared memory, 64 columns at a time, so that 8 lanes write
      // 128 consecutive bytes of one row (a lane writing its own row touches 32
      // lines an instruction: 4096 clk a tile).
      const float w = f < 0 ? 0.f : pair_weight<MODE>(p, f);
      const int n0 = nblk * kRows;
      // 16 bytes at a time where rows are on 16 bytes and the 128 columns exist
      const bool whole = (p.ldy & 7) == 0 && (reinterpret_cast<uintptr_t>(p.y) & 15) == 0 && n0 + kRows <= p.N;
      uint8_t *out = smem + kWideStages * kWideStage + (warp - 4) * kWideOut;
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float lo, hi;
            f2_unpack(acc[part * 32 + c * 4 + i], lo, hi);
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[i]) : "f"(hi * w), "f"(lo * w));
          }
          *reinterpret_cast<uint4 *>(out + lane * 128 + ((c ^ (lane & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        __syncwarp();
        const int chunk = lane & 7, n = n0 + part * 64 + chunk * 8;
#pragma unroll
        for (int i0 = 0; i0 < 8; i0 += 2) {
          uint4 o[2];
          int fr[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = (i0 + i) * 4 + (lane >> 3);
            fr[i] = __shfl_sync(0xFFFFFFFFu, f, r);
            o[i] = *reinterpret_cast<const uint4 *>(out + r * 128 + ((chunk ^ (r & 7)) << 4));
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (fr[i] < 0) continue;
            uint16_t *dst = p.y + (size_t)fr[i] * p.ldy + n;
            if (whole) {
              *reinterpret_cast<uint4 *>(dst) = o[i];
            } else {
              const uint32_t v[4] = {o[i].x, o[i].y, o[i].z, o[i].w};
#pragma unroll
              for (int j = 0; j < 8; ++j)
                if (n + j < p.N) dst[j] = (uint16_t)(v[j >> 1] >> (16 * (j & 1)));
            }
          }
        }
      }
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

int make_maps(const Fp8Args &a, const uint8_t *x, long long rows, long long ldx, int w_box_rows, int x_box_rows,
              Fp8Maps *maps) {
  if (int st = stream::encode_u8(&maps->w, a.w, 3, a.K, a.N, a.E, a.ldw, (uint64_t)a.ldw * a.N, w_box_rows)) return st;
  return stream::encode_u8(&maps->x, x, 2, a.K, rows, 1, ldx, 0, x_box_rows);
}

// The wide kernel's warps trade registers after the launch: the shares must
// fit what the block was launched with, or the trade would wait forever.
template <typename Kernel>
bool register_shares_fit(Kernel kernel) {
  cudaFuncAttributes attr;
  if (cudaFuncGetAttributes(&attr, (const void *)kernel) != cudaSuccess) return false;
  return attr.numRegs * kWideThreads >= 128 * kWideRegsIssue + 256 * kWideRegsEpilogue;
}

// Clusters of this shape that are resident at once; asked once for each shape.
template <typename Kernel>
int resident_clusters(Kernel kernel, const Fp8Cfg &cfg, int threads, const DeviceInfo &dev) {
  if (cfg.cluster == 1) return dev.sm_count;
  struct Entry {
    const void *kernel;
    int device, cluster, smem, clusters;
  };
  static std::mutex mu;
  static Entry known[64];
  static int n = 0;
  std::lock_guard<std::mutex> lock(mu);
  for (int i = 0; i < n; ++i)
    if (known[i].kernel == (const void *)kernel && known[i].device == dev.device && known[i].cluster == cfg.cluster && known[i].smem == cfg.smem_bytes)
      return known[i].clusters;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)cfg.cluster, 1, 1);
  lc.blockDim = dim3(threads, 1, 1);
  lc.dynamicSmemBytes = cfg.smem_bytes;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cfg.cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  int clusters = 0;
  if (cudaOccupancyMaxActiveClusters(&clusters, (const void *)kernel, &lc) != cudaSuccess) {
    cudaGetLastError();   // a failed query leaves no sticky error
    clusters = 0;
  }
  if (clusters < 1) clusters = std::max(1, dev.sm_count / cfg.cluster / 2);
  if (n < 64) known[n++] = {(const void *)kernel, dev.device, cfg.cluster, cfg.smem_bytes, clusters};
  return clusters;
}

// Upper bound of the call's units (skipped ones included).
long long block_bound(const Fp8Args &a, Fp8Mode mode, int bt) {
  if (mode == kFp8Dense) return ((long long)a.pairs + bt - 1) / bt;
  if (mode == kFp8Naive) return a.pairs;
  return std::min<long long>(a.max_blocks, fused_block_bound(a.pairs, 1, a.E, 1, a.block)) * (a.block / bt);
}

// Upper bound of the wide kernel's tiles of rows.
long long tile_bound(const Fp8Args &a, bool sorted) {
  return sorted ? a.pairs / kTileRows + std::min(a.E, a.pairs) : ((long long)a.pairs + kTileRows - 1) / kTileRows;
}

template <int BT, int MODE>
int launch_narrow(const Fp8Args &a, const DeviceInfo &dev, cudaStream_t stream) {
  using C = Narrow<BT>;
  Fp8Cfg cfg = {};
  cfg.nt = (a.N + kRows - 1) / kRows;
  const long long items = block_bound(a, (Fp8Mode)MODE, BT) * cfg.nt;
  if (items <= 0) return 0;
  if (int st = allow_dynamic_smem((const void *)fp8_narrow_kernel<BT, MODE>)) return st;
  if (MODE == kFp8Sorted && a.block > BT) cfg.list = kListUnits;
  // Clusters that split K: while there are too few items for the SMs, as large
  // as leaves each CTA two groups and every item a cluster of its own.  A ring
  // no longer than a CTA's share lets more clusters fit (of 8 CTAs with 200 KB
  // each: 15).  (Pairs that split the last of several rounds cost more than
  // they gave: gpt-oss-shaped w2 decode 146 us against 140.)
  auto shape = [&](int cs) {
    cfg.cluster = cs;
    const int list_bytes = cfg.list * 4;
    const int fixed = kScaleSlots * C::kScaleRow * 4 + (cs > 1 ? C::kRedBytes : 0) + list_bytes + (int)sizeof(NarrowCtrl) + 128;
    const int share = items * cs <= dev.sm_count ? ((a.KB + cs - 1) / cs + 1) / 2 : kMaxRing;
    cfg.stages = std::max(2, std::min(share, std::min(kMaxRing, (200 * 1024 - fixed) / C::kStage)));
    cfg.off_scale = cfg.stages * C::kStage;
    cfg.off_red = cfg.off_scale + kScaleSlots * C::kScaleRow * 4;
    cfg.off_list = cfg.off_red + (cs > 1 ? C::kRedBytes : 0);
    cfg.off_ctrl = cfg.off_list + list_bytes;
    cfg.smem_bytes = cfg.off_ctrl + (int)sizeof(NarrowCtrl);
    return resident_clusters(fp8_narrow_kernel<BT, MODE>, cfg, kNarrowThreads, dev);
  };
  int cs = 1;
  while (cs < 8 && items * cs * 2 <= dev.sm_count && a.KB >= cs * 4) cs *= 2;
  int fit = shape(cs);
  while (cs > 1 && fit < items) fit = shape(cs /= 2);
  const unsigned clusters = (unsigned)std::min<long long>(items, std::min(fit, dev.sm_count / cs));
  Fp8Maps maps;
  if (int st = make_maps(a, a.x, a.rows, a.ldx, kRows, MODE == kFp8Dense ? BT : 1, &maps)) return st;
  return launch_dependent(fp8_narrow_kernel<BT, MODE>, clusters * cs, kNarrowThreads, cs, cfg.smem_bytes, stream, maps, a,
                          cfg);
}

template <int MODE>
int launch_wide(const Fp8Args &a, void *workspace, const DeviceInfo &dev, cudaStream_t stream) {
  Fp8Cfg cfg = {};
  cfg.nt = (a.N + kWideN - 1) / kWideN;
  const long long rows = (long long)a.max_blocks * a.block;
  const long long tiles = tile_bound(a, MODE == kFp8Sorted);
  if (tiles <= 0) return 0;
  cfg.stages = kWideStages;
  cfg.off_ctrl = kWideStages * kWideStage + 8 * kWideOut;
  cfg.smem_bytes = cfg.off_ctrl + (int)sizeof(WideCtrl);
  static const bool fits = register_shares_fit(fp8_wide_kernel<MODE>);
  if (!fits) return MOE_LORA_ERR_LAUNCH;
  if (int st = allow_dynamic_smem((const void *)fp8_wide_kernel<MODE>)) return st;
  Fp8Maps maps;
  WideArgs g = {};
  if (MODE == kFp8Dense) {
    if (int st = make_maps(a, a.x, a.rows, a.ldx, kHalf / 2, kRows, &maps)) return st;
  } else {
    const WideSpace w = wide_space(rows, a.K);
    uint8_t *base = static_cast<uint8_t *>(workspace);
    g.tiles = reinterpret_cast<WideTile *>(base + w.tiles);
    if (int st = make_maps(a, base + w.x, rows, w.ld, kHalf / 2, kRows, &maps)) return st;
    if (int st = launch_dependent(fp8_gather_kernel, (unsigned)std::min<long long>((rows + 7) / 8, dev.sm_count * 8ll),
                                  kGatherThreads, 1, 0, stream, a, reinterpret_cast<WideTile *>(base + w.tiles),
                                  base + w.x, w.ld))
      return st;
  }
  const long long items = tiles * cfg.nt;   // (the sorted arrays' own tiles are no more, but for entries that no align writes)
  const unsigned grid = 2 * (unsigned)std::min<long long>(items, dev.sm_count / 2);
  return launch_dependent(fp8_wide_kernel<MODE>, grid, kWideThreads, 2, cfg.smem_bytes, stream, maps, a, g, cfg);
}

}  // namespace

// Up to this many bytes of weights, calls of single pairs or of at most 16 rows
// run the kernel that streams the weight through registers: it starts in half
// the time (2048 x 2048 and one row: 2.5 us against 4.9), but has fewer bytes
// in flight (8192 x 8192: 19 us against 16).
constexpr double kStreamBytes = 32e6;

// Sorted calls run the wide kernel from 20 pairs an expert on (on average), the
// narrow one, in units of 16, below.  Below, a call is bound by the weight's
// bytes, and tiles of 256 rows and the gather cost more than they give; above,
// an expert's units read its weight again and again.  128 experts of 2048 x
// 1536, us narrow / wide: 4 pairs an expert 66 / 86, 8 68 / 89, 16 76 / 92, 32
// 123 / 95, 64 220 / 100; with a skewed router 4 57 / 74, 8 71 / 89, 16 89 / 96.
// (Units of 32 and 64 were slower than of 16 wherever the narrow kernel wins:
// 92 us at 16 pairs an expert, also over gathered rows.)
// That is one weight's shape: K and N are not in the rule, though the bytes that
// a unit reads again and the cost of a tile grow with them.
// The narrow one also while a round of its items covers the output (16 experts
// of 1024 x 1024 and 128 pairs: 10 us, 13 wide).  A round is a GB300's 152 SMs,
// not the current device's: the workspace's size is asked for on hosts without one.
constexpr long long kRoundItems = 152;
bool fp8_sorted_is_wide(const Fp8Args &a) {
  const long long units = a.pairs / 16 + std::min(a.E, a.pairs);
  return a.pairs >= 20ll * a.E && units * ((a.N + kRows - 1) / kRows) > kRoundItems;
}

size_t fp8_sorted_workspace(const Fp8Args &a) {
  return fp8_sorted_is_wide(a) ? wide_space((long long)a.max_blocks * a.block, a.K).bytes : 0;
}

bool fp8_items_fit(const Fp8Args &a, Fp8Mode mode) {
  if (mode == kFp8Dense ? a.pairs > 64 : mode == kFp8Sorted && fp8_sorted_is_wide(a))
    return tile_bound(a, mode == kFp8Sorted) * ((a.N + kWideN - 1) / kWideN) <= INT32_MAX / 16;
  // every unit that the sorted arrays can hold, whatever they hold
  const long long units = mode == kFp8Sorted ? (long long)a.max_blocks * (a.block / 16) : block_bound(a, mode, 16);
  return units * ((a.N + kRows - 1) / kRows) <= INT32_MAX;
}

int launch_fp8_matmul(const Fp8Args &a, Fp8Mode mode, void *workspace, const DeviceInfo &dev, cudaStream_t s) {
  const bool small = (mode == kFp8Naive ? (double)a.pairs : 1.0) * a.N * a.K <= kStreamBytes;
  if (mode == kFp8Naive) return small ? launch_fp8_stream(a, mode, dev, s) : launch_narrow<16, kFp8Naive>(a, dev, s);
  if (mode == kFp8Sorted) {
    if (fp8_sorted_is_wide(a)) return launch_wide<kFp8Sorted>(a, workspace, dev, s);
    return launch_narrow<16, kFp8Sorted>(a, dev, s);
  }
  if (small && a.pairs <= 16) return launch_fp8_stream(a, mode, dev, s);
  if (a.pairs <= 16) return launch_narrow<16, kFp8Dense>(a, dev, s);
  if (a.pairs <= 32) return launch_narrow<32, kFp8Dense>(a, dev, s);
  // The narrow kernel while one round of its 64 x 128 items covers the output
  // (192 x 4096 x 4096: 14.2 us, 16.2 wide), else the wide one (192 x 8192 x
  // 8192: 27 us, 41 narrow).
  const long long items = ((a.pairs + 63ll) / 64) * ((a.N + kRows - 1) / kRows);
  if (a.pairs <= 64 || items <= dev.sm_count) return launch_narrow<64, kFp8Dense>(a, dev, s);
  return launch_wide<kFp8Dense>(a, nullptr, dev, s);
}

}  // namespace moe_lora
