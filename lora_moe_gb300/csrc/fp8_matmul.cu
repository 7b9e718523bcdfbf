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
// Two kernels, both persistent, with a warp that loads (TMA), a warp that
// issues the MMAs and epilogue warps:
//   narrow  the weight on the 128 rows of the MMA, 16 to 64 pairs on its
//           columns: few pairs for each weight (decode), bound by the weight's
//           bytes.  A cluster of CTAs may split K, its partial sums exchanged
//           through distributed shared memory in a fixed order.
//   wide    128 pairs on the rows, 256 output columns: bound by the tensor cores.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "device_utils.cuh"
#include "fp8.h"
#include "stream_pipeline.cuh"

namespace moe_lora {

namespace {

constexpr int kRows = 128;                     // M of every tcgen05.mma here
constexpr int kTileBytes = kRows * kFp8Group;  // 128 rows of one group: 16 KB, one swizzle row of 128 bytes each

struct Fp8Maps {
  CUtensorMap w;   // [E][N][K], box 1 x 128 x 128
  CUtensorMap x;   // [rows][K], box BT x 128 (dense) or 1 x 128 (gathered)
};

// Launch shape of a call.
struct Fp8Cfg {
  int stages;      // operand ring
  int nt;          // output tiles along N
  int cluster;     // CTAs that split K (narrow)
  int off_scale, off_red, off_ctrl;
  int smem_bytes;
};

// The blocks of a call: on the device for the sorted arrays.
template <int MODE>
__device__ __forceinline__ int num_blocks(const Fp8Args &p, int bt) {
  if (MODE == kFp8Dense) return (p.pairs + bt - 1) / bt;
  if (MODE == kFp8Naive) return p.pairs;
  const int n = __ldg(p.num_tokens_post_padded) / bt;
  return n < 0 ? 0 : (n > p.max_blocks ? p.max_blocks : n);
}
// Expert of block b, or -1 where the id is out of range (the block is skipped).
template <int MODE>
__device__ __forceinline__ int block_expert(const Fp8Args &p, int b) {
  if (MODE == kFp8Dense) return 0;
  const int e = MODE == kFp8Sorted ? __ldg(p.expert_ids + b) : __ldg(p.topk_ids + b);
  return (unsigned)e < (unsigned)p.E ? e : -1;
}
// Pair at position t of block b, or -1.  `bt` positions a block.
template <int MODE>
__device__ __forceinline__ int block_pair(const Fp8Args &p, int b, int t, int bt) {
  if (MODE == kFp8Naive) return t == 0 ? b : -1;
  int f;
  if (MODE == kFp8Dense) f = b * bt + t;
  else f = __ldg(p.sorted_token_ids + (size_t)b * bt + t);
  return (unsigned)f < (unsigned)p.pairs ? f : -1;
}
template <int MODE>
__device__ __forceinline__ int pair_row(const Fp8Args &p, int f) {
  return MODE == kFp8Dense || p.x_per_pair ? f : f / p.topk;
}
// Report the entries of the sorted arrays that are out of range.
template <int MODE>
__device__ __forceinline__ void flag_block(const Fp8Args &p, int b, int t, int bt) {
  if (MODE != kFp8Sorted) return;
  if ((unsigned)__ldg(p.sorted_token_ids + (size_t)b * bt + t) > (unsigned)p.pairs) flag_error(p.err, MOE_LORA_DEVERR_PAIR_ID);
}
template <int MODE>
__device__ __forceinline__ float pair_weight(const Fp8Args &p, int f) {
  return MODE != kFp8Dense && p.topk_weights ? __ldg(p.topk_weights + f) : 1.f;
}

// ------------------------------------------------------------------ narrow

constexpr int kNarrowThreads = 256;
constexpr int kMaxRing = 12;
constexpr int kScaleSlots = 16;   // ring of scale rows, one group each

template <int BT>
struct Narrow {
  static constexpr int kStage = kTileBytes + BT * kFp8Group;
  static constexpr int kScaleRow = BT + 4;    // BT row scales and the weight's, padded to 16 bytes
  static constexpr int kBufs = 4;             // accumulators in tensor memory
  static constexpr int kCols = kBufs * BT;    // power of two, >= 32
  static constexpr int kRedBytes = BT * kRows * 4;   // one exchange buffer: every rank's partial sums of this CTA's columns
};

struct NarrowCtrl {
  uint64_t full[kMaxRing], empty[kMaxRing];
  uint64_t sfull[kScaleSlots], sempty[kScaleSlots];
  uint64_t tfull[4], tempty[4];
  uint64_t red_full[2], red_empty[2];
  uint32_t tmem;
  int abort;
};

template <int BT, int MODE>
__global__ void __launch_bounds__(kNarrowThreads, 1)
    fp8_narrow_kernel(const __grid_constant__ Fp8Maps maps, const Fp8Args p, const Fp8Cfg cfg) {
  using C = Narrow<BT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  NarrowCtrl &ctl = *reinterpret_cast<NarrowCtrl *>(smem + cfg.off_ctrl);
  float *scales = reinterpret_cast<float *>(smem + cfg.off_scale);
  volatile int *abort = &ctl.abort;
  const int cs = cfg.cluster, rank = blockIdx.x % cs;   // (a cluster is cs consecutive CTAs)
  const int cid = blockIdx.x / cs, nclusters = gridDim.x / cs;

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
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ctl.red_full[s], 1);
      mbar_init(&ctl.red_empty[s], cs);
    }
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
  if (cs > 1) {   // peers' barriers are initialised before anything is sent to them
    cluster_arrive_release();
    cluster_wait();
  }
  const uint32_t tmem = ctl.tmem;
  const int items = num_blocks<MODE>(p, BT) * cfg.nt;
  const int kb0 = (int)((long long)p.KB * rank / cs), kb1 = (int)((long long)p.KB * (rank + 1) / cs);

  if (warp == 0) {
    // ---------------- operands: the weight's tile, and the pairs' rows
    int s = 0;
    uint32_t ph = 0;
    for (int it = cid; it < items; it += nclusters) {
      const int b = it / cfg.nt, nt = it - b * cfg.nt, e = block_expert<MODE>(p, b);
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
      for (int kb = kb0; kb < kb1; ++kb) {
        mbar_wait(&ctl.empty[s], ph ^ 1, abort, p.err);
        uint8_t *st = smem + (size_t)s * C::kStage;
        if (lane == 0) {
          mbar_arrive_expect_tx(&ctl.full[s], kTileBytes + groups * 4 * kFp8Group);
          tma_load_3d(st, &maps.w, kb * kFp8Group, nt * kRows, e, &ctl.full[s]);
          if (MODE == kFp8Dense) tma_load_2d(st + kTileBytes, &maps.x, kb * kFp8Group, b * BT, &ctl.full[s]);
        }
        __syncwarp();
        if (MODE != kFp8Dense && mine)
          tma_gather4(st + kTileBytes + lane * 4 * kFp8Group, &maps.x, kb * kFp8Group, row, &ctl.full[s]);
        if (++s == cfg.stages) { s = 0; ph ^= 1; }
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA: each group of 128 columns into an accumulator of its own
    if (lane == 0) {
      constexpr uint32_t idesc = make_idesc_e4m3(kRows, BT);
      int s = 0, a = 0;
      uint32_t ph = 0, aph = 0;
      for (int it = cid; it < items; it += nclusters) {
        if (block_expert<MODE>(p, it / cfg.nt) < 0) continue;
        for (int kb = kb0; kb < kb1; ++kb) {
          mbar_wait(&ctl.tempty[a], aph ^ 1, abort, p.err);
          mbar_wait(&ctl.full[s], ph, abort, p.err);
          tc_fence_after();
          const uint32_t st = smem_addr(smem + (size_t)s * C::kStage);
#pragma unroll
          for (int k = 0; k < kFp8Group / 32; ++k)
            tc_mma_f8(tmem + a * BT, make_sdesc_sw128(st + k * 32), make_sdesc_sw128(st + kTileBytes + k * 32), idesc,
                      k > 0);
          tc_commit(&ctl.empty[s]);
          tc_commit(&ctl.tfull[a]);
          if (++s == cfg.stages) { s = 0; ph ^= 1; }
          if (++a == C::kBufs) { a = 0; aph ^= 1; }
        }
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    // ---------------- scales: a row of BT + 1 for each group
    int s = 0;
    uint32_t ph = 0;
    for (int it = cid; it < items; it += nclusters) {
      const int b = it / cfg.nt, nt = it - b * cfg.nt, e = block_expert<MODE>(p, b);
      if (e < 0) {
        if (lane == 0 && nt == 0 && rank == 0) flag_error(p.err, MOE_LORA_DEVERR_EXPERT_ID);
        continue;
      }
      constexpr int kPer = (BT + 31) / 32;
      const float *src[kPer];
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int t = j * 32 + lane;
        int f = -1;
        if (t < BT) {
          f = block_pair<MODE>(p, b, t, BT);
          if (nt == 0 && rank == 0) flag_block<MODE>(p, b, t, BT);
        }
        src[j] = f < 0 ? nullptr : p.x_scales + (size_t)pair_row<MODE>(p, f) * p.KB;
      }
      const float *sw = p.w_scales + ((size_t)e * p.NB + nt) * p.KB;
      for (int kb = kb0; kb < kb1; ++kb) {
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
  } else if (warp >= 4) {
    // ---------------- epilogue: this thread's weight row, BT pairs
    const int row = (warp - 4) * 32 + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)(warp - 4) << 21);   // lane offset 32 * quarter in bits 16..31
    int s = 0, a = 0;
    uint32_t sph = 0, aph = 0;
    int red = 0;
    uint32_t rph = 0;
    for (int it = cid; it < items; it += nclusters) {
      const int b = it / cfg.nt, nt = it - b * cfg.nt;
      if (block_expert<MODE>(p, b) < 0) continue;
      float acc[BT];
#pragma unroll
      for (int c = 0; c < BT; ++c) acc[c] = 0.f;
      for (int kb = kb0; kb < kb1; ++kb) {
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
      // partial sums, in rank order (one position: rank 0 does).
      const int tc = MODE == kFp8Naive ? 1 : BT / cs, lg = __ffs(tc) - 1;
      const uint32_t red_base = smem_addr(smem + cfg.off_red) + red * C::kRedBytes;
      const bool receives = MODE != kFp8Naive || rank == 0;
      if (row == 0 && receives) mbar_arrive_expect_tx(&ctl.red_full[red], (MODE == kFp8Naive ? cs : BT) * kRows * 4);
      mbar_wait_cluster(&ctl.red_empty[red], rph ^ 1, abort, p.err);
      if constexpr (MODE == kFp8Naive) {
        st_async_f1(cluster_map(red_base + (rank * kRows + row) * 4, 0), acc[0],
                    cluster_map(smem_addr(&ctl.red_full[red]), 0));
      } else {
#pragma unroll
        for (int c = 0; c < BT; c += 2) {
          const int q = c >> lg, tl = c - (q << lg);
          st_async_f2(cluster_map(red_base + (((rank * tc + tl) >> 1) * kRows + row) * 8, q), acc[c], acc[c + 1],
                      cluster_map(smem_addr(&ctl.red_full[red]), q));
        }
      }
      if (receives) {
        mbar_wait_cluster(&ctl.red_full[red], rph, abort, p.err);
        const float *buf = reinterpret_cast<const float *>(smem + cfg.off_red + red * C::kRedBytes);
        if constexpr (MODE == kFp8Naive) {
          float v = 0.f;
          for (int q = 0; q < cs; ++q) v += buf[q * kRows + row];
          store(b, v);
        } else {
          for (int tl = 0; tl < tc; tl += 2) {
            float v0 = 0.f, v1 = 0.f;
            for (int q = 0; q < cs; ++q) {
              const float2 u = *reinterpret_cast<const float2 *>(buf + (((q * tc + tl) >> 1) * kRows + row) * 2);
              v0 += u.x;
              v1 += u.y;
            }
            store(block_pair<MODE>(p, b, rank * tc + tl, BT), v0);
            store(block_pair<MODE>(p, b, rank * tc + tl + 1, BT), v1);
          }
        }
      }
      // the buffer may be written again once every rank has read its own
      named_barrier(1, 128);
      if (row < cs) mbar_arrive_remote(cluster_map(smem_addr(&ctl.red_empty[red]), row));
      if (++red == 2) { red = 0; rph ^= 1; }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
  if (cs > 1) {   // no CTA leaves while a peer may still arrive on its barriers
    cluster_arrive_release();
    cluster_wait();
  }
}

// ------------------------------------------------------------------ wide

constexpr int kWideThreads = 384;
constexpr int kWideN = 256;
constexpr int kWideStage = kTileBytes + kWideN * kFp8Group;   // 48 KB
constexpr int kWideStages = 4;
constexpr int kWideRegsIssue = 56, kWideRegsEpilogue = 216;   // registers a thread: loading and MMA warps, epilogue warps

struct WideCtrl {
  uint64_t full[kWideStages], empty[kWideStages];
  uint64_t tfull[2], tempty[2];
  uint32_t tmem;
  int abort;
};

template <int MODE>
__global__ void __launch_bounds__(kWideThreads, 1)
    fp8_wide_kernel(const __grid_constant__ Fp8Maps maps, const Fp8Args p, const Fp8Cfg cfg) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  WideCtrl &ctl = *reinterpret_cast<WideCtrl *>(smem + cfg.off_ctrl);
  volatile int *abort = &ctl.abort;
  constexpr int BT = kRows;

  if (tid == 0) {
    for (int s = 0; s < kWideStages; ++s) {
      mbar_init(&ctl.full[s], 1);
      mbar_init(&ctl.empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ctl.tfull[s], 1);
      mbar_init(&ctl.tempty[s], 8);
    }
    ctl.abort = 0;
    fence_barrier_init();
    prefetch_tensor_map(&maps.w);
    prefetch_tensor_map(&maps.x);
  }
  if (warp == 1) {
    tmem_alloc(&ctl.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem;
  const int nb = num_blocks<MODE>(p, BT);
  const long long items = (long long)nb * cfg.nt;   // blocks fastest: CTAs at work share the weight's tiles

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kWideRegsIssue));
    if (warp == 0) {
      int s = 0;
      uint32_t ph = 0;
      for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        const int nt = (int)(it / nb), b = (int)(it - (long long)nt * nb), e = block_expert<MODE>(p, b);
        if (e < 0) continue;
        int row[4];
        bool mine = false;
        if (MODE != kFp8Dense) {
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
        for (int kb = 0; kb < p.KB; ++kb) {
          mbar_wait(&ctl.empty[s], ph ^ 1, abort, p.err);
          uint8_t *st = smem + (size_t)s * kWideStage;
          if (lane == 0) {
            mbar_arrive_expect_tx(&ctl.full[s], kWideN * kFp8Group + groups * 4 * kFp8Group);
            tma_load_3d(st + kTileBytes, &maps.w, kb * kFp8Group, nt * kWideN, e, &ctl.full[s]);
            tma_load_3d(st + 2 * kTileBytes, &maps.w, kb * kFp8Group, nt * kWideN + kRows, e, &ctl.full[s]);
            if (MODE == kFp8Dense) tma_load_2d(st, &maps.x, kb * kFp8Group, b * BT, &ctl.full[s]);
          }
          __syncwarp();
          if (MODE != kFp8Dense && mine)
            tma_gather4(st + lane * 4 * kFp8Group, &maps.x, kb * kFp8Group, row, &ctl.full[s]);
          if (++s == kWideStages) { s = 0; ph ^= 1; }
        }
      }
    } else if (warp == 1 && lane == 0) {
      constexpr uint32_t idesc = make_idesc_e4m3(kRows, kWideN);
      int s = 0, a = 0;
      uint32_t ph = 0, aph = 0;
      for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        if (block_expert<MODE>(p, (int)(it % nb)) < 0) continue;
        for (int kb = 0; kb < p.KB; ++kb) {
          mbar_wait(&ctl.tempty[a], aph ^ 1, abort, p.err);
          mbar_wait(&ctl.full[s], ph, abort, p.err);
          tc_fence_after();
          const uint32_t st = smem_addr(smem + (size_t)s * kWideStage);
#pragma unroll
          for (int k = 0; k < kFp8Group / 32; ++k)
            tc_mma_f8(tmem + a * kWideN, make_sdesc_sw128(st + k * 32), make_sdesc_sw128(st + kTileBytes + k * 32),
                      idesc, k > 0);
          tc_commit(&ctl.empty[s]);
          tc_commit(&ctl.tfull[a]);
          if (++s == kWideStages) { s = 0; ph ^= 1; }
          if (++a == 2) { a = 0; aph ^= 1; }
        }
      }
    } else if (warp == 2 && MODE == kFp8Sorted) {
      // the ids that are out of range, reported once
      for (int b = blockIdx.x; b < nb; b += gridDim.x) {
        if (block_expert<MODE>(p, b) < 0) {
          if (lane == 0) flag_error(p.err, MOE_LORA_DEVERR_EXPERT_ID);
          continue;
        }
        for (int t = lane; t < BT; t += 32) flag_block<MODE>(p, b, t, BT);
      }
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kWideRegsEpilogue));
    // this thread's pair, one half (128 columns: one scale) of the output tile
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const uint32_t lane_addr = tmem + ((uint32_t)quarter << 21) + half * 128;
    int a = 0;
    uint32_t aph = 0;
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
      const int nt = (int)(it / nb), b = (int)(it - (long long)nt * nb), e = block_expert<MODE>(p, b);
      if (e < 0) continue;
      const int f = block_pair<MODE>(p, b, quarter * 32 + lane, BT);
      const int nblk = nt * 2 + half;
      const float *sx = f < 0 ? nullptr : p.x_scales + (size_t)pair_row<MODE>(p, f) * p.KB;
      const float *sw = nblk < p.NB ? p.w_scales + ((size_t)e * p.NB + nblk) * p.KB : nullptr;
      float acc[128];
#pragma unroll
      for (int c = 0; c < 128; ++c) acc[c] = 0.f;
      float sx0 = sx ? __ldg(sx) : 0.f, sw0 = sw ? __ldg(sw) : 0.f;
      for (int kb = 0; kb < p.KB; ++kb) {
        const float sc = sx0 * sw0;
        if (kb + 1 < p.KB) {
          sx0 = sx ? __ldg(sx + kb + 1) : 0.f;
          sw0 = sw ? __ldg(sw + kb + 1) : 0.f;
        }
        mbar_wait(&ctl.tfull[a], aph, abort, p.err);
        tc_fence_after();
#pragma unroll
        for (int c0 = 0; c0 < 128; c0 += 32) {
          uint32_t v[32];
          tmem_ld32(lane_addr + a * kWideN + c0, v);
          tc_wait_ld();
          tc_pin(v);
#pragma unroll
          for (int c = 0; c < 32; ++c) acc[c0 + c] += __uint_as_float(v[c]) * sc;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.tempty[a]);
        if (++a == 2) { a = 0; aph ^= 1; }
      }
      if (f >= 0) {
        const float w = pair_weight<MODE>(p, f);
        const int n0 = nblk * kRows;
        uint16_t *dst = p.y + (size_t)f * p.ldy + n0;
        if (n0 + 128 <= p.N && (reinterpret_cast<uintptr_t>(dst) & 15) == 0) {
#pragma unroll
          for (int c = 0; c < 128; c += 8) {
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[i]) : "f"(acc[c + 2 * i + 1] * w), "f"(acc[c + 2 * i] * w));
            *reinterpret_cast<uint4 *>(dst + c) = make_uint4(o[0], o[1], o[2], o[3]);
          }
        } else {
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (n0 + c < p.N) dst[c] = float_to_bf16_bits(acc[c] * w);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ launch

int make_maps(const Fp8Args &a, int x_box_rows, Fp8Maps *maps) {
  if (int st = stream::encode_u8(&maps->w, a.w, 3, a.K, a.N, a.E, a.ldw, (uint64_t)a.ldw * a.N, kRows)) return st;
  return stream::encode_u8(&maps->x, a.x, 2, a.K, a.rows, 1, a.ldx, 0, x_box_rows);
}

// The wide kernel's warps trade registers after the launch: the shares must
// fit what the block was launched with, or the trade would wait forever.
template <typename Kernel>
bool register_shares_fit(Kernel kernel) {
  cudaFuncAttributes attr;
  if (cudaFuncGetAttributes(&attr, (const void *)kernel) != cudaSuccess) return false;
  return attr.numRegs * kWideThreads >= 128 * kWideRegsIssue + 256 * kWideRegsEpilogue;
}

template <typename Kernel>
int launch(Kernel kernel, const Fp8Maps &maps, const Fp8Args &a, const Fp8Cfg &cfg, unsigned grid, int threads,
           cudaStream_t stream) {
  if (cudaFuncSetAttribute((const void *)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, cfg.smem_bytes) !=
      cudaSuccess)
    return MOE_LORA_ERR_LAUNCH;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(grid, 1, 1);
  lc.blockDim = dim3(threads, 1, 1);
  lc.dynamicSmemBytes = cfg.smem_bytes;
  lc.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cfg.cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, kernel, maps, a, cfg) == cudaSuccess ? 0 : MOE_LORA_ERR_LAUNCH;
}

// Upper bound of the call's blocks.
long long block_bound(const Fp8Args &a, Fp8Mode mode, int bt) {
  if (mode == kFp8Dense) return ((long long)a.pairs + bt - 1) / bt;
  if (mode == kFp8Naive) return a.pairs;
  return std::min<long long>(a.max_blocks, fused_block_bound(a.pairs, 1, a.E, 1, bt));
}

template <int BT, int MODE>
int launch_narrow(const Fp8Args &a, const DeviceInfo &dev, cudaStream_t stream) {
  using C = Narrow<BT>;
  Fp8Cfg cfg = {};
  cfg.nt = (a.N + kRows - 1) / kRows;
  const long long items = block_bound(a, (Fp8Mode)MODE, BT) * cfg.nt;
  if (items <= 0) return 0;
  if (items > INT32_MAX) return MOE_LORA_ERR_UNSUPPORTED;
  // K is split while there are too few items for the SMs and each CTA keeps two groups
  int cs = 1;
  while (cs < 8 && items * cs * 2 <= dev.sm_count && a.KB >= cs * 4) cs *= 2;
  cfg.cluster = cs;
  const int fixed = kScaleSlots * C::kScaleRow * 4 + (cs > 1 ? 2 * C::kRedBytes : 0) + (int)sizeof(NarrowCtrl) + 128;
  cfg.stages = std::min(kMaxRing, (200 * 1024 - fixed) / C::kStage);
  cfg.off_scale = cfg.stages * C::kStage;
  cfg.off_red = cfg.off_scale + kScaleSlots * C::kScaleRow * 4;
  cfg.off_ctrl = cfg.off_red + (cs > 1 ? 2 * C::kRedBytes : 0);
  cfg.smem_bytes = cfg.off_ctrl + (int)sizeof(NarrowCtrl);
  const unsigned clusters = (unsigned)std::min<long long>(items, dev.sm_count / cs);
  Fp8Maps maps;
  if (int st = make_maps(a, MODE == kFp8Dense ? BT : 1, &maps)) return st;
  return launch(fp8_narrow_kernel<BT, MODE>, maps, a, cfg, clusters * cs, kNarrowThreads, stream);
}

template <int MODE>
int launch_wide(const Fp8Args &a, const DeviceInfo &dev, cudaStream_t stream) {
  Fp8Cfg cfg = {};
  cfg.nt = (a.N + kWideN - 1) / kWideN;
  const long long items = block_bound(a, (Fp8Mode)MODE, kRows) * cfg.nt;
  if (items <= 0) return 0;
  cfg.cluster = 1;
  cfg.stages = kWideStages;
  cfg.off_ctrl = kWideStages * kWideStage;
  cfg.smem_bytes = cfg.off_ctrl + (int)sizeof(WideCtrl);
  static const bool fits = register_shares_fit(fp8_wide_kernel<MODE>);
  if (!fits) return MOE_LORA_ERR_LAUNCH;
  Fp8Maps maps;
  if (int st = make_maps(a, MODE == kFp8Dense ? kRows : 1, &maps)) return st;
  return launch(fp8_wide_kernel<MODE>, maps, a, cfg, (unsigned)std::min<long long>(items, dev.sm_count), kWideThreads,
                stream);
}

}  // namespace

int launch_fp8_matmul(const Fp8Args &a, Fp8Mode mode, const DeviceInfo &dev, cudaStream_t s) {
  if (mode == kFp8Naive) return launch_narrow<16, kFp8Naive>(a, dev, s);
  if (mode == kFp8Sorted) {
    switch (a.block) {
      case 16: return launch_narrow<16, kFp8Sorted>(a, dev, s);
      case 32: return launch_narrow<32, kFp8Sorted>(a, dev, s);
      case 64: return launch_narrow<64, kFp8Sorted>(a, dev, s);
      case 128: return launch_wide<kFp8Sorted>(a, dev, s);
      default: return MOE_LORA_ERR_UNSUPPORTED;
    }
  }
  if (a.pairs <= 16) return launch_narrow<16, kFp8Dense>(a, dev, s);
  if (a.pairs <= 32) return launch_narrow<32, kFp8Dense>(a, dev, s);
  if (a.pairs <= 256) return launch_narrow<64, kFp8Dense>(a, dev, s);
  return launch_wide<kFp8Dense>(a, dev, s);
}

}  // namespace moe_lora
