// narrow.cuh -- what the narrow kernels of the products (8-bit and bf16) share:
// the list of units that hold pairs, and a CTA's items; and the bf16 kernel's
// sum of partial results over a cluster of any size whose CTAs split K.  (The
// 8-bit kernel's clusters are powers of two, its own sums unrolled for each:
// 37 x 2880 x 2880 in 6.4 us, 6.7 with join_ranks() below.)
#pragma once

#include <type_traits>

#include "blocks.cuh"
#include "device_utils.cuh"

namespace moe_lora {

constexpr int kRows = 128;            // rows of an accumulator: lanes of tensor memory
constexpr int kNarrowThreads = 256;
constexpr int kListUnits = 2048;

// The units of a sorted call that hold pairs, in order: where a block is
// several units, most of a decode batch's hold none, and every CTA would look
// each of them up for every tile of N (256 tokens, blocks of 64: 97 us against
// 76 in blocks of 16, which need no list).  By the whole CTA.
template <int BT>
__device__ __forceinline__ void list_units(const PairBlocks &p, int units, int *list, int *warp_live, int *live, int tid) {
  const int lane = tid & 31, warp = tid >> 5;
  int n = 0;   // (the same in every thread)
  for (int base = 0; base < units; base += kNarrowThreads) {
    const int b = base + tid;
    const int e = b < units ? block_expert<kSorted>(p, b, BT) : kNoPairs;
    const uint32_t has = __ballot_sync(0xFFFFFFFFu, e >= 0);
    if (lane == 0) warp_live[warp] = __popc(has);
    __syncthreads();
    int at = n;
    for (int w = 0; w < kNarrowThreads / 32; ++w) {
      if (w < warp) at += warp_live[w];
      n += warp_live[w];
    }
    if (e >= 0) list[at + __popc(has & ((1u << lane) - 1))] = b;
    __syncthreads();
  }
  if (tid == 0) *live = n;
  __syncthreads();
}

// Most items of a call: NarrowWork steps past the last by up to a grid, which has a CTA an SM at most.
constexpr long long kMostItems = INT32_MAX - (1 << 16);

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

// Units of W neighbouring positions of a tile of BT: 4, or 2 where a cluster of
// cs CTAs has more than BT / 4; rank q of the cluster has the units [U * q / cs,
// U * (q + 1) / cs).
__host__ __device__ constexpr int join_width(int BT, int cs) { return BT / 4 >= cs ? 4 : 2; }
__device__ __forceinline__ int join_first(int BT, int cs, int rank) {
  const int W = join_width(BT, cs);
  return BT / W * rank / cs * W;
}
// Bytes that join_ranks() needs in each CTA (SINGLE: one position).
__host__ __device__ constexpr int join_bytes(int BT, int cs, bool single) {
  return single ? cs * kRows * 4
                : (BT / join_width(BT, cs) + cs - 1) / cs * join_width(BT, cs) * cs * kRows * 4;
}

// The sums over a cluster of cs > 1 CTAs of their acc (this thread's row, BT
// positions), each passed to emit(first position, W sums) in the CTA that has
// them; by the 128 epilogue threads.  A rank sums its positions of every
// rank's partial sums, in rank order (SINGLE: position 0, by rank 0).  There is
// one item at most, so that the buffer `red` is used once, and every CTA waits
// for all that is sent to it: nothing reaches a CTA that has left.  Waits for the cluster's
// first barrier phase (every CTA has initialised its barriers) itself.
template <int BT, bool SINGLE, typename Emit>
__device__ __forceinline__ void join_ranks(const float (&acc)[BT], int cs, int rank, int row, uint8_t *red,
                                           uint64_t *red_full, volatile int *abort, int32_t *err, Emit emit) {
  const uint32_t red_base = smem_addr(red), red_bar = smem_addr(red_full);
  if constexpr (SINGLE) {
    if (row == 0 && rank == 0) mbar_arrive_expect_tx(red_full, cs * kRows * 4);
    cluster_wait();
    st_async_f1(cluster_map(red_base + (rank * kRows + row) * 4, 0), acc[0], cluster_map(red_bar, 0));
    if (rank != 0) return;
    mbar_wait_cluster(red_full, 0, abort, err);
    float v[1] = {0.f};
    for (int q = 0; q < cs; ++q) v[0] += reinterpret_cast<const float *>(red)[q * kRows + row];
    emit(0, v);
  } else {
    auto run = [&](auto width) {
      constexpr int W = decltype(width)::value, U = BT / W;
      const uint32_t inv = (65535u + cs) / cs;   // x / cs is x * inv >> 16 for the x here, at most 128
      auto start = [&](int q) { return (int)(U * q * inv >> 16); };   // rank q's first unit
      const int first = start(rank), own = start(rank + 1) - first;
      if (row == 0) mbar_arrive_expect_tx(red_full, own * cs * W * kRows * 4);
      cluster_wait();
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int q = ((u + 1) * cs - 1) / U, s = start(q), at = u - s, of = start(q + 1) - s;
        const uint32_t dst = cluster_map(red_base + ((rank * of + at) * kRows + row) * W * 4, q), bar = cluster_map(red_bar, q);
        if constexpr (W == 4)
          st_async_v4(dst, make_float4(acc[4 * u], acc[4 * u + 1], acc[4 * u + 2], acc[4 * u + 3]), bar);
        else
          st_async_f2(dst, acc[2 * u], acc[2 * u + 1], bar);
      }
      mbar_wait_cluster(red_full, 0, abort, err);
      const float *buf = reinterpret_cast<const float *>(red) + row * W;
#pragma unroll 1   // (code that runs once a launch is fetched as it runs)
      for (int u = 0; u < own; ++u) {
        float v[W];
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = 0.f;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          if (q >= cs) break;
          const float *src = buf + (q * own + u) * kRows * W;
          if constexpr (W == 4) {
            const float4 x = *reinterpret_cast<const float4 *>(src);
            v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
          } else {
            const float2 x = *reinterpret_cast<const float2 *>(src);
            v[0] += x.x, v[1] += x.y;
          }
        }
        emit((first + u) * W, v);
      }
    };
    if constexpr (BT == 16) {
      if (cs > 4) return run(std::integral_constant<int, 2>());
    }
    run(std::integral_constant<int, 4>());
  }
}

}  // namespace moe_lora
