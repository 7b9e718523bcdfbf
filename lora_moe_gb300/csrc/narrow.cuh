// narrow.cuh -- what the narrow kernels of the products (8-bit and bf16) share:
// the list of units that hold pairs, a CTA's items, and the sum of partial
// results over a cluster whose CTAs split K.
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

// The sums over a cluster of cs > 1 CTAs of their acc (this thread's row, BT
// positions), passed to store(first position, sums) 1, 2 or 4 at a time in one of
// them; by the 128 epilogue threads.  Rank q sums the positions [q * tc, (q + 1) * tc) of every
// rank's partial sums, in rank order (SINGLE: position 0, by rank 0).  There is
// one item at most, so that the buffer `red` (BT * kRows floats; SINGLE: cs *
// kRows) is used once, and every CTA waits for all that is sent to it: nothing
// reaches a CTA that has left.  Waits for the cluster's first barrier phase (every CTA has
// initialised its barriers) itself.
template <int BT, bool SINGLE, typename Store>
__device__ __forceinline__ void join_ranks(const float (&acc)[BT], int cs, int rank, int row, uint8_t *red,
                                           uint64_t *red_full, volatile int *abort, int32_t *err, Store store) {
  const int tc = SINGLE ? 1 : BT / cs, lg = __ffs(tc) - 1;
  const uint32_t red_base = smem_addr(red), red_bar = smem_addr(red_full);
  const bool receives = !SINGLE || rank == 0;
  if (row == 0 && receives) mbar_arrive_expect_tx(red_full, (SINGLE ? cs : BT) * kRows * 4);
  cluster_wait();
  if constexpr (SINGLE) {
    st_async_f1(cluster_map(red_base + (rank * kRows + row) * 4, 0), acc[0], cluster_map(red_bar, 0));
  } else if (tc >= 4) {
#pragma unroll
    for (int c = 0; c < BT; c += 4) {
      const int q = c >> lg, quad = (c - (q << lg)) >> 2;
      st_async_v4(cluster_map(red_base + (((rank * tc) >> 2) + quad) * kRows * 16 + row * 16, q),
                  make_float4(acc[c], acc[c + 1], acc[c + 2], acc[c + 3]), cluster_map(red_bar, q));
    }
  } else {   // two positions a rank
#pragma unroll
    for (int c = 0; c < BT; c += 2)
      st_async_f2(cluster_map(red_base + (rank * kRows + row) * 8, c >> 1), acc[c], acc[c + 1],
                  cluster_map(red_bar, c >> 1));
  }
  if (!receives) return;
  mbar_wait_cluster(red_full, 0, abort, err);
  const float *buf = reinterpret_cast<const float *>(red);
  auto finish = [&](auto ranks) {
    constexpr int CS = decltype(ranks)::value;
    if constexpr (SINGLE) {
      float v[1];
      sum_ranks<CS>(buf, 1, 0, row, v);
      store(0, v);
    } else if constexpr (BT / CS >= 4) {
#pragma unroll 4
      for (int quad = 0; quad < BT / CS / 4; ++quad) {
        float v[4];
        sum_ranks<CS>(buf, BT / CS / 4, quad, row, v);
        store(rank * (BT / CS) + quad * 4, v);
      }
    } else {
      float v[2];
      sum_ranks<CS>(buf, 1, 0, row, v);
      store(rank * 2, v);
    }
  };
  if (cs == 2) finish(std::integral_constant<int, 2>());
  else if (cs == 4) finish(std::integral_constant<int, 4>());
  else finish(std::integral_constant<int, 8>());
}

}  // namespace moe_lora
