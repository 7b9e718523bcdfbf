// blocks.cuh -- how the products (8-bit and bf16) find their work: units of
// positions (rows of a dense call, positions of a sorted block, single pairs of
// the naive assignment), their expert and their pairs.
#pragma once

#include <stdint.h>

#include <algorithm>

#include "device_utils.cuh"
#include "internal.h"

namespace moe_lora {

// Dense: one expert, one block per `block` rows, pair f is row f.
enum ProductMode { kDense = 0, kSorted = 1, kNaive = 2 };

// The pairs of a product, as validated by the C-ABI layer.
struct PairBlocks {
  const float *topk_weights;  // fp32 [pairs] or null
  const int32_t *sorted_token_ids, *expert_ids, *num_tokens_post_padded;   // sorted
  const int32_t *topk_ids;                                                 // naive
  int32_t *err;               // may be null
  int pairs, topk, E;
  int block;                  // pairs per block (sorted)
  int max_blocks;             // blocks that the sorted arrays hold
  int x_per_pair;             // row of pair f is f, else f / topk
};

// Upper bound of a call's units (skipped ones included).
inline long long unit_bound(const PairBlocks &a, ProductMode mode, int bt) {
  if (mode == kDense) return ((long long)a.pairs + bt - 1) / bt;
  if (mode == kNaive) return a.pairs;
  return std::min<long long>(a.max_blocks, fused_block_bound(a.pairs, 1, a.E, 1, a.block)) * (a.block / bt);
}

constexpr int kTileRows = 256;   // most rows of the wide kernels' tiles
// Upper bound of the wide kernels' tiles of `rows` rows.
inline long long tile_bound(const PairBlocks &a, bool sorted, int rows) {
  return sorted ? a.pairs / rows + std::min(a.E, a.pairs) : ((long long)a.pairs + rows - 1) / rows;
}

// Blocks that the sorted arrays hold.
__device__ __forceinline__ int num_blocks(const PairBlocks &p) {
  const int n = load_global(p.num_tokens_post_padded) / p.block;
  return n < 0 ? 0 : (n > p.max_blocks ? p.max_blocks : n);
}
// The narrow kernel's units of bt positions: a block of the sorted arrays is
// `block / bt` of them.
template <int MODE>
__device__ __forceinline__ int num_units(const PairBlocks &p, int bt) {
  if (MODE == kDense) return (p.pairs + bt - 1) / bt;
  if (MODE == kNaive) return p.pairs;
  return num_blocks(p) * (p.block / bt);
}
constexpr int kBadExpert = -1, kNoPairs = -2;
// Expert of unit b; negative where the unit is skipped: its id is out of
// range, or its first position holds the sentinel and it does not begin a
// block (a block's pairs precede its sentinels).
template <int MODE>
__device__ __forceinline__ int block_expert(const PairBlocks &p, int b, int bt) {
  if (MODE == kDense) return 0;
  const int e = MODE == kSorted ? load_global(p.expert_ids + b / (p.block / bt)) : load_global(p.topk_ids + b);
  if ((unsigned)e >= (unsigned)p.E) return kBadExpert;
  if (MODE == kSorted && b % (p.block / bt) && load_global(p.sorted_token_ids + (size_t)b * bt) == p.pairs) return kNoPairs;
  return e;
}
// Pair at position t of block b, or -1.  `bt` positions a block.
template <int MODE>
__device__ __forceinline__ int block_pair(const PairBlocks &p, int b, int t, int bt) {
  if (MODE == kNaive) return t == 0 ? b : -1;
  int f;
  if (MODE == kDense) f = b * bt + t;
  else f = load_global(p.sorted_token_ids + (size_t)b * bt + t);
  return (unsigned)f < (unsigned)p.pairs ? f : -1;
}
template <int MODE>
__device__ __forceinline__ int pair_row(const PairBlocks &p, int f) {
  return MODE == kDense || p.x_per_pair ? f : f / p.topk;
}
// Report what is out of range in unit b, whose block_expert() is e; by one warp.
template <int MODE>
__device__ __forceinline__ void flag_unit(const PairBlocks &p, int b, int bt, int e, int lane) {
  if (MODE == kDense) return;
  if (e == kBadExpert) {
    if (lane == 0) flag_error(p.err, MOE_LORA_DEVERR_EXPERT_ID);
    return;
  }
  if constexpr (MODE == kSorted)
    for (int t = lane; t < bt; t += 32) {
      const int f = load_global(p.sorted_token_ids + (size_t)b * bt + t);
      // neither a pair nor the sentinel, or (in a skipped unit) a pair after a sentinel
      if ((unsigned)f > (unsigned)p.pairs || (e == kNoPairs && f != p.pairs)) flag_error(p.err, MOE_LORA_DEVERR_PAIR_ID);
    }
}
template <int MODE>
__device__ __forceinline__ float pair_weight(const PairBlocks &p, int f) {
  return MODE != kDense && p.topk_weights ? load_global(p.topk_weights + f) : 1.f;
}

}  // namespace moe_lora
