// fp8_blocks.cuh -- how the 8-bit products find their work: units of positions
// (rows of a dense call, positions of a sorted block, single pairs of the naive
// assignment), their expert and their pairs.
#pragma once

#include <stdint.h>

#include "device_utils.cuh"
#include "fp8.h"

namespace moe_lora {

// Blocks that the sorted arrays hold.
__device__ __forceinline__ int num_blocks(const Fp8Args &p) {
  const int n = load_global(p.num_tokens_post_padded) / p.block;
  return n < 0 ? 0 : (n > p.max_blocks ? p.max_blocks : n);
}
// The narrow kernel's units of bt positions: a block of the sorted arrays is
// `block / bt` of them.
template <int MODE>
__device__ __forceinline__ int num_units(const Fp8Args &p, int bt) {
  if (MODE == kFp8Dense) return (p.pairs + bt - 1) / bt;
  if (MODE == kFp8Naive) return p.pairs;
  return num_blocks(p) * (p.block / bt);
}
constexpr int kBadExpert = -1, kNoPairs = -2;
// Expert of unit b; negative where the unit is skipped: its id is out of
// range, or its first position holds the sentinel and it does not begin a
// block (a block's pairs precede its sentinels).
template <int MODE>
__device__ __forceinline__ int block_expert(const Fp8Args &p, int b, int bt) {
  if (MODE == kFp8Dense) return 0;
  const int e = MODE == kFp8Sorted ? load_global(p.expert_ids + b / (p.block / bt)) : load_global(p.topk_ids + b);
  if ((unsigned)e >= (unsigned)p.E) return kBadExpert;
  if (MODE == kFp8Sorted && b % (p.block / bt) && load_global(p.sorted_token_ids + (size_t)b * bt) == p.pairs) return kNoPairs;
  return e;
}
// Pair at position t of block b, or -1.  `bt` positions a block.
template <int MODE>
__device__ __forceinline__ int block_pair(const Fp8Args &p, int b, int t, int bt) {
  if (MODE == kFp8Naive) return t == 0 ? b : -1;
  int f;
  if (MODE == kFp8Dense) f = b * bt + t;
  else f = load_global(p.sorted_token_ids + (size_t)b * bt + t);
  return (unsigned)f < (unsigned)p.pairs ? f : -1;
}
template <int MODE>
__device__ __forceinline__ int pair_row(const Fp8Args &p, int f) {
  return MODE == kFp8Dense || p.x_per_pair ? f : f / p.topk;
}
// Report what is out of range in unit b, whose block_expert() is e; by one warp.
template <int MODE>
__device__ __forceinline__ void flag_unit(const Fp8Args &p, int b, int bt, int e, int lane) {
  if (MODE == kFp8Dense) return;
  if (e == kBadExpert) {
    if (lane == 0) flag_error(p.err, MOE_LORA_DEVERR_EXPERT_ID);
    return;
  }
  if constexpr (MODE == kFp8Sorted)
    for (int t = lane; t < bt; t += 32) {
      const int f = load_global(p.sorted_token_ids + (size_t)b * bt + t);
      // neither a pair nor the sentinel, or (in a skipped unit) a pair after a sentinel
      if ((unsigned)f > (unsigned)p.pairs || (e == kNoPairs && f != p.pairs)) flag_error(p.err, MOE_LORA_DEVERR_PAIR_ID);
    }
}
template <int MODE>
__device__ __forceinline__ float pair_weight(const Fp8Args &p, int f) {
  return MODE != kFp8Dense && p.topk_weights ? load_global(p.topk_weights + f) : 1.f;
}

}  // namespace moe_lora
