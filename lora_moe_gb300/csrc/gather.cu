// gather.cu -- the rows of the sorted pairs, gathered once into the order of
// sorted_token_ids: the wide kernels read each of them N / 256 times, and TMA
// fetches gathered rows four at a time at 80 clk each, cp.async by the 8-bit
// kernel's own warps at 40 % of the tensor cores' time.  CTA 0 also lists the
// tiles of at most tile_rows rows of one expert.  Bound by the rows' bytes.
#include <cuda_runtime.h>

#include <algorithm>

#include "device_utils.cuh"
#include "gather.h"
#include "launch.cuh"

namespace moe_lora {

namespace {

constexpr int kGatherThreads = 256;

__global__ void __launch_bounds__(kGatherThreads)
    gather_kernel(const PairBlocks p, const uint8_t *x, long long row_bytes, long long bytes, int tile_rows, WideTile *tiles,
                  uint8_t *xg, long long ld) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bs = p.block;
  wait_for_prior_grid();
  let_next_grid_start();
  const int nb = num_blocks(p);
  if (blockIdx.x == 0) {
    // Tile list.  Blocks of one expert are neighbours: a run.  A block heads a
    // tile when the blocks before it in its run are a multiple of tile_rows rows; the
    // last block of a tile writes it down.
    __shared__ int warp_last[kGatherThreads / 32], warp_heads[kGatherThreads / 32], carry_first, carry_heads;
    if (tid == 0) carry_first = carry_heads = 0;
    __syncthreads();
    const int per_tile = tile_rows / bs;
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
    const int xr = pair_row<kSorted>(p, f);
    const uint8_t *src = x + xr * row_bytes;
    uint8_t *dst = xg + (size_t)r * ld;
    const long long whole = bytes / 16;
    // (four loads on their way: 8192 rows of 4096 bytes 13.3 us with one, 10.2 with four)
    for (long long c = lane; c < whole; c += 4 * 32) {
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i * 32 < whole) v[i] = load_global(reinterpret_cast<const uint4 *>(src) + c + i * 32);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i * 32 < whole) reinterpret_cast<uint4 *>(dst)[c + i * 32] = v[i];
    }
    for (long long c = whole * 16 + lane; c < bytes; c += 32) dst[c] = load_global(src + c);
  }
}

}  // namespace

GatherSpace gather_space(long long rows, long long bytes) {
  GatherSpace w;
  w.ld = (bytes + 127) / 128 * 128;
  // at most a tile for each of the sorted arrays' smallest blocks, and the count
  w.x = ((size_t)(rows / 16 + 1) * sizeof(WideTile) + sizeof(WideTile) + 127) / 128 * 128;
  w.bytes = w.x + (size_t)rows * w.ld;
  return w;
}

int launch_gather(const PairBlocks &a, const void *x, long long row_bytes, long long bytes, int tile_rows, void *workspace,
                  const DeviceInfo &dev, cudaStream_t stream) {
  const long long rows = (long long)a.max_blocks * a.block;
  const GatherSpace w = gather_space(rows, bytes);
  uint8_t *base = static_cast<uint8_t *>(workspace);
  return launch_dependent(gather_kernel, (unsigned)std::min<long long>((rows + 7) / 8, dev.sm_count * 8ll),
                          kGatherThreads, 1, 0, stream, a, static_cast<const uint8_t *>(x), row_bytes, bytes,
                          tile_rows, reinterpret_cast<WideTile *>(base), base + w.x, w.ld);
}

}  // namespace moe_lora
