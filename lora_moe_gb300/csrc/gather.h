// gather.h -- the rows of a sorted call's pairs in the order of its blocks, for
// the wide kernels.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "blocks.cuh"
#include "internal.h"

namespace moe_lora {

// Neighbouring rows of one expert, from row row0 of the gathered ones.
struct WideTile {
  int row0, rows, expert, pad;
};

// The workspace: the tiles (their count in the first one's row0), then the rows.
struct GatherSpace {
  size_t x, bytes;   // offset of the rows; all of it
  long long ld;      // bytes from row to row
};
GatherSpace gather_space(long long rows, long long bytes);   // rows: capacity of the sorted arrays in whole blocks
// Rows of `bytes` bytes, row_bytes apart; tiles of at most tile_rows, a multiple of the block.
int launch_gather(const PairBlocks &a, const void *x, long long row_bytes, long long bytes, int tile_rows, void *workspace,
                  const DeviceInfo &dev, cudaStream_t stream);

}  // namespace moe_lora
