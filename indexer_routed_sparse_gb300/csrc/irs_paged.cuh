// The list of tiles of the paged decode and the parts that its runs leave, shared by the kernels that
// write and join them. The design stands in irs_paged.cu.
#pragma once

#include "irs_internal.h"

namespace irs {

namespace {

constexpr int kTile = 16;              // positions a tile (two 8-column halves of the score product)
constexpr int kHeads = 16;             // query heads a tile (rows of the products)
constexpr int kMaxPagedCtas = 160;
constexpr int kMaxWarps = 8;
constexpr int kMinTiles = 4;           // a warp's run has at least this many: a part is as large as two tiles

// Workspace: prefix sums of the sequences' tile counts, then two parts for every run and head
// (the sequence it starts in, the one it ends in): rows of Dv sums, then maxima, then sums.
__host__ __device__ inline size_t paged_prefix_bytes(int B) { return ((size_t)(B + 1) * 8 + 255) & ~size_t(255); }
__host__ __device__ inline size_t paged_part_floats(int Dv) { return (size_t)kHeads * (Dv + 2); }

// Tiles of a run.
__device__ __forceinline__ int64_t paged_share(int64_t total, int workers) {
  const int64_t q = (total + workers - 1) / workers;
  return q < kMinTiles ? kMinTiles : q;
}

}  // namespace

}  // namespace irs
