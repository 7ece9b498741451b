// The order in which output tiles are dealt to workgroups.
#pragma once

#include "tpf_internal.hpp"

namespace tpf {

// Tile u of a row range (shard-major) -> (shard, tm, tn).  Within a shard the
// tiles go in groups of kGroupM tile-rows, column by column, so that tiles
// running at the same time share A and B panels (the 32 tiles an XCD runs
// at once cover 8 row panels x 4 column panels; measured about 1 % faster
// than groups of 4 rows, groups of 2 or 16 slower).
constexpr int kGroupM = 8;

__device__ __forceinline__ void tile_coords(int u, int tiles_m, int tiles_n, int& shard, int& tm, int& tn) {
  const int per_shard = tiles_m * tiles_n;
  shard = u / per_shard;
  const int t = u - shard * per_shard;
  const int group = t / (kGroupM * tiles_n);
  const int first = group * kGroupM;
  const int gsize = min(kGroupM, tiles_m - first);
  const int w = t - first * tiles_n;
  tm = first + w % gsize;
  tn = w / gsize;
}

// Block b of a grid of `total` blocks -> task index.  Blocks are dealt to the
// XCDs round-robin (block b runs on XCD b % 8), so the tasks are split into
// kXcds contiguous shares and block b takes task b / 8 of share b % 8: each
// XCD's L2 then sees a contiguous run of tiles.
__device__ __forceinline__ int xcd_task(int b, int total) {
  const int x = b & (kXcds - 1), i = b / kXcds;
  return x * (total / kXcds) + min(x, total % kXcds) + i;
}

}  // namespace tpf
