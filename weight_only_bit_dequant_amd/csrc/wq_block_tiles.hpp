// Which tile of a block-scaled product a workgroup owns: index arithmetic that
// the kernels and a host test share.
#pragma once

#include "wq_block_internal.hpp"

#define WQ_HD __host__ __device__ inline

namespace wq {

// Place of workgroup b of G in an order that the XCDs share out in contiguous
// pieces (workgroup b runs on XCD b % 8, and each XCD has its own L2).
WQ_HD int xcd_order(int b, int G) {
  const int q = G >> 3, r = G & 7, x = b & 7;
  return x * q + (x < r ? x : r) + (b >> 3);
}

// Tile idx of gx x rows: bands of 4 column tiles, row tile by row tile, so that
// tiles in flight on one XCD share operands both ways.
struct At {
  int tx, ty;
};
WQ_HD At place(int idx, int gx, int rows) {
  const int band = idx / (4 * rows), in = idx - band * 4 * rows, left = gx - 4 * band, wide = left < 4 ? left : 4, ty = in / wide;
  return {4 * band + in - ty * wide, ty};
}

// Tiles of the last round that are split, where split ones are faster.
WQ_HD int rest_of_round(bool split, int tiles) {
  const int rest = tiles % kRound;
  return !split || tiles < kRound || rest > kMostRest ? 0 : rest;
}

// Row tiles that a device counted, held to the number that the grid is for:
// decreasing offsets can count to more than that, past what an int holds even,
// and must not name a column tile outside the weights.  (Offsets in order never
// count to more.)
WQ_HD int held(int total, int bound) { return (uint32_t)total > (uint32_t)bound ? bound : total; }

// Workgroup b's tile of gx column tiles x `total` row tiles, the rest of a round
// in `parts` pieces each (1: none is split); part: of a split tile, else -1.
// False: past them all.  `bound`: the row tiles that the grid is for.
WQ_HD bool tile_at(int b, int gx, int total, int bound, int parts, At& p, int& part) {
  const int rows = held(total, bound);
  const int rest = rest_of_round(parts > 1, gx * rows), whole = gx * rows - rest;
  if (b >= whole + parts * rest) return false;
  part = -1;
  if (b < whole) {
    p = place(xcd_order(b, whole), gx, rows);
  } else {
    const int i = xcd_order(b - whole, parts * rest);
    p = place(whole + i / parts, gx, rows);
    part = i % parts;
  }
  return true;
}

// The same of a stream: consecutive workgroups of an XCD take the row tiles of
// one column tile, which share its weights.
WQ_HD bool stream_at(int b, int gx, int total, int bound, At& p) {
  const int rows = held(total, bound);
  if (b >= gx * rows) return false;
  const int tile = xcd_order(b, gx * rows);
  p = {tile / rows, tile % rows};
  return true;
}

}  // namespace wq
