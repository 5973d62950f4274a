// Row tiles of products whose rows are sorted by expert, and the layout of
// operand rows in LDS: what the 8-bit products (block-scaled FP8, INT8) share.
#pragma once

#include "wq_block_tiles.hpp"
#include "wq_kernel_common.hpp"

namespace wq {

constexpr uint32_t kOut = 0xFFFFFFF0u;  // at or past the end of every buffer here (sizes < 2^32, multiples of 16)

// Inclusive sum over the lanes: shifts within rows of 16, then each row's last
// lane to the next row and the first half's to the second (DPP row_shr and
// row_bcast; a lane without a source adds 0).
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
  return v;
}

// The experts' row tiles, BM rows each, numbered through all experts; lane l
// holds expert e0 + l of a stretch of 64.  Offsets are clamped to [0, T].
struct RowTile {
  int e, t0, end;  // expert, its rows [t0, end) of this tile and after
};
struct RowTiles {
  const int32_t* off;
  int E, T, BM;
  int lo, hi, first, tiles, total;  // the first stretch; all tiles

  // lane's expert of a stretch whose tiles come after `before` others; returns the number up to its end
  __device__ __forceinline__ int stretch(int e0, int before, int& l, int& h, int& f, int& n) const {
    const int e = e0 + (int)(threadIdx.x & 63);
    l = h = 0;
    if (e < E) {
      l = min(max(off[e], 0), T);
      h = min(max(off[e + 1], l), T);
    }
    n = (h - l + BM - 1) / BM;
    const int upto = wave_scan(n);
    f = before + upto - n;
    return before + __builtin_amdgcn_readlane(upto, 63);
  }
  __device__ __forceinline__ RowTiles(const int32_t* o, int experts, int rows, int bm) : off(o), E(experts), T(rows), BM(bm) {
    total = stretch(0, 0, lo, hi, first, tiles);
    for (int e0 = 64; e0 < E; e0 += 64) {
      int l, h, f, n;
      total = stretch(e0, total, l, h, f, n);
    }
  }
  // tile ti < total; every lane of the wave gets the same answer
  __device__ __forceinline__ RowTile find(int ti) const {
    int l = lo, h = hi, f = first, n = tiles;
    for (int e0 = 0;;) {
      const uint64_t hit = __ballot(ti >= f && ti < f + n);
      if (hit) {
        const int at = __builtin_ctzll(hit);
        return {e0 + at, __builtin_amdgcn_readlane(l, at) + (ti - __builtin_amdgcn_readlane(f, at)) * BM,
                __builtin_amdgcn_readlane(h, at)};
      }
      const int before = __builtin_amdgcn_readlane(f, 63) + __builtin_amdgcn_readlane(n, 63);
      e0 += 64;
      if (e0 >= E) return {0, 0, 0};  // not reached for ti < total
      stretch(e0, before, l, h, f, n);
    }
  }
};

// LDS slot of 16-byte chunk k of row r: the four lane groups' reads of 16 rows
// then fall on distinct banks.
__device__ __forceinline__ int blk_pos(int r, int k) { return k ^ (((r >> 1) & 1) | (r & 4)); }

// Row tiles of bm rows; for experts a bound on their number: every expert that has rows may end in a partial tile.
inline int64_t row_tiles(bool grouped, int T, int E, int64_t bm) {
  if (!grouped) return (T + bm - 1) / bm;
  return (T + (int64_t)(E < T ? E : T) * (bm - 1)) / bm;
}

// A launch holds fewer than 2^32 threads (and its workgroups are numbered by ints).
inline bool too_many(int64_t groups, int threads) { return groups >= ((int64_t)1 << 32) / threads || groups >= INT32_MAX; }

}  // namespace wq
