// Host check of the block-scaled products' tile arithmetic (wq_block_tiles.hpp):
// every tile has one owner, and no number of row tiles that a device may count,
// wrapped sums of invalid offsets included, gives a tile outside the grid's.
#include <climits>
#include <cstdio>
#include <vector>

#include "wq_block_tiles.hpp"

static int fails = 0;

static void check(bool ok, const char* what, int gx, int total, int bound, int parts, int b) {
  if (!ok && fails++ < 10) std::printf("%s: gx %d total %d bound %d parts %d workgroup %d\n", what, gx, total, bound, parts, b);
}

// workgroups of a grid, all of a small one, else its ends and steps between
static std::vector<int> groups(long long n) {
  std::vector<int> v;
  const long long step = n < 200000 ? 1 : n / 1000 | 1;
  for (long long b = 0; b < n; b += step) v.push_back((int)b);
  for (long long b = n > 64 ? n - 64 : 0; b < n; ++b) v.push_back((int)b);
  return v;
}

static void valid(int gx, int total, int bound, int parts) {
  const long long n = (long long)gx * bound + (parts - 1) * wq::kMostRest;
  std::vector<int> seen((size_t)gx * total * parts, 0);
  for (long long b = 0; b < n; ++b) {
    wq::At p;
    int part;
    if (!wq::tile_at((int)b, gx, total, bound, parts, p, part)) continue;
    const bool in = p.tx >= 0 && p.tx < gx && p.ty >= 0 && p.ty < total && part >= -1 && part < parts;
    check(in, "tile", gx, total, bound, parts, (int)b);
    if (!in) continue;
    for (int i = 0; i < parts; ++i)
      if (part < 0 || part == i) ++seen[((size_t)p.tx * total + p.ty) * parts + i];
  }
  for (int s : seen) check(s == 1, "owners of a tile", gx, total, bound, parts, s);
  std::vector<int> got((size_t)gx * total, 0);
  for (long long b = 0; b < (long long)gx * bound; ++b) {
    wq::At p;
    if (!wq::stream_at((int)b, gx, total, bound, p)) continue;
    const bool in = p.tx >= 0 && p.tx < gx && p.ty >= 0 && p.ty < total;
    check(in, "stream", gx, total, bound, 1, (int)b);
    if (in) ++got[(size_t)p.tx * total + p.ty];
  }
  for (int s : got) check(s == 1, "owners of a stream's tile", gx, total, bound, 1, s);
}

static void any_total(int gx, int total, int bound, int parts) {
  for (int b : groups((long long)gx * bound + (parts - 1) * wq::kMostRest)) {
    wq::At p;
    int part;
    if (wq::tile_at(b, gx, total, bound, parts, p, part))
      check(p.tx >= 0 && p.tx < gx && p.ty >= 0 && p.ty < bound && part >= -1 && part < parts, "any tile", gx, total, bound, parts, b);
    if (wq::stream_at(b, gx, total, bound, p))
      check(p.tx >= 0 && p.tx < gx && p.ty >= 0 && p.ty < bound, "any stream", gx, total, bound, parts, b);
  }
}

int main() {
  for (int parts : {1, 2, 4}) {
    for (int gx : {1, 2, 3, 4, 5, 7, 16, 29, 32})
      for (int bound : {1, 2, 9, 17, 64, 130, 300})
        for (int total : {0, 1, bound / 2, bound - 1, bound}) valid(gx, total, bound, parts);
    for (int gx : {1, 3, 4, 30, 1024, 1 << 19})
      for (int bound : {1, 9, 300, 1 << 11})
        for (int total : {INT_MIN, INT_MIN + 1, -(1 << 30), -(1 << 29), -100, -1, bound + 1, 4 * bound, 1 << 20, 1 << 28, 1 << 29, 1 << 30,
                          (1 << 30) + 1, 0x7FFFFF00, INT_MAX})
          if ((long long)gx * bound + 3 * wq::kMostRest < INT_MAX) any_total(gx, total, bound, parts);
  }
  if (fails) std::printf("%d failures\n", fails);
  return fails != 0;
}
