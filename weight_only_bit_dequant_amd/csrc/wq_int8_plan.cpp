// Which kernel form an 8-bit integer product runs.  Plain C++ with no device
// code: tests ask for the form of a size by wq_int8_form and so cannot come to
// run another one than they mean when the rule changes.
//
// Each form's time is a formula in its tiles and in the blocks of 128 K; the form
// with the least time is run.  The constants are fitted to the choices over 611 plain
// shapes and 290 grouped ones, random and powers of two (1 to 8192 rows, 256 to 8192
// columns and K, weights from memory, graphs of back-to-back launches): over the
// same shapes the chosen form takes 1.1 % more than the best one on average, 22 % at
// worst; over a quarter of them that a fit to the others left out, 1.4 and 2.0 %.  The
// constants have the shape of what they are named for and no more: none is a measured
// time or rate by itself.  To fit them again, time every form at such shapes (graphs of
// 20 calls, weights that do not stay in the caches) and change one constant at a time
// while the mean of log(time of the chosen form / of the best), plus 0.4 of its root mean
// square, falls.  What the formulas do not see is how uneven the experts are, and that T may be more than
// there are rows.
#include <cmath>

#include "wq_int8_internal.hpp"

namespace wq {

namespace {

// LDS tiles, bn x bm, `at_once` of them on the chip.  Time of a launch in us:
//   2 + rounds (start + look + blocks per_block) + end
// with per_block falling over `half` of itself to `few`, and the end to nothing, as a
// round is half full and then empties (where two tiles share a CU, a half is one to
// each: 1024 x 4096 x 4096 in 256 tiles takes 24 us, in 128 of twice the size 31); no
// less than 2.5 and the weights of all experts that have rows at `memory`.
// `look`: for the tile of an expert.  `split`: what K % 128 != 0 adds to a block, whose
// rows then lie across two cache lines.
struct TileCost {
  Int8Form form;
  int bn, bm, at_once;
  float start, per_block, few, half, memory, look, end, split;  // memory: 10^6 bytes a microsecond, as fitted
};
const TileCost kTiles[] = {{kI8Tile256, 256, 256, 256, 7.76f, 1.58f, 0.121f, 0.83f, 3.87f, 0.367f, 0.026f, 0.0115f},
                           {kI8Tile256x128, 256, 128, 256, 3.47f, 0.903f, 0.598f, 0.669f, 5.44f, 0.177f, 1.2f, 0.246f},
                           {kI8Tile128, 128, 128, 512, 1.49f, 1.14f, 0.399f, 0.513f, 7.46f, 0.411f, 3.96f, 0.272f},
                           {kI8Tile128x64, 128, 64, 256, 1.87f, 0.382f, 0.661f, 0.831f, 4.68f, 0.777f, 0.354f, 0.147f},
                           {kI8Tile64, 64, 64, 512, 1.36f, 0.486f, 0.431f, 0.621f, 5.32f, 0.813f, 1.41f, 0.159f},
                           {kI8Tile32x64, 32, 64, 256, 1.71f, 0.171f, 0.805f, 0.842f, 4.44f, 0.32f, 0.0261f, 0.349f}};

// Streams, bn x bm: start + each n + blocks (per_run + more n), n tiles.  Dot
// products, bn columns (four waves) x 1: the same in runs of K that a wave has
// under way at once.
struct StreamCost {
  Int8Form form;
  int bn, bm, run;  // K of a run
  int most, most_grouped, most_tiles;  // rows (of an expert, on average) and tiles of several rows that it is for
  float start, each, per_run, more, memory;
};
constexpr int kAny = 1 << 30;
const StreamCost kStreams[] = {{kI8Stream16, 16, 16, 128, 128, 20, 512, 3.02f, 0.00144f, 0.0511f, 0.000152f, 4.58f},
                               {kI8Stream16Deep, 16, 16, 128, 128, 20, 512, 3.05f, 0.00251f, 0.0295f, 0.000175f, 4.75f},
                               {kI8Stream32, 32, 16, 128, 128, 64, kAny, 2.91f, 0.00169f, 0.172f, 0.000202f, 5.31f},
                               {kI8Stream16x32, 16, 32, 128, 512, 64, kAny, 3.21f, 0.00143f, 0.0537f, 0.000282f, 2.28f},
                               {kI8Dot2, 8, 1, 8192, 4, 1, kAny, 3.03f, 0.002f, 0.276f, 0.00252f, 7.97f},
                               {kI8Dot4, 16, 1, 4096, 4, 1, kAny, 1.33f, 0.0000340f, 1.14f, 0.00329f, 7.62f},
                               {kI8Dot8, 32, 1, 2048, 4, 1, kAny, 1.91f, 0.f, 1.01f, 0.00326f, 7.66f}};

const char* const kNames[] = {"dot 2", "dot 4", "dot 8", "stream 16x16", "stream 16x16 deep", "stream 32x16", "stream 16x32", "tile 256x256",
                              "tile 256x128", "tile 128x128", "tile 128x64", "tile 64x64", "tile 32x64"};
static_assert(sizeof(kNames) / sizeof(kNames[0]) == kI8Forms, "a name for each form");

float up(float a, float b) { return ceilf(a / b); }

}  // namespace

Int8Form int8_form(bool grouped, int T, int E, int N, int K) {
  const int groups = grouped ? (E < T ? E : T) : 1;
  const int rows = (T + groups - 1) / groups;  // of an expert, on average (T for a plain Linear)
  const float blocks = (float)((K + 127) / 128), bytes = (float)N * (float)K * (float)groups;
  Int8Form best = kI8Tile256;
  float least = INFINITY;
  auto take = [&](Int8Form form, float t, float memory) {
    t = fmaxf(t, 2.5f + bytes / (memory * 1e6f));
    if (t < least) best = form, least = t;
  };
  for (const StreamCost& f : kStreams) {
    // (a few rows of a stream's 16 cost what all do; the dot products' weights are read again for each row)
    if (rows > (grouped ? f.most_grouped : f.most)) continue;
    const float bm = (float)f.bm;
    const float m = f.bm == 1 ? (float)T : grouped ? (float)groups * fmaxf(1.f, (float)rows / bm + 0.5f) : up((float)rows, bm);
    const float n = up((float)N, (float)f.bn) * m;
    if (!grouped && rows > f.bm && n > (float)f.most_tiles) continue;
    take(f.form, f.start + f.each * n + up((float)K, (float)f.run) * (f.per_run + f.more * n), f.memory);
  }
  for (const TileCost& f : kTiles) {
    // an expert's last row tile is half full on average
    const float m = grouped ? fmaxf(1.f, (float)rows / (float)f.bm + 0.5f) : up((float)rows, (float)f.bm);
    const float n = up((float)N, (float)f.bn) * (float)groups * m, at = (float)f.at_once;
    const float whole = up(n, at) - 1.f, full = (n - whole * at) / at;
    const float start = f.start + (grouped ? f.look : 0.f), step = blocks * f.per_block * (K % 128 ? 1.f + f.split : 1.f);
    const float part = full < 0.5f ? f.few + (f.half - f.few) * 2.f * full : f.half + (1.f - f.half) * (2.f * full - 1.f);
    take(f.form, 2.f + whole * (start + step) + start + step * part + f.end * fminf(1.f, n / at), f.memory);
  }
  return best;
}

}  // namespace wq

extern "C" const char* wq_int8_form(int64_t T, int64_t E, int64_t N, int64_t K) {
  if (T <= 0) return "";
  return wq::kNames[wq::int8_form(E > 0, (int)T, E > 0 ? (int)E : 1, (int)N, (int)K)];
}
