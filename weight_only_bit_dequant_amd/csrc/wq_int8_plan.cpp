// Which kernel form an 8-bit integer product runs.  Plain C++ with no device
// code: tests ask for the form of a size by wq_int8_form and so cannot come to
// run another one than they mean when the rule changes.
//
// Each form's time is a formula in its tiles and in the blocks of 128 K; the form
// with the least time is run.  The constants are fitted to the times of all
// forms over 130 random shapes and 120 grouped ones (1 to 8192 rows, 256 to 8192
// columns and K, weights from memory, graphs of back-to-back launches); over the
// same shapes the chosen form took 4 % more than the best one on average, 30 % at
// worst.  What the formulas do not see is how uneven the experts are, and that T
// may be more than there are rows.
#include <cmath>

#include "wq_int8_internal.hpp"

namespace wq {

namespace {

// LDS tiles, bn x bm, `at_once` of them on the chip.  Time of a launch in us:
//   2 + rounds (start + look + blocks per_block) + end
// with per_block falling to `few` of itself, and the end to nothing, as a round
// empties; no less than the weights of all experts that have rows from memory.
// `look`: for the tile of an expert.
struct TileCost {
  Int8Form form;
  int bn, bm, at_once;
  float start, per_block, few, end, look, memory;  // memory in TB/s
};
const TileCost kTiles[] = {{kI8Tile256, 256, 256, 256, 7.25f, 1.58f, 0.47f, 0.f, 0.f, 4.9f},
                           {kI8Tile256x128, 256, 128, 256, 3.47f, 1.01f, 0.36f, 1.63f, 1.04f, 4.5f},
                           {kI8Tile128, 128, 128, 512, 2.52f, 1.24f, 0.18f, 3.12f, 0.03f, 5.1f},
                           {kI8Tile128x64, 128, 64, 256, 2.16f, 0.424f, 0.566f, 0.51f, 0.58f, 4.35f},
                           {kI8Tile64, 64, 64, 512, 1.73f, 0.459f, 0.277f, 1.35f, 0.45f, 4.4f},
                           {kI8Tile32x64, 32, 64, 256, 1.56f, 0.191f, 0.570f, 0.385f, 0.26f, 3.65f}};

// Streams, bn x 16: start + each n + blocks (per_block + more n), n tiles.
// Dot products, bn columns (four waves) x 1: the same in runs of K that a wave
// has under way at once.
struct StreamCost {
  Int8Form form;
  int bn, bm, run;  // K of a run
  float start, each, per_run, more, memory;
};
const StreamCost kStreams[] = {{kI8Stream16, 16, 16, 128, 3.01f, 0.00186f, 0.0544f, 0.000140f, 4.1f},
                               {kI8Stream16Deep, 16, 16, 128, 2.96f, 0.0034f, 0.0415f, 0.0001f, 3.8f},
                               {kI8Stream32, 32, 16, 128, 2.93f, 0.00283f, 0.135f, 0.00013f, 4.9f},
                               {kI8Dot2, 8, 1, 8192, 2.69f, 0.00143f, 0.221f, 0.00187f, 4.0f},
                               {kI8Dot4, 16, 1, 4096, 1.96f, 0.f, 1.133f, 0.00311f, 5.4f},
                               {kI8Dot8, 32, 1, 2048, 2.25f, 0.f, 1.052f, 0.00339f, 6.0f}};

const char* const kNames[] = {"dot 2", "dot 4", "dot 8", "stream 16x16", "stream 16x16 deep", "stream 32x16", "tile 256x256",
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
    // (a few rows of the stream's 16 cost what all do; the dot products' weights are read again for each row)
    if (f.bm == 1 ? rows > (grouped ? 1 : 2) : rows > (grouped ? 20 : 160)) continue;
    const float m = f.bm == 1 ? (float)T : grouped ? (float)groups * fmaxf(1.f, (float)rows / 16.f + 0.5f) : up((float)rows, 16.f);
    const float n = up((float)N, (float)f.bn) * m;
    take(f.form, f.start + f.each * n + up((float)K, (float)f.run) * (f.per_run + f.more * n), f.memory);
  }
  for (const TileCost& f : kTiles) {
    // an expert's last row tile is half full on average
    const float m = grouped ? fmaxf(1.f, (float)rows / (float)f.bm + 0.5f) : up((float)rows, (float)f.bm);
    const float n = up((float)N, (float)f.bn) * (float)groups * m, at = (float)f.at_once;
    const float whole = up(n, at) - 1.f, full = (n - whole * at) / at;
    const float start = f.start + (grouped ? f.look : 0.f), step = blocks * f.per_block;
    take(f.form, 2.f + whole * (start + step) + start + step * (f.few + (1.f - f.few) * full) + f.end * fminf(1.f, n / at), f.memory);
  }
  return best;
}

}  // namespace wq

extern "C" const char* wq_int8_form(int64_t T, int64_t E, int64_t N, int64_t K) {
  if (T <= 0) return "";
  return wq::kNames[wq::int8_form(E > 0, (int)T, E > 0 ? (int)E : 1, (int)N, (int)K)];
}
