// Which kernel form an 8-bit integer product runs.  Plain C++ with no device
// code: tests ask for the form of a size by wq_int8_form and so cannot come to
// run another one than they mean when the rule changes.
//
// Each form's time is a formula in its tiles and in the blocks of 128 K; the form
// with the least time is run.  The constants are fitted to the times of all
// forms over 200 random shapes and 120 grouped ones (1 to 8192 rows, 256 to 8192
// columns and K, weights from memory, graphs of back-to-back launches); over the
// same shapes the chosen form took 3 % more than the best one on average, a third
// at worst.  What the formulas do not see is how uneven the experts are, and that T
// may be more than there are rows.
#include <cmath>

#include "wq_int8_internal.hpp"

namespace wq {

namespace {

// LDS tiles, bn x bm, `at_once` of them on the chip.  Time of a launch in us:
//   2 + rounds (start + look + blocks per_block) + end
// with per_block falling to `few` of itself, and the end to nothing, as a round
// empties; no less than the weights of all experts that have rows from memory.
// `look`: for the tile of an expert.  `split`: what K % 128 != 0 adds to a block, whose
// rows then lie across two cache lines.
struct TileCost {
  Int8Form form;
  int bn, bm, at_once;
  float start, per_block, few, memory, look, end, split;  // memory in TB/s
};
const TileCost kTiles[] = {{kI8Tile256, 256, 256, 256, 6.34f, 1.70f, 0.39f, 6.3f, 0.f, 0.f, 0.02f},
                           {kI8Tile256x128, 256, 128, 256, 3.51f, 0.975f, 0.34f, 4.8f, 1.30f, 0.86f, 0.20f},
                           {kI8Tile128, 128, 128, 512, 2.60f, 1.20f, 0.166f, 5.1f, 0.17f, 2.45f, 0.20f},
                           {kI8Tile128x64, 128, 64, 256, 2.18f, 0.400f, 0.62f, 4.4f, 0.69f, 0.03f, 0.23f},
                           {kI8Tile64, 64, 64, 512, 1.64f, 0.460f, 0.286f, 4.6f, 0.48f, 0.81f, 0.31f},
                           {kI8Tile32x64, 32, 64, 256, 1.56f, 0.174f, 0.61f, 3.6f, 0.25f, 0.24f, 0.30f}};

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
const StreamCost kStreams[] = {{kI8Stream16, 16, 16, 128, 64, 20, 512, 3.03f, 0.00138f, 0.0500f, 0.00017f, 4.0f},
                               {kI8Stream16Deep, 16, 16, 128, 64, 20, 512, 2.97f, 0.00266f, 0.0373f, 0.00016f, 3.9f},
                               {kI8Stream32, 32, 16, 128, 64, 40, kAny, 2.94f, 0.00233f, 0.127f, 0.00017f, 4.75f},
                               {kI8Stream16x32, 16, 32, 128, 200, 40, kAny, 3.20f, 0.00158f, 0.0545f, 0.00026f, 3.4f},
                               {kI8Dot2, 8, 1, 8192, 4, 1, kAny, 2.20f, 0.00161f, 0.744f, 0.00172f, 3.85f},
                               {kI8Dot4, 16, 1, 4096, 4, 1, kAny, 1.70f, 0.f, 1.21f, 0.00326f, 5.7f},
                               {kI8Dot8, 32, 1, 2048, 4, 1, kAny, 2.10f, 0.f, 0.94f, 0.00309f, 5.7f}};

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
    take(f.form, 2.f + whole * (start + step) + start + step * (f.few + (1.f - f.few) * full) + f.end * fminf(1.f, n / at), f.memory);
  }
  return best;
}

}  // namespace wq

extern "C" const char* wq_int8_form(int64_t T, int64_t E, int64_t N, int64_t K) {
  if (T <= 0) return "";
  return wq::kNames[wq::int8_form(E > 0, (int)T, E > 0 ? (int)E : 1, (int)N, (int)K)];
}
