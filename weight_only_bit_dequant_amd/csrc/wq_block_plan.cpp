// Which kernel form a block-scaled product runs.  Plain C++ with no device code:
// tests ask for the form of a size by wq_block_form and so cannot come to run
// another one than they mean when the rule changes.
#include <cmath>

#include "wq_block_internal.hpp"

namespace wq {

namespace {

// Forms for many rows, widest first.  Time of a launch in us: 2.5 + rounds (start + blocks per_block), a round being
// `at_once` tiles.  Fitted to N = 4096 with M of one full round at 32 scale blocks of K and M = 4096 at 4 (us: 63 and
// 16.5, 36.5 and 18.3, 23.7 and 21.9, 14.9 and 37, 11.3 and 54, 16.6 and 28.5).  A last round that is not full takes
// down to 85 % of that, the fewer its tiles, and split into 128 x 128 theirs and 2 us.  Over 276 random shapes,
// plain and grouped, the form with the least time by this took 0.6 % more than the best one on average, 9 % at worst.
struct Cost {
  BlockForm form;
  int bn, bm, at_once;
  float start, per_block;
  bool split;  // the rest of a round in 128 x 128
};
const Cost kCosts[] = {{kTile256, 256, 256, 256, 7.4f, 1.66f, true},
                       {kTile256x128, 256, 128, 256, 3.6f, 0.96f, true},
                       {kTile128, 128, 128, 256, 2.5f, 0.58f, false},
                       {kTile128x64, 128, 64, 256, 3.1f, 0.29f, false},
                       {kTile64, 64, 64, 256, 2.4f, 0.20f, false},
                       {kTile64One, 64, 64, 512, 1.7f, 0.39f, false}};

const char* const kNames[] = {"stream 16x16", "stream 16x16 deep", "stream 32x16 eight", "stream 32x16", "stream 32x32",
                              "stream 64x16", "tile 256x256", "tile 256x128", "tile 128x128", "tile 128x64",
                              "tile 64x64", "tile 64x64 one"};
static_assert(sizeof(kNames) / sizeof(kNames[0]) == kBlockForms, "a name for each form");

}  // namespace

// Times in us, of graphs of back-to-back launches.
BlockForm block_form(bool grouped, int T, int E, int N, int K) {
  const int groups = grouped ? (E < T ? E : T) : 1;
  const int rows = (T + groups - 1) / groups;  // of an expert, on average (T for a plain Linear)
  const int kb = (K + 127) / 128;
  // Few rows: streamed.  Columns and rows to a workgroup by the number of 16 x 16 tiles: few keep the chip filled best
  // one to a workgroup, in eight waves where K is long enough for them; many share what they read and, of experts,
  // look for their rows less often.
  const int64_t cols = (N + 15) / 16;
  // Long and narrow: a wave's trips to memory one after the other are the time, so two of its blocks are under way
  // (4 x 2344 x 7552: 6.05 against 7.0; of 1 row, N = 512, 1024, 2048 and 2560: K = 8192 5.4, 5.5, 5.8 and 6.2 against
  // 6.4, 6.5, 6.8 and 6.9, K = 16384 8.1 to 9.8 against 9.9 to 11.1; 16 and 32 rows gain 0.7 to 0.9 and 1.3 to 1.4).
  // Not where the stream itself is the time: N = 4096 gets nothing at K = 8192 and 16384 (1 row 8.0 against 7.9, 12.5
  // against 12.4) and loses 0.1 to 0.2 below.  The bounds lie inside what was measured, not at its edge: K = 4096 and
  // 5120 would gain 0.1 to 0.5 too at N <= 2560, and N between 2560 and 4096 is not measured.
  const bool deep = kb >= 44 && N <= 2560;
  if (grouped && rows <= 16) {
    // (1 x 2 of 32, 1440 x 1920: 4.2 against 5.4 with 64 columns; 10 x 1 of 4, 3856 x 3184: 8.4 against 8.9 with 32 and
    // 10.5 with 64; 6 x 2 of 16, 928 x 544: 4.2 with 32 against 4.6; 16 x 4 of 32, 2048 x 2048: 15.2 with 32, 16.6 with
    // 64, 17.2 with 16; 128 x 4 of 64, 1536 x 2048: 29.0 with 64, 30.7 with 32, 44 with 16, 30 in 256 x 128 tiles.
    // 32 and 64 columns are close: with 4608 to 6144 tiles, 4 rows each of 64 experts, 64 are 0 to 5 % behind)
    // What this rule does not see is how uneven the experts are, and that T may be more than there are rows: 1024 rows
    // of 64 experts, 1536 x 2048, take 42.5 evenly and 50.6 where one has 961 of them (256 x 128 tiles 44.4).
    const int64_t tiles = cols * groups;
    if (tiles <= 256 && deep) return kStream16Deep;
    if (tiles <= 256 || (tiles < 1024 && kb >= 16)) return kStream16;
    if (tiles < 5120) return kStream32;
    return kStream64;
  }
  if (!grouped && rows <= 64) {
    // (1 x 4096 x 3072: 4.9 against 5.4 with 32 columns, 6.2 in four waves; 39 x 1592 x 3456: 4.8 with 32 in eight waves
    // against 5.0 in four and 5.4 with 16; 4 x 7895 x 512: 3.75 with 32 in four waves against 4.0; 56 x 2672 x 1744 5.0
    // against 5.9; 32 x 8192 x 8192: 13.1 with four waves, 14.4 with eight, 16.2 with 16 columns; 64 x 8192 x 8192:
    // 16.5 with 32 x 32, 21.6 with 32 x 16)
    const int64_t tiles = cols * ((rows + 15) / 16);
    if (tiles <= 256) return deep ? kStream16Deep : kStream16;
    if (tiles < 1024 && kb >= 16) return kStream32Eight;
    if (tiles <= 1024 || rows <= 16) return kStream32;
    return kStream32x32;
  }
  // (T = 8192 with 200 rows of 64 experts takes 39.2 in 256 x 128 tiles, 33.1 in the stream that T = 200 gets.)
  // More rows: the form with the least time, but no less than the memory's (weights, for experts those of all that
  // have rows), where the widest does best: fewer workgroups look for their rows (31 rows each of 64 experts, 1536 x
  // 2048: 45 with 256 x 128 tiles against 52-56 with the others).
  const float blocks = (float)kb, memory = 2.5f + (float)N * (float)K * (float)groups / 4.8e6f;
  auto tiles = [&](int bn, int bm) {  // an expert's last row tile is half full on average
    const float m = grouped ? (float)rows / (float)bm + 0.5f : (float)((rows + bm - 1) / bm);
    return (float)((N + bn - 1) / bn) * (float)groups * (m > 1.f ? m : 1.f);
  };
  // Experts' tiles look for their rows first: 1 us a round, 2 in the stream's many workgroups.
  const float look = grouped ? 1.0f : 0.0f;
  const Cost* best = nullptr;
  float least = 0.f;
  for (const Cost& f : kCosts) {
    const float n = tiles(f.bn, f.bm), whole = ceilf(n / (float)f.at_once) - 1.f, rest = n - whole * (float)f.at_once;
    // (two tiles share a CU only when there are more than 256)
    const float per = f.at_once == 512 && n <= 256.f ? 0.25f : f.per_block, round = f.start + look + blocks * per;
    float last = round * (0.85f + 0.15f * rest / (float)f.at_once);
    if (f.split && whole > 0.f && rest <= (float)kMostRest)
      last = 2.f + ceilf(rest / kRound * (float)(f.bn * f.bm / (128 * 128))) * (2.5f + look + blocks * 0.58f);
    const float t = fmaxf(2.5f + whole * round + last, memory);
    if (!best || t < 0.97f * least) best = &f, least = t;
  }
  // The stream of 32 x 32 tiles keeps the chip filled where those are too few: 142 x 1224 x 3120 6.2 against 11.0,
  // 94 x 2795 x 6144 11.1 against 14.8, 128 x 4096 x 4096 9.8 against 10.6; 256 x 4096 x 4096 16.7 against 11.3,
  // 697 x 1512 x 640 8.5 against 6.6.
  const float n = tiles(32, 32);
  const float t = fmaxf(3.0f + 2.f * look + 0.0045f * fmaxf(0.f, n - 300.f) + blocks * (0.09f + 0.00022f * n), memory);
  if (t < 0.97f * least) return kStream32x32;
  return best->form;
}

}  // namespace wq

extern "C" const char* wq_block_form(int64_t T, int64_t E, int64_t N, int64_t K) {
  if (T <= 0) return "";
  return wq::kNames[wq::block_form(E > 0, (int)T, E > 0 ? (int)E : 1, (int)N, (int)K)];
}
