// 8-bit integer GEMMs: Y = (Xq . Wq^T) * Xs * Ws for one weight or, with rows
// sorted by expert, for many.
//
// The matrix cores sum the codes' products in int32, exactly, in whatever order:
// forms that split K give the same bits as those that do not.  The weights are
// operand A, so that a lane holds neighbouring columns n of one row m: one
// activation scale, four weight scales, 8 bytes of bf16 output at a time.
//
// What bounds them, in us of graphs of calls whose weights come from memory:
//   1 x 4096 x 4096, 16.8 MB                5.5 by dot products: the launch and one trip to memory
//   48 rows of 64 experts, 1408 x 2048      11: the weights' stream, 98 MB, some of them from the Infinity Cache
//   2800 rows of 64 experts, 1536 x 2048    43: the weights' stream, 4.9 TB/s
//   333 x 5003 x 2064                       12: 17 steps of 0.4, loads beyond L2 with 96 KB under way; 4 of launch, first loads
//                                           and stores; rows across two cache lines (K % 128 != 0) are 1.6 of them
//   4096 x 2048 x 5632                      42 alone, 47 in a row: the matrix cores, busy 70 %, and the power limit
//   8192 x 8192 x 8192                      424, 2.6 POP/s: the power limit (1.82 GHz, the matrix cores busy 80 % at that
//                                           clock); their MFMAs on registers alone reach 3.5 POP/s with random codes
#include "wq_int8_internal.hpp"
#include "wq_row_tiles.hpp"

namespace wq {

namespace {

typedef __attribute__((ext_vector_type(4))) int i32x4;
typedef __attribute__((ext_vector_type(16))) int i32x16;
typedef __attribute__((ext_vector_type(4), aligned(2))) uint32_t u32x4_any;

__device__ __forceinline__ i32x4 as_i32(u32x4 v) { return __builtin_bit_cast(i32x4, v); }

// Lane (g, c) of A: 16 codes of weight row c, of B: 16 codes of activation row
// c, both at K 16 g .. 16 g + 15; D[4g + r][c] in element r.
__device__ __forceinline__ i32x4 mfma16(u32x4 w, u32x4 x, i32x4 acc) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(as_i32(w), as_i32(x), acc, 0, 0, 0);
}
// The same of 32 rows: lane (h, c), h = lane / 32, holds K 16 h .. 16 h + 15 of
// row c; D[8 q + 4 h + r][c] in element 4 q + r.
__device__ __forceinline__ i32x16 mfma32(u32x4 w, u32x4 x, i32x16 acc) {
  return __builtin_amdgcn_mfma_i32_32x32x32_i8(as_i32(w), as_i32(x), acc, 0, 0, 0);
}

__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  return (uint32_t)f32_to_bf16(lo) | ((uint32_t)f32_to_bf16(hi) << 16);
}

// An output before its rounding to bf16, each operation rounded by itself: joined into a multiply-add, as the compiler does
// where it may, the bias would meet an unrounded product in some forms and not in others, and a row's bits go by the number
// of rows beside it.  Without a bias kNoBias is added, which leaves every value as it is, -0 too.
constexpr uint16_t kNoBias = 0x8000;  // -0
__device__ __forceinline__ float output(int sum, float xs, float ws, float bias) {
#pragma clang fp contract(off)
  return (float)sum * xs * ws + bias;
}

// ---------------------------------------------------------------- single rows: dot products
// A wave owns C columns of one row; its lanes split K, 16 codes of every 1024
// each, so that one instruction reads 1 KiB of one weight row, and multiply by
// v_dot4_i32_i8.  All loads of a run of kAhead KiB are under way at once: where
// C weight rows fit a run, a product is one trip to memory (1 x 4096 x 4096: 5.5
// us with C = 4, 6.0 with 2, 7.2 with 8, 6.1 as a stream of 16 rows, 15 of them
// none).  Of two rows the weights come twice, the second time from L2: 6.0 us; a
// wave for two or four rows at a time took 6.5 and 9.8.
constexpr int kAhead = 16;

template <int C>
__global__ __launch_bounds__(256) void k_int8_dot(Int8GemmArgs a, int gx, int gy) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int N = a.N, K = a.K;
  RowTile t;
  At p;
  if (a.offsets) {
    const RowTiles all(a.offsets, a.E, a.T, 1);
    if (!stream_at(blockIdx.x, gx, all.total, gy, p)) return;  // the grid is for a bound on their number
    t = all.find(p.ty);
  } else {
    stream_at(blockIdx.x, gx, gy, gy, p);
    t = {0, p.ty, a.M};
  }
  const int n0 = (p.tx * 4 + wave) * C, cols = min(C, N - n0);
  if (cols <= 0) return;
  const uint32_t src = a.rows ? (uint32_t)__builtin_amdgcn_readfirstlane(a.rows[t.t0]) : (uint32_t)t.t0;
  const bool has = src < (uint32_t)a.M;  // a row from elsewhere reads as zeros
  const __amdgpu_buffer_rsrc_t Wr = make_rsrc(a.Wq + ((int64_t)t.e * N + n0) * K, (uint32_t)cols * (uint32_t)K);
  const __amdgpu_buffer_rsrc_t Xr = make_rsrc(a.Xq + (int64_t)(has ? src : 0) * K, has ? (uint32_t)K : 0u);
  // lane i's column at the end
  const int n = n0 + min(lane, cols - 1);
  const float xs = has ? a.Xs[src] : 0.f, ws = a.Ws[(int64_t)t.e * N + n];
  const float bias = bf16_to_f32(a.bias ? a.bias[n] : kNoBias);

  constexpr int U = kAhead / C;  // KiB of a row at a time
  int acc[C] = {};
  for (int k = 16 * lane; k < K + 16 * lane; k += 1024 * U) {
    u32x4 w[U][C], x[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < C; ++i) w[u][i] = bload128(Wr, k + 1024 * u < K ? (uint32_t)i * (uint32_t)K + k + 1024 * u : kOut);
#pragma unroll
    for (int u = 0; u < U; ++u) x[u] = bload128(Xr, (uint32_t)(k + 1024 * u));  // past the row: zeros
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < C; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i] = __builtin_amdgcn_sdot4((int)w[u][i][r], (int)x[u][r], acc[i], false);
  }
  int sum = 0;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int s = __builtin_amdgcn_readlane(wave_scan(acc[i]), 63);
    sum = lane == i ? s : sum;
  }
  if (lane < cols) {
    a.Y[(int64_t)t.t0 * N + n] = f32_to_bf16(output(sum, xs, ws, bias));
  }
}

// ---------------------------------------------------------------- few rows: weight stream
// A workgroup owns 16 NT columns x 16 MT rows and all of K; its W waves split
// K, each a run of 128-byte blocks.  A wave copies a block's rows into a slot of
// its own in LDS (buffer_load ... lds, 8 whole 128-byte rows per instruction) and
// reads them back as operands; SL slots are blocks under way.  Waves meet once,
// to add up their sums.  Bound by the weights' stream and, below some 10 MB, by
// the trips to memory.  16 columns where the weights are few, so that more
// workgroups read them; 32 rows at once rather than the weights twice.
template <int NT, int MT, int W, int SL>
struct StreamT {
  static constexpr int SLOT = (NT + MT) * 2048, L = 2 * (NT + MT);  // bytes and loads per block
  static constexpr int PART = W * 16 * MT * 16 * NT * 4;
  static constexpr int SMEM = SL * W * SLOT > PART ? SL * W * SLOT : PART;
};

template <int NT, int MT, int W, int SL>
__global__ __launch_bounds__(W * 64) void k_int8_stream(Int8GemmArgs a, int gx, int gy) {
  using S = StreamT<NT, MT, W, SL>;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, c = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int N = a.N, K = a.K, KB = (K + 127) >> 7;
  RowTile t;
  At p;
  if (a.offsets) {
    const RowTiles all(a.offsets, a.E, a.T, 16 * MT);
    if (!stream_at(blockIdx.x, gx, all.total, gy, p)) return;  // the grid is for a bound on their number
    t = all.find(p.ty);
  } else {
    stream_at(blockIdx.x, gx, gy, gy, p);
    t = {0, p.ty * 16 * MT, a.M};
  }
  const int n0 = p.tx * 16 * NT;

  const __amdgpu_buffer_rsrc_t Wr =
      make_rsrc(a.Wq + ((int64_t)t.e * N + n0) * K, (uint32_t)min(16 * NT, N - n0) * (uint32_t)K);
  const __amdgpu_buffer_rsrc_t Xr = a.rows ? make_rsrc(a.Xq, (uint32_t)((int64_t)a.M * K))
                                           : make_rsrc(a.Xq + (int64_t)t.t0 * K, (uint32_t)min(16 * MT, t.end - t.t0) * (uint32_t)K);
  // load l of a block: rows 8 l + lane / 8 (weights first), chunk kc16 / 16 of the row; rows past the end read zeros
  const int lr = lane >> 3, kc16 = 16 * blk_pos(lr, lane & 7);
  uint32_t voff[S::L];
#pragma unroll
  for (int l = 0; l < S::L; ++l) {
    const int r = 8 * l + lr;
    voff[l] = (uint32_t)(l < 2 * NT ? (n0 + r < N ? r : -1) : (t.t0 + r - 16 * NT < t.end ? r - 16 * NT : -1));
  }
  uint32_t limit = 0x7FFFFFFFu;  // source rows from here on read as zeros
  if (a.rows) {
    limit = (uint32_t)a.M;
#pragma unroll
    for (int l = 2 * NT; l < S::L; ++l)
      if ((int)voff[l] >= 0) voff[l] = (uint32_t)a.rows[t.t0 + voff[l]];
  }
#pragma unroll
  for (int l = 0; l < S::L; ++l)
    voff[l] = voff[l] < (l < 2 * NT ? 0x7FFFFFFFu : limit) ? voff[l] * (uint32_t)K + kc16 : kOut;

  unsigned char* slot0 = smem + wave * SL * S::SLOT;
  auto issue = [&](int kt, int at) {
    unsigned char* slot = slot0 + at * S::SLOT;
#pragma unroll
    for (int l = 0; l < S::L; ++l)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(l < 2 * NT ? Wr : Xr,
                                               (__attribute__((address_space(3))) void*)(slot + l * 1024), 16,
                                               (int)(kt * 128 + kc16 < K ? voff[l] : kOut), kt * 128, 0, 0);
  };
  const int flo = c * 128 + blk_pos(c, 2 * g) * 16;
  struct Pair {
    u32x4 v[2];  // K 32 g .. 32 g + 31 of a row, for both operands
  };
  auto frag = [&](int at, int i) {
    const unsigned char* p = slot0 + at * S::SLOT + i * 2048;
    return Pair{{*reinterpret_cast<const u32x4*>(p + flo), *reinterpret_cast<const u32x4*>(p + (flo ^ 16))}};
  };

  i32x4 acc[NT][MT] = {};
  const int per = (KB + W - 1) / W, first = wave * per, n = min(KB, first + per) - first;
#pragma unroll
  for (int u = 0; u < SL; ++u)
    if (u < n) issue(first + u, u);
  int at = 0;
  for (int u = 0; u < n; ++u) {
    constexpr int NEWER = (SL - 1) * S::L;  // loads that may still be under way
    if (SL > 1 && u + SL <= n)
      __builtin_amdgcn_s_waitcnt(kWaitVm0 | (NEWER & 15) | ((NEWER >> 4) << 14));
    else
      __builtin_amdgcn_s_waitcnt(kWaitVm0);
    asm volatile("" ::: "memory");
    Pair A[NT], B[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j) B[j] = frag(at, NT + j);
#pragma unroll
    for (int i = 0; i < NT; ++i) A[i] = frag(at, i);
    __builtin_amdgcn_s_waitcnt(kWaitLgkm0);  // the slot has been read
    asm volatile("" ::: "memory");
    if (u + SL < n) issue(first + u + SL, at);
    at = at + 1 == SL ? 0 : at + 1;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[i][j] = mfma16(A[i].v[h], B[j].v[h], acc[i][j]);
  }

  __syncthreads();  // the slots are no longer used
  int(*part)[16 * MT][16 * NT] = reinterpret_cast<int(*)[16 * MT][16 * NT]>(smem);
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) *reinterpret_cast<i32x4*>(&part[wave][16 * j + c][16 * i + 4 * g]) = acc[i][j];
  __syncthreads();
  // four columns of a row per thread
  for (int q = tid; q < 16 * MT * 4 * NT; q += W * 64) {
    const int row = q / (4 * NT), col = 4 * (q % (4 * NT)), m = t.t0 + row, n = n0 + col;
    if (m >= t.end || n >= N) continue;
    const uint32_t src = a.rows ? (uint32_t)a.rows[m] : (uint32_t)m;
    const float xs = src < (uint32_t)a.M ? a.Xs[src] : 0.f;
    i32x4 s = *reinterpret_cast<const i32x4*>(&part[0][row][col]);
#pragma unroll
    for (int v = 1; v < W; ++v) s += *reinterpret_cast<const i32x4*>(&part[v][row][col]);
    float y[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int nr = min(n + r, N - 1);
      y[r] = output(s[r], xs, a.Ws[(int64_t)t.e * N + nr], bf16_to_f32(a.bias ? a.bias[nr] : kNoBias));
    }
    uint16_t* p = a.Y + (int64_t)m * N + n;
    if ((N & 3) == 0) {
      *reinterpret_cast<u32x2*>(p) = u32x2{pack(y[0], y[1]), pack(y[2], y[3])};
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n + r < N) p[r] = f32_to_bf16(y[r]);
    }
  }
}

// ---------------------------------------------------------------- LDS-tiled kernel
// A workgroup of WN x WM waves owns BN columns x BM rows of Y; K advances 128 per
// step, four MFMAs deep.  Operand rows go from memory straight into LDS
// (buffer_load ... lds: lane i's 16 bytes land at the wave's base + 16 i), 8
// whole rows of 128 bytes per instruction; the 16-byte chunks of row r are
// XOR-swizzled by r / 2 % 8, by the choice of the chunk that each lane loads, so
// that 32 rows' reads of one chunk fall on distinct banks (conflicts: 3 % of the
// cycles).  Steps of 64 load half cache lines: 128 x 128 tiles 534 -> 681 us at 8192^3.
//
// LDS is a ring of UNITS units, a step's weights or its activations in turn, so
// that 160 KB hold two and a half steps of a 256 x 256 tile: the loads of two are
// always under way or landed while one is multiplied.  Smaller tiles have five
// steps, as their loads' way is long against a step (deeper rings: no change).
//
// A wave owns 32 TN x 32 TM of the tile.  Its fragments of a quarter step (K = 32)
// are read while the quarter before is multiplied, in two sets of registers.  When
// the last quarter's have been read the waves meet, at the step's one barrier:
// its units are free, the next step's have landed.  The last quarter's MFMAs cover
// its first reads of the next step; the refill is spread over SPAN quarters (all in
// one: 465 us, 441 spread, at 8192^3).  Eight waves, two to a SIMD: four take as long
// on whole tiles (4096 x 2048 x 5632 in 256 x 128: 47 us both) and longer where some
// of them have no rows (333 x 5000 x 2048: 14.5 and 16.8).
//
// With KS > 1, KS such groups of waves split K, each with its own ring, and add
// up their sums in LDS at the end: tiles too few to fill the chip finish sooner.
template <int BN_, int BM_, int WN_, int WM_, int KS_, int UNITS_, int SPAN_ = 4>
struct Tile {
  static constexpr int BN = BN_, BM = BM_, WN = WN_, WM = WM_, KS = KS_, UNITS = UNITS_, SPAN = SPAN_;
  static constexpr int WAVES = WN * WM, THREADS = KS * WAVES * 64, TN = BN / (32 * WN), TM = BM / (32 * WM);
  static constexpr int GROUP = UNITS * (BN + BM) * 64, MAIN = KS * GROUP;
  static constexpr int PITCH = TN * 64 + 16;  // output tile row in LDS
  static constexpr int PART = BN * 4 + 16;    // row of sums in LDS (KS > 1)
  static constexpr int OUT = KS > 1 ? KS * BM * PART : WAVES * TM * 32 * PITCH;
  static constexpr int LAST = OUT + (2 * BN + BM) * 4;  // with the columns' scales and biases and the rows' scales
  static constexpr int SMEM = MAIN > LAST ? MAIN : LAST, ON_CU = 160 * 1024 / SMEM;  // workgroups on a CU
  static_assert(BN % (8 * WAVES) == 0 && BM % (8 * WAVES) == 0, "whole loads");
  static_assert(WAVES % 2 == 0, "the swizzle of a wave's loads goes by its parity");
  static_assert(UNITS >= 4 && (UNITS % 2 == 0 || BN == BM), "a ring of units of one size, or of pairs");
};

// TAIL: K % 128 != 0, chunks past K read zeros.  (Without it the loads carry no
// mask; those of steps past the end read the last block again, unused.)
template <class T, bool TAIL>
__device__ __forceinline__ void tile(const Int8GemmArgs& a, const RowTile t, const int n0) {
  constexpr int BN = T::BN, BM = T::BM, WN = T::WN, KS = T::KS, U = T::UNITS;
  constexpr int TN = T::TN, TM = T::TM, W = T::WAVES;
  constexpr int LJW = BN / (8 * W), LJX = BM / (8 * W), LJ = LJW + LJX;  // loads per wave and step: weights, activations
  extern __shared__ __attribute__((aligned(16))) unsigned char shared[];
  const int group = KS > 1 ? __builtin_amdgcn_readfirstlane((int)threadIdx.x / (W * 64)) : 0;
  const int tid = (int)threadIdx.x - group * W * 64, lane = tid & 63;  // within the group
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  unsigned char* smem = shared + group * T::GROUP;
  const int h = lane >> 5, c = lane & 31;
  const int wn = wave % WN, wm = wave / WN;
  const int N = a.N, K = a.K, KB = (K + 127) >> 7;

  // load j of this wave: rows (j * W + wave) * 8 + lane / 8 of the weights, then of the activations; chunk kc16 / 16
  const int lr = lane >> 3, kc16 = 16 * ((lane & 7) ^ (4 * (wave & 1) + (lr >> 1)));
  const __amdgpu_buffer_rsrc_t Wr =
      make_rsrc(a.Wq + ((int64_t)t.e * N + n0) * K, (uint32_t)min(BN, N - n0) * (uint32_t)K);
  const __amdgpu_buffer_rsrc_t Xr = a.rows ? make_rsrc(a.Xq, (uint32_t)((int64_t)a.M * K))
                                           : make_rsrc(a.Xq + (int64_t)t.t0 * K, (uint32_t)min(BM, t.end - t.t0) * (uint32_t)K);
  const uint32_t have = (uint32_t)(t.end - t.t0);
  uint32_t voff[LJ];  // rows past the end read as zeros, without a request to memory
#pragma unroll
  for (int j = 0; j < LJ; ++j) {
    const int r = (j * W + wave) * 8 + lr;
    voff[j] = (uint32_t)(j < LJW ? r : r - BN);
  }
  // this thread's share of the scales: of column i, the bias of column i - BN, of row i - 2 BN
  constexpr int SCALES = 2 * BN + BM, PER = (SCALES + T::THREADS - 1) / T::THREADS;
  uint32_t src[PER];
#pragma unroll
  for (int u = 0; u < PER; ++u) src[u] = (uint32_t)(t.t0 + min(max((int)threadIdx.x + u * T::THREADS - 2 * BN, 0), (int)have - 1));
  uint32_t limit = have;  // source rows from here on read as zeros too
  if (a.rows) {
    limit = (uint32_t)a.M;
#pragma unroll
    for (int j = LJW; j < LJ; ++j) {
      const uint32_t row = (uint32_t)a.rows[t.t0 + min(voff[j], have - 1)];
      voff[j] = voff[j] < have ? row : 0xFFFFFFFFu;
    }
#pragma unroll
    for (int u = 0; u < PER; ++u) src[u] = (uint32_t)a.rows[src[u]];
  }
#pragma unroll
  for (int j = 0; j < LJ; ++j) voff[j] = j < LJW || voff[j] < limit ? voff[j] * (uint32_t)K + kc16 : kOut;
  // this group's steps: blocks k0 .. k0 + mine - 1, of `per` that the groups meet for
  const int per = (KB + KS - 1) / KS, k0 = group * per, mine = max(0, min(per, KB - k0));

  // The ring's unit i holds step i / 2's weights (i even) or activations, at place i % U.
  auto place = [](int i) { return (i & 1) * BN * 128 + (i >> 1) * (BN + BM) * 128; };  // i < U
  constexpr int RING = U % 2 ? U * BN * 128 : place(U);
  auto issue1 = [&](int n, int at, int j) {  // load j of step n, its unit at `at`
    const int kt = min(k0 + n, KB - 1), jj = j < LJW ? j : j - LJW;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        j < LJW ? Wr : Xr, (__attribute__((address_space(3))) void*)(smem + at + (jj * W + wave) * 1024), 16,
        (int)(!TAIL || kt * 128 + kc16 < K ? voff[j] : kOut), kt * 128, 0, 0);
  };
  // Once step n's units, at wo and xo, are free they take units 2 n + U and 2 n + U + 1, by LJ loads spread over SPAN
  // quarter steps: its last one, then those of the step after.  (All in one quarter they fill the memory pipe's queue
  // and the waves stall on it.)
  constexpr int Q = TN * TM, LAST = 3;
  auto slot = [](int l) { return l * Q * T::SPAN / LJ; };
  auto refill = [&](int n, int wo, int xo, int l) {
    if constexpr (U % 2) {
      if (l < LJX) issue1(n + (U - 1) / 2, wo, LJW + l);
      else issue1(n + (U + 1) / 2, xo, l - LJX);
    } else {
      issue1(n + U / 2, l < LJW ? wo : xo, l);
    }
  };
  // loads that may be under way when a step's are needed: those of the U - 4 units after it
  constexpr int NEWER = U % 2 ? (U - 5) / 2 * LJ + LJW : (U - 4) / 2 * LJ;
#pragma unroll
  for (int j = 0; j < LJ; ++j) issue1(0, j < LJW ? place(0) : place(1), j);
  // the scales, for the end, kept in registers until LDS is free
  float raw[PER];
  uint32_t rawb[PER];
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    const int i = (int)threadIdx.x + u * T::THREADS, n = min(n0 + (i < BN ? i : i - BN), N - 1);
    raw[u] = *(i < 2 * BN ? a.Ws + (int64_t)t.e * N + n : a.Xs + min(src[u], (uint32_t)a.M - 1));
    rawb[u] = a.bias ? a.bias[n] : kNoBias;
  }
#pragma unroll
  for (int i = 2; i < U - 2; ++i)
#pragma unroll
    for (int j = 0; j < LJ; ++j)
      if ((j >= LJW) == (i & 1)) issue1(i >> 1, place(i), j);
  int pwo = place(U - 2), pxo = place(U - 1);  // the units of the step before
#pragma unroll
  for (int l = 0; l < LJ; ++l)
    if (slot(l) < Q) refill(-1, pwo, pxo, l);

  // operand fragments: rows 32 i + c of the wave's part, K 32 s + 16 h .. + 15 of the step
  const int flo = c * 128 + (h ^ ((c >> 1) & 7)) * 16;
  auto frag = [&](int at, int s, int i) { return *reinterpret_cast<const u32x4*>(smem + at + i * 4096 + (flo ^ (32 * s))); };

  // this wave's loads but for the newest have landed, and its LDS reads; meet the others
#define WQ_MEET(N)                                                                                        \
  do {                                                                                                    \
    __builtin_amdgcn_s_waitcnt((kWaitVm0 & kWaitLgkm0) | ((N) & 15) | (((N) >> 4) << 14));                \
    asm volatile("s_barrier" ::: "memory");                                                               \
  } while (0)

  i32x16 acc[TN][TM] = {};
  // Waves whose rows or columns are all past the end only load and meet.
  const bool live = t.t0 + wm * TM * 32 < t.end && n0 + wn * TN * 32 < N;
  auto after = [](int at) { return at + 2 * (RING / U) < RING ? at + 2 * (RING / U) : at + 2 * (RING / U) - RING; };
  const int fw = wn * TN * 4096, fx = wm * TM * 4096;
  constexpr int F = TN + TM;
  WQ_MEET(NEWER);
  int wo = place(0), xo = place(1);
  if (live) {
    struct Operands {
      u32x4 a[TN], b[TM];
    } set[2];
#pragma unroll
    for (int i = 0; i < TN; ++i) set[0].a[i] = frag(wo + fw, 0, i);
#pragma unroll
    for (int j = 0; j < TM; ++j) set[0].b[j] = frag(xo + fx, 0, j);
    for (int n = 0; n < mine; ++n) {
      const int nwo = after(wo), nxo = after(xo);
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        Operands &now = set[s & 1], &next = set[(s & 1) ^ 1];
        if (s == LAST) WQ_MEET(NEWER);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
#pragma unroll
          for (int f = 0; f < F; ++f)  // next operands in the order of their use, early in the quarter
            if (q == f * Q / (2 * F)) {
              const int ns = (s + 1) & 3, wat = (s == LAST ? nwo : wo) + fw, xat = (s == LAST ? nxo : xo) + fx;
              if (f == 0) next.a[0] = frag(wat, ns, 0);
              else if (f <= TM) next.b[f - 1] = frag(xat, ns, f - 1);
              else next.a[f - TM] = frag(wat, ns, f - TM);
            }
          acc[q / TM][q % TM] = mfma32(now.a[q / TM], now.b[q % TM], acc[q / TM][q % TM]);
#pragma unroll
          for (int l = 0; l < LJ; ++l) {
            if (s == LAST && slot(l) == q) refill(n, wo, xo, l);
            if (s < LAST && slot(l) == (s + 1) * Q + q) refill(n - 1, pwo, pxo, l);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      pwo = wo, pxo = xo;
      wo = nwo, xo = nxo;
    }
  } else {
    for (int n = 0; n < mine; ++n) {
#pragma unroll
      for (int l = 0; l < LJ; ++l)
        if (slot(l) >= Q) refill(n - 1, pwo, pxo, l);
      WQ_MEET(NEWER);
#pragma unroll
      for (int l = 0; l < LJ; ++l)
        if (slot(l) < Q) refill(n, wo, xo, l);
      pwo = wo, pxo = xo;
      wo = after(wo), xo = after(xo);
    }
  }
  for (int n = mine; n < per; ++n) WQ_MEET(0);
#undef WQ_MEET

  __builtin_amdgcn_s_waitcnt(kWaitVm0 & kWaitLgkm0);
  asm volatile("s_barrier" ::: "memory");  // the ring is no longer used
  float* scales = reinterpret_cast<float*>(shared + T::OUT);
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    const int i = (int)threadIdx.x + u * T::THREADS;
    if (i < SCALES) scales[i] = i < BN ? raw[u] : i < 2 * BN ? bf16_to_f32((uint16_t)rawb[u]) : src[u] < (uint32_t)a.M ? raw[u] : 0.f;
  }
  if constexpr (KS == 1) __syncthreads();
  const bool vec = (N & 7) == 0;
  auto put = [&](int m, int n, u32x4 v) {  // 8 columns of a row
    if (m >= t.end) return;
    uint16_t* y = a.Y + (int64_t)m * N + n;
    if (vec) {
      if (n < N) __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(y));
    } else if (n + 8 <= N) {
      *reinterpret_cast<u32x4_any*>(y) = v;  // (rows of an odd width start anywhere; element by element 333 x 5003 x 2064 takes 4 us more)
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (n + e < N) y[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
    }
  };
  const float *ws = scales, *bs = scales + BN, *xs = scales + 2 * BN;

  if constexpr (KS > 1) {
    // the groups' sums meet in LDS, 8 columns of a row per thread
    const int col = wn * TN * 32 + 4 * h, row = wm * TM * 32 + c;
    unsigned char* own = shared + group * (BM * T::PART);
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<i32x4*>(own + (row + 32 * j) * T::PART + (col + 32 * i + 8 * q) * 4) =
              i32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
    __syncthreads();
    for (int q = threadIdx.x; q < BM * BN / 8; q += T::THREADS) {
      const int r = q / (BN / 8), n = 8 * (q % (BN / 8));
      u32x4 v;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        i32x4 s = {0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < KS; ++k) s += *reinterpret_cast<const i32x4*>(shared + (k * BM + r) * T::PART + n * 4 + 16 * half);
        const f32x4 w = *reinterpret_cast<const f32x4*>(ws + n + 4 * half), b = *reinterpret_cast<const f32x4*>(bs + n + 4 * half);
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = output(s[e], xs[r], w[e], b[e]);
        v[2 * half] = pack(y[0], y[1]);
        v[2 * half + 1] = pack(y[2], y[3]);
      }
      put(t.t0 + r, n0 + n, v);
    }
  } else {
    // wave tiles leave through LDS as 16-byte row pieces
    unsigned char* et = shared + wave * (TM * 32 * T::PITCH);
    const int nw = wn * TN * 32, mw = wm * TM * 32;
    float xm[TM];
#pragma unroll
    for (int j = 0; j < TM; ++j) xm[j] = xs[mw + 32 * j + c];
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = nw + 32 * i + 8 * q + 4 * h;
        const f32x4 w = *reinterpret_cast<const f32x4*>(ws + n), b = *reinterpret_cast<const f32x4*>(bs + n);
#pragma unroll
        for (int j = 0; j < TM; ++j) {
          float y[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) y[r] = output(acc[i][j][4 * q + r], xm[j], w[r], b[r]);
          *reinterpret_cast<u32x2*>(et + (32 * j + c) * T::PITCH + (32 * i + 8 * q + 4 * h) * 2) =
              u32x2{pack(y[0], y[1]), pack(y[2], y[3])};
        }
      }
    __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
    asm volatile("" ::: "memory");
    constexpr int LPR = TN * 4, RPI = 64 / LPR;  // lanes per row, rows per store instruction
#pragma unroll
    for (int q = 0; q < TM * 32 / RPI; ++q) {
      const int row = RPI * q + lane / LPR, col = 8 * (lane % LPR);
      put(t.t0 + mw + row, n0 + nw + col, *reinterpret_cast<const u32x4*>(et + row * T::PITCH + col * 2));
    }
  }
}

// Tiles B in whole rounds of the chip, one to a CU; the rest of them, where that
// is at most half a round, in tiles S, which take less time (S = B: none).
template <class B, class S, bool TAIL>
__global__ __launch_bounds__(B::THREADS, B::THREADS / 256 * (B::ON_CU < 2 ? 1 : 2)) void k_int8_tile(Int8GemmArgs a, int gx, int gy) {
  static_assert(B::THREADS == S::THREADS, "one launch");
  constexpr int PX = B::BN / S::BN, PARTS = PX * (B::BM / S::BM);
  const int b = blockIdx.x;
  At p;
  int part;
  RowTile t;
  if (a.offsets) {
    const RowTiles all(a.offsets, a.E, a.T, B::BM);
    if (!tile_at(b, gx, all.total, gy, PARTS, p, part)) return;
    t = all.find(p.ty);
  } else {
    tile_at(b, gx, gy, gy, PARTS, p, part);  // (the grid is exact)
    t = {0, p.ty * B::BM, a.M};
  }
  if constexpr (PARTS > 1) {
    if (part >= 0) {
      t.t0 += S::BM * (part / PX);
      const int n0 = p.tx * B::BN + S::BN * (part % PX);
      if (t.t0 < t.end && n0 < a.N) tile<S, TAIL>(a, t, n0);
      return;
    }
  }
  tile<B, TAIL>(a, t, p.tx * B::BN);
}

int64_t row_tiles(const Int8GemmArgs& a, int64_t bm) { return wq::row_tiles(a.offsets != nullptr, a.T, a.E, bm); }

template <class B, class S>
hipError_t tile_launch(const Int8GemmArgs& a, hipStream_t s) {
  constexpr int smem = B::SMEM > S::SMEM ? B::SMEM : S::SMEM, parts = B::BN * B::BM / (S::BN * S::BM);
  static_assert(smem <= 160 * 1024, "LDS of a CU");
  const int64_t gx = (a.N + B::BN - 1) / B::BN, gy = row_tiles(a, B::BM);
  if (too_many(gx * gy + parts * kMostRest, B::THREADS)) return hipErrorInvalidConfiguration;
  // (of experts the kernel counts the tiles)
  const int64_t rest = a.offsets ? (parts > 1 ? kMostRest : 0) : rest_of_round(parts > 1, (int)(gx * gy));
  static SmemAllowed allowed[2];
  const bool tail = a.K % 128 != 0;
  const auto kern = tail ? k_int8_tile<B, S, true> : k_int8_tile<B, S, false>;
  hipError_t e = allow_smem(kern, smem, allowed[tail]);
  if (e != hipSuccess) return e;
  return launch(kern, dim3((unsigned)(gx * gy + (parts - 1) * rest)), B::THREADS, smem, s, a, (int)gx, (int)gy);
}

template <int NT, int MT, int W, int SL = 1>
hipError_t stream_launch(const Int8GemmArgs& a, hipStream_t s) {
  constexpr int smem = StreamT<NT, MT, W, SL>::SMEM;
  static_assert(smem <= 65536, "no leave needed for the LDS size");
  const int64_t gx = (a.N + 16 * NT - 1) / (16 * NT), gy = row_tiles(a, 16 * MT);
  if (too_many(gx * gy, W * 64)) return hipErrorInvalidConfiguration;
  return launch(k_int8_stream<NT, MT, W, SL>, dim3((unsigned)(gx * gy)), W * 64, smem, s, a, (int)gx, (int)gy);
}

template <int C>
hipError_t dot_launch(const Int8GemmArgs& a, hipStream_t s) {
  const int64_t gx = (a.N + 4 * C - 1) / (4 * C), gy = row_tiles(a, 1);
  if (too_many(gx * gy, 256)) return hipErrorInvalidConfiguration;
  return launch(k_int8_dot<C>, dim3((unsigned)(gx * gy)), 256, 0, s, a, (int)gx, (int)gy);
}

using Tile256 = Tile<256, 256, 2, 4, 1, 5, 3>;
using Tile256x128 = Tile<256, 128, 4, 2, 1, 6, 3>;
using Tile128 = Tile<128, 128, 4, 2, 1, 5, 3>;
using Tile128x64 = Tile<128, 64, 4, 2, 1, 10>;
using Tile64 = Tile<64, 64, 2, 2, 1, 10>;
using Tile32x64 = Tile<32, 64, 1, 2, 2, 8>;

hipError_t run_form(Int8Form form, const Int8GemmArgs& a, hipStream_t s) {
  switch (form) {
    case kI8Dot2: return dot_launch<2>(a, s);
    case kI8Dot4: return dot_launch<4>(a, s);
    case kI8Dot8: return dot_launch<8>(a, s);
    case kI8Stream16: return stream_launch<1, 1, 8>(a, s);
    case kI8Stream16Deep: return stream_launch<1, 1, 8, 2>(a, s);
    case kI8Stream32: return stream_launch<2, 1, 4>(a, s);
    case kI8Stream16x32: return stream_launch<1, 2, 8>(a, s);
    case kI8Tile256: return tile_launch<Tile256, Tile128>(a, s);
    case kI8Tile256x128: return tile_launch<Tile256x128, Tile128>(a, s);
    case kI8Tile128: return tile_launch<Tile128, Tile128>(a, s);
    case kI8Tile128x64: return tile_launch<Tile128x64, Tile128x64>(a, s);
    case kI8Tile64: return tile_launch<Tile64, Tile64>(a, s);
    case kI8Tile32x64: return tile_launch<Tile32x64, Tile32x64>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_int8_gemm(const Int8GemmArgs& a, hipStream_t s) {
  return run_form(int8_form(a.offsets != nullptr, a.T, a.E, a.N, a.K), a, s);
}

}  // namespace wq
