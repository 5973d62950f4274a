// Block-scaled FP8 GEMMs: Y = deq(X) . deq(W)^T for one weight or, with rows
// sorted by expert, for many.
//
// One v_mfma_f32_16x16x128_f8f6f4 is exactly one scale block deep: with a zero
// addend it gives the sum of the block's products, which the VALU scales and
// adds to the fp32 sum (one fused multiply-add per output and block).  The
// weights are operand A, so a lane's four results are four columns n of one
// row m: one activation scale, one weight scale, 8 bytes of bf16 output.
//
// The matrix cores' sum is not that of 128 exact products in fp32: the eight of
// each 8 consecutive K are aligned to 2^e, e the largest sum of two codes'
// exponents (at least -6 each; zero products take no part), and cut towards zero
// below 2^(e - 13).  Found by probing the instruction; four 16x16x32 of FP8 give
// the same bits.
//
// Times in the comments are of graphs of back-to-back launches, cold weights but
// for what the Infinity Cache holds.  Cards differ by some 3 %, and calls from the
// host one by one let a kernel that power bounds run faster than graphs of it
// do (8192 rows of 8 experts, 4096 x 4096: 148.6 against 154.6).
#include "wq_block_tiles.hpp"
#include "wq_kernel_common.hpp"

namespace wq {

namespace {

typedef __attribute__((ext_vector_type(8))) int i32x8;

constexpr uint32_t kOut = 0xFFFFFFF0u;  // at or past the end of every buffer here (sizes < 2^32, multiples of 16)

// lane (g, c) of A: 32 codes of weight row c, of B: 32 codes of activation row
// c, both at K 32g .. 32g+31; D[4g + r][c] in element r.  (Scale operands 0
// select the instruction without block scales.)
__device__ __forceinline__ f32x4 mfma_blk(i32x8 w, i32x8 x) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

__device__ __forceinline__ i32x8 join(u32x4 lo, u32x4 hi) {
  return i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

// CH scales from p on (4-byte aligned); with fewer than CH blocks in a row
// (KB < CH, p the row's start) the last one again.
template <int CH>
struct Scales {
  float v[CH];
};
template <int CH>
__device__ __forceinline__ Scales<CH> load_scales(const float* p, int KB) {
  typedef float vec __attribute__((ext_vector_type(CH)));
  typedef float vecu __attribute__((ext_vector_type(CH), aligned(4)));
  Scales<CH> s;
  if (KB >= CH) {
    const vec v = *reinterpret_cast<const vecu*>(p);
#pragma unroll
    for (int i = 0; i < CH; ++i) s.v[i] = v[i];
  } else {
#pragma unroll
    for (int i = 0; i < CH; ++i) s.v[i] = p[min(i, KB - 1)];
  }
  return s;
}

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

// ---------------------------------------------------------------- few rows: weight stream
// A workgroup owns 16 NT columns x 16 MT rows and all of K; its W waves split
// K, each a run of scale blocks.  A wave copies a block's rows into a slot of
// its own in LDS (buffer_load ... lds, 8 whole 128-byte rows per instruction)
// and reads them back as operands: loaded as operands, 16 rows of 64 bytes per
// instruction, rows a power of two apart took twice as long (16 x 512 x 8192:
// 11.3 against 4.9 us).  Waves meet once, to add up their sums.  A wave has SL
// slots, blocks under way: one, and more workgroups on a CU, does as well as two
// or three (32 x 4096 x 3072 5.5 us either way) but where few workgroups have long
// runs.  What bounds it is the weights' stream (64 rows of 32 experts, 2048 x 2048:
// 118 MB in 15.2 us, some of them from the Infinity Cache) and, below some 10 MB,
// the trips to memory: 1 x 4096 x 3072 takes 4.7 us, 12.6 MB at 2.7 TB/s.
constexpr int kRun = 8;  // blocks whose scales a wave holds at a time

template <int NT, int MT, int W, int SL>
struct StreamT {
  static constexpr int SLOT = (NT + MT) * 2048, L = 2 * (NT + MT);  // bytes and loads per block
  static constexpr int PART = W * 16 * MT * 16 * NT * 4;
  static constexpr int SMEM = SL * W * SLOT > PART ? SL * W * SLOT : PART;
};

template <int NT, int MT, int W, int SL>
__global__ __launch_bounds__(W * 64) void k_block_stream(BlockGemmArgs a, int gx, int gy) {
  using S = StreamT<NT, MT, W, SL>;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, c = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int N = a.N, K = a.K, KB = (K + 127) >> 7, NBLK = (N + 127) >> 7;
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
  int src[MT];  // source row of operand row 16 j + c, -1: none
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const int m = t.t0 + 16 * j + c;
    src[j] = m < t.end ? m : -1;
  }
#pragma unroll
  for (int l = 0; l < S::L; ++l) {
    const int r = 8 * l + lr;
    voff[l] = (uint32_t)(l < 2 * NT ? (n0 + r < N ? r : -1) : (t.t0 + r - 16 * NT < t.end ? r - 16 * NT : -1));
  }
  uint32_t limit = 0x7FFFFFFFu;  // source rows from here on read as zeros
  if (a.rows) {
    limit = (uint32_t)a.M;
#pragma unroll
    for (int j = 0; j < MT; ++j)
      if (src[j] >= 0) src[j] = a.rows[src[j]];
#pragma unroll
    for (int l = 2 * NT; l < S::L; ++l)
      if ((int)voff[l] >= 0) voff[l] = (uint32_t)a.rows[t.t0 + voff[l]];
  }
#pragma unroll
  for (int l = 0; l < S::L; ++l)
    voff[l] = voff[l] < (l < 2 * NT ? 0x7FFFFFFFu : limit) ? voff[l] * (uint32_t)K + kc16 : kOut;
  const float* sa[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) sa[j] = a.Xs + (int64_t)((uint32_t)src[j] < (uint32_t)a.M ? src[j] : 0) * KB;
  const float* sb = a.Ws + ((int64_t)t.e * NBLK + n0 / 128) * KB;  // 16 NT columns lie in one block

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
  auto frag = [&](int at, int i) {
    const unsigned char* p = slot0 + at * S::SLOT + i * 2048;
    return join(*reinterpret_cast<const u32x4*>(p + flo), *reinterpret_cast<const u32x4*>(p + (flo ^ 16)));
  };

  f32x4 acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int per = (KB + W - 1) / W, end = min(KB, (wave + 1) * per);
  for (int k0 = wave * per; k0 < end; k0 += kRun) {
    const int n = min(kRun, end - k0);
    // scales of kRun blocks from `first` on, so that none is read past the row; block k0 + u is number u + back
    const int first = max(0, min(k0, KB - kRun)), back = k0 - first;
    const Scales<kRun> bv = load_scales<kRun>(sb + first, KB);
    Scales<kRun> av[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      av[j] = load_scales<kRun>(sa[j] + first, KB);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < SL; ++u)
      if (u < n) issue(k0 + u, u);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int u = 0; u < kRun; ++u) av[j].v[u] = (uint32_t)src[j] < (uint32_t)a.M ? av[j].v[u] * bv.v[u] : 0.f;
#pragma unroll
    for (int u = 0; u < kRun; ++u) {
      if (u < n) {
        constexpr int NEWER = (SL - 1) * S::L;  // loads that may still be under way
        if (SL > 1 && u + SL <= n)
          __builtin_amdgcn_s_waitcnt(kWaitVm0 | (NEWER & 15) | ((NEWER >> 4) << 14));
        else
          __builtin_amdgcn_s_waitcnt(kWaitVm0);
        asm volatile("" ::: "memory");
        i32x8 B[MT];
        float sc[MT];
#pragma unroll
        for (int j = 0; j < MT; ++j) {
          B[j] = frag(u % SL, NT + j);
          sc[j] = av[j].v[0];
#pragma unroll
          for (int v = 1; v < kRun; ++v) sc[j] = u + back == v ? av[j].v[v] : sc[j];
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const i32x8 A = frag(u % SL, i);
#pragma unroll
          for (int j = 0; j < MT; ++j) {
            const f32x4 p = mfma_blk(A, B[j]);
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(p[r], sc[j], acc[i][j][r]);
          }
        }
        __builtin_amdgcn_s_waitcnt(kWaitLgkm0);  // the slot has been read
        asm volatile("" ::: "memory");
        if (u + SL < n) issue(k0 + u + SL, u % SL);
      }
    }
  }

  __syncthreads();  // the slots are no longer used
  float(*part)[16 * MT][16 * NT] = reinterpret_cast<float(*)[16 * MT][16 * NT]>(smem);
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) *reinterpret_cast<f32x4*>(&part[wave][16 * j + c][16 * i + 4 * g]) = acc[i][j];
  __syncthreads();
  // four columns of a row per thread, the waves' sums in order
  for (int q = tid; q < 16 * MT * 4 * NT; q += W * 64) {
    const int row = q / (4 * NT), col = 4 * (q % (4 * NT)), m = t.t0 + row, n = n0 + col;
    if (m >= t.end || n >= N) continue;
    f32x4 y = *reinterpret_cast<const f32x4*>(&part[0][row][col]);
#pragma unroll
    for (int v = 1; v < W; ++v) y += *reinterpret_cast<const f32x4*>(&part[v][row][col]);
    if (a.bias) {
#pragma unroll
      for (int r = 0; r < 4; ++r) y[r] += bf16_to_f32(a.bias[min(n + r, N - 1)]);
    }
    uint16_t* p = a.Y + (int64_t)m * N + n;
    if ((N & 3) == 0) {
      *reinterpret_cast<u32x2*>(p) = u32x2{(uint32_t)f32_to_bf16(y[0]) | ((uint32_t)f32_to_bf16(y[1]) << 16),
                                           (uint32_t)f32_to_bf16(y[2]) | ((uint32_t)f32_to_bf16(y[3]) << 16)};
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n + r < N) p[r] = f32_to_bf16(y[r]);
    }
  }
}

// ---------------------------------------------------------------- LDS-tiled kernel
// A workgroup of WN x WM waves owns BN columns x BM rows of Y; K advances one
// scale block (128) per step.  Operand rows go from memory straight into LDS
// (buffer_load ... lds: lane i's 16 bytes land at the wave's base + 16 i), 8
// whole rows of 128 bytes per instruction, NS stages deep, chunks of a row
// XOR-swizzled by the choice of the chunk each lane reads (blk_pos).
//
// With KS > 1, KS such groups of waves split K, each with its own stages, and add
// up their sums in LDS at the end: tiles too few to fill the chip finish sooner.
//
// The scales come the same way, 8 steps' at a time and two buffers deep: 8 rows
// x 8 scales per instruction, in LDS row r's scale of step k at 8 r + (k + r / 8
// % 2) % 8 (16 rows on distinct banks).  Through registers their wait drained
// the loads under way every few steps (256 x 4096 x 4096: 13.9 us, 11.7 without
// any scales).
//
// Step with two or three stages (larger tiles): a wave holds its TM activation
// fragments and streams its TN weight fragments, read two ahead; each meets TM
// MFMAs, and the VALU scales and adds every result three MFMAs later.  All LDS
// reads of a stage are done two fragments before the step's end; there the waves
// meet at the step's one barrier, and the last two fragments' MFMAs cover the
// first reads of the next stage.
// Step with four stages (smaller tiles, whose MFMAs are too few to cover reads
// within the step): every fragment is read a whole step ahead into a second set
// of registers; the waves meet at the step's start and refill the stage of the
// step before.
//
// 8192 x 8192 x 8192 in 256 x 256: 442 us, 2.49 PFLOP/s, the matrix cores busy 72
// % of the time at the clock that the power limit leaves (a plain library product
// of the same codes, without scales: 350-365 us).  300 x 6152 x 4096 in 128 x 64:
// 14.9 us: 16 steps of 0.58 us in each of the two groups, and 5.6 us for launch,
// filling the stages, joining the groups' sums and storing.  A tile's operands,
// 786 KB, take 6.8 us at the 115 GB/s that a CU reads from L2, 0.43 of a step's
// 0.58: that read is the larger part, the rest of a step its latency.
constexpr int kScaleSteps = 8;

template <int BN_, int BM_, int WN_, int WM_, int NS_, int KS_>
struct Tile {
  static constexpr int BN = BN_, BM = BM_, WN = WN_, WM = WM_, NS = NS_, KS = KS_, THREADS = KS * WN * WM * 64;
  static constexpr int WAVES = WN * WM, TN = BN / (16 * WN), TM = BM / (16 * WM);
  static constexpr int STAGE = (BN + BM) * 128;
  static constexpr int NB = BN / 128 ? BN / 128 : 1;  // 128-column blocks
  static constexpr int SROWS = BM / (8 * WAVES);          // scale loads per wave
  static constexpr int SBUF = BM * 4 * kScaleSteps + 256;  // scales of rows, then of columns
  static constexpr int PITCH = TN * 32 + 16;  // output tile row in LDS
  static constexpr int PART = BN * 4 + 16;    // row of fp32 sums in LDS (KS > 1)
  static constexpr int OUT = KS > 1 ? KS * BM * PART : WAVES * TM * 16 * PITCH;
  static constexpr int PARK = WAVES * 64 * 4 * SROWS;  // offsets of the scale loads
  static constexpr int GROUP = NS * STAGE + 2 * SBUF + PARK;
  static constexpr int MAIN = KS * GROUP;
  static constexpr int SMEM = MAIN > OUT ? MAIN : OUT;
  static_assert(BN % (8 * WAVES) == 0 && BM % (8 * WAVES) == 0, "whole loads of 8 rows");
  static_assert(WAVES % 2 == 0 && NB <= 8 && NS < kScaleSteps, "scale buffers");
};

// TAIL: K % 128 != 0, chunks past K read zeros.  (Without it the loads carry no
// mask; those of steps past the end read the last block again, unused.)
template <class T, bool TAIL>
__device__ __forceinline__ void tile(const BlockGemmArgs& a, const RowTile t, const int n0) {
  constexpr int BN = T::BN, BM = T::BM, WN = T::WN, WM = T::WM, NS = T::NS, KS = T::KS;
  constexpr int TN = T::TN, TM = T::TM, W = T::WAVES;
  constexpr int LJW = BN / (8 * W), LJ = (BN + BM) / (8 * W);  // loads per wave and step: weights, all
  extern __shared__ __attribute__((aligned(16))) unsigned char shared[];
  const int group = KS > 1 ? __builtin_amdgcn_readfirstlane((int)threadIdx.x / (W * 64)) : 0;
  const int tid = (int)threadIdx.x - group * W * 64, lane = tid & 63;  // within the group
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  unsigned char* smem = shared + group * T::GROUP;
  unsigned char* sc = smem + NS * T::STAGE;
  const int g = lane >> 4, c = lane & 15;
  const int wn = wave % WN, wm = wave / WN;
  const int N = a.N, K = a.K, KB = (K + 127) >> 7, NBLK = (N + 127) >> 7;

  // load j of this wave: rows (j * W + wave) * 8 + lane / 8 of the stage, weights first; chunk kc of the row
  const int lr = lane >> 3, kc16 = 16 * blk_pos(lr, lane & 7);
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
  uint32_t limit = have;  // source rows from here on read as zeros too
  if (a.rows) {
    limit = (uint32_t)a.M;
#pragma unroll
    for (int j = LJW; j < LJ; ++j) {
      const uint32_t row = (uint32_t)a.rows[t.t0 + min(voff[j], have - 1)];
      voff[j] = voff[j] < have ? row : 0xFFFFFFFFu;
    }
  }
  // the loads of scales take the same rows as those of activations
  const int KB4 = KB * 4, kpos = ((lane & 7) - (wave & 1)) & 7;
  uint32_t* park = reinterpret_cast<uint32_t*>(sc + 2 * T::SBUF) + tid;  // kept in LDS: registers are short
#pragma unroll
  for (int j = 0; j < T::SROWS; ++j) park[j * W * 64] = voff[LJW + j] < limit ? voff[LJW + j] * (uint32_t)KB4 : kOut;
#pragma unroll
  for (int j = 0; j < LJ; ++j)
    voff[j] = j < LJW || voff[j] < limit ? voff[j] * (uint32_t)K + kc16 : kOut;
  // this group's steps: blocks k0 .. k0 + per - 1 (steps past those count nothing: their scales are zero)
  constexpr bool AHEAD = NS > 3;  // steps in pairs
  const int per = (KB + KS - 1) / KS, steps = AHEAD ? (per + 1) & ~1 : per;
  const int k0 = group * per;
  auto issue1 = [&](int kt, int st, int j) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        j < LJW ? Wr : Xr, (__attribute__((address_space(3))) void*)(smem + st * T::STAGE + (j * W + wave) * 1024), 16,
        (int)(!TAIL || kt * 128 + kc16 < K ? voff[j] : kOut), min(kt, KB - 1) * 128, 0, 0);
  };

  // scales of this group's steps 8 ch .. 8 ch + 7 (past the blocks the last one's), into buffer ch % 2
  const __amdgpu_buffer_rsrc_t Sr =
      a.rows ? make_rsrc(a.Xs, (uint32_t)((int64_t)a.M * KB4))
             : make_rsrc(a.Xs + (int64_t)t.t0 * KB, (uint32_t)min(BM, t.end - t.t0) * (uint32_t)KB4);
  const __amdgpu_buffer_rsrc_t Vr = make_rsrc(a.Ws + ((int64_t)t.e * NBLK + n0 / 128) * KB,
                                              (uint32_t)min(T::NB, NBLK - n0 / 128) * (uint32_t)KB4);
  auto fetch_scales = [&](int ch) {
    unsigned char* to = sc + (ch & 1) * T::SBUF;
    const int at = k0 + kScaleSteps * ch;
#pragma unroll
    for (int j = 0; j < T::SROWS; ++j) {
      const uint32_t row = park[j * W * 64];
      __builtin_amdgcn_raw_ptr_buffer_load_lds(Sr, (__attribute__((address_space(3))) void*)(to + (j * W + wave) * 256), 4,
                                               (int)(row == kOut ? kOut : row + 4u * min(at + kpos, KB - 1)), 0, 0, 0);
    }
    if (wave == 0)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          Vr, (__attribute__((address_space(3))) void*)(to + BM * 4 * kScaleSteps), 4,
          (int)(lr < T::NB ? (uint32_t)(lr * KB4) + 4u * min(at + (lane & 7), KB - 1) : kOut), 0, 0, 0);
  };

  // operand fragments: rows 16 i + c of the wave's part, K 32 g .. 32 g + 31 = chunks 2g, 2g + 1
  const int flo = c * 128 + blk_pos(c, 2 * g) * 16;
  const unsigned char* fw = smem + wn * TN * 2048;
  const unsigned char* fx = smem + BN * 128 + wm * TM * 2048;
  auto frag = [&](const unsigned char* base, int st, int i) {
    const unsigned char* p = base + st * T::STAGE + i * 2048;
    return join(*reinterpret_cast<const u32x4*>(p + flo), *reinterpret_cast<const u32x4*>(p + (flo ^ 16)));
  };
  const unsigned char* sx = sc + (wm * TM * 16 + c) * 4 * kScaleSteps;
  const unsigned char* sw = sc + BM * 4 * kScaleSteps + wn * TN * 16 / 128 * 4 * kScaleSteps;
  // a step's scales: the lane's rows' and the column block's, multiplied once they have landed (a step past the
  // blocks multiplies zeros)
  struct StepScales {
    float s[TM], w;
  };
  auto read_scales = [&](int n, StepScales& v) {
    const int buf = (n / kScaleSteps & 1) * T::SBUF, k = n % kScaleSteps;
    v.w = *reinterpret_cast<const float*>(sw + buf + 4 * k);
#pragma unroll
    for (int j = 0; j < TM; ++j)
      v.s[j] = *reinterpret_cast<const float*>(sx + buf + j * 64 * kScaleSteps + 4 * ((k + (c >> 3)) & 7));
  };
  auto join_scales = [&](int n, StepScales& v) {
#pragma unroll
    for (int j = 0; j < TM; ++j) v.s[j] = (KS == 1 && !AHEAD) || (n < per && k0 + n < KB) ? v.s[j] * v.w : 0.f;
  };

  f32x4 acc[TN][TM];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  fetch_scales(0);
#pragma unroll
  for (int st = 0; st < NS - 1; ++st)
#pragma unroll
    for (int j = 0; j < LJ; ++j) issue1(k0 + st, st, j);

  // Waves whose rows or columns are all past the end only load and meet: the
  // others have their share of the matrix cores and of LDS (32000 rows of 64
  // experts, 2048 x 2048: 174 us against 186; 8192 of 8, 4096 x 4096: 152.5
  // against 156.5; sizes without such waves within 1 %).
  const bool live = t.t0 + wm * TM * 16 < t.end && n0 + wn * TN * 16 < N;

  // products, scaled and added LAG MFMAs after they were made: fewer, and the VALU would wait for their results
  constexpr int LAG = 3, Q = TN * TM;
  f32x4 p[LAG + 1];
  auto add = [&](int q, const StepScales& v) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      acc[q / TM][q % TM][r] = __builtin_fmaf(p[q % (LAG + 1)][r], v.s[q % TM], acc[q / TM][q % TM][r]);
  };
  auto settle = [&] {
    // the sums are due here: the compiler would sink the scaling past the branch between the steps and keep the
    // step's products in registers
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j) asm volatile("" : "+v"(acc[i][j]));
  };
  // this wave's loads but for the newest N have landed, and its LDS reads; meet the others
#define WQ_MEET(N)                                                                                        \
  do {                                                                                                    \
    __builtin_amdgcn_s_waitcnt((kWaitVm0 & kWaitLgkm0) | ((N) & 15) | (((N) >> 4) << 14));                \
    asm volatile("s_barrier" ::: "memory");                                                               \
  } while (0)

  if constexpr (AHEAD) {
    WQ_MEET((NS - 2) * LJ);
    struct Operands {
      i32x8 a[TN], b[TM];
      StepScales s;
    } set[2];
#pragma unroll
    for (int i = 0; i < TN; ++i) set[0].a[i] = frag(fw, 0, i);
#pragma unroll
    for (int j = 0; j < TM; ++j) set[0].b[j] = frag(fx, 0, j);
    read_scales(0, set[0].s);
    // step n on `now`, reading step n + 1's operands into `next`; `pst`, `nst`: the stages of the step before and of
    // the next one
    auto step = [&](int n, int pst, int nst, Operands& now, Operands& next) {
      WQ_MEET((NS - 3) * LJ);
      join_scales(n, now.s);
      read_scales(n + 1, next.s);
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        constexpr int F = TN + TM;
#pragma unroll
        for (int f = 0; f < F; ++f)  // next operands in the order of their use, spread over the step
          if (q == f * Q / F) {
            if (f == 0) next.a[0] = frag(fw, nst, 0);
            else if (f <= TM) next.b[f - 1] = frag(fx, nst, f - 1);
            else next.a[f - TM] = frag(fw, nst, f - TM);
          }
        p[q % (LAG + 1)] = mfma_blk(now.a[q / TM], now.b[q % TM]);
        if (q >= LAG) add(q - LAG, now.s);
#pragma unroll
        for (int l = 0; l < LJ; ++l)
          if (q == l * Q / LJ) issue1(k0 + n - 1 + NS, pst, l);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int q = Q - LAG; q < Q; ++q) add(q, now.s);
      settle();
    };
    auto after = [](int st) { return st + 1 == NS ? 0 : st + 1; };
    if (live) {
      for (int n = 0, pst = NS - 1, st = 0; n < steps; n += 2) {
        const int st1 = after(st), st2 = after(st1);
        step(n, pst, st1, set[0], set[1]);
        step(n + 1, st, st2, set[1], set[0]);
        if (n % kScaleSteps == 0) fetch_scales(n / kScaleSteps + 1);
        pst = st1;
        st = st2;
      }
    } else {
      for (int n = 0, pst = NS - 1; n < steps; ++n) {
        WQ_MEET((NS - 3) * LJ);
#pragma unroll
        for (int l = 0; l < LJ; ++l) issue1(k0 + n - 1 + NS, pst, l);
        if (n % kScaleSteps == 1) fetch_scales(n / kScaleSteps + 1);
        pst = after(pst);
      }
    }
  } else {
    WQ_MEET(0);
    // A freed stage's loads are spread over SPAN fragments' MFMAs (two of the
    // step that frees it, the rest of the next one): issued in one go they fill
    // the memory pipe's queue and the waves stall on it.
    constexpr int SPAN = TN >= 8 ? 4 : TN - 1;
    auto slot = [](int l) { return l * SPAN / LJ; };
#pragma unroll
    for (int l = 0; l < LJ; ++l)
      if (slot(l) < 2) issue1(k0 + NS - 1, NS - 1, l);

    // ring of weight fragments: fragment i in slot i % R, so that the next step's
    // first two find slots 0 and 1 free at the end of this step
    constexpr int R = TN % 3 == 2 ? 3 : 4;
    static_assert(TN % R == 2 || TN % R == 0, "slots 0 and 1 are free in time");
    i32x8 A[R], B[TM];
    StepScales S;
    A[0] = frag(fw, 0, 0);
#pragma unroll
    for (int j = 0; j < TM; ++j) B[j] = frag(fx, 0, j);
    read_scales(0, S);
    A[1] = frag(fw, 0, 1);
    // step n; `pst`, `st`, `nst`: the stages of the last, this and the next one
    auto step = [&](int n, int pst, int st, int nst) {
      const int kt = k0 + n;
      constexpr int MEET = (TN - 2) * TM;
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int i = q / TM, j = q % TM;
        if (j == 0 && i + 2 < TN) A[(i + 2) % R] = frag(fw, st, i + 2);
        if (q == MEET) WQ_MEET((NS - 2) * LJ);  // every read of this stage has been made: meet, then refill it
        p[q % (LAG + 1)] = mfma_blk(A[i % R], B[j]);
        if (q == LAG - 1) join_scales(n, S);
        if (q >= LAG) add(q - LAG, S);
#pragma unroll
        for (int l = 0; l < LJ; ++l) {
          // in a slot's first MFMAs, one load each
          const int at = slot(l), nth = l - (at * LJ + SPAN - 1) / SPAN;
          if (j == min(nth, TM - 1)) {
            if (at < 2 && i == TN - 2 + at) issue1(kt + NS, st, l);
            if (at >= 2 && i == at - 2) issue1(kt + NS - 1, pst, l);
          }
        }
        if (q == MEET + TM - 1) A[0] = frag(fw, nst, 0);
        if (i == TN - 1) B[j] = frag(fx, nst, j);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int q = Q - LAG; q < Q; ++q) add(q, S);
      settle();
      A[1] = frag(fw, nst, 1);
      read_scales(n + 1, S);
      __builtin_amdgcn_sched_barrier(0);
    };
    auto after = [](int st) { return st + 1 == NS ? 0 : st + 1; };
    if (live) {
      for (int n = 0, pst = NS - 1, st = 0; n < steps; ++n) {
        const int nst = after(st);
        step(n, pst, st, nst);
        if (n % kScaleSteps == 0) fetch_scales(n / kScaleSteps + 1);
        pst = st;
        st = nst;
      }
    } else {
      for (int n = 0, pst = NS - 1, st = 0; n < steps; ++n) {
#pragma unroll
        for (int l = 0; l < LJ; ++l)
          if (slot(l) >= 2) issue1(k0 + n + NS - 1, pst, l);
        WQ_MEET((NS - 2) * LJ);
#pragma unroll
        for (int l = 0; l < LJ; ++l)
          if (slot(l) < 2) issue1(k0 + n + NS, st, l);
        if (n % kScaleSteps == 0) fetch_scales(n / kScaleSteps + 1);
        pst = st;
        st = after(st);
      }
    }
  }
#undef WQ_MEET

  __builtin_amdgcn_s_waitcnt(kWaitVm0 & kWaitLgkm0);
  asm volatile("s_barrier" ::: "memory");  // the stages are no longer used
  const bool vec = (N & 7) == 0;
  auto put = [&](int m, int n, u32x4 v) {  // 8 columns of a row
    if (m >= t.end) return;
    uint16_t* y = a.Y + (int64_t)m * N + n;
    if (vec) {
      if (n < N) __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(y));
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (n + e < N) y[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
    }
  };
  auto bias = [&](int n) { return a.bias ? bf16_to_f32(a.bias[min(n, N - 1)]) : 0.f; };
  auto pack = [](float lo, float hi) { return (uint32_t)f32_to_bf16(lo) | ((uint32_t)f32_to_bf16(hi) << 16); };

  if constexpr (KS > 1) {
    // the groups' sums meet in LDS and are added in order, 8 columns of a row per thread
    const int col = wn * TN * 16 + 4 * g, row = wm * TM * 16 + c;
    unsigned char* mine = shared + group * (BM * T::PART);
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j)
        *reinterpret_cast<f32x4*>(mine + (row + 16 * j) * T::PART + (col + 16 * i) * 4) = acc[i][j];
    __syncthreads();
    for (int q = threadIdx.x; q < BM * BN / 8; q += KS * W * 64) {
      const int r = q / (BN / 8), n = 8 * (q % (BN / 8));
      f32x4 y[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          y[h] += *reinterpret_cast<const f32x4*>(shared + (k * BM + r) * T::PART + n * 4 + 16 * h);
      u32x4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[e] = pack(y[e >> 1][2 * (e & 1)] + bias(n0 + n + 2 * e), y[e >> 1][2 * (e & 1) + 1] + bias(n0 + n + 2 * e + 1));
      put(t.t0 + r, n0 + n, v);
    }
  } else {
    // wave tiles leave through LDS as 16-byte row pieces
    unsigned char* et = shared + wave * (TM * 16 * T::PITCH);
    const int nw = n0 + wn * TN * 16, mw = t.t0 + wm * TM * 16;
#pragma unroll
    for (int i = 0; i < TN; ++i) {
      float b[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) b[r] = bias(nw + 16 * i + 4 * g + r);
#pragma unroll
      for (int j = 0; j < TM; ++j)
        *reinterpret_cast<u32x2*>(et + (16 * j + c) * T::PITCH + (16 * i + 4 * g) * 2) =
            u32x2{pack(acc[i][j][0] + b[0], acc[i][j][1] + b[1]), pack(acc[i][j][2] + b[2], acc[i][j][3] + b[3])};
    }
    __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
    asm volatile("" ::: "memory");
    constexpr int LPR = TN * 2, RPI = 64 / LPR;  // lanes per row, rows per store instruction
#pragma unroll
    for (int q = 0; q < TM * 16 / RPI; ++q) {
      const int row = RPI * q + lane / LPR, col = 8 * (lane % LPR);
      put(mw + row, nw + col, *reinterpret_cast<const u32x4*>(et + row * T::PITCH + col * 2));
    }
  }
}

// Tiles B in whole rounds of the chip, one to a CU; the rest of them, where that
// is at most half a round, in tiles S, which take less time (S = B: none).
// 4352 x 4096 x 4096, 272 tiles of 256 x 256: 77 us, 92 with the last 16 whole;
// 8192 rows of 8 experts, 4096 x 4096: 155 against 169 (before waves without rows
// were left out); 2000 rows of 64 experts, 1536 x 2048 (256 x 128): 42.9 against
// 44.8.  128 x 128 tiles gain as much from a split, but never so that they beat
// the other forms.
//
// Experts: the tiles there are, not the bound that the grid is for, so that the
// XCDs share them out evenly (5604 rows of 16 experts, 3424 x 3072: 111 us by
// the bound).
template <class B, class S, bool TAIL>
__global__ __launch_bounds__(B::THREADS, 2) void k_block_tile(BlockGemmArgs a, int gx, int gy) {
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

}  // namespace

// Row tiles of bm rows; for experts a bound on their number: every expert that has rows may end in a partial tile.
static int64_t row_tiles(const BlockGemmArgs& a, int64_t bm) {
  if (!a.offsets) return (a.M + bm - 1) / bm;
  return (a.T + (int64_t)(a.E < a.T ? a.E : a.T) * (bm - 1)) / bm;
}

// A launch holds fewer than 2^32 threads (and its workgroups are numbered by ints).
static bool too_many(int64_t groups, int threads) { return groups >= ((int64_t)1 << 32) / threads || groups >= INT32_MAX; }

template <class B, class S>
static hipError_t tile_launch(const BlockGemmArgs& a, hipStream_t s) {
  constexpr int smem = B::SMEM > S::SMEM ? B::SMEM : S::SMEM, parts = B::BN * B::BM / (S::BN * S::BM);
  static_assert(smem <= 160 * 1024, "LDS of a CU");
  const int64_t gx = (a.N + B::BN - 1) / B::BN, gy = row_tiles(a, B::BM);
  if (too_many(gx * gy + parts * kMostRest, B::THREADS)) return hipErrorInvalidConfiguration;
  // (of experts the kernel counts the tiles)
  const int64_t rest = a.offsets ? (parts > 1 ? kMostRest : 0) : rest_of_round(parts > 1, (int)(gx * gy));
  static SmemAllowed allowed[2];
  const bool tail = a.K % 128 != 0;
  const auto kern = tail ? k_block_tile<B, S, true> : k_block_tile<B, S, false>;
  hipError_t e = allow_smem(kern, smem, allowed[tail]);
  if (e != hipSuccess) return e;
  return launch(kern, dim3((unsigned)(gx * gy + (parts - 1) * rest)), B::THREADS, smem, s, a, (int)gx, (int)gy);
}

template <int NT, int MT, int W, int SL = 1>
static hipError_t stream_launch(const BlockGemmArgs& a, hipStream_t s) {
  constexpr int smem = StreamT<NT, MT, W, SL>::SMEM;
  static_assert(smem <= 65536, "no leave needed for the LDS size");
  const int64_t gx = (a.N + 16 * NT - 1) / (16 * NT), gy = row_tiles(a, 16 * MT);
  if (too_many(gx * gy, W * 64)) return hipErrorInvalidConfiguration;
  return launch(k_block_stream<NT, MT, W, SL>, dim3((unsigned)(gx * gy)), W * 64, smem, s, a, (int)gx, (int)gy);
}

using Tile256 = Tile<256, 256, 2, 4, 2, 1>;
using Tile256x128 = Tile<256, 128, 4, 2, 3, 1>;
using Tile128 = Tile<128, 128, 2, 4, 4, 1>;
using Tile128x64 = Tile<128, 64, 2, 2, 3, 2>;
using Tile64 = Tile<64, 64, 2, 2, 4, 2>;
using Tile64One = Tile<64, 64, 2, 2, 4, 1>;

hipError_t launch_block_gemm(const BlockGemmArgs& a, hipStream_t s) {
  switch (block_form(a.offsets != nullptr, a.T, a.E, a.N, a.K)) {
    case kStream16: return stream_launch<1, 1, 8>(a, s);
    case kStream16Deep: return stream_launch<1, 1, 8, 2>(a, s);
    case kStream32Eight: return stream_launch<2, 1, 8>(a, s);
    case kStream32: return stream_launch<2, 1, 4>(a, s);
    case kStream32x32: return stream_launch<2, 2, 4>(a, s);
    case kStream64: return stream_launch<4, 1, 4>(a, s);
    case kTile256: return tile_launch<Tile256, Tile128>(a, s);
    case kTile256x128: return tile_launch<Tile256x128, Tile128>(a, s);
    case kTile128: return tile_launch<Tile128, Tile128>(a, s);
    case kTile128x64: return tile_launch<Tile128x64, Tile128x64>(a, s);
    case kTile64: return tile_launch<Tile64, Tile64>(a, s);
    case kTile64One: return tile_launch<Tile64One, Tile64One>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace wq
