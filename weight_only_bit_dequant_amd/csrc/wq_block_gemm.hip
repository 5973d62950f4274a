// Block-scaled FP8 GEMMs: Y = deq(X) . deq(W)^T for one weight or, with rows
// sorted by expert, for many.
//
// One v_mfma_f32_16x16x128_f8f6f4 is exactly one scale block deep: with a zero
// addend it gives the block's products summed in fp32, which the VALU scales
// and adds to the fp32 sum (one fused multiply-add per output and block).  The
// weights are operand A, so a lane's four results are four columns n of one
// row m: one activation scale, one weight scale, 8 bytes of bf16 output.
#include "wq_block_internal.hpp"
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

// Row tile `ti` of the experts' row tiles, BM rows each, numbered through all
// experts: expert e (-1: no such tile), its rows [t0, end).  Offsets are
// clamped to [0, T].  Every lane of the wave gets the same answer.
struct RowTile {
  int e, t0, end;
};
__device__ __forceinline__ RowTile row_tile(const int32_t* off, int E, int T, int BM, int ti) {
  const int lane = threadIdx.x & 63;
  int before = 0;  // tiles of the experts before this stretch of 64
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + lane;
    int lo = 0, hi = 0;
    if (e < E) {
      lo = min(max(off[e], 0), T);
      hi = min(max(off[e + 1], lo), T);
    }
    const int tiles = (hi - lo + BM - 1) / BM;
    int upto = tiles;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(upto, d);
      if (lane >= d) upto += v;
    }
    const int first = before + upto - tiles;
    const uint64_t hit = __ballot(ti >= first && ti < first + tiles);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      const int elo = __builtin_amdgcn_readlane(lo, l), ehi = __builtin_amdgcn_readlane(hi, l);
      return {e0 + l, elo + (ti - __builtin_amdgcn_readlane(first, l)) * BM, ehi};
    }
    before += __builtin_amdgcn_readlane(upto, 63);
  }
  return {-1, 0, 0};
}

// ---------------------------------------------------------------- direct kernel
// 4 waves x 16 columns, 16 rows, all of K; operands straight from memory.
__global__ __launch_bounds__(256) void k_block_direct(BlockGemmArgs a) {
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int N = a.N, K = a.K, KB = (K + 127) / 128, NB = (N + 127) / 128;
  RowTile t = a.offsets ? row_tile(a.offsets, a.E, a.T, 16, blockIdx.y)
                        : RowTile{0, (int)blockIdx.y * 16, a.M};
  if (t.e < 0) return;
  const int n0 = blockIdx.x * 64 + wave * 16;
  if (n0 >= N) return;
  const uint8_t* W = a.Wq + ((int64_t)t.e * N + n0) * K;
  const float* Ws = a.Ws + ((int64_t)t.e * NB + n0 / 128) * KB;
  const int m = t.t0 + c;
  const bool mok = m < t.end;
  const int src = mok ? (a.rows ? a.rows[m] : m) : 0;
  const bool sok = mok && (uint32_t)src < (uint32_t)a.M;
  const uint8_t* X = a.Xq + (int64_t)(sok ? src : 0) * K;
  const float* Xs = a.Xs + (int64_t)(sok ? src : 0) * KB;
  const bool nok = n0 + c < N;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int kb = 0; kb < KB; ++kb) {
    u32x4 w[2] = {}, x[2] = {};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = kb * 128 + 32 * g + 16 * h;
      if (k < K && nok) w[h] = *reinterpret_cast<const u32x4*>(W + (int64_t)c * K + k);
      if (k < K && sok) x[h] = *reinterpret_cast<const u32x4*>(X + k);
    }
    const float s = (sok ? Xs[kb] : 0.f) * Ws[kb];
    const f32x4 p = mfma_blk(join(w[0], w[1]), join(x[0], x[1]));
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[r] = __builtin_fmaf(p[r], s, acc[r]);
  }
  if (!mok) return;
  const int n = n0 + 4 * g;
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (n + r < N) a.Y[(int64_t)m * N + n + r] = f32_to_bf16(acc[r] + (a.bias ? bf16_to_f32(a.bias[n + r]) : 0.f));
}

// ---------------------------------------------------------------- LDS-tiled kernel
// A workgroup of WN x WM waves owns BN columns x BM rows of Y; K advances one
// scale block (128) per step.  Operand rows go from memory straight into LDS
// (buffer_load ... lds: lane i's 16 bytes land at the wave's base + 16 i), 8
// whole rows of 128 bytes per instruction, NS stages deep, chunks of a row
// XOR-swizzled by the choice of the chunk each lane reads (blk_pos).
//
// The products sa * sb of the tile's scales wait in LDS too, four steps at a
// time ([buffer][128-column block][row][4]): the BM first threads load four
// scales of one activation row at once, which costs a quarter of the line
// requests of one load per step.
//
// Step: a wave holds its TM activation fragments and streams its TN weight
// fragments, read two fragments ahead; each meets TM MFMAs, and the VALU scales
// and adds every result three MFMAs later.  All LDS reads of a stage are done two
// fragments before the step's end; there the waves meet at the step's one
// barrier, and the last two fragments' MFMAs cover the first reads of the next
// stage.
constexpr int kScaleSteps = 4;

// LDS slot of 16-byte chunk k of row r: the four lane groups' reads of 16 rows
// then fall on distinct banks.
__device__ __forceinline__ int blk_pos(int r, int k) { return k ^ (((r >> 1) & 1) | (r & 4)); }

template <int BN, int BM, int WN, int WM, int NS>
struct TileT {
  static constexpr int WAVES = WN * WM, TN = BN / (16 * WN), TM = BM / (16 * WM);
  static constexpr int STAGE = (BN + BM) * 128;
  static constexpr int NB = BN / 128 ? BN / 128 : 1;  // 128-column blocks
  static constexpr int SBUF = NB * BM * 4 * kScaleSteps;
  static constexpr int PITCH = TN * 32 + 16;  // output tile row in LDS
  static constexpr int OUT = WAVES * TM * 16 * PITCH;
  static constexpr int MAIN = NS * STAGE + 2 * SBUF;
  static constexpr int SMEM = MAIN > OUT ? MAIN : OUT;
  static_assert(BM <= WAVES * 64, "a thread per row of scales");
  static_assert(BN % (8 * WAVES) == 0 && BM % (8 * WAVES) == 0, "whole loads of 8 rows");
};

template <int BN, int BM, int WN, int WM, int NS>
__global__ __launch_bounds__(WN* WM * 64, 2) void k_block_tile(BlockGemmArgs a, int gx, int gy) {
  using T = TileT<BN, BM, WN, WM, NS>;
  constexpr int TN = T::TN, TM = T::TM, W = T::WAVES;
  constexpr int LJW = BN / (8 * W), LJ = (BN + BM) / (8 * W);  // loads per wave and step: weights, all
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  float* sc = reinterpret_cast<float*>(smem + NS * T::STAGE);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, c = lane & 15;
  const int wn = wave % WN, wm = wave / WN;
  const int N = a.N, K = a.K, KB = (K + 127) >> 7, NBLK = (N + 127) >> 7;

  // XCD-aware tile order: workgroup b runs on XCD b % 8; each XCD takes a
  // contiguous piece of an order that fills bands of 4 column tiles row tile
  // by row tile, so tiles in flight on one L2 share operands both ways
  int tx, ty;
  {
    const int G = gx * gy, b = blockIdx.x, q = G >> 3, r = G & 7, x = b & 7;
    const int idx = x * q + min(x, r) + (b >> 3);
    const int band = idx / (4 * gy), in = idx - band * 4 * gy, wide = min(4, gx - 4 * band);
    ty = in / wide;
    tx = 4 * band + in - ty * wide;
  }
  RowTile t{0, ty * BM, a.M};
  if (a.offsets) {
    t = row_tile(a.offsets, a.E, a.T, BM, ty);
    if (t.e < 0) return;
  }
  const int n0 = tx * BN;

  // load j of this wave: rows (j * W + wave) * 8 + lane / 8 of the stage, weights first; chunk kc of the row
  const int lr = lane >> 3, kc16 = 16 * blk_pos(lr, lane & 7);
  const __amdgpu_buffer_rsrc_t Wr =
      make_rsrc(a.Wq + ((int64_t)t.e * N + n0) * K, (uint32_t)min(BN, N - n0) * (uint32_t)K);
  const __amdgpu_buffer_rsrc_t Xr = a.rows ? make_rsrc(a.Xq, (uint32_t)((int64_t)a.M * K))
                                           : make_rsrc(a.Xq + (int64_t)t.t0 * K, (uint32_t)min(BM, t.end - t.t0) * (uint32_t)K);
  uint32_t voff[LJ];  // rows past the end repeat the last
#pragma unroll
  for (int j = 0; j < LJ; ++j) {
    const int r = (j * W + wave) * 8 + lr;
    voff[j] = (uint32_t)(j < LJW ? min(r, N - n0 - 1) : min(r - BN, t.end - t.t0 - 1));
  }
  const int srow = t.t0 + min(tid, t.end - t.t0 - 1);  // the row whose scales thread tid < BM stages
  int ssrc = srow;
  uint32_t limit = 0xFFFFFFFFu;  // source rows from here on read as zeros
  if (a.rows) {
    limit = (uint32_t)a.M;
    ssrc = a.rows[srow];
#pragma unroll
    for (int j = LJW; j < LJ; ++j) voff[j] = (uint32_t)a.rows[t.t0 + voff[j]];
  }
#pragma unroll
  for (int j = 0; j < LJ; ++j)
    voff[j] = j < LJW || voff[j] < limit ? voff[j] * (uint32_t)K + kc16 : kOut;
  auto issue1 = [&](int kt, int st, int j) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        j < LJW ? Wr : Xr, (__attribute__((address_space(3))) void*)(smem + st * T::STAGE + (j * W + wave) * 1024), 16,
        (int)(kt * 128 + kc16 < K ? voff[j] : kOut), min(kt, KB - 1) * 128, 0, 0);
  };

  // scales of steps [first(ch), first(ch) + 4): thread `tid` owns row tid
  const float* sa = nullptr;  // its activation row's scales (null: a row without any)
  if (tid < BM && (uint32_t)ssrc < (uint32_t)a.M) sa = a.Xs + (int64_t)ssrc * KB;
  const float* sb = a.Ws + ((int64_t)t.e * NBLK + n0 / 128) * KB;
  auto first = [&](int ch) { return max(0, min(kScaleSteps * ch, KB - kScaleSteps)); };
  typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
  auto load4 = [&](const float* p) {
    if (KB >= kScaleSteps) return f32x4(*reinterpret_cast<const f32x4u*>(p));
    return f32x4{p[0], p[min(1, KB - 1)], p[min(2, KB - 1)], p[KB - 1]};
  };
  f32x4 sav, sbv[T::NB];
  auto load_scales = [&](int ch) {
    sav = f32x4{0.f, 0.f, 0.f, 0.f};
    if (sa) {
      sav = load4(sa + first(ch));
#pragma unroll
      for (int q = 0; q < T::NB; ++q) sbv[q] = load4(sb + (int64_t)min(q, NBLK - 1 - n0 / 128) * KB + first(ch));
    }
  };
  auto store_scales = [&](int ch) {
    if (tid < BM) {
#pragma unroll
      for (int q = 0; q < T::NB; ++q)
        *reinterpret_cast<f32x4*>(sc + ((ch & 1) * T::NB + q) * BM * kScaleSteps + tid * kScaleSteps) =
            sa ? sav * sbv[q] : f32x4{0.f, 0.f, 0.f, 0.f};
    }
  };

  // operand fragments: rows 16 i + c of the wave's part, K 32 g .. 32 g + 31 = chunks 2g, 2g + 1
  const int flo = c * 128 + blk_pos(c, 2 * g) * 16;
  const unsigned char* fw = smem + wn * TN * 2048;
  const unsigned char* fx = smem + BN * 128 + wm * TM * 2048;
  auto frag = [&](const unsigned char* base, int st, int i) {
    const unsigned char* p = base + st * T::STAGE + i * 2048;
    return join(*reinterpret_cast<const u32x4*>(p + flo), *reinterpret_cast<const u32x4*>(p + (flo ^ 16)));
  };
  const float* scw = sc + ((wn * TN * 16) / 128 * BM + wm * TM * 16 + c) * kScaleSteps;
  auto scale = [&](int kt, int i) {
    const int ch = kt / kScaleSteps;
    return scw[(ch & 1) * T::NB * BM * kScaleSteps + i * 16 * kScaleSteps + kt - first(ch)];
  };

  f32x4 acc[TN][TM];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  load_scales(0);
#pragma unroll
  for (int st = 0; st < NS - 1; ++st)
#pragma unroll
    for (int j = 0; j < LJ; ++j) issue1(st, st, j);
  store_scales(0);
  __builtin_amdgcn_s_waitcnt(kWaitVm0 & kWaitLgkm0);
  asm volatile("s_barrier" ::: "memory");
  // A freed stage's loads are spread over SPAN fragments' MFMAs (two of the
  // step that frees it, the rest of the next one): issued in one go they fill
  // the memory pipe's queue and the waves stall on it.
  constexpr int SPAN = TN >= 8 ? TN - 2 : TN - 1;
  auto slot = [](int l) { return l * SPAN / LJ; };
#pragma unroll
  for (int l = 0; l < LJ; ++l)
    if (slot(l) < 2) issue1(NS - 1, NS - 1, l);

  // ring of weight fragments: fragment i in slot i % R, so that the next step's
  // first two find slots 0 and 1 free at the end of this step
  constexpr int R = TN % 3 == 2 ? 3 : 4;
  static_assert(TN % R == 2 || TN % R == 0, "slots 0 and 1 are free in time");
  i32x8 A[R], B[TM];
  // products, scaled and added LAG MFMAs after they were made: fewer, and the VALU would wait for their results
  constexpr int LAG = 3;
  f32x4 p[LAG + 1];
  float s[TM];
  A[0] = frag(fw, 0, 0);
#pragma unroll
  for (int j = 0; j < TM; ++j) {
    B[j] = frag(fx, 0, j);
    s[j] = scale(0, j);
  }
  A[1] = frag(fw, 0, 1);
  auto add = [&](int q) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      acc[q / TM][q % TM][r] = __builtin_fmaf(p[q % (LAG + 1)][r], s[q % TM], acc[q / TM][q % TM][r]);
  };
  // one step; `pst`, `st`, `nst`: the stages of the last, this and the next one
  auto step = [&](int kt, int pst, int st, int nst) {
    constexpr int Q = TN * TM, MEET = (TN - 2) * TM;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int i = q / TM, j = q % TM;
      if (j == 0 && i + 2 < TN) A[(i + 2) % R] = frag(fw, st, i + 2);
      if (q == MEET) {
        // every read of this stage has been made: meet, then refill it
        __builtin_amdgcn_s_waitcnt((kWaitVm0 & kWaitLgkm0) | ((NS - 2) * LJ & 15) | (((NS - 2) * LJ >> 4) << 14));
        asm volatile("s_barrier" ::: "memory");
        const int sub = kt & (kScaleSteps - 1);
        if (sub == 0) load_scales(kt / kScaleSteps + 1);
        if (sub == 2) store_scales(kt / kScaleSteps + 1);
      }
      p[q % (LAG + 1)] = mfma_blk(A[i % R], B[j]);
      if (q >= LAG) add(q - LAG);
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
    for (int q = Q - LAG; q < Q; ++q) add(q);
    A[1] = frag(fw, nst, 1);
#pragma unroll
    for (int j = 0; j < TM; ++j) s[j] = scale(min(kt + 1, KB - 1), j);
    __builtin_amdgcn_sched_barrier(0);
  };
  for (int kt = 0, pst = NS - 1, st = 0; kt < KB; ++kt) {
    const int nst = st + 1 == NS ? 0 : st + 1;
    step(kt, pst, st, nst);
    pst = st;
    st = nst;
  }

  // output: wave tiles leave through LDS as 16-byte row pieces
  __builtin_amdgcn_s_waitcnt(kWaitVm0 & kWaitLgkm0);
  asm volatile("s_barrier" ::: "memory");
  unsigned char* et = smem + wave * (TM * 16 * T::PITCH);
  const int nw = n0 + wn * TN * 16, mw = t.t0 + wm * TM * 16;
#pragma unroll
  for (int i = 0; i < TN; ++i) {
    float b[4] = {0.f, 0.f, 0.f, 0.f};
    if (a.bias) {
#pragma unroll
      for (int r = 0; r < 4; ++r) b[r] = bf16_to_f32(a.bias[min(nw + 16 * i + 4 * g + r, N - 1)]);
    }
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      u32x2 v;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        v[h] = (uint32_t)f32_to_bf16(acc[i][j][2 * h] + b[2 * h]) |
               ((uint32_t)f32_to_bf16(acc[i][j][2 * h + 1] + b[2 * h + 1]) << 16);
      *reinterpret_cast<u32x2*>(et + (16 * j + c) * T::PITCH + (16 * i + 4 * g) * 2) = v;
    }
  }
  __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
  asm volatile("" ::: "memory");
  constexpr int LPR = TN * 2, RPI = 64 / LPR;  // lanes per row, rows per store instruction
  const bool vec = (N & 7) == 0;
#pragma unroll
  for (int q = 0; q < TM * 16 / RPI; ++q) {
    const int row = RPI * q + lane / LPR, col = 8 * (lane % LPR);
    const u32x4 v = *reinterpret_cast<const u32x4*>(et + row * T::PITCH + col * 2);
    const int m = mw + row, n = nw + col;
    if (m < t.end) {
      uint16_t* y = a.Y + (int64_t)m * N + n;
      if (vec) {
        if (n < N) __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(y));
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (n + e < N) y[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
      }
    }
  }
}

}  // namespace

template <int BN, int BM, int WN, int WM, int NS>
static hipError_t tile_launch(const BlockGemmArgs& a, hipStream_t s) {
  using T = TileT<BN, BM, WN, WM, NS>;
  static std::atomic<int> allowed{0};
  const auto kern = k_block_tile<BN, BM, WN, WM, NS>;
  hipError_t e = allow_smem(kern, T::SMEM, allowed);
  if (e != hipSuccess) return e;
  const int64_t gx = (a.N + BN - 1) / BN;
  const int64_t gy = a.offsets ? (a.T + (int64_t)(a.E < a.T ? a.E : a.T) * (BM - 1)) / BM : (a.M + BM - 1) / BM;
  kern<<<(unsigned)(gx * gy), WN * WM * 64, T::SMEM, s>>>(a, (int)gx, (int)gy);
  return hipGetLastError();
}

hipError_t launch_block_gemm(const BlockGemmArgs& a, hipStream_t s) {
  if (a.T >= 1024) return tile_launch<256, 256, 2, 4, 2>(a, s);
  if (a.T >= 128) return tile_launch<128, 128, 2, 2, 2>(a, s);
  // row tiles of 16: every expert with rows may end in a partial one
  const int64_t tiles = a.offsets ? (a.T + (int64_t)(a.E < a.T ? a.E : a.T) * 15) / 16 : (a.M + 15) / 16;
  k_block_direct<<<dim3((unsigned)((a.N + 63) / 64), (unsigned)tiles), 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace wq
