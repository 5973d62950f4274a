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
// c, both at K 32g .. 32g+31; D[4g + r][c] in element r.  Unit block scales.
__device__ __forceinline__ f32x4 mfma_blk(i32x8 w, i32x8 x) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 127, 0, 127);
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

}  // namespace

hipError_t launch_block_gemm(const BlockGemmArgs& a, hipStream_t s) {
  // row tiles of 16: every expert with rows may end in a partial one
  const int64_t tiles = a.offsets ? (a.T + (int64_t)(a.E < a.T ? a.E : a.T) * 15) / 16 : (a.M + 15) / 16;
  k_block_direct<<<dim3((unsigned)((a.N + 63) / 64), (unsigned)tiles), 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace wq
