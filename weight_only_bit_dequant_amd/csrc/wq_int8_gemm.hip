// 8-bit integer GEMMs: Y = (Xq . Wq^T) * Xs * Ws for one weight or, with rows
// sorted by expert, for many.
//
// v_mfma_i32_16x16x64_i8 sums 64 products in int32, exactly.  The weights are
// operand A, so a lane's four results are four columns n of one row m: one
// activation scale, four weight scales, 8 bytes of bf16 output.
#include "wq_int8_internal.hpp"
#include "wq_row_tiles.hpp"

namespace wq {

namespace {

typedef __attribute__((ext_vector_type(4))) int i32x4;

// lane (g, c) of A: 16 codes of weight row c, of B: 16 codes of activation row
// c, both at K 16g .. 16g+15; D[4g + r][c] in element r
__device__ __forceinline__ i32x4 mfma_i8(u32x4 w, u32x4 x, i32x4 acc) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, w), __builtin_bit_cast(i32x4, x), acc, 0, 0, 0);
}

// A wave owns 16 columns x 16 rows of Y and all of K; operands come straight
// from memory.
__global__ __launch_bounds__(256) void k_int8_simple(Int8GemmArgs a, int gx, int gy) {
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  RowTile t;
  At p;
  if (a.offsets) {
    const RowTiles all(a.offsets, a.E, a.T, 16);
    if (!stream_at(blockIdx.x, gx, all.total, gy, p)) return;
    t = all.find(p.ty);
  } else {
    stream_at(blockIdx.x, gx, gy, gy, p);
    t = {0, p.ty * 16, a.M};
  }
  const int n0 = p.tx * 64 + wave * 16, m = t.t0 + c;
  if (n0 >= a.N) return;
  int src = m < t.end ? m : -1;
  if (a.rows && src >= 0) src = a.rows[src];
  const bool has = (uint32_t)src < (uint32_t)a.M;
  const uint8_t* x = a.Xq + (int64_t)(has ? src : 0) * a.K;
  const bool wide = n0 + c < a.N;
  const uint8_t* w = a.Wq + ((int64_t)t.e * a.N + (wide ? n0 + c : n0)) * a.K;
  i32x4 acc = {0, 0, 0, 0};
  for (int k = 0; k < a.K; k += 64) {
    const bool in = k + 16 * g < a.K;
    const u32x4 zero = {0, 0, 0, 0};
    const u32x4 wv = in && wide ? *reinterpret_cast<const u32x4*>(w + k + 16 * g) : zero;
    const u32x4 xv = in && has ? *reinterpret_cast<const u32x4*>(x + k + 16 * g) : zero;
    acc = mfma_i8(wv, xv, acc);
  }
  if (m >= t.end) return;
  const float xs = has ? a.Xs[src] : 0.f;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int n = n0 + 4 * g + r;
    if (n >= a.N) continue;
    float y = (float)acc[r] * xs * a.Ws[(int64_t)t.e * a.N + n];
    if (a.bias) y += bf16_to_f32(a.bias[n]);
    a.Y[(int64_t)m * a.N + n] = f32_to_bf16(y);
  }
}

}  // namespace

hipError_t launch_int8_gemm(const Int8GemmArgs& a, hipStream_t s) {
  const int64_t gx = (a.N + 63) / 64, gy = row_tiles(a.offsets != nullptr, a.T, a.E, 16);
  if (too_many(gx * gy, 256)) return hipErrorInvalidConfiguration;
  return launch(k_int8_simple, dim3((unsigned)(gx * gy)), 256, 0, s, a, (int)gx, (int)gy);
}

}  // namespace wq
