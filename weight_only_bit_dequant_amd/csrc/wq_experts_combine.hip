// Weighted sum of the experts' rows at each token.
#include "wq_experts_internal.hpp"
#include "wq_row_tiles.hpp"
#include "wq_rows.hpp"

namespace wq {

namespace {

constexpr int kCols = 512;  // columns of a wave, 8 to a lane

// A wave owns kCols columns of one token.  VEC: whole 16-byte pieces; otherwise
// (N % 8 != 0, so that rows start anywhere) a lane's columns lie 64 apart.
template <bool VEC>
__global__ __launch_bounds__(256) void k_combine(CombineArgs a, int pieces, uint32_t waves) {
  const uint32_t w = blockIdx.x * 4u + (uint32_t)__builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  if (w >= waves) return;
  const int lane = threadIdx.x & 63;
  const int m = (int)(w / (uint32_t)pieces);
  const int64_t n0 = (int64_t)(w % (uint32_t)pieces) * kCols;
  const int32_t* places = a.places + (int64_t)m * a.top;
  const float* weights = a.weights + (int64_t)m * a.top;
  auto col = [&](int i) { return VEC ? n0 + 8 * lane + i : n0 + lane + 64 * i; };
  auto load = [&](const uint16_t* row) {
    F8 y{};
    if constexpr (VEC) {
      if (col(0) < a.N) y = unpack8(*reinterpret_cast<const u32x4*>(row + col(0)));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (col(i) < a.N) y.v[i] = bf16_to_f32(row[col(i)]);
    }
    return y;
  };
  F8 sum{};
  for (int j = 0; j < a.top; ++j) {
    const int p = places[j];
    if ((uint32_t)p >= (uint32_t)a.T) continue;
    const F8 y = load(a.Y + (int64_t)p * a.N);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum.v[i] = __builtin_fmaf(weights[j], y.v[i], sum.v[i]);
  }
  if (a.base) {
    const F8 b = load(a.base + (int64_t)m * a.N);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum.v[i] += b.v[i];
  }
  uint16_t* out = a.out + (int64_t)m * a.N;
  if constexpr (VEC) {
    if (col(0) < a.N) *reinterpret_cast<u32x4*>(out + col(0)) = pack8(sum);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col(i) < a.N) out[col(i)] = f32_to_bf16(sum.v[i]);
  }
}

}  // namespace

hipError_t launch_combine(const CombineArgs& a, hipStream_t s) {
  const int64_t pieces = (a.N + kCols - 1) / kCols, waves = pieces * a.M, groups = (waves + 3) / 4;
  if (too_many(groups, 256)) return hipErrorInvalidConfiguration;
  return launch(a.N % 8 ? k_combine<false> : k_combine<true>, dim3((unsigned)groups), 256, 0, s, a, (int)pieces, (uint32_t)waves);
}

}  // namespace wq
