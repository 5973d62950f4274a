// Weighted sum of the experts' rows at each token.
#include <type_traits>

#include "wq_experts_internal.hpp"
#include "wq_row_tiles.hpp"
#include "wq_rows.hpp"

namespace wq {

namespace {

constexpr int kCols = 512;  // columns of a wave, 8 to a lane
constexpr int64_t kInfinityCache = (int64_t)256 << 20;

typedef __attribute__((ext_vector_type(4), aligned(2))) uint32_t u32x4_any;  // rows of an odd width start anywhere

// A wave owns kCols columns of one token and adds up its rows in registers, AHEAD
// of them under way at once.  Places and weights are the wave's, so that a row
// is one descriptor, of no bytes for a choice without a place.  Bound by memory:
// 8192 x 8 rows of 4096 and a base, 672 MB, in 106 us, 6.3 TB/s.
//   AHEAD: 4 where there are no more choices (16 x 4 of 2048: 2.5 us, 2.9 with 8),
//     else 8; one row after the other took 7.8 us for 512 x 8 of 4096, 6.8 so
//   STREAM: rows are read past the caches' replacement.  Y larger than the
//     Infinity Cache (256 MB) has left it since it was written and would push out
//     what is still of use: 130 -> 106 us at 537 MB.  Smaller it is there: 8192 x 2 of
//     4096, 134 MB, 31.8 us, 36.3 as a stream.
//   WHOLE: N % 8 == 0.  Rows of other widths start anywhere; 16-byte accesses take
//     that (2048 x 8 of 5003: 36 us, 72 element by element)
template <bool WHOLE, int AHEAD, bool STREAM>
__global__ __launch_bounds__(256) void k_combine(CombineArgs a, int pieces, uint32_t waves) {
  const uint32_t w = blockIdx.x * 4u + (uint32_t)__builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  if (w >= waves) return;
  const int lane = threadIdx.x & 63;
  const int m = (int)(w / (uint32_t)pieces);
  const int64_t N = a.N, n0 = (int64_t)(w % (uint32_t)pieces) * kCols, n = n0 + 8 * lane;
  const int32_t* places = a.places + (int64_t)m * a.top;
  const float* weights = a.weights + (int64_t)m * a.top;
  const uint16_t* base = a.base ? a.base + (int64_t)m * N : nullptr;
  uint16_t* out = a.out + (int64_t)m * N;
  if (WHOLE ? n < N : n + 8 <= N) {
    u32x4 b = {0, 0, 0, 0};
    if (base) b = WHOLE ? *reinterpret_cast<const u32x4*>(base + n) : *reinterpret_cast<const u32x4_any*>(base + n);
    F8 sum{};
    for (int j0 = 0; j0 < a.top; j0 += AHEAD) {
      u32x4 y[AHEAD];
      float f[AHEAD];
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        const int p = j0 + j < a.top ? places[j0 + j] : -1;
        const bool has = (uint32_t)p < (uint32_t)a.T;
        const __amdgpu_buffer_rsrc_t row = make_rsrc(a.Y + (has ? (int64_t)p : 0) * N + n0, has ? (uint32_t)min(N - n0, (int64_t)kCols) * 2u : 0u);
        y[j] = STREAM ? bload128_nt(row, 16u * (uint32_t)lane) : bload128(row, 16u * (uint32_t)lane);
        f[j] = has ? weights[j0 + j] : 0.f;
      }
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        const F8 v = unpack8(y[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum.v[i] = __builtin_fmaf(f[j], v.v[i], sum.v[i]);
      }
    }
    const F8 v = unpack8(b);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum.v[i] += v.v[i];
    const u32x4 r = pack8(sum);
    if constexpr (WHOLE) *reinterpret_cast<u32x4*>(out + n) = r;
    else *reinterpret_cast<u32x4_any*>(out + n) = r;
  } else if (!WHOLE) {
    for (int64_t c = n; c < N; ++c) {  // fewer than 8, of one lane
      float sum = 0.f;
      for (int j = 0; j < a.top; ++j) {
        const int p = places[j];
        if ((uint32_t)p < (uint32_t)a.T) sum = __builtin_fmaf(weights[j], bf16_to_f32(a.Y[(int64_t)p * N + c]), sum);
      }
      out[c] = f32_to_bf16(base ? sum + bf16_to_f32(base[c]) : sum);
    }
  }
}

}  // namespace

hipError_t launch_combine(const CombineArgs& a, hipStream_t s) {
  const int64_t pieces = (a.N + kCols - 1) / kCols, waves = pieces * a.M, groups = (waves + 3) / 4;
  if (too_many(groups, 256)) return hipErrorInvalidConfiguration;
  const bool stream = (int64_t)a.T * a.N * 2 > kInfinityCache;
  auto pick = [&](auto ahead, auto past) {
    constexpr int A = decltype(ahead)::value;
    constexpr bool S = decltype(past)::value;
    return a.N % 8 ? k_combine<false, A, S> : k_combine<true, A, S>;
  };
  using Four = std::integral_constant<int, 4>;
  using Eight = std::integral_constant<int, 8>;
  const auto kern = a.top <= 4 ? (stream ? pick(Four{}, std::true_type{}) : pick(Four{}, std::false_type{}))
                               : (stream ? pick(Eight{}, std::true_type{}) : pick(Eight{}, std::false_type{}));
  return launch(kern, dim3((unsigned)groups), 256, 0, s, a, (int)pieces, (uint32_t)waves);
}

}  // namespace wq
