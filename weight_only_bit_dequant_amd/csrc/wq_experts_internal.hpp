// Internal launch interface of the experts' routing (wq_experts_api.hip to
// wq_experts_route.hip and wq_experts_combine.hip).  Launchers assume their
// arguments were validated by the ABI layer.
#pragma once

#include <hip/hip_runtime.h>

#include "wq_block_internal.hpp"
#include "wq_experts.h"

namespace wq {

struct RouteArgs {
  const void* logits;
  int64_t ld;
  const float* bias;     // [E] or null
  const uint8_t* valid;  // [M] or null
  int32_t* ids;
  float* weights;
  int32_t* offsets;
  int32_t* rows;
  int32_t* places;
  uint16_t* counts;  // workspace: choices of each stretch of tokens by expert
  int M, E, top, groups, keep;
  float scale;
  bool half, sigmoid, pairs, renormalize;
};

// Tokens in stretches, one to a workgroup: `passes` times `span` tokens each, at
// most 2^16 - 64 in all (a stretch's counts have 16 bits).  Few tokens are spread
// over the chip, a wave to each; many share a wave.  Four waves to a workgroup, one
// to a SIMD, as long as the second launch has no more stretches to add up for it:
// 256 of 256 experts in groups 14.9 -> 11.5 us, 1000 15.2 -> 14.3, 900 of 60 10.2 -> 9.4.
constexpr int kWaves = 4, kFewSpan = 16, kSpan = 64, kMaxStretches = 256, kMaxPasses = 1023;
struct Stretches {
  int span, passes, count;
};
inline Stretches stretches(int64_t M) {
  if (M > kFewSpan && M <= kWaves * kMaxStretches) return {kWaves, 1, (int)((M + kWaves - 1) / kWaves)};
  if (M <= kFewSpan * kMaxStretches) return {kFewSpan, 1, M ? (int)((M + kFewSpan - 1) / kFewSpan) : 1};
  const int64_t all = (M + kSpan - 1) / kSpan, even = (all + kMaxStretches - 1) / kMaxStretches;
  const int64_t passes = even < kMaxPasses ? even : kMaxPasses;
  return {kSpan, (int)passes, (int)((all + passes - 1) / passes)};
}
// Counts of a stretch, whole words.
inline __host__ __device__ int counts_pitch(int E) { return (E + 1) & ~1; }

hipError_t launch_route(const RouteArgs& a, hipStream_t s);

struct CombineArgs {
  const uint16_t* Y;
  const int32_t* places;
  const float* weights;
  const uint16_t* base;  // or null
  uint16_t* out;
  int64_t N;
  int T, M, top;
};
hipError_t launch_combine(const CombineArgs& a, hipStream_t s);

}  // namespace wq
