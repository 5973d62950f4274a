// Internal launch interface of the experts' routing (wq_experts_api.hip to
// wq_experts_route.hip and wq_experts_combine.hip).  Launchers assume their
// arguments were validated by the ABI layer.
#pragma once

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
  int32_t* counts;  // workspace: choices of each stretch of tokens by expert
  int M, E, top, groups, keep;
  float scale;
  bool half, sigmoid, pairs, renormalize;
};

// Tokens in stretches, one to a workgroup: `passes` times kPassTokens each.
constexpr int kPassTokens = 64, kMaxStretches = 256;
struct Stretches {
  int passes, count;
};
inline Stretches stretches(int64_t M) {
  const int64_t all = (M + kPassTokens - 1) / kPassTokens;
  const int64_t passes = all ? (all + kMaxStretches - 1) / kMaxStretches : 1;
  return {(int)passes, (int)((all + passes - 1) / passes)};
}

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
