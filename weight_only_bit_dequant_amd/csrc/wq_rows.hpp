// Elements of bf16 rows in a lane's registers: what the row operators of the
// 8-bit formats (block-scaled FP8, INT8) share.
#pragma once

#include "wq_kernel_common.hpp"

namespace wq {

struct F8 {
  float v[8];
};

__device__ __forceinline__ F8 unpack8(u32x4 w) {
  F8 f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f.v[2 * i] = bitsf(w[i] << 16);
    f.v[2 * i + 1] = bitsf(w[i] & 0xFFFF0000u);
  }
  return f;
}

__device__ __forceinline__ u32x4 pack8(const F8& f) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = (uint32_t)f32_to_bf16(f.v[2 * i]) | ((uint32_t)f32_to_bf16(f.v[2 * i + 1]) << 16);
  return w;
}

// max |y| as an integer: the bits of nonnegative floats are in their order,
// and a NaN's lie above infinity's, so a NaN is the largest.
__device__ __forceinline__ uint32_t absmax8(const F8& y) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, fbits(y.v[i]) & 0x7FFFFFFFu);
  return m;
}

}  // namespace wq
