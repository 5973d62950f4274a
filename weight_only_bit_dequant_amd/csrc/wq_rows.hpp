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

// silu(g) u = g / (1 + exp(-g)) u within a few fp32 ulp (of the fp32 formula's own
// rounding size; a code may fall to either side of a tie of both).
//   exp(-g) = 2^t, t = -g log2 e with the constant in two parts (Cody and
//   Waite's reduction), the hardware's 2^x for what is left beside a whole number;
//   the quotient is g' r with one correction by its remainder (a Newton step on
//   the quotient), r the hardware's reciprocal of d' (1 ulp).  d' = 2^-8 (1 + exp(-g)) and g' = 2^-8 g: r stays a
//   normal number up to the largest d (reciprocals below 2^-126 read as 0).
// Below -88.6 exp(-g) leaves fp32 and the result is -0 (its size is below
// 3e-37); above 90 exp(-g) no longer counts and the result is g.  Both are g
// times 0 or 1, so that +infinity stays one and -infinity (an infinity over an
// infinity) and NaN give NaN: the quotient's correction would make NaN of both
// infinities.
// Two library calls (expf and division) took 45 instructions an element, more
// than the memory's time (8192 x 8192: 75 us; so 63 to 67.5).
__device__ __forceinline__ float silu_mul(float g, float u) {
  constexpr float L = -1.4426950216293335f, Ll = -1.9259629911e-8f;  // -log2 e = L + Ll
  constexpr float far = -88.6f;
  const float x = __builtin_amdgcn_fmed3f(g, far, 90.0f);
  const float hi = x * L;
  const float lo = __builtin_fmaf(x, Ll, __builtin_fmaf(x, L, -hi));
  const float whole = __builtin_rintf(hi);
  const float e = __builtin_ldexpf(__builtin_amdgcn_exp2f((hi - whole) + lo), (int)whole);
  const float d = __builtin_fmaf(e, 0.00390625f, 0.00390625f), n = g * 0.00390625f;
  const float r = __builtin_amdgcn_rcpf(d);
  const float q = n * r;
  float v = __builtin_fmaf(__builtin_fmaf(-q, d, n), r, q);
  asm("" : "+v"(v));  // a select, not a branch around the quotient for each element
  return (x == g ? v : g * (g > 0.0f ? 1.0f : 0.0f)) * u;
}

}  // namespace wq
