// 8-bit integer quantizers: activation rows, gated activation, weights (whose
// rows are the output channels).  One scale a row, so a row belongs to WPR waves
// and stays in their registers from its one read to its one write: lane l of
// wave w holds chunks w * 64 + l + 64 * WPR * j (8 elements each) for j < CPT.
// The row's maximum goes round a wave's lanes by shuffles and round the waves
// through LDS.
#include "wq_int8_internal.hpp"
#include "wq_row_tiles.hpp"
#include "wq_rows.hpp"

namespace wq {

namespace {

constexpr float kTiny = 1.17549435e-38f;  // 2^-126, the floor of a scale

template <int WPR>
constexpr int rows_per_group() {  // four waves or one row
  return WPR >= 3 ? 1 : 4 / WPR;
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, d));
  return v;
}

// max over a row's WPR waves, whose maxima lie in part[first ..]
template <int WPR>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* part, int wave, int lane) {
  v = wave_max(v);
  if constexpr (WPR > 1) {
    if (lane == 0) part[wave] = v;
    __syncthreads();
    const int first = wave / WPR * WPR;
    v = part[first];
#pragma unroll
    for (int w = 1; w < WPR; ++w) v = max(v, part[first + w]);
  }
  return v;
}

struct RowScale {
  float s, inv, rest;  // inv + rest = 1 / s to some 48 bits
  bool bad;            // an infinity or a NaN among the row
};
__device__ __forceinline__ RowScale row_scale(uint32_t amax_bits) {
  RowScale r;
  r.bad = amax_bits >= 0x7F800000u;
  r.s = bitsf(r.bad ? 0 : amax_bits) / 127.0f;
  r.s = r.s < kTiny ? kTiny : r.s;
  r.inv = 1.0f / r.s;
  r.rest = __builtin_fmaf(-r.s, r.inv, 1.0f) * r.inv;
  return r;
}

// Codes of y / s, the quotient IEEE division's but for rare last bits, at a third of its
// instructions: y * (1 / s) and one correction by its remainder, or, of gated rows, y times
// 1 / s in two parts, one instruction less (4096 x 5632: 20.4 us, 21.0).  (Of bf16 rows a
// thousandth of the quotients are within an ulp of a tie: y * (1 / s) alone takes two in three
// of those to the other side.  Of 23 million gated values 11 have another code by it than the
// fp32 formula gives, 3 so; it saves 0.9 us.)  Adding 1.5 * 2^23 rounds to a whole number,
// ties to even, whose low byte is the sum's.  |y / s| < 127.5 by the choice of s.
template <bool GATE>
__device__ __forceinline__ u32x2 codes8(const F8& y, const RowScale& r) {
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (GATE) {
      b[i] = fbits(__builtin_fmaf(y.v[i], r.inv, y.v[i] * r.rest) + 12582912.0f);
    } else {
      const float v = y.v[i] * r.inv;
      b[i] = fbits(__builtin_fmaf(__builtin_fmaf(-v, r.s, y.v[i]), r.inv, v) + 12582912.0f);
    }
  }
  u32x2 w;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = __builtin_amdgcn_perm(b[4 * h + 1], b[4 * h], 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(b[4 * h + 3], b[4 * h + 2], 0x04000C0Cu);
    w[h] = r.bad ? 0u : lo | hi;
  }
  return w;
}

// silu(g) u = g / (1 + exp(-g)) u of a bf16 gate, within 10 2^-24 of itself (all 65536 gates: 2.3 ulp of
// silu at most, 0.075 on average; fp32's exp, sum and quotient 1.75 and 0.063).
//   exp(-g) = 2^(-g L) (1 - g C), L = log2 e cut to 16 bits, so that its product with the 8 bits of g is exact
//     and 2^x gets its argument unrounded; C = (log2 e - L) ln 2, and (g C)^2 / 2, less than 1.6 2^-24, is left out
//   the quotient is g' / d' with g' = 2^-8 g, d' = 2^-8 (1 + exp(-g)), on the hardware's reciprocal (an ulp): it
//     reads reciprocals below 2^-126 as 0, and d' stays below 2^120
// Below -88.72 exp(-g) leaves fp32 and the result is -0, as the formula has it there.  Infinite gates may give
// NaN for an infinity: their row holds neither codes nor a scale.  4096 x 5632 20.4 us; with one rounding of the
// exponent (up to 55 ulp off) 18.8, with the quotient corrected by its remainder (1 code in 23 million differs
// from the formula's, 3 so) 21.6, by expf and division 32.
__device__ __forceinline__ float silu_mul(float g, float u) {
  constexpr float L = 369.328125f, C = 0.00125145476f;  // 2^8 times the constants above
  const float n = g * 0.00390625f;
  const float p = __builtin_amdgcn_exp2f(n * -L);
  const float e = __builtin_fmaf(p, n * -C, p);
  return n * __builtin_amdgcn_rcpf(__builtin_fmaf(e, 0.00390625f, 0.00390625f)) * u;
}

__device__ __forceinline__ float stored(const RowScale& r) { return r.bad ? __builtin_nanf("") : r.s; }

// Bound by memory: 8192 x 8192 in 29.4 us (6.8 TB/s), gated 61.6 (5.45 TB/s), 4096 x 5632 gated 20.5 (5.6 TB/s); a few
// rows by the launch and one trip to memory, 2.6 us.
template <bool GATE, int WPR, int CPT>
__global__ __launch_bounds__(rows_per_group<WPR>() * WPR * 64) void k_int8_rows(const uint16_t* X, int64_t ldx, int M,
                                                                                int K, uint8_t* Xq, float* Xs) {
  constexpr int RPW = rows_per_group<WPR>();
  __shared__ uint32_t part[RPW * WPR];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int64_t row = (int64_t)blockIdx.x * RPW + wave / WPR;
  const bool live = row < M;
  const int64_t m = live ? row : 0;
  const uint32_t bytes = live ? (uint32_t)K * 2u : 0u;
  const __amdgpu_buffer_rsrc_t Xr = make_rsrc(X + m * ldx, bytes);
  const __amdgpu_buffer_rsrc_t Ur = make_rsrc(X + m * ldx + (GATE ? K : 0), bytes);
  const uint32_t c0 = (uint32_t)((wave % WPR) * 64 + lane);

  u32x4 xw[CPT], uw[CPT];
#pragma unroll
  for (int j = 0; j < CPT; ++j) xw[j] = bload128(Xr, (c0 + 64u * WPR * j) * 16u);  // past the row: zeros
  if constexpr (GATE) {
#pragma unroll
    for (int j = 0; j < CPT; ++j) uw[j] = bload128(Ur, (c0 + 64u * WPR * j) * 16u);
  }
  F8 y[CPT];
  uint32_t amax = 0;
#pragma unroll
  for (int j = 0; j < CPT; ++j) {
    y[j] = unpack8(xw[j]);
    if constexpr (GATE) {
      const F8 u = unpack8(uw[j]);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[j].v[i] = silu_mul(y[j].v[i], u.v[i]);
    }
    amax = max(amax, absmax8(y[j]));
  }
  const RowScale r = row_scale(row_max<WPR>(amax, part, wave, lane));
#pragma unroll
  for (int j = 0; j < CPT; ++j) {
    const uint32_t c = c0 + 64u * WPR * j;
    if (live && c * 8u < (uint32_t)K) *reinterpret_cast<u32x2*>(Xq + m * K + c * 8u) = codes8<GATE>(y[j], r);
  }
  if (live && c0 == 0) Xs[m] = stored(r);
}

// Rows too long for the registers of 16 waves: read twice.
template <bool GATE>
__global__ __launch_bounds__(1024) void k_int8_long_rows(const uint16_t* X, int64_t ldx, int K, uint8_t* Xq, float* Xs) {
  __shared__ uint32_t part[16];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int64_t m = blockIdx.x;
  const uint16_t* x = X + m * ldx;
  auto at = [&](int k) {
    F8 y = unpack8(*reinterpret_cast<const u32x4*>(x + k));
    if constexpr (GATE) {
      const F8 u = unpack8(*reinterpret_cast<const u32x4*>(x + K + k));
#pragma unroll
      for (int i = 0; i < 8; ++i) y.v[i] = silu_mul(y.v[i], u.v[i]);
    }
    return y;
  };
  uint32_t amax = 0;
  for (int k = 8 * (int)threadIdx.x; k < K; k += 8192) amax = max(amax, absmax8(at(k)));
  const RowScale r = row_scale(row_max<16>(amax, part, wave, lane));
  for (int k = 8 * (int)threadIdx.x; k < K; k += 8192) *reinterpret_cast<u32x2*>(Xq + m * K + k) = codes8<GATE>(at(k), r);
  if (threadIdx.x == 0) Xs[m] = stored(r);
}

template <bool GATE, int WPR, int CPT>
hipError_t rows_launch(const uint16_t* X, int64_t ldx, int64_t M, int64_t K, uint8_t* Xq, float* Xs, hipStream_t s) {
  constexpr int rows = rows_per_group<WPR>(), threads = rows * WPR * 64;
  const int64_t groups = (M + rows - 1) / rows;
  if (too_many(groups, threads)) return hipErrorInvalidConfiguration;
  return launch(k_int8_rows<GATE, WPR, CPT>, dim3((unsigned)groups), threads, 0, s, X, ldx, (int)M, (int)K, Xq, Xs);
}

template <bool GATE>
hipError_t quant_rows(const uint16_t* X, int64_t ldx, int64_t M, int64_t K, uint8_t* Xq, float* Xs, hipStream_t s) {
  // the narrowest form that holds a row: one chunk to a lane in up to 8 waves, then two, then four
  const int64_t chunks = K / 8;
  if (chunks <= 64) return rows_launch<GATE, 1, 1>(X, ldx, M, K, Xq, Xs, s);
  if (chunks <= 128) return rows_launch<GATE, 2, 1>(X, ldx, M, K, Xq, Xs, s);
  if (chunks <= 192) return rows_launch<GATE, 3, 1>(X, ldx, M, K, Xq, Xs, s);
  if (chunks <= 256) return rows_launch<GATE, 4, 1>(X, ldx, M, K, Xq, Xs, s);
  if (chunks <= 384) return rows_launch<GATE, 6, 1>(X, ldx, M, K, Xq, Xs, s);
  if (chunks <= 512) return rows_launch<GATE, 4, 2>(X, ldx, M, K, Xq, Xs, s);
  if (chunks <= 768) return rows_launch<GATE, 6, 2>(X, ldx, M, K, Xq, Xs, s);
  if (chunks <= 1024) return rows_launch<GATE, 8, 2>(X, ldx, M, K, Xq, Xs, s);
  if (chunks <= 2048) return rows_launch<GATE, 16, 2>(X, ldx, M, K, Xq, Xs, s);
  if (chunks <= 4096) return rows_launch<GATE, 16, 4>(X, ldx, M, K, Xq, Xs, s);
  if (too_many(M, 1024)) return hipErrorInvalidConfiguration;
  return launch(k_int8_long_rows<GATE>, dim3((unsigned)M), 1024, 0, s, X, ldx, (int)K, Xq, Xs);
}

}  // namespace

hipError_t launch_int8_quant_rows(bool gate, const uint16_t* X, int64_t ldx, int64_t M, int64_t K, uint8_t* Xq,
                                  float* Xs, hipStream_t s) {
  return gate ? quant_rows<true>(X, ldx, M, K, Xq, Xs, s) : quant_rows<false>(X, ldx, M, K, Xq, Xs, s);
}

}  // namespace wq
