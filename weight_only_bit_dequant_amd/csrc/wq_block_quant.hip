// Block-scaled FP8 quantizers and the operators that end in one: activation
// rows, residual addition + RMS norm, gated activation, weights.
//
// All of them read bf16 and write E4M3 codes with one fp32 scale for 128
// elements along K, so a 16-lane row of a wave is one scale block: each lane
// holds 8 consecutive elements (one 16-byte load, one 8-byte store of codes)
// and the block's maximum goes round the 16 lanes by DPP row rotations,
// without LDS.
#include "wq_block_internal.hpp"
#include "wq_kernel_common.hpp"

namespace wq {

namespace {

constexpr float kTiny = 1.17549435e-38f;  // 2^-126, the floor of a scale

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

// max of v over the 16 lanes of a DPP row (rotations by 8, 4, 2, 1)
__device__ __forceinline__ uint32_t max_row16(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xF, 0xF, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xF, 0xF, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xF, 0xF, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xF, 0xF, true));
  return v;
}

// max |y| as an integer: the bits of nonnegative floats are in their order,
// and a NaN's lie above infinity's, so a NaN is the largest.
__device__ __forceinline__ uint32_t absmax8(const F8& y) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, fbits(y.v[i]) & 0x7FFFFFFFu);
  return m;
}

__device__ __forceinline__ float block_scale(uint32_t amax_bits) {
  const float s = bitsf(amax_bits) / 448.0f;
  return s < kTiny ? kTiny : s;  // a NaN stays
}

// E4M3 codes of y / s, the quotient as y * (1 / s) and one correction by its
// remainder: IEEE division's result but for rare last bits, at a third of its
// instructions.  (y * (1 / s) alone rounds four times as many codes to the
// other neighbour as the fp32 definition does.)  |y / s| <= 448 by the choice
// of s, so nothing is clamped.  Over an infinite s the quotient is y * 0 already
// (a zero, NaN for an infinite y): its remainder, 0 * s off, would be NaN for all.
__device__ __forceinline__ u32x2 codes8(const F8& y, float s) {
  const float inv = 1.0f / s, back = s < __builtin_inff() ? s : 0.0f;
  F8 q;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float v = y.v[i] * inv;
    q.v[i] = __builtin_copysignf(__builtin_fmaf(__builtin_fmaf(-v, back, y.v[i]), inv, v), v);  // (-0 would become 0)
  }
  return u32x2{e4m3_pack4(q.v[0], q.v[1], q.v[2], q.v[3]), e4m3_pack4(q.v[4], q.v[5], q.v[6], q.v[7])};
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

// ---------------------------------------------------------------- activation rows, gated activation
// One lane per 8 elements, one 16-lane row per scale block; the blocks of all
// rows are numbered through, so short rows share a workgroup.  Bound by memory:
// the gate over 8192 x 8192 moves its 338 MB in 63 to 67.5 us, 5.0 to 5.3 TB/s (a
// copy of that size 4.8); non-temporal loads, 512 threads and two blocks to a lane were
// no faster.  64 x 2048 takes 2.6 us, 1 above an empty launch: one trip.
// The row of a block is blk / KB as a product: with 2^sh < KB <= 2^(sh + 1) and
// magic = ceil(2^(32 + sh) / KB), exact for blk < 2^31 (KB = 1: magic = 0).
template <bool GATE>
__global__ __launch_bounds__(256) void k_block_quant_rows(const uint16_t* __restrict__ X, int64_t ldx, uint32_t nblk,
                                                          uint32_t KB, uint32_t magic, uint32_t sh, uint32_t K,
                                                          uint8_t* __restrict__ Xq, float* __restrict__ Xs) {
  const uint32_t blk = blockIdx.x * 16u + (threadIdx.x >> 4);
  if (blk >= nblk) return;  // whole 16-lane rows leave together
  const uint32_t m = magic ? __umulhi(blk, magic) >> sh : blk, k = (blk - m * KB) * 128u + (threadIdx.x & 15u) * 8u;
  const bool in = k < K;  // K % 16 == 0: a lane's 8 elements are inside or outside together
  F8 y{};
  if (in) {
    const uint16_t* p = X + (int64_t)m * ldx + k;
    const F8 x = unpack8(*reinterpret_cast<const u32x4*>(p));
    if constexpr (GATE) {
      const F8 u = unpack8(*reinterpret_cast<const u32x4*>(p + K));
#pragma unroll
      for (int i = 0; i < 8; ++i) y.v[i] = silu_mul(x.v[i], u.v[i]);
    } else {
      y = x;
    }
  }
  const float s = block_scale(max_row16(absmax8(y)));
  if (in) {
    *reinterpret_cast<u32x2*>(Xq + (int64_t)m * K + k) = codes8(y, s);
    if ((threadIdx.x & 15u) == 0) Xs[blk] = s;
  }
}

// ---------------------------------------------------------------- residual addition + RMS norm
// A row belongs to WPR waves and stays in their registers from its one read to
// its one write: lane l of wave w holds chunks w * 64 + l + 64 * WPR * j
// (8 elements each) for j < CPT, so its 16-lane rows are scale blocks.  The
// sum of squares crosses lanes by shuffles and waves through LDS.  Bound by
// memory: 16384 x 8192 moves 941 MB in 160 to 164 us, 5.7 to 5.9 TB/s (a copy 4.8; two passes
// over a row would read 537 MB again); a row of 4096 takes 2.6 to 3.0 us, one trip and
// one meeting of its waves above an empty launch (1.6 us).
template <int WPR>
constexpr int norm_rows() {  // rows per workgroup: four waves or one row
  return WPR >= 3 ? 1 : 4 / WPR;
}

template <int WPR, int CPT>
__global__ __launch_bounds__(norm_rows<WPR>() * WPR * 64) void k_block_norm(BlockNormArgs a) {
  constexpr int RPW = norm_rows<WPR>();
  __shared__ float part[RPW * WPR];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int64_t row = (int64_t)blockIdx.x * RPW + wave / WPR;
  const bool live = row < a.M;
  const int64_t m = live ? row : 0;
  const uint32_t K = (uint32_t)a.K, rb = live ? K * 2u : 0u;
  const __amdgpu_buffer_rsrc_t Xr = make_rsrc(a.X + m * a.ldx, rb);
  const __amdgpu_buffer_rsrc_t Rr = make_rsrc(a.residual ? a.residual + m * K : a.X, a.residual ? rb : 0u);
  const __amdgpu_buffer_rsrc_t Gr = make_rsrc(a.gain, K * 2u);
  const uint32_t c0 = (uint32_t)((wave % WPR) * 64 + lane);

  u32x4 xw[CPT], rw[CPT], gw[CPT];
#pragma unroll
  for (int j = 0; j < CPT; ++j) xw[j] = bload128(Xr, (c0 + 64u * WPR * j) * 16u);  // past the row: zeros
  if (a.residual) {
#pragma unroll
    for (int j = 0; j < CPT; ++j) rw[j] = bload128(Rr, (c0 + 64u * WPR * j) * 16u);
  }
#pragma unroll
  for (int j = 0; j < CPT; ++j) gw[j] = bload128(Gr, (c0 + 64u * WPR * j) * 16u);

  F8 h[CPT];
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < CPT; ++j) {
    h[j] = unpack8(xw[j]);
    if (a.residual) {
      const F8 r = unpack8(rw[j]);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[j].v[i] += r.v[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += h[j].v[i] * h[j].v[i];
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) ss += __shfl_xor(ss, d);
  if constexpr (WPR > 1) {
    if (lane == 0) part[wave] = ss;
    __syncthreads();
    ss = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) ss += part[wave / WPR * WPR + w];
  }
  const float rstd = 1.0f / sqrtf(ss / (float)a.K + a.eps);

  const uint32_t KB = (K + 127u) / 128u;
#pragma unroll
  for (int j = 0; j < CPT; ++j) {
    const uint32_t c = c0 + 64u * WPR * j;
    const bool in = live && c * 8u < K;
    const F8 g = unpack8(gw[j]);
    F8 y;
#pragma unroll
    for (int i = 0; i < 8; ++i) y.v[i] = h[j].v[i] * rstd * g.v[i];
    if (!in) y = F8{};  // a row of NaN or infinite rstd must not reach the tail lanes of its last block
    const float s = block_scale(max_row16(absmax8(y)));
    if (in) {
      if (a.residual_out) *reinterpret_cast<u32x4*>(a.residual_out + m * K + c * 8u) = pack8(h[j]);
      if (a.y_out) *reinterpret_cast<u32x4*>(a.y_out + m * K + c * 8u) = pack8(y);
      *reinterpret_cast<u32x2*>(a.Xq + m * K + c * 8u) = codes8(y, s);
      if ((lane & 15) == 0) a.Xs[m * KB + c / 16u] = s;
    }
  }
}

// ---------------------------------------------------------------- weights
// One workgroup per 128 x 128 block: 16 lanes read a row of it, 16 rows at a
// time.  Runs once per weight.
__global__ __launch_bounds__(256) void k_block_quant_weight(const uint16_t* __restrict__ W, int N, int K,
                                                            uint8_t* __restrict__ codes, float* __restrict__ scales) {
  __shared__ uint32_t part[4];
  const int kb = blockIdx.x, nb = blockIdx.y, KB = gridDim.x, NB = gridDim.y;
  const int64_t base = (int64_t)blockIdx.z * N * K;
  const int k = kb * 128 + (threadIdx.x & 15) * 8;
  F8 y[8];
  uint32_t amax = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int n = nb * 128 + 16 * j + (int)(threadIdx.x >> 4);
    y[j] = F8{};
    if (n < N && k < K) y[j] = unpack8(*reinterpret_cast<const u32x4*>(W + base + (int64_t)n * K + k));
    amax = max(amax, absmax8(y[j]));
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) amax = max(amax, (uint32_t)__shfl_xor((int)amax, d));
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = amax;
  __syncthreads();
  const float s = block_scale(max(max(part[0], part[1]), max(part[2], part[3])));
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int n = nb * 128 + 16 * j + (int)(threadIdx.x >> 4);
    if (n < N && k < K) *reinterpret_cast<u32x2*>(codes + base + (int64_t)n * K + k) = codes8(y[j], s);
  }
  if (threadIdx.x == 0) scales[((int64_t)blockIdx.z * NB + nb) * KB + kb] = s;
}

}  // namespace

hipError_t launch_block_quant_rows(bool gate, const uint16_t* X, int64_t ldx, int64_t M, int64_t K, uint8_t* Xq,
                                   float* Xs, hipStream_t s) {
  const uint32_t KB = (uint32_t)((K + 127) / 128), nblk = (uint32_t)M * KB;
  const unsigned grid = (nblk + 15u) / 16u;
  uint32_t sh = 0, magic = 0;
  if (KB > 1) {
    while ((2u << sh) < KB) ++sh;
    magic = (uint32_t)((((uint64_t)1 << (32 + sh)) + KB - 1) / KB);
  }
  return launch(gate ? k_block_quant_rows<true> : k_block_quant_rows<false>, dim3(grid), 256, 0, s, X, ldx, nblk, KB, magic,
                sh, (uint32_t)K, Xq, Xs);
}

template <int WPR, int CPT>
static hipError_t norm_launch(const BlockNormArgs& a, hipStream_t s) {
  constexpr int rows = norm_rows<WPR>();
  return launch(k_block_norm<WPR, CPT>, dim3((unsigned)((a.M + rows - 1) / rows)), rows * WPR * 64, 0, s, a);
}

hipError_t launch_block_norm(const BlockNormArgs& a, hipStream_t s) {
  // The narrowest form that holds a row: one chunk to a lane in up to 6 waves (rows to 3072), two in 4 to 8 (to 8192),
  // four above.  A row of 8192 in 8 waves x 2 chunks takes 163 us against 166 in 4 x 4 and 179 in 16 x 1 (16384 rows),
  // 3.7 against 4.3 us (64 rows).
  const int chunks = (a.K + 127) / 128 * 16;  // whole 16-lane rows
  if (chunks <= 64) return norm_launch<1, 1>(a, s);
  if (chunks <= 128) return norm_launch<2, 1>(a, s);
  if (chunks <= 192) return norm_launch<3, 1>(a, s);
  if (chunks <= 256) return norm_launch<4, 1>(a, s);
  if (chunks <= 384) return norm_launch<6, 1>(a, s);
  if (chunks <= 512) return norm_launch<4, 2>(a, s);
  if (chunks <= 768) return norm_launch<6, 2>(a, s);
  if (chunks <= 1024) return norm_launch<8, 2>(a, s);
  if (chunks <= 2048) return norm_launch<8, 4>(a, s);
  return norm_launch<16, 4>(a, s);
}

hipError_t launch_block_quant_weight(const uint16_t* W, int64_t E, int64_t N, int64_t K, uint8_t* codes,
                                     float* scales, hipStream_t s) {
  const dim3 grid((unsigned)((K + 127) / 128), (unsigned)((N + 127) / 128), (unsigned)E);
  return launch(k_block_quant_weight, grid, 256, 0, s, W, (int)N, (int)K, codes, scales);
}

}  // namespace wq
