// Routing of tokens to experts: scores, groups, the `top` largest choices with
// their weights, and the stable order of all choices by expert.
//
// L lanes of a wave hold a token's experts, q <= R of them each, in the order of
// the experts: the lowest index among equal choices is the lowest lane's lowest.
// With groups (a power of two of them, up to L) L / groups lanes hold a group.
// Choices are compared as integer keys in the order of the numbers: 0 for what
// cannot be picked, above it -max .. +infinity, above those NaN.  Without a bias
// the key is the logit's, exact; with one it is that of score + bias in fp64, so
// that choices next to each other are in the order of the definition (an fp32
// score is off by 2^-24, and one token in some thousand has choices that near).
//
// The order needs no atomics whose order counts: of each `span` tokens a bit mask
// of those that picked an expert gives every choice its rank among them (the bits
// below its own) and the expert its count.  A few tokens take one launch of one
// workgroup; more take two: the first writes counts of each stretch of tokens, in
// the second each workgroup adds up the counts before its own.
//
// What bounds it: 16384 tokens of 256 experts (sigmoid, bias, the best 4 of 8 groups)
// take 20 us in the first launch, instructions: of some 1500 for four tokens a third
// are the scores in fp64, a third the order in each lane and the eight picks (the next
// tokens' logits fetched ahead, four scores' chains side by side: no change).  The second
// takes 8 us, a few trips to memory.  By the logits alone the first takes 12 us.  One
// token takes 4.9 us, 2.5 of them the launch, one trip to memory, and the picks one
// after the other.
#include <type_traits>
#include <utility>

#include "wq_experts_internal.hpp"
#include "wq_row_tiles.hpp"

namespace wq {

namespace {

constexpr int kOrderThreads = 512;
constexpr uint16_t kNone = 0xFFFF;

// ---------------------------------------------------------------- keys

// Logits as integers in their order: 0 for -infinity (not to be picked), above
// it -max .. +infinity, above those NaN.
struct Narrow {
  typedef uint32_t T;
  static constexpr T kNot = 0;
  __device__ __forceinline__ static T of(float c) {
    const uint32_t u = fbits(c + 0.0f);  // -0 is 0
    return c != c ? ~0u : c == -__builtin_inff() ? 0u : u ^ (uint32_t)(((int32_t)u >> 31) | (int32_t)0x80000000);
  }
  __device__ __forceinline__ static float logit(T k) {
    return k == ~0u ? __builtin_nanf("") : k == 0 ? -__builtin_inff() : bitsf(k ^ (k >> 31 ? 0x80000000u : ~0u));
  }
  __device__ __forceinline__ static T max(T a, T b) { return a > b ? a : b; }
  __device__ __forceinline__ static T min(T a, T b) { return a < b ? a : b; }
  __device__ __forceinline__ static T sum(T a, T) { return a; }  // (pairs are never narrow)
};
// Choices as fp64 numbers: what is not to be picked, +infinity and NaN are powers of
// two (2^1010, negative, 2^1000 and 2^1010; choices of fp32 biases are far below them).
struct Wide {
  typedef double T;
  static constexpr T kNaN = 0x1p1010, kNot = -kNaN, kMost = 0x1p1000;
  // (the instructions themselves: the compiler's fmax first makes each operand that might be a signalling NaN a quiet one)
  __device__ __forceinline__ static T max(T a, T b) {
    asm("v_max_f64 %0, %1, %2" : "=v"(a) : "v"(a), "v"(b));
    return a;
  }
  __device__ __forceinline__ static T min(T a, T b) {
    asm("v_min_f64 %0, %1, %2" : "=v"(a) : "v"(a), "v"(b));
    return a;
  }
  __device__ __forceinline__ static T of(double c) {
    const double m = max(min(c, kMost), kNot);
    return c != c ? kNaN : m;
  }
  __device__ __forceinline__ static T sum(T a, T b) {  // of a group's two largest, a >= b
    return b == kNot ? a : a > kMost ? a : min(a + b, kMost);
  }
};

// Choices with their expert's number in the low BITS bits (the lowest expert the largest): no two experts' are equal, and
// the number comes with the choice through maxima and sorting.  Choices that differ in those bits alone are told apart
// afterwards (`unsure` below).
template <int BITS>
struct Numbered {
  static constexpr uint32_t MASK = (1u << BITS) - 1;
  // (of negative numbers the smallest number is the largest)
  __device__ __forceinline__ static uint32_t turned(u32x2 u) { return (uint32_t)((int32_t)u.y >> 31); }
  __device__ __forceinline__ static double of(double c, int e) {
    u32x2 u = __builtin_bit_cast(u32x2, c);
    u.x = (u.x & ~MASK) | (~((uint32_t)e ^ turned(u)) & MASK);
    return __builtin_bit_cast(double, u);
  }
  __device__ __forceinline__ static int expert(double v) {
    const u32x2 u = __builtin_bit_cast(u32x2, v);
    return (int)(~(u.x ^ turned(u)) & MASK);
  }
  __device__ __forceinline__ static double choice(double v) {
    u32x2 u = __builtin_bit_cast(u32x2, v);
    u.x &= ~MASK;
    return __builtin_bit_cast(double, u);
  }
};

// The D largest of R numbers, in descending order, in v[0 .. D): blocks of D by Batcher's odd-even merge sort, then
// each next block's largest: of two ordered blocks the larger of v[i] and w[D - 1 - i], a bitonic sequence, merged.
template <int R, int D>
__device__ __forceinline__ void largest(double (&v)[R]) {
  auto order = [&](int i, int j) {
    const double a = v[i], b = v[j];
    v[i] = Wide::max(a, b);
    v[j] = Wide::min(a, b);
  };
#pragma unroll
  for (int b = 0; b < R; b += D) {
#pragma unroll
    for (int p = 1; p < D; p *= 2)
#pragma unroll
      for (int k = p; k >= 1; k /= 2)
#pragma unroll
        for (int i = 0; i + k < D; ++i)
          if (i % (2 * k) >= k % p && (i - k % p) % (2 * k) < k && i / (2 * p) == (i + k) / (2 * p)) order(b + i, b + i + k);
    if (b == 0) continue;
#pragma unroll
    for (int i = 0; i < D; ++i) v[i] = Wide::max(v[i], v[b + D - 1 - i]);
#pragma unroll
    for (int k = D / 2; k >= 1; k /= 2)
#pragma unroll
      for (int i = 0; i < D; ++i)
        if (!(i & k)) order(i, i | k);
  }
}

// ---------------------------------------------------------------- across lanes

// The two largest keys, of n lanes.
template <class K>
struct Two {
  typename K::T a, b;
  __device__ __forceinline__ void add(typename K::T k) {
    b = K::max(b, K::min(a, k));
    a = K::max(a, k);
  }
};
// The value of another lane: DPP within a row of 16 lanes.
template <int CTRL, typename T>
__device__ __forceinline__ T dpp(T v) {
  if constexpr (sizeof(T) == 8) {
    const u32x2 u = __builtin_bit_cast(u32x2, v);
    return __builtin_bit_cast(T, u32x2{(uint32_t)__builtin_amdgcn_update_dpp(0, (int)u.x, CTRL, 0xF, 0xF, true),
                                       (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u.y, CTRL, 0xF, 0xF, true)});
  } else {
    return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
  }
}
template <int CTRL, class K>
__device__ __forceinline__ Two<K> dpp(Two<K> v) {
  return {dpp<CTRL>(v.a), dpp<CTRL>(v.b)};
}
// f(1) .. f(15), as constants.
template <typename F, int... I>
__device__ __forceinline__ void unroll_of(F f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I + 1>{}), ...);
}
template <typename F>
__device__ __forceinline__ void unroll16(F f) {
  unroll_of(f, std::make_integer_sequence<int, 15>{});
}
template <typename T>
__device__ __forceinline__ T read_lane(T v, int lane) {
  if constexpr (sizeof(T) == 8) {
    const u32x2 u = __builtin_bit_cast(u32x2, v);
    return __builtin_bit_cast(T, u32x2{(uint32_t)__builtin_amdgcn_readlane((int)u.x, lane), (uint32_t)__builtin_amdgcn_readlane((int)u.y, lane)});
  } else {
    return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
  }
}
// v and its counterpart of the other half of 32 (HALF = 16) or 64 (32) lanes, in both halves alike.
template <int HALF, typename T>
__device__ __forceinline__ void halves(T v, T& a, T& b) {
  auto one = [](uint32_t x, uint32_t& p, uint32_t& q) {
    const auto r = HALF == 16 ? __builtin_amdgcn_permlane16_swap(x, x, false, false) : __builtin_amdgcn_permlane32_swap(x, x, false, false);
    p = r[0], q = r[1];
  };
  if constexpr (sizeof(T) == 8) {
    const u32x2 u = __builtin_bit_cast(u32x2, v);
    uint32_t p[2], q[2];
    one(u.x, p[0], q[0]);
    one(u.y, p[1], q[1]);
    a = __builtin_bit_cast(T, u32x2{p[0], p[1]});
    b = __builtin_bit_cast(T, u32x2{q[0], q[1]});
  } else {
    uint32_t p, q;
    one(__builtin_bit_cast(uint32_t, v), p, q);
    a = __builtin_bit_cast(T, p);
    b = __builtin_bit_cast(T, q);
  }
}
template <int HALF, class K>
__device__ __forceinline__ void halves(Two<K> v, Two<K>& a, Two<K>& b) {
  halves<HALF>(v.a, a.a, b.a);
  halves<HALF>(v.b, a.b, b.b);
}
// op over the n lanes (a power of two) that share lane / n, in all of them.
template <typename T, typename F>
__device__ __forceinline__ T over(T v, int n, F op) {
  if (n > 1) v = op(v, dpp<0xB1>(v));   // lane ^ 1
  if (n > 2) v = op(v, dpp<0x4E>(v));   // lane ^ 2
  if (n > 4) v = op(v, dpp<0x141>(v));  // mirrored in 8
  if (n > 8) v = op(v, dpp<0x140>(v));  // mirrored in 16
  T a, b;
  if (n > 16) halves<16>(v, a, b), v = op(a, b);
  if (n > 32) halves<32>(v, a, b), v = op(a, b);
  return v;
}
template <class K>
__device__ __forceinline__ typename K::T max_over(typename K::T v, int n) {
  return over(v, n, [](auto a, auto b) { return K::max(a, b); });
}
template <typename T>
__device__ __forceinline__ T sum_over(T v, int n) {
  return over(v, n, [](T a, T b) { return a + b; });
}

// What makes a group's value, of its n lanes' two largest: the two largest of all, or the largest and none.
template <class K>
__device__ __forceinline__ Two<K> best_over(Two<K> t, int n, bool pairs) {
  if (!pairs) return {max_over<K>(t.a, n), K::kNot};
  return over(t, n, [](Two<K> x, Two<K> y) { return Two<K>{K::max(x.a, y.a), K::max(K::min(x.a, y.a), K::max(x.b, y.b))}; });
}
template <class K>
__device__ __forceinline__ typename K::T group_value(Two<K> t, int n, bool pairs) {
  const Two<K> r = best_over<K>(t, n, pairs);
  return K::sum(r.a, r.b);
}

// ---------------------------------------------------------------- fp64 scores

// exp(x), -800 <= x <= 800 (beyond fp64's range 0 and infinity): x = n ln 2 + r, |r| <= ln 2 / 2, ln 2 in two parts
// (Cody and Waite's reduction), exp(r) by its series to r^12 / 12! (the rest is below 2^-52), times 2^n.  The library's
// takes twice the instructions, and 16 scores a lane are most of this kernel's.
__device__ __forceinline__ double exp64(double x) {
  const double n = __builtin_rint(x * 1.4426950408889634);
  const double r = __builtin_fma(n, -1.9082149292705877e-10, __builtin_fma(n, -0.6931471803691238, x));
  // (the multiply-add as an instruction: the compiler's takes each constant into the result's registers first)
  auto step = [&](double p, double k) {
    asm("v_fma_f64 %0, %1, %2, %3" : "=v"(p) : "v"(p), "v"(r), "s"(k));
    return p;
  };
  double p = 1.0 / 479001600.0;
  constexpr double c[] = {1.0 / 39916800.0, 1.0 / 3628800.0, 1.0 / 362880.0, 1.0 / 40320.0, 1.0 / 5040.0, 1.0 / 720.0,
                          1.0 / 120.0,      1.0 / 24.0,      1.0 / 6.0,      0.5,           1.0,          1.0};
#pragma unroll
  for (double k : c) p = step(p, k);
  return __builtin_ldexp(p, (int)n);
}
// c ? a : b without a branch around what a takes, or an index of c.
__device__ __forceinline__ double either(bool c, double a, double b) {
  asm("" : "+v"(a));
  asm("" : "+v"(b));
  return c ? a : b;
}
// 1 / (1 + exp(-l)) of a number, the same for all below kFar, where exp(-l) leaves fp64's range.  The reciprocal is the
// hardware's with two Newton steps.
constexpr float kFar = -709.78265f;  // the last fp32 number above -1024 ln 2
__device__ __forceinline__ double sigmoid_of_number(float l) {
  const double d = 1.0 + exp64(-(double)__builtin_amdgcn_fmed3f(l, kFar, 800.0f));
  double r = __builtin_amdgcn_rcp(d);
  r = __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
  return __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
}
// The same, NaN for NaN, 0 below kFar.
__device__ __forceinline__ double sigmoid64(float l) {
  return either(l != l, __builtin_nan(""), either(l < kFar, 0.0, sigmoid_of_number(l)));
}
// exp(l - peak) of a finite peak, 0 for l of -infinity.
__device__ __forceinline__ double below_finite_peak(float l, float peak) {
  return exp64(Wide::max((double)l - (double)peak, -800.0));
}
// The same, NaN where either is NaN or the peak +infinity.
__device__ __forceinline__ double below_peak64(float l, float peak) {
  const double e = below_finite_peak(l, peak);
  return either(l == -__builtin_inff(), 0.0, either(l != l, __builtin_nan(""), e + ((double)peak - (double)peak)));
}

// ---------------------------------------------------------------- picking

struct Layout {
  int q, lanes, per;  // experts of a lane, lanes of a group, experts of a group
  bool whole;         // every lane has a multiple of 4 experts
};

__device__ __forceinline__ float logit_at(const RouteArgs& a, int64_t m, int e) {
  const int64_t at = m * a.ld + e;
  return a.half ? bf16_to_f32(static_cast<const uint16_t*>(a.logits)[at]) : static_cast<const float*>(a.logits)[at];
}

// Exclusive sum over the workgroup's threads, `total[w]` for the waves' sums.
__device__ __forceinline__ int block_before(int v, int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int upto = wave_scan(v);
  if (lane == 63) total[wave] = upto;
  __syncthreads();
  const int waves = lane < wave ? total[lane & 15] : 0;  // (at most 16)
  return upto - v + __builtin_amdgcn_readlane(wave_scan(waves), 63);
}

// A choice on its way to the second launch: its expert and its rank among its
// stretch's choices of that expert, -1 for none.
constexpr int kRankBits = 16;

// n <= R fp32 (or bf16) numbers from byte offset `at` on, `fill` past them.  No
// branch but the uniform ones: each would wait for the loads before it.
// `whole`: n is a multiple of 4 in every lane.
template <int R>
__device__ __forceinline__ void load_run(__amdgpu_buffer_rsrc_t from, uint32_t at, int n, bool half, bool whole, float fill, float* to) {
  if (R >= 4 && whole) {
    u32x4 w[(R + 3) / 4];
#pragma unroll
    for (int r = 0; r < R; r += 4) {
      if (half) {
        const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(from, (int)(r < n ? at + 2 * r : kOut), 0, 0);
        w[r / 4].x = v.x, w[r / 4].y = v.y;
      } else {
        w[r / 4] = bload128(from, r < n ? at + 4 * r : kOut);
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const u32x4 v = w[r / 4];
      const float wide = bitsf(v[r & 3]), narrow = bitsf(r & 1 ? v[(r & 3) >> 1] & 0xFFFF0000u : v[(r & 3) >> 1] << 16);
      to[r] = r < n ? (half ? narrow : wide) : fill;
    }
  } else {
    uint32_t w[R];
#pragma unroll
    for (int r = 0; r < R; ++r) w[r] = half ? bload16(from, r < n ? at + 2 * r : kOut) << 16 : bload32(from, r < n ? at + 4 * r : kOut);
#pragma unroll
    for (int r = 0; r < R; ++r) to[r] = r < n ? bitsf(w[r]) : fill;
  }
}

// Groups before this lane's: of a larger value, or an equal one and a lower index.
template <int L, class K>
__device__ __forceinline__ int better_groups(typename K::T v, int group, int lanes, int groups, int lane) {
  int better = 0;
  if constexpr (L == 16) {
    unroll16([&](auto by) {  // the values of lanes by, by ... further, round the row
      constexpr int BY = decltype(by)::value;
      if (BY % lanes) return;  // (uniform)
      const typename K::T o = dpp<0x120 + BY>(v);
      const int g = dpp<0x120 + BY>(group);  // (from all lanes, not those with a tie alone)
      better += o > v || (o == v && g < group);
    });
  } else {
    for (int g = 0; g < groups; ++g) {
      typename K::T o;
      if constexpr (L == 64) o = read_lane(v, g * lanes);
      else o = __shfl(v, lane / L * L + g * lanes);
      better += o > v || (o == v && g < group);
    }
  }
  return better;
}

// Of group values known to lie in [lo, hi]: how many other groups are surely better, and how many may be, or be equal.
template <int L>
__device__ __forceinline__ void rank_groups(double lo, double hi, int lanes, int groups, int lane, int& surely, int& maybe) {
  surely = maybe = 0;
  auto against = [&](double olo, double ohi) {
    surely += olo > hi;
    maybe += ohi >= lo;
  };
  if constexpr (L == 16) {
    unroll16([&](auto by) {
      constexpr int BY = decltype(by)::value;
      if (BY % lanes) return;  // (uniform)
      against(dpp<0x120 + BY>(lo), dpp<0x120 + BY>(hi));
    });
  } else {
    for (int g = 0; g < groups; ++g) against(__shfl(lo, lane / L * L + g * lanes), __shfl(hi, lane / L * L + g * lanes));
    --maybe;  // (itself)
  }
}

// D = 0: each pick looks through all choices of the lanes.  D > 0, of fp64 choices: each lane orders its D largest (as many
// as are picked, or all it has) first, and a pick is the largest of the lanes' first ones.  The numbers in the choices' low
// bits may have put near ones in the wrong order there; where they can have, the wave does its tokens again as D = 0 does:
//   a group's value lies within 2^-42 of the size of its choices from what they are without those bits; it is unsure
//     whether a group stays if it depends on where (a relative bound above 2^(BITS - 52), and 2^-1000 for subnormal ones)
//   picks go on for as long as the next is equal to the last in all other bits, so that all such are seen; neighbours
//     that are equal so have to have the same logit and bias: then they are equal, and the lowest index is first
//   a lane whose D ordered choices are all picked may have had more of them
// 16384 of 256 experts by biased scores: 25.0 us, 29.4 with D = 0, in groups 26.7 and 31.7; of 512 43 and 53.  The checks are
// 0.2 to 0.8 us of it (of 512 3, for registers).  Groups of the same value at the border are done again: with bf16 logits and
// no bias, or few values of one, 31 us in pairs, 38 by the largest.  By logits, whose keys take half the registers, ordering
// makes 20.2 us 19.5 for 8 picks and 26.6 31.3 for 16.
template <int L, int R, int D, class K, bool LOOSE, int THREADS>
__global__ __launch_bounds__(THREADS) void k_route(RouteArgs a, Layout at, int span, int passes) {
  typedef typename K::T T;
  constexpr bool WIDE = sizeof(T) == 8;
  constexpr int AT_ONCE = THREADS / L;  // tokens
  __shared__ uint64_t mask[WQ_MAX_EXPERTS];
  __shared__ int base[WQ_MAX_EXPERTS];
  __shared__ uint16_t picks[kSpan * WQ_MAX_TOP];
  __shared__ int total[THREADS / 64];
  extern __shared__ __attribute__((aligned(16))) unsigned char loose[];  // keys of loose groups: [AT_ONCE][groups]
  const int tid = threadIdx.x, l = tid % L, slot = tid / L;
  const int E = a.E, top = a.top;
  const bool alone = gridDim.x == 1 && passes == 1;  // this workgroup has all tokens
  for (int e = tid; e < E; e += THREADS) mask[e] = 0, base[e] = 0;
  __syncthreads();

  // this lane's experts: first .. first + mine - 1
  const int in_group = l % at.lanes, group = l / at.lanes;
  const int first = group * at.per + in_group * at.q;
  const int mine = max(0, min(at.q, min(at.per - in_group * at.q, E - first)));
  T bias[WIDE ? R : 1];  // kNot past a lane's experts
  if constexpr (WIDE) {
    float b[R];
    load_run<R>(make_rsrc(a.bias, a.bias ? (uint32_t)E * 4u : 0u), (uint32_t)first * 4u, mine, false, at.whole, -__builtin_inff(), b);
#pragma unroll
    for (int r = 0; r < R; ++r) bias[r] = K::of((double)b[r]);
  }

  for (int pass = 0; pass < passes; ++pass) {
    const int64_t m0 = ((int64_t)blockIdx.x * passes + pass) * span;
    if (m0 >= a.M) break;
    const int tokens = (int)min((int64_t)span, (int64_t)a.M - m0);
    const __amdgpu_buffer_rsrc_t rows = make_rsrc(static_cast<const char*>(a.logits) + m0 * a.ld * (a.half ? 2 : 4),
                                                  ((uint32_t)(tokens - 1) * (uint32_t)a.ld + (uint32_t)E) * (a.half ? 2u : 4u));
    for (int sub = 0; sub < tokens; sub += AT_ONCE) {
      const int t = sub + slot;
      const int64_t m = m0 + t;
      const bool live = t < tokens && (!a.valid || a.valid[m]);
      uint32_t biggest;  // key of the row's largest logit
      double sum;
      float peak;
      int pick;  // of lane j: the j-th largest choice
      float x;   // its logit
      for (bool whole = D == 0;; whole = true) {  // whether choices are compared in all their bits
        T key[R];
        biggest = 0, sum = 0.0;
        // (as if new each time: kept through the loop, what comes of them takes registers that are not there)
        int token = t, from = first, count = live ? mine : 0;
        if constexpr (D > 0) asm volatile("" : "+v"(token), "+v"(from), "+v"(count));
        {
          float logit[R];
          load_run<R>(rows, ((uint32_t)token * (uint32_t)a.ld + (uint32_t)from) * (a.half ? 2u : 4u), count, a.half, at.whole,
                      WIDE && a.sigmoid && live ? 0.f : -__builtin_inff(), logit);
          if (!a.sigmoid || !WIDE) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
              const uint32_t k = Narrow::of(logit[r]);
              if constexpr (!WIDE) key[r] = k;
              biggest = max(biggest, k);
            }
            biggest = max_over<Narrow>(biggest, L);
          }
          peak = Narrow::logit(biggest);
          if constexpr (WIDE) {
            // choices of numbers; infinities and NaN, if the wave has any, after that (a logit of +infinity has the score 1)
            constexpr int kNaNs = 0x003, kBelow = 0x004, kAbove = 0x200;
            bool odd;
            if (a.sigmoid) {
              odd = false;
#pragma unroll
              for (int r = 0; r < R; ++r) {
                key[r] = sigmoid_of_number(logit[r]) + bias[r];
                odd |= __builtin_amdgcn_classf(logit[r], kNaNs | kBelow);
                if (r % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // (16 at once would not fit the registers)
              }
            } else {
#pragma unroll
              for (int r = 0; r < R; ++r) {
                sum += key[r] = below_finite_peak(logit[r], peak);
                if (r % 4 == 3) __builtin_amdgcn_sched_barrier(0);
              }
              sum = sum_over(sum, L);
              const double part = 1.0 / sum;
              odd = __builtin_amdgcn_classf(peak, kNaNs | kBelow | kAbove);
#pragma unroll
              for (int r = 0; r < R; ++r) {
                key[r] = __builtin_fma(key[r], part, bias[r]);
                odd |= __builtin_amdgcn_classf(logit[r], kBelow);
              }
            }
            if (__any(odd)) {
              const bool all = !a.sigmoid && __builtin_amdgcn_classf(peak, kNaNs | kAbove);
#pragma unroll
              for (int r = 0; r < R; ++r)
                key[r] = either(logit[r] == -__builtin_inff(), K::kNot, either(all || logit[r] != logit[r], K::kNaN, key[r]));
            }
          } else if (!a.sigmoid && !a.renormalize) {
            // (fp32's exponentials and sum leave the weights up to 2.5 2^-24 off and take 22.9 us for 16384 of 256 experts, 25.2 so)
#pragma unroll
            for (int r = 0; r < R; ++r) {
              sum += below_finite_peak(logit[r], peak);
              if (r % 4 == 3) __builtin_amdgcn_sched_barrier(0);
            }
            sum = sum_over(sum, L);
          }
        }

        pick = -1, x = 0.f;
        if constexpr (D > 0) {
          if (!whole) {
            typedef Numbered<__builtin_ctz(L * R)> N;
#pragma unroll
            for (int r = 0; r < R; ++r) key[r] = N::of(key[r], from + r);
            largest<R, D>(key);
            bool unsure = false;
            if (a.groups > 1) {
              const Two<K> best = best_over<K>(Two<K>{N::choice(key[0]), N::choice(key[1])}, at.lanes, a.pairs);
              const double value = K::sum(best.a, best.b), size = __builtin_fabs(best.a) + (best.b == K::kNot ? 0.0 : __builtin_fabs(best.b));
              const double off = __builtin_fma(size, 0x1p-42, 0x1p-1000);
              int surely, maybe;
              rank_groups<L>(value - off, value + off, at.lanes, a.groups, tid & 63, surely, maybe);
              unsure = best.a != K::kNot && surely < a.keep && maybe >= a.keep;
              if (maybe >= a.keep) {
#pragma unroll
                for (int r = 0; r < D; ++r) key[r] = K::kNot;
              }
            }
            const double held = key[D - 1];  // the least of this lane that can be picked
            double own = K::kNot, last = K::kNot;
            auto next = [&] {
              const double best = max_over<K>(key[0], L);
              const bool taken = key[0] == best;
#pragma unroll
              for (int r = 0; r < D; ++r) key[r] = either(taken, r + 1 < D ? key[r + 1] : K::kNot, key[r]);
              return best;
            };
            for (int j = 0; j < top; ++j) {
              last = next();
              own = l == j ? last : own;
            }
            double least = last;
            for (int j = top;; ++j) {
              const double best = max_over<K>(key[0], L);
              const bool more = N::choice(best) == N::choice(last) && N::choice(last) != K::kNot;
              if (!__any(more)) break;
              if (j == L) {
                unsure |= more;
                break;
              }
              next();
              own = more && l == j ? best : own;
              least = more ? best : least;
            }
            if constexpr (D < R) unsure |= N::choice(held) != K::kNot && held >= least;
            const bool has = N::choice(own) != K::kNot;
            const double before = L == 16 ? dpp<0x111>(own) : __shfl(own, (tid & 63) - 1);
            const bool near = l > 0 && has && N::choice(own) == N::choice(before);
            if (__any(near)) {
              const float mine_l = has ? logit_at(a, m, N::expert(own)) : 0.f, mine_b = has && a.bias ? a.bias[N::expert(own)] : 0.f;
              const float before_l = __shfl(mine_l, (tid & 63) - 1), before_b = __shfl(mine_b, (tid & 63) - 1);
              unsure |= near && !(mine_l == before_l && mine_b == before_b);
            }
            if (__any(unsure)) continue;
            if (l < top && has) pick = N::expert(own);
            break;
          }
        }
        {
          if (a.groups > 1) {
            if constexpr (!LOOSE) {
              Two<K> two{K::kNot, K::kNot};
#pragma unroll
              for (int r = 0; r < R; ++r) two.add(key[r]);
              const T v = group_value<K>(two, at.lanes, a.pairs);
              if (better_groups<L, K>(v, group, at.lanes, a.groups, tid & 63) >= a.keep) {
#pragma unroll
                for (int r = 0; r < R; ++r) key[r] = K::kNot;
              }
            } else {
              T* value = reinterpret_cast<T*>(loose) + slot * a.groups;
              const int size = E / a.groups;
              for (int g = 0; g < a.groups; ++g) {
                Two<K> t2{K::kNot, K::kNot};
#pragma unroll
                for (int r = 0; r < R; ++r)
                  if ((first + r) / size == g) t2.add(key[r]);
                const T v = group_value<K>(t2, L, a.pairs);
                if (l == 0) value[g] = v;
              }
              __syncthreads();
#pragma unroll
              for (int r = 0; r < R; ++r) {
                if (r >= mine) continue;
                const int own = (first + r) / size;
                const T v = value[own];
                int better = 0;
                for (int g = 0; g < a.groups; ++g) better += value[g] > v || (value[g] == v && g < own);
                if (better >= a.keep) key[r] = K::kNot;
              }
              __syncthreads();
            }
          }

          for (int j = 0; j < top; ++j) {
            T best = key[0];
#pragma unroll
            for (int r = 1; r < R; ++r) best = K::max(best, key[r]);
            best = max_over<K>(best, L);
            uint32_t e = ~0u;  // the lowest expert of that key
#pragma unroll
            for (int r = R - 1; r >= 0; --r) e = key[r] == best ? (uint32_t)(from + r) : e;
            if constexpr (L == 64) {
              e = __builtin_amdgcn_readlane(e, __builtin_ctzll(__ballot(e != ~0u)));
            } else {
              e = over(e, L, [](uint32_t p, uint32_t q) { return p < q ? p : q; });
            }
            if (l == j && best != K::kNot) {
              pick = (int)e;
              if constexpr (!WIDE) x = Narrow::logit(best);
            }
#pragma unroll
            for (int r = 0; r < R; ++r) key[r] = (uint32_t)(from + r) == e ? K::kNot : key[r];
          }
        }
        break;
      }
      if (WIDE && pick >= 0) x = logit_at(a, m, pick);

      double s = 0.0;
      if (pick >= 0) s = a.sigmoid ? sigmoid64(x) : below_peak64(x, peak);
      if (a.renormalize) {
        const double all = sum_over(s, L);
        s = all == 0.0 ? 0.0 : s / all;
      } else if (!a.sigmoid) {
        s /= sum;
      }
      if (l < top) {
        if (t < tokens) {
          a.ids[m * top + l] = pick;
          a.weights[m * top + l] = pick >= 0 ? (float)((double)a.scale * s) : 0.f;
        }
        picks[t * top + l] = pick >= 0 ? (uint16_t)pick : kNone;
        if (pick >= 0) atomicOr((unsigned long long*)&mask[pick], 1ull << t);
      }
    }
    __syncthreads();

    if (alone) {
      // offsets, then places and rows at once; a thread has PER experts
      constexpr int PER = WQ_MAX_EXPERTS / THREADS;
      int n[PER], sum = 0;
#pragma unroll
      for (int u = 0; u < PER; ++u) {
        const int e = tid * PER + u;
        n[u] = e < E ? __builtin_popcountll(mask[e]) : 0;
        sum += n[u];
      }
      int before = block_before(sum, total);
#pragma unroll
      for (int u = 0; u < PER; ++u) {
        const int e = tid * PER + u;
        if (e < E) {
          base[e] = before;
          a.offsets[e] = before;
          before += n[u];
          if (e == E - 1) a.offsets[E] = before;
        }
      }
      __syncthreads();
    }
    for (int i = tid; i < tokens * top; i += THREADS) {
      const int t = i / top;
      const int e = picks[i];
      int p = -1;
      if (e != kNone) {
        p = base[e] + __builtin_popcountll(mask[e] & ((1ull << t) - 1));
        if (alone) a.rows[p] = t;
        else p |= e << kRankBits;
      }
      a.places[m0 * top + i] = p;
    }
    if (!alone) {
      __syncthreads();
      for (int e = tid; e < E; e += THREADS) {
        base[e] += __builtin_popcountll(mask[e]);
        mask[e] = 0;
      }
      __syncthreads();
    }
  }
  if (!alone)
    for (int e = tid; e < E; e += THREADS) a.counts[(int64_t)blockIdx.x * counts_pitch(E) + e] = (uint16_t)base[e];
}

// ---------------------------------------------------------------- the order of many stretches

__global__ __launch_bounds__(kOrderThreads) void k_route_order(RouteArgs a, int tokens) {
  __shared__ int before[WQ_MAX_EXPERTS], all[WQ_MAX_EXPERTS], total[kOrderThreads / 64];
  const int tid = threadIdx.x, E = a.E, top = a.top, n = gridDim.x, b = blockIdx.x;
  const int64_t m0 = (int64_t)b * tokens;
  const int choices = (int)min((int64_t)tokens, (int64_t)a.M - m0) * top;
  int32_t* places = a.places + m0 * top;
  int next = tid < choices ? places[tid] : -1;  // (under way with the counts)
  for (int e = tid; e < E; e += kOrderThreads) before[e] = 0, all[e] = 0;
  __syncthreads();
  // two experts to a thread, so that few loads, all under way at once, take a stretch's counts
  const int words = counts_pitch(E) / 2, wide = (words + 63) / 64 * 64, slices = kOrderThreads / wide, slice = tid / wide, w = tid % wide;
  if (slice < slices && w < words) {
    int x[2] = {0, 0}, y[2] = {0, 0};
    constexpr int AHEAD = 32;
    const uint32_t* counts = reinterpret_cast<const uint32_t*>(a.counts) + w;
    for (int i = slice; i < n; i += AHEAD * slices) {
      uint32_t c[AHEAD];
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) c[u] = i + u * slices < n ? counts[(int64_t)(i + u * slices) * words] : 0;
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int lo = (int)(c[u] & 0xFFFFu), hi = (int)(c[u] >> 16);
        const bool earlier = i + u * slices < b;
        y[0] += lo, y[1] += hi;
        x[0] += earlier ? lo : 0, x[1] += earlier ? hi : 0;
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (2 * w + k < E) {
        atomicAdd(&before[2 * w + k], x[k]);
        atomicAdd(&all[2 * w + k], y[k]);
      }
  }
  __syncthreads();
  constexpr int PER = WQ_MAX_EXPERTS / kOrderThreads;  // experts of a thread
  int each[PER], sum = 0;
#pragma unroll
  for (int u = 0; u < PER; ++u) sum += each[u] = tid * PER + u < E ? all[tid * PER + u] : 0;
  int start = block_before(sum, total);
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    const int e = tid * PER + u;
    if (e < E) {
      before[e] += start;
      if (b == 0) a.offsets[e] = start;
      start += each[u];
      if (b == 0 && e == E - 1) a.offsets[E] = start;
    }
  }
  __syncthreads();
  for (int i = tid; i < choices;) {
    const int c = next, at = i;
    i += kOrderThreads;
    next = i < choices ? places[i] : -1;
    if (c == -1) continue;
    const int p = before[(uint32_t)c >> kRankBits] + (c & ((1 << kRankBits) - 1));
    places[at] = p;
    a.rows[p] = (int32_t)(m0 + at / top);
  }
}

template <int L, int R, int D, class K, int THREADS, bool LOOSE>
hipError_t launch_one(const RouteArgs& a, const Layout& at, const Stretches& st, hipStream_t s) {
  const size_t smem = LOOSE ? (size_t)(THREADS / L) * a.groups * sizeof(typename K::T) : 0;
  return launch(k_route<L, R, D, K, LOOSE, THREADS>, dim3((unsigned)st.count), THREADS, smem, s, a, at, st.span, st.passes);
}
template <int L, int R, int THREADS, bool LOOSE = false>
hipError_t route_launch(const RouteArgs& a, const Layout& at, const Stretches& st, bool wide, hipStream_t s) {
  // (16 fp64 keys a lane do not fit the registers that 16 waves on a CU leave: 16384 of 256 experts 31.1 us, 28.9 with 8; of
  // 512 45.0, 43.2 with 8)
  constexpr int WIDE_THREADS = R == 16 && L < 64 ? THREADS / 2 : THREADS;
  if (!wide) return launch_one<L, R, 0, Narrow, THREADS, LOOSE>(a, at, st, s);
  if constexpr (L < 64 && R >= 8) {
    if (a.top <= 4) return launch_one<L, R, 4, Wide, WIDE_THREADS, LOOSE>(a, at, st, s);
    if (a.top <= 8) return launch_one<L, R, 8, Wide, WIDE_THREADS, LOOSE>(a, at, st, s);
  }
  return launch_one<L, R, L < 64 && R >= 4 ? R : 0, Wide, WIDE_THREADS, LOOSE>(a, at, st, s);
}

__global__ void k_no_tokens(int32_t* offsets, int n) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) offsets[i] = 0;
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t s) {
  if (a.M == 0) return launch(k_no_tokens, dim3(1), 256, 0, s, a.offsets, a.E + 1);
  const bool wide = a.bias || a.pairs;
  Stretches st = stretches(a.M);
  // one launch of one workgroup where that takes no longer than two: 64 tokens of 128 experts 8.9 us, 9.3 in two, 17 8.4 and
  // 9.0; 64 of 256 11.3 and 9.8, of 1024 34 and 12; by biased scores, 64 of 256 in groups 20 and 11
  if (a.M > kFewSpan && a.M <= kSpan && a.E <= 128 && !wide) st = {kSpan, 1, 1};
  const bool on_lanes = (a.groups & (a.groups - 1)) == 0;
  auto fits = [&](int lanes, int regs, Layout& at) {
    if (a.top > lanes || (on_lanes && a.groups > lanes)) return false;
    const int groups = on_lanes ? a.groups : 1;
    at.per = a.E / groups;
    at.lanes = lanes / groups;
    at.q = (at.per + at.lanes - 1) / at.lanes;
    at.whole = at.q % 4 == 0 && at.per % 4 == 0;
    return at.q <= regs;
  };
  Layout at;
  hipError_t e = hipErrorInvalidValue;
#define WQ_ROUTE(L, R, T) \
  if (fits(L, R, at)) e = route_launch<L, R, T>(a, at, st, wide, s)
  if (!on_lanes) {
    const bool waves = st.span == kWaves;
    if (fits(64, 4, at)) e = waves ? route_launch<64, 4, 256, true>(a, at, st, wide, s) : route_launch<64, 4, 1024, true>(a, at, st, wide, s);
    else if (fits(64, 16, at)) e = waves ? route_launch<64, 16, 256, true>(a, at, st, wide, s) : route_launch<64, 16, 1024, true>(a, at, st, wide, s);
  } else if (a.M <= 4 || st.span == kWaves) {
    // a token to a wave, in a workgroup of no more waves than that takes: 1 token of 128 experts 5.1 us, 6.2 with 16 waves
    WQ_ROUTE(64, 1, 256);
    else WQ_ROUTE(64, 2, 256);
    else WQ_ROUTE(64, 4, 256);
    else WQ_ROUTE(64, 16, 256);
  } else if (st.span == kFewSpan) {
    WQ_ROUTE(64, 1, 1024);
    else WQ_ROUTE(64, 2, 1024);
    else WQ_ROUTE(64, 4, 1024);
    else WQ_ROUTE(64, 16, 1024);
  } else {
    // the fewest lanes that hold a token's experts, in the fewest registers
    WQ_ROUTE(16, 1, 1024);
    else WQ_ROUTE(16, 2, 1024);
    else WQ_ROUTE(16, 4, 1024);
    else WQ_ROUTE(16, 8, 1024);
    else WQ_ROUTE(16, 16, 1024);
    else WQ_ROUTE(32, 16, 1024);
    else WQ_ROUTE(64, 16, 1024);
  }
#undef WQ_ROUTE
  if (e != hipSuccess || (st.count == 1 && st.passes == 1)) return e;
  return launch(k_route_order, dim3((unsigned)st.count), kOrderThreads, 0, s, a, st.span * st.passes);
}

}  // namespace wq
