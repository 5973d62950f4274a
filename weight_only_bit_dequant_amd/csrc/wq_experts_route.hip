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
// The order needs no atomics whose order counts: of each kPassTokens tokens a bit
// mask of those that picked an expert gives every choice its rank among them
// (the bits below its own) and the expert its count.  Up to kPassTokens tokens
// take one launch of one workgroup; more take two: the first writes counts of
// each stretch of tokens, in the second each workgroup adds up the counts before
// its own.
#include "wq_experts_internal.hpp"
#include "wq_row_tiles.hpp"

namespace wq {

namespace {

constexpr int kThreads = 1024;
constexpr uint16_t kNone = 0xFFFF;

// ---------------------------------------------------------------- keys

__device__ __forceinline__ uint32_t key_of(float c) {
  const uint32_t u = fbits(c + 0.0f);  // -0 is 0
  return c != c ? ~0u : c == -__builtin_inff() ? 0u : u ^ (uint32_t)(((int32_t)u >> 31) | (int32_t)0x80000000);
}
__device__ __forceinline__ uint64_t key_of(double c) {
  const uint64_t u = __builtin_bit_cast(uint64_t, c + 0.0);
  return c != c ? ~0ull : c == -__builtin_inf() ? 0ull : u ^ (uint64_t)(((int64_t)u >> 63) | (int64_t)0x8000000000000000ull);
}
__device__ __forceinline__ float value_of(uint32_t k) {
  const uint32_t u = k ^ (k >> 31 ? 0x80000000u : ~0u);
  return k == ~0u ? __builtin_nanf("") : k == 0 ? -__builtin_inff() : bitsf(u);
}
__device__ __forceinline__ double value_of(uint64_t k) {
  const uint64_t u = k ^ (k >> 63 ? 0x8000000000000000ull : ~0ull);
  return k == ~0ull ? __builtin_nan("") : k == 0 ? -__builtin_inf() : __builtin_bit_cast(double, u);
}

// Over the first `n` (a power of two) of the lanes that share lane / n.
template <typename T>
__device__ __forceinline__ T max_over(T v, int n) {
  for (int d = 1; d < n; d <<= 1) {
    const T o = __shfl_xor(v, d);
    v = v > o ? v : o;
  }
  return v;
}
template <typename T>
__device__ __forceinline__ T sum_over(T v, int n) {
  for (int d = 1; d < n; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

// The two largest keys, and those of two such pairs.
template <typename K>
struct Two {
  K a, b;
  __device__ __forceinline__ void add(K k) {
    b = k > a ? a : k > b ? k : b;
    a = k > a ? k : a;
  }
};
template <typename K>
__device__ __forceinline__ Two<K> two_over(Two<K> t, int n) {
  for (int d = 1; d < n; d <<= 1) {
    const K oa = __shfl_xor(t.a, d), ob = __shfl_xor(t.b, d);
    const K low = t.a > oa ? oa : t.a;
    t.a = t.a > oa ? t.a : oa;
    t.b = t.b > ob ? t.b : ob;
    t.b = t.b > low ? t.b : low;
  }
  return t;
}
template <typename K>
__device__ __forceinline__ K group_value(Two<K> t, bool pairs) {
  if (!pairs || t.b == 0) return t.a;
  return key_of(value_of(t.a) + value_of(t.b));
}

// ---------------------------------------------------------------- picking

struct Layout {
  int q, lanes, per;  // experts of a lane, lanes of a group, experts of a group
  bool loose;         // groups that do not fall on lanes
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
  int before = upto - v;
  for (int w = 0; w < wave; ++w) before += total[w];
  return before;
}

template <int L, int R, bool WIDE>
__global__ __launch_bounds__(kThreads) void k_route(RouteArgs a, Layout at, int passes) {
  using K = std::conditional_t<WIDE, uint64_t, uint32_t>;
  constexpr int AT_ONCE = kThreads / L;  // tokens
  static_assert(kPassTokens % AT_ONCE == 0, "whole rounds of a pass");
  __shared__ uint64_t mask[WQ_MAX_EXPERTS];
  __shared__ int base[WQ_MAX_EXPERTS];
  __shared__ uint16_t picks[kPassTokens * WQ_MAX_TOP];
  __shared__ int total[kThreads / 64];
  extern __shared__ __attribute__((aligned(16))) unsigned char loose[];  // keys of loose groups: [AT_ONCE][groups]
  const int tid = threadIdx.x, l = tid % L, slot = tid / L;
  const int E = a.E, top = a.top;
  const bool alone = gridDim.x == 1 && passes == 1;  // this workgroup has all tokens
  for (int e = tid; e < E; e += kThreads) mask[e] = 0, base[e] = 0;
  __syncthreads();

  // this lane's experts: first .. first + mine - 1
  const int in_group = l % at.lanes, group = l / at.lanes;
  const int first = group * at.per + in_group * at.q;
  const int mine = max(0, min(at.q, min(at.per - in_group * at.q, E - first)));
  const uint64_t seg = (L == 64 ? ~0ull : ((1ull << (L & 63)) - 1)) << ((tid & 63) / L * L);

  for (int pass = 0; pass < passes; ++pass) {
    const int64_t m0 = ((int64_t)blockIdx.x * passes + pass) * kPassTokens;
    for (int sub = 0; sub < kPassTokens; sub += AT_ONCE) {
      const int t = sub + slot;
      const int64_t m = m0 + t;
      const bool live = m < a.M && (!a.valid || a.valid[m]);
      K key[R];
      uint32_t biggest = 0;  // key of the row's largest logit
      float logit[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        logit[r] = live && r < mine ? logit_at(a, m, first + r) : -__builtin_inff();
        biggest = max(biggest, key_of(logit[r]));
      }
      biggest = max_over(biggest, L);
      const float peak = value_of(biggest);
      double sum = 0.0;
      if constexpr (WIDE) {
        double s[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const bool on = logit[r] != -__builtin_inff();
          if (a.sigmoid) {
            s[r] = 1.0 / (1.0 + exp(-(double)logit[r]));
          } else {
            s[r] = on ? exp((double)logit[r] - (double)peak) : 0.0;
            sum += s[r];
          }
        }
        if (!a.sigmoid) {
          sum = sum_over(sum, L);
#pragma unroll
          for (int r = 0; r < R; ++r) s[r] /= sum;
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
          key[r] = r < mine && logit[r] != -__builtin_inff() ? key_of(s[r] + (a.bias ? (double)a.bias[first + r] : 0.0)) : 0;
      } else {
        float part = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          key[r] = key_of(logit[r]);
          if (!a.sigmoid && !a.renormalize) part += logit[r] == -__builtin_inff() ? 0.f : expf(logit[r] - peak);
        }
        sum = sum_over(part, L);
      }

      if (a.groups > 1) {
        Two<K> two{0, 0};
        if (!at.loose) {
#pragma unroll
          for (int r = 0; r < R; ++r) two.add(key[r]);
          const K v = group_value(two_over(two, at.lanes), a.pairs);
          int better = 0;
          for (int g = 0; g < a.groups; ++g) {
            const K o = __shfl(v, (tid & 63) / L * L + g * at.lanes);
            better += o > v || (o == v && g < group);
          }
          if (better >= a.keep) {
#pragma unroll
            for (int r = 0; r < R; ++r) key[r] = 0;
          }
        } else {
          K* value = reinterpret_cast<K*>(loose) + slot * a.groups;
          const int size = E / a.groups;
          for (int g = 0; g < a.groups; ++g) {
            Two<K> t2{0, 0};
#pragma unroll
            for (int r = 0; r < R; ++r)
              if ((first + r) / size == g) t2.add(key[r]);
            const K v = group_value(two_over(t2, L), a.pairs);
            if (l == 0) value[g] = v;
          }
          __syncthreads();
#pragma unroll
          for (int r = 0; r < R; ++r) {
            if (r >= mine) continue;
            const int own = (first + r) / size;
            const K v = value[own];
            int better = 0;
            for (int g = 0; g < a.groups; ++g) better += value[g] > v || (value[g] == v && g < own);
            if (better >= a.keep) key[r] = 0;
          }
          __syncthreads();
        }
      }

      int pick = -1;  // of lane j: the j-th largest choice
      for (int j = 0; j < top; ++j) {
        K best = 0;
        int br = 0;
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (key[r] > best) best = key[r], br = r;
        const K all = max_over(best, L);
        const uint64_t holders = __ballot(best == all) & seg;
        const int winner = __builtin_ctzll(holders);
        const int e = __shfl(first + br, winner);
        if (l == j && all != 0) pick = e;
        if ((tid & 63) == winner) {
#pragma unroll
          for (int r = 0; r < R; ++r) key[r] = r == br ? 0 : key[r];
        }
      }

      double s = 0.0;
      if (pick >= 0) {
        const double x = logit_at(a, m, pick);
        // (a peak of +infinity makes every score NaN, those of finite logits too)
        s = a.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - (double)peak) + ((double)peak - (double)peak);
      }
      if (a.renormalize) {
        const double all = sum_over(s, L);
        s = all == 0.0 ? 0.0 : s / all;
      } else if (!a.sigmoid) {
        s /= sum;
      }
      if (l < top) {
        if (m < a.M) {
          a.ids[m * top + l] = pick;
          a.weights[m * top + l] = pick >= 0 ? (float)((double)a.scale * s) : 0.f;
        }
        picks[t * top + l] = pick >= 0 ? (uint16_t)pick : kNone;
        if (pick >= 0) atomicOr((unsigned long long*)&mask[pick], 1ull << t);
      }
    }
    __syncthreads();

    if (alone) {
      // offsets, then places and rows at once
      const int n = tid < E ? __builtin_popcountll(mask[tid]) : 0;
      const int before = block_before(n, total);
      if (tid < E) {
        base[tid] = before;
        a.offsets[tid] = before;
        if (tid == E - 1) a.offsets[E] = before + n;
      }
      __syncthreads();
    }
    for (int i = tid; i < kPassTokens * top; i += kThreads) {
      const int t = i / top;
      if (m0 + t >= a.M) break;
      const int e = picks[i];
      int p = -1;
      if (e != kNone) {
        p = base[e] + __builtin_popcountll(mask[e] & ((1ull << t) - 1));
        if (alone) a.rows[p] = t;
      }
      a.places[m0 * top + i] = p;  // (more than one stretch: the rank within this one)
    }
    if (!alone) {
      __syncthreads();
      for (int e = tid; e < E; e += kThreads) {
        base[e] += __builtin_popcountll(mask[e]);
        mask[e] = 0;
      }
      __syncthreads();
    }
  }
  if (!alone)
    for (int e = tid; e < E; e += kThreads) a.counts[(int64_t)blockIdx.x * E + e] = base[e];
}

// ---------------------------------------------------------------- the order of many stretches

__global__ __launch_bounds__(kThreads) void k_route_order(RouteArgs a, int passes) {
  __shared__ int before[WQ_MAX_EXPERTS], all[WQ_MAX_EXPERTS], total[kThreads / 64];
  const int tid = threadIdx.x, E = a.E, top = a.top, n = gridDim.x, b = blockIdx.x;
  for (int e = tid; e < E; e += kThreads) before[e] = 0, all[e] = 0;
  __syncthreads();
  const int wide = (E + 63) / 64 * 64, slices = kThreads / wide, slice = tid / wide, e = tid % wide;
  if (slice < slices && e < E) {
    int x = 0, y = 0;
    for (int i = slice; i < n; i += slices) {
      const int c = a.counts[(int64_t)i * E + e];
      y += c;
      x += i < b ? c : 0;
    }
    atomicAdd(&before[e], x);
    atomicAdd(&all[e], y);
  }
  __syncthreads();
  const int mine = tid < E ? all[tid] : 0;
  const int start = block_before(mine, total);
  if (tid < E) {
    before[tid] += start;
    if (b == 0) {
      a.offsets[tid] = start;
      if (tid == E - 1) a.offsets[E] = start + mine;
    }
  }
  __syncthreads();
  const int64_t m0 = (int64_t)b * passes * kPassTokens;
  const int tokens = (int)min((int64_t)passes * kPassTokens, (int64_t)a.M - m0);
  for (int i = tid; i < tokens * top; i += kThreads) {
    const int pick = a.ids[m0 * top + i];
    if (pick < 0) continue;
    const int p = before[pick] + a.places[m0 * top + i];
    a.places[m0 * top + i] = p;
    a.rows[p] = (int32_t)(m0 + i / top);
  }
}

template <int L, int R>
hipError_t route_launch(const RouteArgs& a, const Layout& at, const Stretches& st, bool wide, hipStream_t s) {
  const size_t smem = at.loose ? (size_t)(kThreads / L) * a.groups * (wide ? 8 : 4) : 0;
  return launch(wide ? k_route<L, R, true> : k_route<L, R, false>, dim3((unsigned)st.count), kThreads, smem, s, a, at, st.passes);
}

__global__ void k_no_tokens(int32_t* offsets, int n) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) offsets[i] = 0;
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t s) {
  if (a.M == 0) return launch(k_no_tokens, dim3(1), 256, 0, s, a.offsets, a.E + 1);
  const bool wide = a.bias || a.pairs;
  const Stretches st = stretches(a.M);
  // the fewest lanes that hold a token's experts, in the fewest registers
  const bool on_lanes = (a.groups & (a.groups - 1)) == 0;
  auto fits = [&](int lanes, int regs, Layout& at) {
    if (a.top > lanes || (on_lanes && a.groups > lanes)) return false;
    const int groups = on_lanes ? a.groups : 1;
    at.loose = !on_lanes;
    at.per = a.E / groups;
    at.lanes = lanes / groups;
    at.q = (at.per + at.lanes - 1) / at.lanes;
    return at.q <= regs;
  };
  Layout at;
  hipError_t e;
  if (fits(16, 1, at)) e = route_launch<16, 1>(a, at, st, wide, s);
  else if (fits(16, 2, at)) e = route_launch<16, 2>(a, at, st, wide, s);
  else if (fits(16, 4, at)) e = route_launch<16, 4>(a, at, st, wide, s);
  else if (fits(16, 8, at)) e = route_launch<16, 8>(a, at, st, wide, s);
  else if (fits(16, 16, at)) e = route_launch<16, 16>(a, at, st, wide, s);
  else if (fits(32, 4, at)) e = route_launch<32, 4>(a, at, st, wide, s);
  else if (fits(32, 16, at)) e = route_launch<32, 16>(a, at, st, wide, s);
  else if (fits(64, 4, at)) e = route_launch<64, 4>(a, at, st, wide, s);
  else if (fits(64, 16, at)) e = route_launch<64, 16>(a, at, st, wide, s);
  else return hipErrorInvalidValue;
  if (e != hipSuccess || (st.count == 1 && st.passes == 1)) return e;
  return launch(k_route_order, dim3((unsigned)st.count), kThreads, 0, s, a, st.passes);
}

}  // namespace wq
