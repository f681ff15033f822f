// Routing of one token from its logits, by 16 or 64 lanes of a wave (gfx950).
//
//   s = softmax(l) or sigmoid(l);  v = s + b, or the order of l without a balance b
//   groups graded by their best v, or by the sum of their two best (of s without b)
//   the top-k of the best groups' experts by v, equal ones to the lower expert
//
// v is compared as a 64-bit float whose last ten mantissa bits hold the expert: one
// minimum and one maximum order two candidates, index and ties included, and a list
// of K is merged by K maxima and a network of K/2 log2 K pairs.  A logit has 24
// significant bits, so its order is exact; scores with a balance are computed in 64
// bits and compared to 42 of them (in 32 bits, two of 256 balanced scores round to the
// same value about once in 10^4 tokens, and the ids would depend on how).
#pragma once

#include "exl3_internal.hpp"
#include "exl3_wave.hpp"

namespace exl3 {

constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxGroups = 64;
constexpr int kRouteMaxTopk = 16;

// What stands for infinities, NaN (lowest of all experts) and no expert, so that the
// mantissa's last bits are free in every key.
constexpr double kKeyInf = 1e300, kKeyNan = -1.2e300, kKeyNone = -1.7e308;
constexpr uint32_t kKeyPlace = 1023;

// The key of value v at place e: larger for larger v, then for lower e.
__device__ __forceinline__ double route_key(double v, uint32_t e) {
  v = v > kKeyInf ? kKeyInf : v;
  v = v < -kKeyInf ? -kKeyInf : v;
  v = (v != v ? kKeyNan : v) + 0.0;  // -0 is 0
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  const uint32_t place = (int64_t)b < 0 ? e : kKeyPlace - e;
  return __longlong_as_double((long long)((b & ~(uint64_t)kKeyPlace) | place));
}
__device__ __forceinline__ uint32_t route_place(double key) {
  const uint64_t b = (uint64_t)__double_as_longlong(key);
  const uint32_t place = (uint32_t)b & kKeyPlace;
  return (int64_t)b < 0 ? place : kKeyPlace - place;
}
__device__ __forceinline__ double route_value(double key) {
  const uint64_t b = (uint64_t)__double_as_longlong(key) & ~(uint64_t)kKeyPlace;
  const double v = __longlong_as_double((long long)b);
  constexpr double inf = __builtin_huge_val();
  return v >= 0.99e300 ? inf : v <= -1.1e300 ? __builtin_nan("") : v <= -0.99e300 ? -inf : v;
}

// ---------------------------------------------------------------------------
// over the lanes of a token
// ---------------------------------------------------------------------------
typedef uint32_t u32pair_t __attribute__((ext_vector_type(2)));

// The value of the lane N places on in its row of 16.
template <int N>
__device__ __forceinline__ uint32_t row_turn(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + N, 0xF, 0xF, true);
}
template <int N>
__device__ __forceinline__ float row_turn(float v) {
  return __uint_as_float(row_turn<N>(__float_as_uint(v)));
}
template <int N>
__device__ __forceinline__ double row_turn(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  const uint64_t lo = row_turn<N>((uint32_t)b), hi = row_turn<N>((uint32_t)(b >> 32));
  return __longlong_as_double((long long)(hi << 32 | lo));
}

// v of both halves of the wave (HALF), or of both rows of a pair of rows.
template <bool HALF>
__device__ __forceinline__ void both(uint32_t v, uint32_t& a, uint32_t& b) {
  const auto p = HALF ? __builtin_amdgcn_permlane32_swap(v, v, false, false)
                      : __builtin_amdgcn_permlane16_swap(v, v, false, false);
  a = p[0];
  b = p[1];
}
template <bool HALF>
__device__ __forceinline__ void both(float v, float& a, float& b) {
  uint32_t x, y;
  both<HALF>(__float_as_uint(v), x, y);
  a = __uint_as_float(x);
  b = __uint_as_float(y);
}
template <bool HALF>
__device__ __forceinline__ void both(double v, double& a, double& b) {
  const uint64_t w = (uint64_t)__double_as_longlong(v);
  uint32_t x0, x1, y0, y1;
  both<HALF>((uint32_t)w, x0, y0);
  both<HALF>((uint32_t)(w >> 32), x1, y1);
  a = __longlong_as_double((long long)((uint64_t)x1 << 32 | x0));
  b = __longlong_as_double((long long)((uint64_t)y1 << 32 | y0));
}

// op over the token's lanes; every lane ends with the result.
template <int LANES, class T, class Op>
__device__ __forceinline__ T route_all(T v, Op op) {
  v = op(v, row_turn<8>(v));
  v = op(v, row_turn<4>(v));
  v = op(v, row_turn<2>(v));
  v = op(v, row_turn<1>(v));
  if constexpr (LANES == 64) {
    T a, b;
    both<false>(v, a, b);
    v = op(a, b);
    both<true>(v, a, b);
    v = op(a, b);
  }
  return v;
}

// ---------------------------------------------------------------------------
// lists of keys, highest first
// ---------------------------------------------------------------------------
__device__ __forceinline__ void key_order(double& a, double& b) {
  const double hi = __builtin_fmax(a, b), lo = __builtin_fmin(a, b);
  a = hi;
  b = lo;
}

template <int N>
__device__ __forceinline__ void keys_sort(double* v) {
#pragma unroll
  for (int k = 2; k <= N; k *= 2)
#pragma unroll
    for (int j = k / 2; j > 0; j /= 2)
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (!(i & j)) {
          if (!(i & k)) key_order(v[i], v[i | j]);
          else key_order(v[i | j], v[i]);
        }
}

// a: the highest K of two lists of K.
template <int K>
__device__ __forceinline__ void keys_merge(double (&a)[K], const double (&b)[K]) {
#pragma unroll
  for (int i = 0; i < K; ++i) a[i] = __builtin_fmax(a[i], b[K - 1 - i]);
#pragma unroll
  for (int j = K / 2; j > 0; j /= 2)
#pragma unroll
    for (int i = 0; i < K; ++i)
      if (!(i & j)) key_order(a[i], a[i | j]);
}

template <int N, int K>
__device__ __forceinline__ void keys_turn(double (&a)[K]) {
  double b[K];
#pragma unroll
  for (int i = 0; i < K; ++i) b[i] = row_turn<N>(a[i]);
  keys_merge<K>(a, b);
}
template <bool HALF, int K>
__device__ __forceinline__ void keys_both(double (&a)[K]) {
  double b[K];
#pragma unroll
  for (int i = 0; i < K; ++i) both<HALF>(a[i], a[i], b[i]);
  keys_merge<K>(a, b);
}

// ---------------------------------------------------------------------------
// one token
// ---------------------------------------------------------------------------
__device__ __forceinline__ void wave_sync() {  // LDS of other lanes of this wave
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ float sigmoid_f(float l) { return 1.f / (1.f + exp_f(-l)); }

// What a token of grouped routing needs of LDS.
template <int LANES, int VPL>
struct RouteLds {
  double value[LANES * VPL];
  double grade[kRouteMaxGroups];
};

// l[i] is the logit of expert LANES i + lane (any value past the experts).  Lane s
// ends with choice s and its weight.
template <int LANES, int VPL, int K>
__device__ __forceinline__ void route_token(const RouteRule& q, const float (&l)[VPL], int lane,
                                            RouteLds<LANES, VPL>* lds, int& id, float& weight) {
  const auto max_f = [](float a, float b) { return __builtin_fmaxf(a, b); };
  const auto sum_f = [](float a, float b) { return a + b; };
  const bool softmax = q.scoring == 0;
  const bool sums = q.groups > 1 && q.top2;
  float high = -__builtin_huge_valf();  // of the logits, NaN aside
  if (softmax) {
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (LANES * i + lane < q.experts) high = max_f(high, l[i]);
    high = route_all<LANES>(high, max_f);
  }
  double v[VPL];
  if (q.balance || sums) {  // scores in 64 bits
    double total = 1.0;
    if (softmax) {
      total = 0.0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        v[i] = exp((double)l[i] - (double)high);
        if (LANES * i + lane < q.experts) total += v[i];
      }
      total = route_all<LANES>(total, [](double a, double b) { return a + b; });
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = LANES * i + lane;
      const double s = softmax ? v[i] / total : 1.0 / (1.0 + exp(-(double)l[i]));
      v[i] = q.balance && e < q.experts ? s + (double)q.balance[e] : s;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] = (double)l[i];
  }
  if (q.groups > 1) {
    // a group a lane; a group is kept if fewer than topk_groups are graded higher, or as
    // high and before it
#pragma unroll
    for (int i = 0; i < VPL; ++i) lds->value[LANES * i + lane] = route_key(v[i], LANES * i + lane);
    wave_sync();
    for (int g = lane; g < q.groups; g += LANES) {
      double best = kKeyNone, second = kKeyNone;
      for (int j = 0; j < q.group_size; ++j) {
        const double key = lds->value[g * q.group_size + j];
        second = __builtin_fmax(second, __builtin_fmin(best, key));
        best = __builtin_fmax(best, key);
      }
      const double grade = q.top2 ? route_value(best) + route_value(second) : route_value(best);
      lds->grade[g] = route_key(grade, g);
    }
    wave_sync();
    uint64_t kept = 0;
    for (int g0 = 0; g0 < q.groups; g0 += LANES) {
      const int g = g0 + lane;
      bool keep = false;
      if (g < q.groups) {
        const double mine = lds->grade[g];
        int ahead = 0;
        for (int o = 0; o < q.groups; ++o) ahead += lds->grade[o] > mine;
        keep = ahead < q.topk_groups;
      }
      const uint64_t all = __ballot(keep);
      if constexpr (LANES == 64) kept = all;
      else kept |= ((all >> (threadIdx.x & 48)) & 0xFFFFull) << g0;
    }
    wave_sync();
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const uint32_t e = LANES * i + lane;
      const bool in = e < (uint32_t)q.experts && (kept >> ((e * q.group_inverse) >> 20) & 1);
      const double key = route_key(!q.balance ? (double)l[i] : v[i], e);
      v[i] = in ? key : kKeyNone;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = LANES * i + lane;
      v[i] = e < q.experts ? route_key(v[i], e) : kKeyNone;
    }
  }
  double top[K];
  if constexpr (VPL < K) {
    keys_sort<VPL>(v);
#pragma unroll
    for (int i = 0; i < K; ++i) top[i] = i < VPL ? v[i < VPL ? i : 0] : kKeyNone;
  } else {
    keys_sort<K>(v);
#pragma unroll
    for (int i = 0; i < K; ++i) top[i] = v[i];
#pragma unroll
    for (int c = K; c < VPL; c += K) {
      double next[K];
      keys_sort<K>(v + c);
#pragma unroll
      for (int i = 0; i < K; ++i) next[i] = v[c + i];
      keys_merge<K>(top, next);
    }
  }
  keys_turn<8>(top);
  keys_turn<4>(top);
  keys_turn<2>(top);
  keys_turn<1>(top);
  if constexpr (LANES == 64) {
    keys_both<false>(top);
    keys_both<true>(top);
  }
  double mine = top[0];
#pragma unroll
  for (int s = 1; s < K; ++s) mine = lane == s ? top[s] : mine;
  id = (int)route_place(mine);
  // its logit, from the lane that holds it
  float chosen = 0.f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const float o = __shfl(l[i], id % LANES, LANES);
    chosen = id / LANES == i ? o : chosen;
  }
  if (softmax) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) sum += LANES * i + lane < q.experts ? exp_f(l[i] - high) : 0.f;
    weight = exp_f(chosen - high) / route_all<LANES>(sum, sum_f);
  } else {
    weight = sigmoid_f(chosen);
  }
  if (q.renormalize) weight = weight / route_all<LANES>(lane < q.topk ? weight : 0.f, sum_f);
  weight *= q.scale;
}

}  // namespace exl3
