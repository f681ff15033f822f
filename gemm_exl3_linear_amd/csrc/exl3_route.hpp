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

// The key of a finite value v at place e: larger for larger v, then for lower e.
__device__ __forceinline__ double route_key_finite(double v, uint32_t e) {
  const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);  // -0 is 0
  const uint32_t sign = (uint32_t)((int32_t)(b >> 32) >> 31);
  return __longlong_as_double((long long)((b & ~(uint64_t)kKeyPlace) | ((kKeyPlace - e) ^ (sign & kKeyPlace))));
}
// The same of any value.
__device__ __forceinline__ double route_key(double v, uint32_t e) {
  const double held = __builtin_fmax(__builtin_fmin(v, kKeyInf), -kKeyInf);
  return route_key_finite(v != v ? kKeyNan : held, e);
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

// The value of another lane of the same row of 16.
template <int CTRL>
__device__ __forceinline__ uint32_t row_move(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}
template <int CTRL>
__device__ __forceinline__ float row_move(float v) {
  return __uint_as_float(row_move<CTRL>(__float_as_uint(v)));
}
template <int CTRL>
__device__ __forceinline__ double row_move(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  const uint64_t lo = row_move<CTRL>((uint32_t)b), hi = row_move<CTRL>((uint32_t)(b >> 32));
  return __longlong_as_double((long long)(hi << 32 | lo));
}
// Of the lane N places on in the row.
template <int N, class T>
__device__ __forceinline__ T row_turn(T v) {
  return row_move<0x120 + N>(v);
}
// Of the lane ^ 1 and of the lane ^ 2.
template <class T>
__device__ __forceinline__ T row_pair(T v) {
  return row_move<0xB1>(v);
}
template <class T>
__device__ __forceinline__ T row_other_pair(T v) {
  return row_move<0x4E>(v);
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

// v + that of the other half of the wave (HALF), or of the other row of a pair of rows.
template <bool HALF, class T>
__device__ __forceinline__ T add_both(T v) {
  T a, b;
  both<HALF>(v, a, b);
  return a + b;
}

// The sum of a token's values; every lane ends with it.  Up to 256 experts one tree for
// 16 lanes and for 64, so that a token's bits do not depend on the number of tokens: fours
// of neighbours in two pairs, then the fours that lie 16 apart, then 8, 4, 2 and 1 apart.
// Zeros past the experts change no sum.
template <int LANES, int VPL, class T>
__device__ __forceinline__ T route_sum(const T (&v)[VPL]) {
  static_assert(LANES == 64 || (VPL >= 4 && VPL <= 16), "16 lanes hold fours of up to 256 experts");
  if constexpr (VPL == 1) {
    T s = v[0] + row_pair(v[0]);
    s += row_other_pair(s);
    s = add_both<false>(add_both<true>(s));
    s += row_turn<8>(s);
    return s + row_turn<4>(s);
  } else if constexpr (VPL == 2) {
    T s = v[0] + v[1];
    s += row_pair(s);
    s = add_both<false>(add_both<true>(s));
    s += row_turn<8>(s);
    s += row_turn<4>(s);
    return s + row_turn<2>(s);
  } else {
    T four[VPL / 4];
#pragma unroll
    for (int c = 0; c < VPL / 4; ++c) four[c] = (v[4 * c] + v[4 * c + 1]) + (v[4 * c + 2] + v[4 * c + 3]);
#pragma unroll
    for (int d = 1; d < VPL / 4; d *= 2)
#pragma unroll
      for (int c = 0; c < VPL / 4; c += 2 * d) four[c] += four[c + d];
    T s = four[0];
    if constexpr (LANES == 64) s = add_both<true>(add_both<false>(s));
    s += row_turn<8>(s);
    s += row_turn<4>(s);
    s += row_turn<2>(s);
    return s + row_turn<1>(s);
  }
}

// ---------------------------------------------------------------------------
// lists of keys, highest first
// ---------------------------------------------------------------------------
__device__ __forceinline__ void key_order(double& a, double& b) {
  const double hi = __builtin_fmax(a, b), lo = __builtin_fmin(a, b);
  a = hi;
  b = lo;
}

// Batcher's odd-even merge sort, highest first (19 pairs for eight).
template <int N>
__device__ __forceinline__ void keys_sort(double* v) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (j + i + k < N && (j + i) / (2 * p) == (j + i + k) / (2 * p)) key_order(v[j + i], v[j + i + k]);
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
// scores in 64 bits
// ---------------------------------------------------------------------------
// e^x for x that is not NaN, to 2^-46 of itself: 2^n 2^f with |f| <= 1/2 and the Taylor
// series of 2^f up to its 11th term (the 12th is at most 2^-47.2, all errors together
// 2^-46.7 in a trial of 1500 f; values are compared to 2^-42, and each term costs every
// score an instruction).  From e^708 on that, below 2^-1074 zero.
__device__ __forceinline__ double exp_d(double x) {
  constexpr double kLog2e = 1.4426950408889634, kLog2eRest = 2.0355273740931033e-17, kLn2 = 0.6931471805599453;
  x = __builtin_fmax(__builtin_fmin(x, 708.0), -760.0);
  const double n = __builtin_rint(x * kLog2e);
  const double f = __builtin_fma(x, kLog2eRest, __builtin_fma(x, kLog2e, -n));
  constexpr double c2 = kLn2 * kLn2 / 2, c3 = c2 * kLn2 / 3, c4 = c3 * kLn2 / 4, c5 = c4 * kLn2 / 5,
                   c6 = c5 * kLn2 / 6, c7 = c6 * kLn2 / 7, c8 = c7 * kLn2 / 8, c9 = c8 * kLn2 / 9,
                   c10 = c9 * kLn2 / 10, c11 = c10 * kLn2 / 11;
  double p = __builtin_fma(f, c11, c10);
  p = __builtin_fma(f, p, c9);
  p = __builtin_fma(f, p, c8);
  p = __builtin_fma(f, p, c7);
  p = __builtin_fma(f, p, c6);
  p = __builtin_fma(f, p, c5);
  p = __builtin_fma(f, p, c4);
  p = __builtin_fma(f, p, c3);
  p = __builtin_fma(f, p, c2);
  p = __builtin_fma(f, p, kLn2);
  p = __builtin_fma(f, p, 1.0);
  return __builtin_ldexp(p, (int)n);
}

// 1 / y for 1 <= y < 2^1023: the instruction's estimate and two Newton steps.
__device__ __forceinline__ double recip_d(double y) {
  double r = __builtin_amdgcn_rcp(y);
  r = __builtin_fma(r, __builtin_fma(-y, r, 1.0), r);
  return __builtin_fma(r, __builtin_fma(-y, r, 1.0), r);
}

// ---------------------------------------------------------------------------
// one token
// ---------------------------------------------------------------------------
__device__ __forceinline__ void wave_sync() {  // LDS of other lanes of this wave
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ float sigmoid_f(float l) { return 1.f / (1.f + exp_f(-l)); }

// A lane's i-th expert: four (or all, if fewer) neighbours a lane.
template <int LANES, int VPL>
__device__ __forceinline__ int route_expert(int i, int lane) {
  constexpr int V = VPL < 4 ? VPL : 4;
  return i / V * (LANES * V) + lane * V + i % V;
}

// The chosen expert's logit from the lane (of 64) that holds it: 0.5 us sooner than a sum
// of shares again (a logit that is in memory comes 0.2 us sooner from there).
template <int VPL>
__device__ __forceinline__ float route_held(const float (&l)[VPL], int chosen) {
  constexpr int V = VPL < 4 ? VPL : 4;
  const int from = chosen / V % 64;
  float at = 0.f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const float o = __shfl(l[i], from);
    at = route_expert<64, VPL>(i, from) == chosen ? o : at;
  }
  return at;
}

// What a token of grouped routing needs of LDS: values, or the two best of four.
template <int LANES, int VPL>
struct RouteLds {
  double value[LANES * VPL];
  double grade[kRouteMaxGroups];
};

// The keys of a lane's values.  (What is not finite is rare, and its instructions, which
// a call of few tokens waits for, stay out of the way.)
template <int LANES, int VPL>
__device__ __forceinline__ void route_keys(double (&v)[VPL], bool finite, int lane) {
  if (__builtin_expect(finite, 1)) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] = route_key_finite(v[i], route_expert<LANES, VPL>(i, lane));
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] = route_key(v[i], route_expert<LANES, VPL>(i, lane));
  }
}

// The groups that are kept, a bit each: fewer than topk_groups are graded higher, or as
// high and before it.  key: a lane's keys.
template <int LANES, int VPL>
__device__ __forceinline__ uint64_t route_groups(const RouteRule& q, const double (&key)[VPL], int lane,
                                                 RouteLds<LANES, VPL>* lds) {
  const bool fours = VPL >= 4 && q.group_size % 4 == 0;  // four neighbours are of one group
  if (fours) {
#pragma unroll
    for (int i = 0; i + 3 < VPL; i += 4) {
      double k[4] = {key[i], key[i + 1], key[i + 2], key[i + 3]};
      key_order(k[0], k[1]);
      key_order(k[2], k[3]);
      double* at = lds->value + route_expert<LANES, VPL>(i, lane) / 2;
      at[0] = __builtin_fmax(k[0], k[2]);
      at[1] = __builtin_fmax(__builtin_fmin(k[0], k[2]), __builtin_fmax(k[1], k[3]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) lds->value[route_expert<LANES, VPL>(i, lane)] = key[i];
  }
  wave_sync();
  for (int g = lane; g < q.groups; g += LANES) {
    double best = kKeyNone, second = kKeyNone;
    const int n = q.group_size / (fours ? 2 : 1);
    const double* at = lds->value + g * n;
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
      second = __builtin_fmax(second, __builtin_fmin(best, at[j]));
      best = __builtin_fmax(best, at[j]);
    }
    lds->grade[g] = route_key(route_value(best) + (q.top2 ? route_value(second) : 0.0), g);
  }
  wave_sync();
  uint64_t kept = 0;
  for (int g0 = 0; g0 < q.groups; g0 += LANES) {
    const int g = g0 + lane;
    const double mine = g < q.groups ? lds->grade[g] : kKeyNone;
    int ahead = 0;
#pragma unroll 4
    for (int o = 0; o < q.groups; ++o) ahead += lds->grade[o] > mine;
    const uint64_t all = __ballot(g < q.groups && ahead < q.topk_groups);
    if constexpr (LANES == 64) kept = all;
    else kept |= ((all >> (threadIdx.x & 48)) & 0xFFFFull) << g0;
  }
  wave_sync();
  return kept;
}

// l[i] is the logit of the lane's i-th expert (any value past the experts); logit(e) gives
// expert e's again, and is asked for experts alone.  Lane s < topk ends with choice s and
// its weight.
template <int LANES, int VPL, int K, class Logit>
__device__ __forceinline__ void route_token(const RouteRule& q, float (&l)[VPL], int lane,
                                            RouteLds<LANES, VPL>* lds, const Logit& logit, int& id, float& weight) {
#pragma clang fp contract(off)  // the same roundings in every instance
  const auto max_f = [](float a, float b) { return __builtin_fmaxf(a, b); };
  const auto sum_f = [](float a, float b) { return a + b; };
  const bool softmax = q.scoring == 0, ragged = q.experts < LANES * VPL;
  float worst = 0.f;  // NaN if a logit is not finite
#pragma unroll
  for (int i = 0; i < VPL; ++i) worst = __builtin_fmaf(l[i], 0.f, worst);
  const bool finite = !__any(worst != 0.f);
  if (ragged) {  // past the experts: nothing to the highest and to the softmax's sum
#pragma unroll
    for (int i = 0; i < VPL; ++i) l[i] = route_expert<LANES, VPL>(i, lane) < q.experts ? l[i] : -__builtin_huge_valf();
  }
  float high = -__builtin_huge_valf(), total = 0.f;  // of the logits (NaN aside) and of the softmax
  if (softmax) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) high = max_f(high, l[i]);
    high = route_all<LANES>(high, max_f);
    float part[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) part[i] = exp_f(l[i] - high);
    total = route_sum<LANES>(part);
  }
  double v[VPL];
  uint64_t kept = ~0ull;
  const auto none_past = [&] {
    if (ragged) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) v[i] = route_expert<LANES, VPL>(i, lane) < q.experts ? v[i] : kKeyNone;
    }
  };
  const bool scores = q.balance || (q.groups > 1 && q.top2);
  if (scores) {  // in 64 bits
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] = exp_d(softmax ? (double)l[i] - (double)high : -(double)l[i]);
    if (softmax) {
      const double scale = total != total ? __builtin_nan("") : recip_d(route_sum<LANES>(v));
#pragma unroll
      for (int i = 0; i < VPL; ++i) v[i] *= scale;
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) v[i] = recip_d(1.0 + v[i]);
      if (!finite) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) v[i] = l[i] != l[i] ? (double)l[i] : v[i];
      }
    }
    if (q.balance) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int e = route_expert<LANES, VPL>(i, lane);
        v[i] += (double)q.balance[e < q.experts ? e : 0];
      }
    }
    double odd = 0.0;  // NaN if a value is not finite
#pragma unroll
    for (int i = 0; i < VPL; ++i) odd = __builtin_fma(v[i], 0.0, odd);
    route_keys<LANES, VPL>(v, !__any(odd != 0.0), lane);
    none_past();
    if (q.groups > 1) kept = route_groups<LANES, VPL>(q, v, lane, lds);
  }
  if (!q.balance) {  // in the order of the logits
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] = (double)l[i];
    route_keys<LANES, VPL>(v, finite, lane);
    none_past();
    if (q.groups > 1 && !scores) kept = route_groups<LANES, VPL>(q, v, lane, lds);
  }
  if (q.groups > 1) {
    const bool fours = VPL >= 4 && q.group_size % 4 == 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      // four neighbours are of the first one's group; places past the experts, which hold
      // none, may lie past 64 groups
      const uint32_t e = route_expert<LANES, VPL>(fours ? i & ~3 : i, lane);
      v[i] = (kept >> (((e * q.group_inverse) >> 20) & 63) & 1) ? v[i] : kKeyNone;
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
  // (a lane past the choices may hold no expert's key, whose place is any)
  const float chosen = q.balance ? logit(lane < q.topk ? id : 0) : (float)route_value(mine);
  weight = softmax ? exp_f(chosen - high) / total : sigmoid_f(chosen);
  if (q.renormalize) weight = weight / route_all<LANES>(lane < q.topk ? weight : 0.f, sum_f);
  weight *= q.scale;
}

}  // namespace exl3
