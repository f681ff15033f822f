// Sums between workgroups and over a wave, and a short exponential, shared by the
// expert layers and the routing.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace exl3 {

// Sums that the last workgroup to arrive takes from the others, which run on
// other XCDs, pass by stores and loads of device scope: those do not stay in an
// XCD's L2, so a wave that has waited for its stores may count itself in.  (Fences
// of device scope write the L2 back and drop it: 1 to 2 us.)
__device__ __forceinline__ void store_shared(float* p, float v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float load_shared(const float* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void wait_stores() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
// Counts one of n in; true for the last, which leaves 0.
__device__ __forceinline__ bool last_in(uint32_t* count, uint32_t n) {
  const bool last = __hip_atomic_fetch_add(count, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == n - 1;
  if (last) __hip_atomic_store(count, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return last;
}

// Reductions over a wave on the vector unit alone: shifts by 1, 2, 4, 8 inside
// the rows of 16 lanes, then row ends to the next row and to the upper half; lane
// 63 ends with the result.  (Six LDS permutes took 6 x 100 cycles a choice.)
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_or_zero(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, ROWS == 0xF);
}
template <class Op>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t v, Op op) {  // 0 is neutral
  v = op(v, dpp_or_zero<0x111, 0xF>(v));
  v = op(v, dpp_or_zero<0x112, 0xF>(v));
  v = op(v, dpp_or_zero<0x114, 0xF>(v));
  v = op(v, dpp_or_zero<0x118, 0xF>(v));
  v = op(v, dpp_or_zero<0x142, 0xA>(v));
  v = op(v, dpp_or_zero<0x143, 0xC>(v));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  return wave_reduce(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
__device__ __forceinline__ float wave_sum_f(float v) {
  return __uint_as_float(wave_reduce(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

// e^x in few instructions: x log2 e with the product's own rounding error, and log2
// e's, put back after the power.  To about an ulp for 2^-125 < e^x < 2^126; past that, where
// a correction could meet an infinity or a subnormal, without it: off by up to 2^-17 of
// the value.  (The routing runs once
// a call, so its instructions come from memory: their number is its time.)
__device__ __forceinline__ float exp_f(float x) {
  constexpr float kLog2e = 1.44269502162933349609375f, kLog2eRest = 1.925963033500e-8f, kLn2 = 0.693147180559945309f;
  const float t = x * kLog2e;
  const float rest = __builtin_fmaf(x, kLog2eRest, __builtin_fmaf(x, kLog2e, -t));
  const float p = __builtin_amdgcn_exp2f(t);
  return t > 126.f || t < -125.f ? p : __builtin_fmaf(p, rest * kLn2, p);
}

}  // namespace exl3
