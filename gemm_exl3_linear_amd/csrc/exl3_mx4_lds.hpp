// Copies from memory straight to LDS, and LDS reads by address (gfx950).
#pragma once

#include "exl3_mx4.hpp"

namespace exl3 {

typedef __attribute__((address_space(3))) uint8_t lds_u8;

__device__ __forceinline__ u32x4_t lds_read16(uint32_t at) {
  return *reinterpret_cast<const __attribute__((address_space(3))) u32x4_t*>((const lds_u8*)(uintptr_t)at);
}
__device__ __forceinline__ u32x2_t lds_read8(uint32_t at) {
  return *reinterpret_cast<const __attribute__((address_space(3))) u32x2_t*>((const lds_u8*)(uintptr_t)at);
}

// 16 (4) bytes a lane from a buffer to LDS: lane l's land at `at` + 16 l (4 l).
// The source needs dword alignment.
// Written as assembly so that the compiler, which cannot tell the stages
// apart, does not wait for it before every LDS read; the kernel waits itself
// before the barrier that hands a stage over.  The LDS address is an operand in M0,
// so the compiler, which writes it there, knows what M0 holds; one wait state lies
// between the two.
__device__ __forceinline__ void lds_copy16(u32x4_t rsrc, uint32_t at, uint32_t lane_off, uint32_t off) {
  asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
               :
               : "v"(lane_off), "s"(rsrc), "s"(off), "{m0}"(at)
               : "memory");
}
__device__ __forceinline__ void lds_copy4(u32x4_t rsrc, uint32_t at, uint32_t lane_off, uint32_t off) {
  asm volatile("s_nop 0\n\tbuffer_load_dword %0, %1, %2 offen lds"
               :
               : "v"(lane_off), "s"(rsrc), "s"(off), "{m0}"(at)
               : "memory");
}

// A lane offset that is past the end of every buffer here.
constexpr uint32_t kPastEnd = 0xFFFFFFF0u;

// Raw buffer descriptor over [p, p + bytes): loads past its end give zeros.
__device__ __forceinline__ u32x4_t buffer_words(const uint8_t* p, uint64_t bytes) {
  const uint64_t at = reinterpret_cast<uint64_t>(p);
  u32x4_t w = {(uint32_t)at, (uint32_t)(at >> 32) & 0xFFFFu, (uint32_t)bytes, (uint32_t)kBufferRsrcWord3};
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = (uint32_t)__builtin_amdgcn_readfirstlane((int)w[i]);
  return w;
}

}  // namespace exl3
