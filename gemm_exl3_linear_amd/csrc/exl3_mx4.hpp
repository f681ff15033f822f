// Device-side building blocks of the MXFP4 kernels (gfx950 / CDNA4, wave64).
//
// Format: a row of k elements (k a multiple of 32) is k/2 bytes of E2M1 codes,
// the even element in the low half of a byte, and k/32 E8M0 scale bytes s, each
// the factor 2^(s - 127) of 32 consecutive elements (255: NaN).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "exl3_device.hpp"

namespace exl3 {

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

constexpr int kMx4Block = 32;          // elements of a scale
constexpr int kMfmaFp4 = 4;            // operand format code of the f8f6f4 matrix instructions
constexpr uint32_t kMx4One = 127;      // scale byte of the factor 1

// 2^(s - 127) as fp32: the byte is the exponent field, but 0 is the subnormal
// 2^-127 and 255 is NaN (both need mantissa bit 22).
__device__ __forceinline__ float mx4_scale(uint32_t s) {
  const uint32_t odd = (s + 1u) & 0xFFu;  // 1 for s = 0, 0 for s = 255
  return __uint_as_float((s << 23) | (odd <= 1u ? 0x00400000u : 0u));
}

// Eight codes times a scale to eight fp16 values.
__device__ __forceinline__ f16x8_t mx4_to_f16(uint32_t codes, float scale = 1.0f) {
  const half2_t a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 0);
  const half2_t b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 1);
  const half2_t c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 2);
  const half2_t d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 3);
  return f16x8_t{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// Eight codes times a scale to eight bf16 values: exact (two significand bits and
// fp32's exponent range) but for magnitudes from 2^128, at scale bytes 253 and 254,
// which become infinities.
__device__ __forceinline__ bf16x8_t mx4_to_bf16(uint32_t codes, float scale) {
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
  const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
  return bf16x8_t{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// One 16 x 16 product over 128 k: lane (r = l % 16, g = l / 16) holds the
// 32 codes of k block g of row r of either operand, and their scale byte.
__device__ __forceinline__ float4_t mfma_mx4(u32x4_t a, uint32_t sa, u32x4_t b, uint32_t sb,
                                             float4_t c) {
  const i32x8_t A = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const i32x8_t B = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, c, kMfmaFp4, kMfmaFp4, 0, (int)sa,
                                                          0, (int)sb);
}

__device__ __forceinline__ u32x4_t load16(const void* p) {
  return *reinterpret_cast<const u32x4_t*>(p);
}

}  // namespace exl3
