// MXFP4 quantisation and its inverse.
//
// Quantisation of a block of 32: with e the largest fp32 exponent field of its
// elements, the scale byte is s = max(e - 2, 0) (the specification's
// 2^(floor(log2 max|x|) - 2); an all-zero or subnormal block gets 0), and the
// codes are x * 2^(127 - s) rounded to E2M1 by the conversion instruction (to
// nearest, ties to even, saturating at 6).  Every step is exact but that one
// rounding, which the format asks for.  e = 255 (a NaN or an infinity) makes
// the block NaN: s = 255, codes 0.
//
// Both kernels are bound by HBM.  A thread takes eight elements, so a wave's
// loads, its 4-byte code stores and its value stores are contiguous; the four
// lanes of a block meet in two quad permutations.  Measured: 4096 x 5120 fp16
// 11.6 us there and 8.7 back (52 MB each), 10007 x 6880 fp32 75 and 63 us (312 MB
// each, 4.2 and 5.0 TB/s; a 2 GiB copy reaches 4.9).  One row of 5120: 1.6 us each,
// a launch.
#include "exl3_internal.hpp"
#include "exl3_mx4.hpp"

namespace exl3 {

constexpr int kMx4QuantThreads = 256;
constexpr int kMx4QuantElems = 8;  // elements per thread

// Largest of the four lanes of a quad.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, kDppXor1, 0xF, 0xF, true);
  v = v > o ? v : o;
  o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, kDppXor2, 0xF, 0xF, true);
  return v > o ? v : o;
}

template <bool F32>
__global__ __launch_bounds__(kMx4QuantThreads) void mx4_quantize_kernel(
    const void* __restrict__ x, int64_t ldx, int64_t chunks, uint32_t row_chunks,
    uint32_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  // chunk: eight consecutive elements; a block's four chunks are one quad, and
  // chunks is a multiple of 4, so a quad is in range as a whole
  const int64_t c = (int64_t)blockIdx.x * kMx4QuantThreads + threadIdx.x;
  if (c >= chunks) return;
  int64_t off = c * kMx4QuantElems;
  if (ldx != (int64_t)row_chunks * kMx4QuantElems) {
    const int64_t row = c / row_chunks;
    off = row * ldx + (c - row * row_chunks) * kMx4QuantElems;
  }
  float v[8];
  if constexpr (F32) {
    const float4_t a = *reinterpret_cast<const float4_t*>(static_cast<const float*>(x) + off);
    const float4_t b = *reinterpret_cast<const float4_t*>(static_cast<const float*>(x) + off + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  } else {
    const f16x8_t h = *reinterpret_cast<const f16x8_t*>(static_cast<const _Float16*>(x) + off);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)h[i];
  }
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __float_as_uint(v[i]) & 0x7FFFFFFFu;
    top = top > b ? top : b;
  }
  const uint32_t e = quad_max(top) >> 23;
  const bool bad = e == 255u;
  const uint32_t s = bad ? 255u : (e > 2u ? e - 2u : 0u);
  const float inv = __uint_as_float((254u - (bad ? 0u : s)) << 23);  // 2^(127 - s), normal
  uint32_t q = 0;
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0] * inv, v[1] * inv, 1.0f, 0);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2] * inv, v[3] * inv, 1.0f, 1);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4] * inv, v[5] * inv, 1.0f, 2);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6] * inv, v[7] * inv, 1.0f, 3);
  codes[c] = bad ? 0u : q;
  if ((threadIdx.x & 3) == 0) scales[c >> 2] = (uint8_t)s;
}

template <bool F32>
__global__ __launch_bounds__(kMx4QuantThreads) void mx4_reconstruct_kernel(
    const uint32_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t chunks,
    uint32_t row_chunks, void* __restrict__ out, int64_t ldo) {
  const int64_t c = (int64_t)blockIdx.x * kMx4QuantThreads + threadIdx.x;
  if (c >= chunks) return;
  int64_t off = c * kMx4QuantElems;
  if (ldo != (int64_t)row_chunks * kMx4QuantElems) {
    const int64_t row = c / row_chunks;
    off = row * ldo + (c - row * row_chunks) * kMx4QuantElems;
  }
  const f16x8_t h = mx4_to_f16(codes[c]);
  const float sc = mx4_scale(scales[c >> 2]);
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = (float)h[i] * sc;  // exact below 2^128
  if constexpr (F32) {
    float* o = static_cast<float*>(out) + off;
    *reinterpret_cast<float4_t*>(o) = float4_t{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<float4_t*>(o + 4) = float4_t{v[4], v[5], v[6], v[7]};
  } else {
    f16x8_t r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = (_Float16)v[i];
    *reinterpret_cast<f16x8_t*>(static_cast<_Float16*>(out) + off) = r;
  }
}

hipError_t launch_mx4_quantize(const void* x, bool f32, int64_t rows, int64_t k, int64_t ldx,
                               uint8_t* codes, uint8_t* scales, hipStream_t s) {
  const int64_t chunks = rows * (k / kMx4QuantElems);
  const dim3 grid((uint32_t)((chunks + kMx4QuantThreads - 1) / kMx4QuantThreads));
  uint32_t* c = reinterpret_cast<uint32_t*>(codes);
  const uint32_t rc = (uint32_t)(k / kMx4QuantElems);
  if (f32)
    hipLaunchKernelGGL((mx4_quantize_kernel<true>), grid, dim3(kMx4QuantThreads), 0, s, x, ldx, chunks, rc, c, scales);
  else
    hipLaunchKernelGGL((mx4_quantize_kernel<false>), grid, dim3(kMx4QuantThreads), 0, s, x, ldx, chunks, rc, c, scales);
  return hipGetLastError();
}

hipError_t launch_mx4_reconstruct(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t k,
                                  void* out, bool f32, int64_t ldo, hipStream_t s) {
  const int64_t chunks = rows * (k / kMx4QuantElems);
  const dim3 grid((uint32_t)((chunks + kMx4QuantThreads - 1) / kMx4QuantThreads));
  const uint32_t* c = reinterpret_cast<const uint32_t*>(codes);
  const uint32_t rc = (uint32_t)(k / kMx4QuantElems);
  if (f32)
    hipLaunchKernelGGL((mx4_reconstruct_kernel<true>), grid, dim3(kMx4QuantThreads), 0, s, c, scales, chunks, rc, out, ldo);
  else
    hipLaunchKernelGGL((mx4_reconstruct_kernel<false>), grid, dim3(kMx4QuantThreads), 0, s, c, scales, chunks, rc, out, ldo);
  return hipGetLastError();
}

}  // namespace exl3
