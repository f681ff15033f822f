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
// Both kernels are bound by HBM.  Quantising, a thread takes eight elements, so a
// wave's loads and its 4-byte code stores are contiguous; the four lanes of a block
// meet in two quad permutations.  Back, a thread stores 16 bytes four times.
// Measured: 4096 x 5120 fp16 12 us there and 10 back (53 MB each, some of it from
// the last-level cache; 14 and 10 over 1.5 GB of tensors in turn), 14000 x 5120 fp32
// 56 and 46 us (325 MB each, 5.8 and 7.0 TB/s; a 2 GiB copy reaches 4.9).  One row of
// 5120: 1.6 to 2 us each, a launch.
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

// Values a thread stores at once (16 bytes), how often, a workgroup's width apart.
template <bool F32>
constexpr int kMx4BackElems = F32 ? 4 : 8;
constexpr int kMx4BackTimes = 4;

// STREAM: values past the caches (kMx4StreamBytes) are stored without a place in
// them, where they would push out what waits to be written: 14000 x 5120 fp32 46 us,
// 57 with (65 with one chunk of 32 bytes a thread); the kernel that follows gains as
// much.  42 MB of values are 8 and 10 us, but what reads them next then takes 1 us
// longer.  (Loads of the quantized values gained nothing so.)
constexpr int64_t kMx4StreamBytes = (int64_t)64 << 20;
template <bool F32, bool STREAM>
__global__ __launch_bounds__(kMx4QuantThreads) void mx4_reconstruct_kernel(
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t chunks,
    uint32_t row_chunks, void* __restrict__ out, int64_t ldo) {
  constexpr int E = kMx4BackElems<F32>;
  const int64_t first = (int64_t)blockIdx.x * (kMx4QuantThreads * kMx4BackTimes) + threadIdx.x;
  uint32_t in[kMx4BackTimes], scale[kMx4BackTimes];
#pragma unroll
  for (int u = 0; u < kMx4BackTimes; ++u) {
    const int64_t c = first + u * kMx4QuantThreads;
    in[u] = scale[u] = 0;
    if (c >= chunks) continue;
    if constexpr (F32)
      in[u] = reinterpret_cast<const uint16_t*>(codes)[c];
    else
      in[u] = reinterpret_cast<const uint32_t*>(codes)[c];
    scale[u] = scales[c / (kMx4Block / E)];
  }
#pragma unroll
  for (int u = 0; u < kMx4BackTimes; ++u) {
    const int64_t c = first + u * kMx4QuantThreads;
    if (c >= chunks) continue;
    int64_t off = c * E;
    if (ldo != (int64_t)row_chunks * E) {
      const int64_t row = c / row_chunks;
      off = row * ldo + (c - row * row_chunks) * E;
    }
    const f16x8_t h = mx4_to_f16(in[u]);
    const float sc = mx4_scale(scale[u]);
    float v[E];
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = (float)h[i] * sc;  // exact below 2^128
    u32x4_t o;
    if constexpr (F32) {
      o = __builtin_bit_cast(u32x4_t, float4_t{v[0], v[1], v[2], v[3]});
    } else {
      f16x8_t r;
#pragma unroll
      for (int i = 0; i < E; ++i) r[i] = (_Float16)v[i];
      o = __builtin_bit_cast(u32x4_t, r);
    }
    u32x4_t* to = reinterpret_cast<u32x4_t*>(static_cast<uint8_t*>(out) + off * (F32 ? 4 : 2));
    if constexpr (STREAM)
      __builtin_nontemporal_store(o, to);
    else
      *to = o;
  }
}

hipError_t launch_mx4_quantize(const void* x, bool f32, int64_t rows, int64_t k, int64_t ldx,
                               uint8_t* codes, uint8_t* scales, hipStream_t s) {
  const int64_t chunks = rows * (k / kMx4QuantElems);
  const dim3 grid((uint32_t)((chunks + kMx4QuantThreads - 1) / kMx4QuantThreads)), block(kMx4QuantThreads);
  uint32_t* c = reinterpret_cast<uint32_t*>(codes);
  const uint32_t rc = (uint32_t)(k / kMx4QuantElems);
  if (f32)
    hipLaunchKernelGGL(mx4_quantize_kernel<true>, grid, block, 0, s, x, ldx, chunks, rc, c, scales);
  else
    hipLaunchKernelGGL(mx4_quantize_kernel<false>, grid, block, 0, s, x, ldx, chunks, rc, c, scales);
  return hipGetLastError();
}

template <bool F32>
static hipError_t reconstruct(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t k, void* out,
                              int64_t ldo, hipStream_t s) {
  constexpr int kGroup = kMx4QuantThreads * kMx4BackTimes;
  const int64_t row_chunks = k / kMx4BackElems<F32>, chunks = rows * row_chunks;
  const dim3 grid((uint32_t)((chunks + kGroup - 1) / kGroup)), block(kMx4QuantThreads);
  const uint32_t rc = (uint32_t)row_chunks;
  if (chunks * 16 >= kMx4StreamBytes)
    hipLaunchKernelGGL((mx4_reconstruct_kernel<F32, true>), grid, block, 0, s, codes, scales, chunks, rc, out, ldo);
  else
    hipLaunchKernelGGL((mx4_reconstruct_kernel<F32, false>), grid, block, 0, s, codes, scales, chunks, rc, out, ldo);
  return hipGetLastError();
}
hipError_t launch_mx4_reconstruct(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t k,
                                  void* out, bool f32, int64_t ldo, hipStream_t s) {
  return f32 ? reconstruct<true>(codes, scales, rows, k, out, ldo, s)
             : reconstruct<false>(codes, scales, rows, k, out, ldo, s);
}

}  // namespace exl3
