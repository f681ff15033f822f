// Products with MXFP4 weights where the weights' bytes bound the time: a
// workgroup takes 16 MG rows by 16 NG columns of the output, its waves split k
// and meet in LDS at the end.
//
// A wave's unit is 256 k: lane (r = l % 16, g = l / 16) loads the two 16-byte
// blocks 8u + g and 8u + 4 + g of weight row r, so the four lanes of a row and
// the two loads cover one whole 128-byte line.  Either 128-k half of a unit is
//  - with 4-bit rows: the operand of one scaled 16x16x128 matrix instruction as
//    loaded (the instruction applies both scales; no arithmetic of our own);
//  - with fp16 rows: after a 4 x 4 transpose between the lane groups
//    (lane_group_transpose) dword j of every lane is a piece of block j, so
//    four 16x16x32 fp16 instructions take one block each, on the unscaled codes
//    (exact in fp16), and one fp32 multiply-add per sum applies the block's
//    scale.  A block's sum is formed before its scale, so any scale byte is
//    exact: weights times scales would leave fp16's range.
// Output columns are the weight rows (matrix operand B), so a lane's sums all
// belong to the column whose scales it loaded.
#pragma once

#include "exl3_mx4.hpp"

namespace exl3 {

constexpr int kMx4UnitK = 256;   // k of one unit
constexpr int kMx4UnitBytes = kMx4UnitK / 2;
constexpr int kMx4UnitBlocks = kMx4UnitK / kMx4Block;

// Codes and scale bytes of one row's unit, as one lane holds them.
struct Mx4Unit {
  u32x4_t half[2];   // blocks 8u + g and 8u + 4 + g
  uint32_t sc[2];    // scale bytes of blocks 8u .. 8u + 3 and 8u + 4 .. 8u + 7
};

// Row `row` of codes (k/2 bytes a row) and scales (kb = k/32 bytes a row),
// unit u; blocks past the row's end read as zeros with scale 1.
__device__ __forceinline__ void mx4_load_unit(const uint8_t* codes, const uint8_t* scales, int kb, int u, int g,
                                              Mx4Unit& t) {
  const uint8_t* c = codes + (int64_t)u * kMx4UnitBytes + 16 * g;
  const uint8_t* s = scales + u * kMx4UnitBlocks;
  if ((u + 1) * kMx4UnitBlocks <= kb) {
    t.half[0] = load16(c);
    t.half[1] = load16(c + 64);
    __builtin_memcpy(t.sc, s, 8);
  } else {
    const int left = kb - u * kMx4UnitBlocks;
    t.half[0] = t.half[1] = u32x4_t{0u, 0u, 0u, 0u};
    if (g < left) t.half[0] = load16(c);
    if (4 + g < left) t.half[1] = load16(c + 64);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      t.sc[h] = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b) t.sc[h] |= (4 * h + b < left ? (uint32_t)s[4 * h + b] : kMx4One) << (8 * b);
    }
  }
}

// Scale byte of block g of half h, in the low byte.
__device__ __forceinline__ uint32_t mx4_own_scale(const Mx4Unit& t, int h, int g) { return t.sc[h] >> (8 * g); }

// fp16 activations of half h of unit u, row x: [j] holds elements 8g .. 8g + 7
// of block j, zeros past the row's end or where the row is not there.
__device__ __forceinline__ void mx4_load_x(const uint16_t* x, bool there, int kb, int u, int h, int g,
                                           f16x8_t (&f)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int b = u * kMx4UnitBlocks + 4 * h + j;
    u32x4_t v = {0u, 0u, 0u, 0u};
    if (there && b < kb) v = load16(x + (int64_t)b * kMx4Block + 8 * g);
    f[j] = __builtin_bit_cast(f16x8_t, v);
  }
}

// acc[mg] += x[mg] times the half h of a unit of 16 weight rows.
template <int MG>
__device__ __forceinline__ void mx4_mma_f16(const f16x8_t (&x)[MG][4], const Mx4Unit& w, int h, float4_t (&acc)[MG]) {
  uint32_t d[4] = {w.half[h].x, w.half[h].y, w.half[h].z, w.half[h].w};
  lane_group_transpose(d);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const f16x8_t b = mx4_to_f16(d[j]);
    const float s = mx4_scale((w.sc[h] >> (8 * j)) & 0xFFu);
#pragma unroll
    for (int mg = 0; mg < MG; ++mg) {
      const float4_t p = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[mg][j], b, float4_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[mg][i] = __builtin_fmaf(p[i], s, acc[mg][i]);
    }
  }
}

}  // namespace exl3
