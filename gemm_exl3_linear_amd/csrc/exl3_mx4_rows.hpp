// Products with MXFP4 weights where the weights' bytes bound the time: a
// workgroup takes 16 MG rows by 16 NG columns of the output, its waves split k
// and meet in LDS at the end.
//
// A wave's unit is 256 k: lane (r = l % 16, g = l / 16) loads the two 16-byte
// blocks 8u + g and 8u + 4 + g of weight row r, so the four lanes of a row and
// the two loads cover one whole 128-byte line.  Either 128-k half of a unit is
//  - with 4-bit rows: the operand of one scaled 16x16x128 matrix instruction as
//    loaded (the instruction applies both scales; no arithmetic of our own);
//  - with fp16 rows: 16 conversions to fp16 (code times scale, exact for scale
//    bytes 104 .. 140) and four 16x16x32 fp16 instructions, the j-th on the j-th
//    dword (piece) of every lane's block.  A wave that met a block with another
//    scale byte takes its whole share again, block by block: the unscaled codes, then
//    the sums by the block's scale (mx4_sum_blocks).
//    Few rows: with at most 16 / P of them, one operand carries P pieces, piece p
//    of row t in operand row p 16 / P + t, and piece p has sums of its own of which
//    only those rows are wanted.  One load then brings P pieces; loads of one
//    piece each, mostly masked, cost as much and bounded the time (5120 -> 17408,
//    one row: 16 us, 12.8 with four pieces; 12.1 with the loads of a whole unit
//    issued without branches).
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

// Where one lane's weight row lies: uniform bases (of a workgroup's first row)
// and 32-bit offsets, which a load takes as they are.
struct Mx4Row {
  const uint8_t* codes;
  const uint8_t* scales;
  uint32_t code_off, scale_off;
};
__device__ __forceinline__ Mx4Row mx4_row(const uint8_t* codes, const uint8_t* scales, int64_t first, uint32_t row,
                                          int kb) {
  return Mx4Row{codes + first * kb * 16, scales + first * kb, row * (uint32_t)kb * 16u, row * (uint32_t)kb};
}

// Unit u of a row of kb blocks; blocks past the row's end read as zeros with
// scale 1.  WHOLE: the unit is known to lie inside (without the branch, the loads of
// several rows and units are issued together).
template <bool WHOLE = false>
__device__ __forceinline__ void mx4_load_unit(const Mx4Row& row, int kb, int u, int g, Mx4Unit& t) {
  const uint32_t c = row.code_off + (uint32_t)(u * kMx4UnitBytes + 16 * g);
  const uint32_t s = row.scale_off + (uint32_t)(u * kMx4UnitBlocks);
  if (WHOLE || (u + 1) * kMx4UnitBlocks <= kb) {
    t.half[0] = load16(row.codes + c);
    t.half[1] = load16(row.codes + c + 64u);
    __builtin_memcpy(t.sc, row.scales + s, 8);
  } else {
    const int left = kb - u * kMx4UnitBlocks;
    t.half[0] = t.half[1] = u32x4_t{0u, 0u, 0u, 0u};
    if (g < left) t.half[0] = load16(row.codes + c);
    if (4 + g < left) t.half[1] = load16(row.codes + c + 64u);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      t.sc[h] = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b)
        t.sc[h] |= (4 * h + b < left ? (uint32_t)row.scales[s + 4 * h + b] : kMx4One) << (8 * b);
    }
  }
}

// Scale byte of block g of half h, in the low byte.
__device__ __forceinline__ uint32_t mx4_own_scale(const Mx4Unit& t, int h, int g) { return t.sc[h] >> (8 * g); }

// Operand rows of fp16 activations: P pieces (1, 2 or 4) of 16 / P rows.
template <int P>
struct Mx4X {
  static constexpr int kRows = 16 / P;  // rows of x
  static constexpr int kLoads = 4 / P;  // operands of one 128-k half
};

// Operand `q` of half h of unit u: lane (r, g) holds 8 elements of block 4 h + g,
// piece q P + r / kRows, of row r % kRows; zeros past the row's end or where the
// row is not there.  x: this lane's row.  WHOLE: the unit lies inside, and a row that
// is not there may hold what it likes.
template <int P, bool WHOLE = false>
__device__ __forceinline__ f16x8_t mx4_load_x(const uint16_t* x, bool there, int kb, int u, int h, int g, int r,
                                              int q) {
  const int b = u * kMx4UnitBlocks + 4 * h + g;
  u32x4_t v = {0u, 0u, 0u, 0u};
  if (WHOLE || (there && b < kb)) v = load16(x + (int64_t)b * kMx4Block + 8 * (q * P + r / Mx4X<P>::kRows));
  return __builtin_bit_cast(f16x8_t, v);
}

// Scale bytes whose blocks are exact in fp16: 0.5 * 2^(104 - 127) = 2^-24, the
// least subnormal, to 6 * 2^(140 - 127) < 65504.
constexpr uint32_t kMx4ScaleLow = 104, kMx4ScaleHigh = 140;

// Whether this lane's block of half h is exact in fp16, and the factor then.
__device__ __forceinline__ bool mx4_fp16_scale(const Mx4Unit& w, int h, int g, float& s) {
  const uint32_t own = mx4_own_scale(w, h, g) & 0xFFu;
  const u32x4_t d = w.half[h];
  const bool zero = ((d.x | d.y | d.z | d.w) & 0x77777777u) == 0;
  const bool exact = own - kMx4ScaleLow <= kMx4ScaleHigh - kMx4ScaleLow;
  s = exact ? __uint_as_float(own << 23) : 1.0f;
  return exact || (zero && own != 255u);
}

// acc += x times the half h of a unit of NG x 16 weight rows; false where this
// lane's blocks are not all exact in fp16, and what was added is of no use.  (A
// block of zeros is, at any scale but NaN.)
template <int MG, int P, int NG>
__device__ __forceinline__ bool mx4_mma_f16(const f16x8_t (&x)[MG][Mx4X<P>::kLoads], const Mx4Unit (&w)[NG], int h,
                                            int g, float4_t (&acc)[NG][MG][P]) {
  bool exact = true;
#pragma unroll
  for (int ng = 0; ng < NG; ++ng) {
    float s;
    exact = mx4_fp16_scale(w[ng], h, g, s) && exact;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const f16x8_t c = mx4_to_f16(w[ng].half[h][j], s);
#pragma unroll
      for (int mg = 0; mg < MG; ++mg)
        acc[ng][mg][j % P] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[mg][j / P], c, acc[ng][mg][j % P], 0, 0, 0);
    }
  }
  return exact;
}

// acc += the same, whatever the scales: block by block the unscaled codes, then
// the sums by the block's scale.  The other blocks are taken out of both operands:
// an infinite x times their zeros would be NaN.
template <int MG, int P, int NG>
__device__ __forceinline__ void mx4_mma_f16_blocks(const f16x8_t (&x)[MG][Mx4X<P>::kLoads], const Mx4Unit (&w)[NG],
                                                   int h, int g, float4_t (&acc)[NG][MG][P]) {
#pragma unroll 1
  for (int b = 0; b < 4; ++b) {
    const uint32_t keep = g == b ? 0xFFFFFFFFu : 0u;
#pragma unroll
    for (int ng = 0; ng < NG; ++ng) {
      const float sb = mx4_scale((w[ng].sc[h] >> (8 * b)) & 0xFFu);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f16x8_t c = mx4_to_f16(w[ng].half[h][j] & keep);
#pragma unroll
        for (int mg = 0; mg < MG; ++mg) {
          const u32x4_t xb = __builtin_bit_cast(u32x4_t, x[mg][j / P]) & keep;
          const float4_t v = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, xb), c,
                                                                    float4_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
          float4_t& a = acc[ng][mg][j % P];
#pragma unroll
          for (int i = 0; i < 4; ++i) a[i] = __builtin_fmaf(v[i], sb, a[i]);
        }
      }
    }
  }
}

// acc = the sums over every `stride`th unit of [first, end) and its halves
// [h0, h1) by that second way, from memory again.  A wave that met a scale
// outside fp16 takes its whole share so: a choice inside the loop cost the common
// case 5 to 10 % (5120 -> 17408, one row: 15.3 us against 14.5).
template <int MG, int P, int NG>
__device__ __forceinline__ void mx4_sum_blocks(const uint16_t* const (&x)[MG], const bool (&there)[MG],
                                               const Mx4Row (&rows)[NG], int kb, int first, int end, int stride, int h0,
                                               int h1, int g, int r, float4_t (&acc)[NG][MG][P]) {
#pragma unroll
  for (int ng = 0; ng < NG; ++ng)
#pragma unroll
    for (int mg = 0; mg < MG; ++mg)
#pragma unroll
      for (int p = 0; p < P; ++p) acc[ng][mg][p] = float4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int u = first; u < end; u += stride) {
    Mx4Unit w[NG];
#pragma unroll
    for (int ng = 0; ng < NG; ++ng) mx4_load_unit(rows[ng], kb, u, g, w[ng]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h < h0 || h >= h1) continue;
      f16x8_t f[MG][Mx4X<P>::kLoads];
#pragma unroll
      for (int mg = 0; mg < MG; ++mg)
#pragma unroll
        for (int i = 0; i < Mx4X<P>::kLoads; ++i) f[mg][i] = mx4_load_x<P>(x[mg], there[mg], kb, u, h, g, r, i);
      mx4_mma_f16_blocks<MG, P, NG>(f, w, h, g, acc);
    }
  }
}

// One 16 x 16 tile of the sums of P pieces: operand row 4 g + i is wanted of
// piece (4 g + i) / kRows only.
template <int P>
__device__ __forceinline__ float4_t mx4_pick(const float4_t (&acc)[P], int g) {
  if constexpr (P == 1) return acc[0];
  float4_t v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = acc[i / Mx4X<P>::kRows][i];
#pragma unroll
    for (int k = 1; k < 4; ++k) v[i] = g == k ? acc[(4 * k + i) / Mx4X<P>::kRows][i] : v[i];
  }
  return v;
}

}  // namespace exl3
