// Sums of 64 x 64 products over k, both operands fp16 rows of contiguous k (gfx950).
//
// Eight waves, over k in stages of 128 that go from memory straight to LDS, three of them
// in flight.  A wave takes 16 of a stage's 128 k for the whole tile, so that LDS is read
// once (a quarter of the tile each would read it twice), and reads the next stage while it
// multiplies this one; the waves' sums meet in LDS at the end.  (Operands loaded by the
// lanes that multiply them, 16 rows an instruction, come at 16 bytes a clock and CU; a
// copy's lanes take whole rows and reach 39.)
//
// LDS: a stage holds rows of 256 bytes, 64 of the one operand and then 64 of the other;
// 16-byte piece c of row r lies at place c ^ (r % 16), so that sixteen rows' pieces c
// cover all 64 banks.
#pragma once

#include "exl3_mx4_lds.hpp"

namespace exl3 {

constexpr int kTile64 = 64;
constexpr int kTile64Waves = 8;
constexpr int kTile64K = 16 * kTile64Waves;                       // of a stage
constexpr int kTile64Ring = 4;                                    // stages of LDS
constexpr int kTile64Stage = 2 * kTile64 * kTile64K * 2;          // bytes
constexpr int kTile64Lds = kTile64Ring * kTile64Stage;
constexpr int kTile64Copies = kTile64Stage / 1024 / kTile64Waves;  // a wave's 1 KB copies of a stage
typedef float float16_t __attribute__((ext_vector_type(16)));

// The row of an operand that this lane copies, the i-th (0, 1) of two.
__device__ __forceinline__ uint32_t tile64_row(int i) {
  return 4 * (2 * (threadIdx.x >> 6) + i) + ((threadIdx.x & 63) >> 4);
}

// sums[wave][64][64] = the waves' sums over stages first .. end - 1 of k elements, in `lds`
// (kTile64Lds bytes, aligned to 1024, free before and after: the call ends with a
// barrier).  Operand o is a buffer rsrc[o]; row[o][i] is the byte offset of the row
// tile64_row(i) of it (kPastEnd: a row of zeros).  What lies past k is taken as 0.
__device__ __forceinline__ float* tile64_sums(const u32x4_t (&rsrc)[2], const uint32_t (&row)[2][2], uint32_t k,
                                              int first, int end, uint8_t* lds) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const uint32_t base = (uint32_t)(uintptr_t)(lds_u8*)lds;
  uint32_t piece[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) piece[i] = 8 * ((lane & 15) ^ (tile64_row(i) & 15));
  const auto fetch = [&](int st) {
    const uint32_t at = base + (uint32_t)(st % kTile64Ring) * kTile64Stage;
#pragma unroll
    for (int o = 0; o < 2; ++o)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool there = (uint32_t)st * kTile64K + piece[i] < k && row[o][i] != kPastEnd;
        lds_copy16(rsrc[o], at + (uint32_t)(2 * kTile64Waves * o + 2 * wave + i) * 1024,
                   there ? row[o][i] + 2 * piece[i] : kPastEnd, (uint32_t)st * kTile64K * 2);
      }
  };
  struct Operands {
    f16x8_t x[2], w[2];
  };
  const uint32_t r = lane & 31, c = 2 * wave + (lane >> 5);
  const uint32_t in_tile = r * 256 + 16 * (c ^ (r & 15));
  const auto read = [&](int st, Operands& o) {
    const uint32_t at = base + (uint32_t)(st % kTile64Ring) * kTile64Stage + in_tile;
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      o.x[a] = __builtin_bit_cast(f16x8_t, lds_read16(at + a * 8192));
      o.w[a] = __builtin_bit_cast(f16x8_t, lds_read16(at + kTile64Stage / 2 + a * 8192));
    }
  };
  float16_t acc[2][2];
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[a][b][i] = 0.f;
  const auto multiply = [&](const Operands& o) {
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int b = 0; b < 2; ++b)
        acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(o.x[a], o.w[b], acc[a][b], 0, 0, 0);
  };
  // Waits until at most the two stages after the next are open here: the next has landed
  // here, and behind the barrier everywhere, and this one's place is read and free.
  static_assert(kTile64Ring == 4 && kTile64Copies == 4, "8 copies of two stages");
  const auto step = [&](int st, const Operands& now, Operands& next) {
    asm volatile("s_waitcnt vmcnt(8) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    fetch(st + kTile64Ring);
    read(st + 1, next);
    multiply(now);
  };
  for (int st = first; st < first + kTile64Ring; ++st) fetch(st);
  asm volatile("s_waitcnt vmcnt(12)\n\ts_barrier" ::: "memory");
  Operands even, odd;
  read(first, even);
  int st = first;  // what is read past the end is never multiplied
  for (; st + 1 < end; st += 2) {
    step(st, even, odd);
    step(st + 1, odd, even);
  }
  if (st < end) multiply(even);
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  float* sums = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        sums[(wave * 64 + 32 * a + 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3)) * 64 + 32 * b + r] = acc[a][b][i];
  __syncthreads();
  return sums;
}

// Element (row, col) of the tile from the waves' sums.
__device__ __forceinline__ float tile64_sum(const float* sums, int row, int col) {
  float v = sums[row * 64 + col];
#pragma unroll
  for (int o = 1; o < kTile64Waves; ++o) v += sums[(o * 64 + row) * 64 + col];
  return v;
}

}  // namespace exl3
