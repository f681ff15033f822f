// exl3_mx4_linear for 17 to 64 rows: fp16 rows shared by a workgroup through
// LDS.
//
// With so many rows the waves can no longer each fetch the rows for their share
// of k (exl3_mx4_rows.hpp): a wave's 16 columns bring 2 KB of weights for 8 KB of
// rows, and the load path, not the weights, bounds the time (37 rows, 17408 ->
// 5120: 34 us).  Here four waves take 32 columns each and the same k, so a
// workgroup fetches the rows once for 128 columns; what is left of k's length is
// shared among workgroups, and their sums are added by mx4_rows_finish.
//
// A stage is 256 k of everything, copied from memory straight to LDS, kept in a
// ring of three or four: a step waits for its own stage only, so that the bytes
// of the others are in flight meanwhile.  The product is that of the few rows
// (mx4_mma_f16).
#include "exl3_internal.hpp"
#include "exl3_mx4_lds.hpp"
#include "exl3_mx4_linear.hpp"

namespace exl3 {

constexpr int kWideWaves = 4, kWideCols = 128, kWideNI = kWideCols / kWideWaves / 16;
constexpr int kWideLine = kMx4UnitK * 2;  // bytes of a row of x in a stage

template <int MG>
__global__ __launch_bounds__(kWideWaves * 64) void mx4_wide_kernel(Mx4RowsArgs q) {
  // a stage: rows of x, lines of codes, and of each weight row four dwords, the
  // first three of which hold its eight scale bytes
  constexpr uint32_t kX = 0, kB = kX + MG * 16 * kWideLine, kS = kB + kWideCols * kMx4UnitBytes,
                     kBytes = kS + kWideCols * 16;
  constexpr int kStages = 160 * 1024 / kBytes < 4 ? 160 * 1024 / kBytes : 4;
  constexpr int kAhead = kStages - 1;
  constexpr int CX = MG * 8 / kWideWaves, CB = kWideCols / 8 / kWideWaves, kCopies = CX + CB + 1;  // a wave's, a stage
  __shared__ __align__(128) uint8_t smem[kStages * kBytes];
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_u8*)smem;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int g = lane >> 4, r = lane & 15;
  const uint32_t tile = blockIdx.x / (uint32_t)q.splits, split = blockIdx.x - tile * (uint32_t)q.splits;
  const int64_t n0 = (int64_t)tile * kWideCols;
  const int kb = q.kb;
  const uint32_t pitch = (uint32_t)kb * 16u, xpitch = (uint32_t)q.lda * 2u;
  const int units = (kb + kMx4UnitBlocks - 1) / kMx4UnitBlocks;
  const int begin = (int)((int64_t)units * split / q.splits), end = (int)((int64_t)units * (split + 1) / q.splits);

  // x: two rows an instruction; chunk c of row i at place c ^ (i & 3), so that
  // the lanes a 16-byte read serves together fall on different banks
  const int64_t left = q.n - n0 < kWideCols ? q.n - n0 : kWideCols;
  const u32x4_t rx = buffer_words(static_cast<const uint8_t*>(q.a), (uint64_t)(q.m - 1) * xpitch + (uint64_t)kb * 64);
  const u32x4_t rb = buffer_words(q.b + n0 * pitch, (uint64_t)left * pitch);
  const u32x4_t rs = buffer_words(q.b_scales + ((n0 * kb) & ~(int64_t)3), ((uint64_t)left * kb + (n0 * kb & 3) + 3) & ~3ull);
  // the row of the c-th instruction is 2 (CX wave + c) + lane / 32: its chunks'
  // order alternates with the parity of CX wave + c
  const uint32_t b_chunk = (lane & 7) ^ ((lane >> 3) & 7), b_off = pitch * (lane >> 3) + 16 * b_chunk;
  const uint32_t s_row = (uint32_t)(n0 * kb & 3) + (uint32_t)(wave * 32 + (lane & 31)) * kb;  // byte of its first scale
  auto copy = [&](uint32_t stage, int u, bool there) {
#pragma unroll
    for (int c = 0; c < CX; ++c) {
      const int pair = wave * CX + c, row = 2 * pair + (lane >> 5);
      const uint32_t chunk = (lane & 31) ^ (row & 3);
      const bool in = there && u * kMx4UnitBlocks + (int)(chunk >> 2) < kb && row < q.m;
      lds_copy16(rx, stage + kX + pair * 1024, in ? xpitch * (lane >> 5) + 16 * chunk : kPastEnd,
                 xpitch * 2 * pair + (uint32_t)u * kWideLine);
    }
    const bool in = there && u * kMx4UnitBlocks + (int)b_chunk < kb;
#pragma unroll
    for (int c = 0; c < CB; ++c)
      lds_copy16(rb, stage + kB + (wave * CB + c) * 1024, in ? b_off : kPastEnd,
                 pitch * 8 * (wave * CB + c) + (uint32_t)u * kMx4UnitBytes);
    if (lane < 32)
      lds_copy16(rs, stage + kS + wave * 32 * 16, there ? s_row & ~3u : kPastEnd, (uint32_t)u * kMx4UnitBlocks);
  };

  float4_t acc[kWideNI][MG][1];
#pragma unroll
  for (int ni = 0; ni < kWideNI; ++ni)
#pragma unroll
    for (int mg = 0; mg < MG; ++mg) acc[ni][mg][0] = float4_t{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](uint32_t stage, int u) {
    Mx4Unit w[kWideNI];
#pragma unroll
    for (int ni = 0; ni < kWideNI; ++ni) {
      const int row = wave * 32 + 16 * ni + r;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        w[ni].half[h] = lds_read16(stage + kB + row * kMx4UnitBytes + (((4 * h + g) ^ (r & 7)) * 16));
      const uint32_t shift = ((uint32_t)(n0 * kb & 3) + (uint32_t)row * kb) & 3u;
      const u32x4_t d = lds_read16(stage + kS + row * 16);
      w[ni].sc[0] = __builtin_amdgcn_alignbyte(d.y, d.x, shift);
      w[ni].sc[1] = __builtin_amdgcn_alignbyte(d.z, d.y, shift);
      if ((u + 1) * kMx4UnitBlocks > kb) {  // what follows a row's end is the next row's
#pragma unroll
        for (int b = 0; b < 8; ++b)
          if (u * kMx4UnitBlocks + b >= kb)
            w[ni].sc[b / 4] = (w[ni].sc[b / 4] & ~(0xFFu << (8 * (b % 4)))) | (kMx4One << (8 * (b % 4)));
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      f16x8_t x[MG][4];
#pragma unroll
      for (int mg = 0; mg < MG; ++mg)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          x[mg][j] = __builtin_bit_cast(
              f16x8_t, lds_read16(stage + kX + (16 * mg + r) * kWideLine + (((4 * (4 * h + g) + j) ^ (r & 3)) * 16)));
#pragma unroll
      for (int ni = 0; ni < kWideNI; ++ni) mx4_mma_f16<MG, 1>(x, w[ni], h, g, acc[ni]);
    }
  };

#pragma unroll
  for (int s = 0; s < kAhead; ++s) copy(lds0 + s * kBytes, begin + s, begin + s < end);
  uint32_t stage = 0;
  for (int u = begin; u < end; ++u) {
    // this wave's copies of the stage are in (those of kAhead - 1 later ones may
    // not be) and its reads of the stage before are done; then everybody's
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kCopies * (kAhead - 1)) : "memory");
    copy(lds0 + (stage == 0 ? kAhead * kBytes : stage - kBytes), u + kAhead, u + kAhead < end);
    multiply(lds0 + stage, u);
    stage = stage == kAhead * kBytes ? 0 : stage + kBytes;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no copy outlives the workgroup's LDS

#pragma unroll
  for (int ni = 0; ni < kWideNI; ++ni) {
    const int64_t col = n0 + wave * 32 + 16 * ni + r;
    if (col >= q.n) continue;
#pragma unroll
    for (int mg = 0; mg < MG; ++mg)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t row = 16 * mg + 4 * g + i;
        if (row >= q.m) continue;
        if (q.splits == 1)
          mx4_store(q, row, col, acc[ni][mg][0][i]);
        else
          q.part[((int64_t)split * q.m + row) * q.n + col] = acc[ni][mg][0][i];
      }
  }
}

hipError_t launch_mx4_wide(Mx4RowsArgs q, int splits, void* ws, hipStream_t s) {
  const uint32_t tiles = (uint32_t)((q.n + kWideCols - 1) / kWideCols);
  q.splits = splits;
  q.part = static_cast<float*>(ws);
  const dim3 grid(tiles * (uint32_t)splits), block(kWideWaves * 64);
  if (q.m <= 32) hipLaunchKernelGGL(mx4_wide_kernel<2>, grid, block, 0, s, q);
  else if (q.m <= 48) hipLaunchKernelGGL(mx4_wide_kernel<3>, grid, block, 0, s, q);
  else hipLaunchKernelGGL(mx4_wide_kernel<4>, grid, block, 0, s, q);
  if (splits > 1) launch_mx4_rows_finish(q, s);
  return hipGetLastError();
}

}  // namespace exl3
