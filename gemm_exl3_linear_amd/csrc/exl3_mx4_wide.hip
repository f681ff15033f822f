// exl3_mx4_linear for more rows and large weights: fp16 rows shared by a
// workgroup through LDS.
//
// With so many rows the waves can no longer each fetch the rows for their share
// of k (exl3_mx4_rows.hpp): a wave's 16 columns bring 2 KB of weights for 8 KB of
// rows, and the load path, not the weights, bounds the time (37 rows, 17408 ->
// 5120: 34 us).  Here four pairs of waves take 32 columns each and the same k, so
// a workgroup fetches the rows once for 128 columns; what is left of k's length
// is shared among workgroups, and their sums are added by mx4_rows_finish.  The
// waves of a pair take the two halves of a unit: one wave a SIMD would leave its
// LDS reads, conversions and matrix instructions one after the other (25 us).
//
// A stage is 256 k of everything, copied from memory straight to LDS, kept in a
// ring of three to six: a step waits for the next stage only, so that the bytes
// of the others are in flight meanwhile.  The waves run in step, so what a step
// does one after the other leaves the rest of the CU idle (copies 500 cycles, LDS
// reads 900, product 1000, of 3000): a quarter of the product is followed by a
// quarter of the copies and by the reads of the next stage into the registers
// that it has freed.  (Quarters of a unit for 64 columns a wave, with fewer LDS
// reads, were 12 % slower; shares of k across the tiles' ends, to fill the chip for
// any number of tiles, 10 %.)
//
// Measured: 37 rows 17408 -> 5120 (49 MB) 22.8 us over three sets of tensors in turn,
// 24.1 over 1 GB of them: 11.3 steps of 1.25 us, 3.4 TB/s of weights, then start, end
// and the second launch.  The copies bound a step: alone they take 1.1 us with 16
// rows and 1.5 with 48, the rest without them 0.95.
#include "exl3_internal.hpp"
#include "exl3_mx4_lds.hpp"
#include "exl3_mx4_linear.hpp"

namespace exl3 {

constexpr int kWideWaves = 8, kWideCols = 128, kWideNI = 2;
constexpr int kWideLine = kMx4UnitK * 2;  // bytes of a row of x in a stage

// What the places of a row's chunks in LDS are turned by: a 16-byte read of one
// chunk of eight rows and the next but three of the same rows then falls on 16
// different places of 256 bytes.
__device__ __forceinline__ uint32_t wide_turn(int row) { return (uint32_t)((row & 3) | ((row & 4) << 1)); }

template <int MG>
__global__ __launch_bounds__(kWideWaves * 64) void mx4_wide_kernel(Mx4RowsArgs q) {
  // a stage: rows of x, lines of codes, and of each weight row four dwords, the
  // first three of which hold its eight scale bytes
  constexpr uint32_t kX = 0, kB = kX + MG * 16 * kWideLine, kS = kB + kWideCols * kMx4UnitBytes,
                     kBytes = kS + kWideCols * 16;
  constexpr int kStages = 160 * 1024 / kBytes;
  constexpr int CX = MG * 8 / kWideWaves, CB = kWideCols / 8 / kWideWaves, kCopies = CX + CB + 1;  // a wave's, a stage
  __shared__ __align__(128) uint8_t smem[kStages * kBytes];
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_u8*)smem;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int g = lane >> 4, r = lane & 15;
  const int h = wave >> 2, cols = (wave & 3) * 32;  // half of a unit, columns of the tile
  const uint32_t tile = blockIdx.x / (uint32_t)q.splits, split = blockIdx.x - tile * (uint32_t)q.splits;
  const int64_t n0 = (int64_t)tile * kWideCols;
  const int kb = q.kb;
  const uint32_t pitch = (uint32_t)kb * 16u, xpitch = (uint32_t)q.lda * 2u;
  const int units = (kb + kMx4UnitBlocks - 1) / kMx4UnitBlocks;
  const int begin = (int)((int64_t)units * split / q.splits), end = (int)((int64_t)units * (split + 1) / q.splits);

  // x: two rows an instruction; chunk c of row i at place c ^ wide_turn(i).  Rows
  // past the last lie past the buffers' ends and read as zeros.
  const int64_t left = q.n - n0 < kWideCols ? q.n - n0 : kWideCols;
  const u32x4_t rx = buffer_words(static_cast<const uint8_t*>(q.a), (uint64_t)(q.m - 1) * xpitch + (uint64_t)kb * 64);
  const u32x4_t rb = buffer_words(q.b + n0 * pitch, (uint64_t)left * pitch);
  const u32x4_t rs = buffer_words(q.b_scales + n0 * kb, ((uint64_t)left * kb + 3) & ~3ull);
  constexpr int kTurns = CX < 4 ? CX : 4;  // the turn of row 2 (CX wave + i) + lane / 32 repeats after four i
  uint32_t x_chunk[kTurns], x_off[kTurns];
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    x_chunk[i] = (uint32_t)(lane & 31) ^ wide_turn(2 * (CX * wave + i) + (lane >> 5));
    x_off[i] = xpitch * (lane >> 5) + 16 * x_chunk[i];
  }
  const uint32_t b_chunk = (lane & 7) ^ ((lane >> 3) & 7), b_off = pitch * (lane >> 3) + 16 * b_chunk;
  const uint32_t s_off = ((uint32_t)(wave * 16 + r) * kb) & ~3u;  // dword of its first scale
  // Copies of unit u, in quarters (0 .. 3; the scales in the last); none of a
  // unit past the end: zeros, from a buffer without bytes.
  struct Copy {
    u32x4_t rx, rb, rs;
    uint32_t x[kTurns], b;
    int u;
  };
  auto plan = [&](int u) {
    Copy c{rx, rb, rs, {}, 0u, u};
    if (u >= end) c.rx.z = c.rb.z = c.rs.z = 0u;
    const int left = kb - u * kMx4UnitBlocks;  // chunks past a row's end: zeros
#pragma unroll
    for (int p = 0; p < kTurns; ++p) c.x[p] = (int)(x_chunk[p] >> 2) < left ? x_off[p] : kPastEnd;
    c.b = (int)b_chunk < left ? b_off : kPastEnd;
    return c;
  };
  auto copy = [&](const Copy& c, int part, uint32_t stage) {
#pragma unroll
    for (int i = 0; i < CX; ++i)
      if (i % 4 == part) {
        const int pair = wave * CX + i;
        lds_copy16(c.rx, stage + kX + pair * 1024, c.x[i % 4],
                   xpitch * 2 * pair + (uint32_t)c.u * kWideLine);
      }
#pragma unroll
    for (int i = 0; i < CB; ++i)
      if ((CX + i) % 4 == part)
        lds_copy16(c.rb, stage + kB + (wave * CB + i) * 1024, c.b,
                   pitch * 8 * (wave * CB + i) + (uint32_t)c.u * kMx4UnitBytes);
    if (part == 3 && lane < 16)
      lds_copy16(c.rs, stage + kS + wave * 16 * 16, s_off, (uint32_t)c.u * kMx4UnitBlocks);
  };

  float4_t acc[kWideNI][MG][1];
#pragma unroll
  for (int ni = 0; ni < kWideNI; ++ni)
#pragma unroll
    for (int mg = 0; mg < MG; ++mg) acc[ni][mg][0] = float4_t{0.f, 0.f, 0.f, 0.f};
  Mx4Unit w[kWideNI], wn[kWideNI];
  f16x8_t x[MG][4];
  auto read_w = [&](Mx4Unit (&t)[kWideNI], uint32_t stage, int u) {
#pragma unroll
    for (int ni = 0; ni < kWideNI; ++ni) {
      const int row = cols + 16 * ni + r;
      t[ni].half[0] = lds_read16(stage + kB + row * kMx4UnitBytes + (((4 * h + g) ^ (r & 7)) * 16));
      // scale bytes 4 h .. 4 h + 3, of three dwords that hold all eight
      const uint32_t shift = ((uint32_t)row * kb) & 3u;
      const u32x2_t d = lds_read8(stage + kS + row * 16 + 4 * h);
      t[ni].sc[0] = __builtin_amdgcn_alignbyte(d.y, d.x, shift);
      if ((u + 1) * kMx4UnitBlocks > kb) {  // what follows a row's end is the next row's
#pragma unroll
        for (int b = 0; b < 4; ++b)
          if (u * kMx4UnitBlocks + 4 * h + b >= kb)
            t[ni].sc[0] = (t[ni].sc[0] & ~(0xFFu << (8 * b))) | (kMx4One << (8 * b));
      }
    }
  };
  auto read_x = [&](int j, uint32_t stage) {
#pragma unroll
    for (int mg = 0; mg < MG; ++mg)
      x[mg][j] = __builtin_bit_cast(
          f16x8_t, lds_read16(stage + kX + (16 * mg + r) * kWideLine +
                              ((uint32_t)(4 * (4 * h + g) + j) ^ wide_turn(r)) * 16));
  };

#pragma unroll
  for (int s = 0; s < kStages; ++s) {
    const Copy c = plan(begin + s);
#pragma unroll
    for (int p = 0; p < 4; ++p) copy(c, p, lds0 + s * kBytes);
  }
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(kCopies * (kStages - 1)) : "memory");
  read_w(w, lds0, begin);
#pragma unroll
  for (int j = 0; j < 4; ++j) read_x(j, lds0);
  uint32_t stage = lds0;  // of unit u
  // Every scale of these columns in fp16.  Those of rows past the last are what
  // follows them in their dword, and have no say.
  bool exact[kWideNI];
#pragma unroll
  for (int ni = 0; ni < kWideNI; ++ni) exact[ni] = true;
  for (int u = begin; u < end; ++u) {
    // this wave's copies of the next stage are in (those of kStages - 2 later
    // ones may not be) and its reads of stage u are done; then everybody's
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kCopies * (kStages - 2)) : "memory");
    const uint32_t next = stage == lds0 + (kStages - 1) * kBytes ? lds0 : stage + kBytes;
    const Copy c = plan(u + kStages);
    float s[kWideNI];
#pragma unroll
    for (int ni = 0; ni < kWideNI; ++ni) exact[ni] = mx4_fp16_scale(w[ni], 0, g, s[ni]) && exact[ni];
    read_w(wn, next, u + 1);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int ni = 0; ni < kWideNI; ++ni) {
        const f16x8_t v = mx4_to_f16(w[ni].half[0][j], s[ni]);
#pragma unroll
        for (int mg = 0; mg < MG; ++mg)
          acc[ni][mg][0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[mg][j], v, acc[ni][mg][0], 0, 0, 0);
      }
      copy(c, j, stage);
      read_x(j, next);
    }
#pragma unroll
    for (int ni = 0; ni < kWideNI; ++ni) w[ni] = wn[ni];
    stage = next;
  }

  bool all_exact = true;
#pragma unroll
  for (int ni = 0; ni < kWideNI; ++ni) all_exact = (exact[ni] || cols + 16 * ni + r >= left) && all_exact;
  if (__builtin_expect(!__all(all_exact), 0)) {
    const uint16_t* xr[MG];
    bool there[MG];
#pragma unroll
    for (int mg = 0; mg < MG; ++mg) {
      there[mg] = 16 * mg + r < q.m;
      xr[mg] = static_cast<const uint16_t*>(q.a) + (there[mg] ? 16 * mg + r : 0) * q.lda;
    }
#pragma unroll
    for (int ni = 0; ni < kWideNI; ++ni) {  // one by one, for fewer registers
      const int row = cols + 16 * ni + r;
      const Mx4Row rows[1] = {mx4_row(q.b, q.b_scales, n0, row < left ? row : (uint32_t)(left - 1), kb)};
      float4_t sums[1][MG][1];
      mx4_sum_blocks<MG, 1, 1>(xr, there, rows, kb, begin, end, 1, h, h + 1, g, r, sums);
#pragma unroll
      for (int mg = 0; mg < MG; ++mg) acc[ni][mg][0] = sums[0][mg][0];
    }
  }

  // the second half's sums to the waves of the first, through LDS
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  float4_t* sums = reinterpret_cast<float4_t*>(smem) + (wave & 3) * (kWideNI * MG * 64) + lane;
  static_assert(4 * kWideNI * MG * 1024 <= kStages * kBytes, "the sums fit");
  if (h == 1) {
#pragma unroll
    for (int i = 0; i < kWideNI * MG; ++i) sums[i * 64] = acc[i / MG][i % MG][0];
  }
  __syncthreads();
  if (h == 1) return;
#pragma unroll
  for (int i = 0; i < kWideNI * MG; ++i) acc[i / MG][i % MG][0] += sums[i * 64];
#pragma unroll
  for (int ni = 0; ni < kWideNI; ++ni) {
    const int64_t col = n0 + cols + 16 * ni + r;
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
  if (q.m <= 16) hipLaunchKernelGGL(mx4_wide_kernel<1>, grid, block, 0, s, q);
  else if (q.m <= 32) hipLaunchKernelGGL(mx4_wide_kernel<2>, grid, block, 0, s, q);
  else if (q.m <= 48) hipLaunchKernelGGL(mx4_wide_kernel<3>, grid, block, 0, s, q);
  else hipLaunchKernelGGL(mx4_wide_kernel<4>, grid, block, 0, s, q);
  if (splits > 1) launch_mx4_rows_finish(q, s);
  return hipGetLastError();
}

}  // namespace exl3
