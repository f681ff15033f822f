// exl3_mx4_linear and exl3_mx4_matmul where few rows or small sizes leave the
// weights' bytes, or the launch, as the bound: workgroups whose waves share k, and
// the choice of the kernel by size.  Measured, as below, in graphs of such calls over
// three sets of tensors in turn: one row 5120 -> 17408 (47 MB) 11.5 us with fp16 rows,
// 11.0 with 4-bit rows; over 1 GB of sets, whose weights come from HBM, 12.5 (3.8 TB/s)
// and 11.8 (4.0); one row 2048 -> 512 3.4 us, of which a launch is 1.6.
#include "exl3_internal.hpp"
#include "exl3_mx4_linear.hpp"

namespace exl3 {

// 16 MG rows (A4: 4-bit, else fp16 in operands of P pieces, P = 1 unless
// MG = 1), 16 NG columns, NW waves.
template <bool A4, int MG, int P, int NG, int NW>
__global__ __launch_bounds__(NW * 64) void mx4_rows_kernel(Mx4RowsArgs q) {
  static_assert(P == 1 || (MG == 1 && !A4), "pieces are for few fp16 rows");
  constexpr int T = MG * NG;
  constexpr int kRows = Mx4X<P>::kRows, kLoads = Mx4X<P>::kLoads;
  __shared__ float4_t part[NW * T * 64];  // 64 KB at most
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int g = lane >> 4, r = lane & 15;
  const uint32_t tm = blockIdx.x / q.col_tiles, tn = blockIdx.x - tm * q.col_tiles;
  const int64_t m0 = (int64_t)tm * (16 * MG), n0 = (int64_t)tn * (16 * NG);
  const int kb = q.kb;

  Mx4Row rb[NG], ra[A4 ? MG : 1];
#pragma unroll
  for (int ng = 0; ng < NG; ++ng) {
    // columns past n are computed and not stored
    const int64_t left = q.n - 1 - n0;
    rb[ng] = mx4_row(q.b, q.b_scales, n0, 16 * ng + r <= left ? 16 * ng + r : (uint32_t)left, kb);
  }
  const uint16_t* xr[MG];
  bool there[MG];
#pragma unroll
  for (int mg = 0; mg < MG; ++mg) {
    const int i = 16 * mg + r % kRows;
    const int64_t left = q.m - 1 - m0;
    there[mg] = i <= left;
    if constexpr (A4)
      ra[mg] = mx4_row(static_cast<const uint8_t*>(q.a), q.a_scales, m0, there[mg] ? i : (uint32_t)left, kb);
    else
      xr[mg] = static_cast<const uint16_t*>(q.a) + (m0 + (there[mg] ? i : 0)) * q.lda;
  }

  float4_t acc[NG][MG][P];
#pragma unroll
  for (int ng = 0; ng < NG; ++ng)
#pragma unroll
    for (int mg = 0; mg < MG; ++mg)
#pragma unroll
      for (int p = 0; p < P; ++p) acc[ng][mg][p] = float4_t{0.f, 0.f, 0.f, 0.f};

  bool exact = true;  // fp16 rows: every scale in fp16
  auto unit = [&](auto whole, int u) {
    constexpr bool W = decltype(whole)::value != 0;
    Mx4Unit w[NG];
#pragma unroll
    for (int ng = 0; ng < NG; ++ng) mx4_load_unit<W>(rb[ng], kb, u, g, w[ng]);
    if constexpr (A4) {
      Mx4Unit x[MG];
#pragma unroll
      for (int mg = 0; mg < MG; ++mg) mx4_load_unit<W>(ra[mg], kb, u, g, x[mg]);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int ng = 0; ng < NG; ++ng)
#pragma unroll
          for (int mg = 0; mg < MG; ++mg)
            acc[ng][mg][0] = mfma_mx4(x[mg].half[h], mx4_own_scale(x[mg], h, g), w[ng].half[h],
                                      mx4_own_scale(w[ng], h, g), acc[ng][mg][0]);
    } else {
      f16x8_t x[2][MG][kLoads];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int mg = 0; mg < MG; ++mg)
#pragma unroll
          for (int i = 0; i < kLoads; ++i) x[h][mg][i] = mx4_load_x<P, W>(xr[mg], there[mg], kb, u, h, g, r, i);
#pragma unroll
      for (int h = 0; h < 2; ++h) exact = mx4_mma_f16<MG, P, NG>(x[h], w, h, g, acc) && exact;
    }
  };
  // whole units without a branch about the row's end (333 rows 2080 -> 1111 7.5 us with,
  // 6.9 without; 16 rows 5120 -> 5120 11.1 / 10.5; two units at a time were no quicker)
  const int whole = kb / kMx4UnitBlocks;
  for (int u = wave; u < whole; u += NW) unit(PowC<1>{}, u);
  if (whole * kMx4UnitBlocks < kb && whole % NW == wave) unit(PowC<0>{}, whole);
  if constexpr (!A4) {
    if (__builtin_expect(!__all(exact), 0))
      mx4_sum_blocks<MG, P, NG>(xr, there, rb, kb, wave, (kb + kMx4UnitBlocks - 1) / kMx4UnitBlocks, NW, 0, 2, g, r,
                                acc);
  }

  // Sum over the waves in wave order.  Lane l of a 16 x 16 tile holds operand rows
  // 4 (l / 16) .. + 3 of column l % 16.
#pragma unroll
  for (int t = 0; t < T; ++t) part[(wave * T + t) * 64 + lane] = mx4_pick<P>(acc[t / MG][t % MG], g);
  __syncthreads();
  for (int e = threadIdx.x; e < T * 64; e += NW * 64) {
    float4_t v = part[e];
#pragma unroll
    for (int w = 1; w < NW; ++w) v += part[w * T * 64 + e];
    const int t = e >> 6, l = e & 63;
    const int64_t col = n0 + 16 * (t / MG) + (l & 15), row = m0 + 16 * (t % MG) + 4 * (l >> 4);
    if constexpr (P > 1) {  // the pieces' sums, in piece order, by the lanes of the first rows
      part[e] = v;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int p = 1; p < P; ++p) {
        const int at = p * kRows;  // operand row of the piece's row 0
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (4 * (l >> 4) + i < kRows) {
            const int o = at + 4 * (l >> 4) + i;
            v[i] += part[(e & ~63) + 16 * (o >> 2) + (l & 15)][o & 3];
          }
      }
    }
    if (col >= q.n) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (row + i >= q.m) break;
      mx4_store(q, row + i, col, v[i]);
    }
  }
}

// y = sum of the splits in order (+ bias), eight splits' loads at a time where
// there are so many (20 rows 17408 -> 1001, 17 splits: 13.2 us, 14.4 with four).
template <int N>
__device__ __forceinline__ void add_splits(const float* p, int64_t size, int& s, int splits, float& v) {
  for (; s + N <= splits; s += N) {
    float w[N];
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = p[(s + i) * size];
#pragma unroll
    for (int i = 0; i < N; ++i) v += w[i];
  }
}
__global__ __launch_bounds__(256) void mx4_rows_finish(Mx4RowsArgs q) {
  const int64_t row = blockIdx.y, col = (int64_t)blockIdx.x * 256 + threadIdx.x, size = q.m * q.n;
  if (col >= q.n) return;
  const float* p = q.part + row * q.n + col;
  float v = 0.f;
  int s = 0;
  add_splits<8>(p, size, s, q.splits, v);
  add_splits<3>(p, size, s, q.splits, v);
  add_splits<1>(p, size, s, q.splits, v);
  mx4_store(q, row, col, v);
}

void launch_mx4_rows_finish(const Mx4RowsArgs& q, hipStream_t s) {
  hipLaunchKernelGGL(mx4_rows_finish, dim3((uint32_t)((q.n + 255) / 256), (uint32_t)q.m), dim3(256), 0, s, q);
}

template <bool A4, int MG, int P, int NG, int NW>
static hipError_t launch_rows(Mx4RowsArgs q, hipStream_t s) {
  q.col_tiles = (uint32_t)((q.n + 16 * NG - 1) / (16 * NG));
  const uint32_t tiles = q.col_tiles * (uint32_t)((q.m + 16 * MG - 1) / (16 * MG));
  hipLaunchKernelGGL((mx4_rows_kernel<A4, MG, P, NG, NW>), dim3(tiles), dim3(NW * 64), 0, s, q);
  return hipGetLastError();
}

// Shares of k of the rows shared through LDS: as many as fill the chip's CUs once,
// two units each at least (us, for 2 / 3 / 4 / 5 / 6 / 8 shares: 37 rows 17408 -> 5120,
// 40 tiles, 42 / 32 / 27 / 25 / 24 / 33; 20 rows 8192 -> 8192, 64 tiles, 22 / 19 / 17 /
// 25 / 24 / 23).
static int wide_splits(int64_t n, int64_t k) {
  const int64_t tiles = (n + 127) / 128, units = (k + kMx4UnitK - 1) / kMx4UnitK;
  int64_t s = 256 / tiles;
  if (s > units / 2) s = units / 2;
  return s < 1 ? 1 : (int)s;
}

// How five rows and more are cut: 16 rows (up to 8 in two pieces) and 16 or 32
// columns a workgroup here, or all rows shared through LDS for 128 columns
// (exl3_mx4_wide.hip).  The estimates, in us, count the launch, a wave's turns over k
// and what further rounds of the CUs add; there, a start and steps that grow with
// the rows, and a second launch for shares of k (up to 8 rows only where it is
// clearly less).  As measured (us, 16 / 32 / LDS):
//    8 rows  5120 ->  2048    6.4    7.8    9.2
//    8 rows  5120 ->  5120   10.2    8.3   12.4
//    8 rows 17408 ->   512   14.4   18.8   10.0
//    6 rows 17408 ->  5120   24.7   18.4   19.2
//   64 rows  2048 ->   512    5.0    5.5   10.7
//   64 rows  5120 ->  2048   14.5   10.1   14.9
//   20 rows   512 ->  8192    4.7    4.3    7.5
//   40 rows 17408 ->    64   21.3   25.7   11.1
//   32 rows  5120 ->  5120   20.3   17.3   15.0
//   16 rows 17408 ->  5120   41.2   27.5   20.2
//   16 rows  5120 ->  5120   14.6   10.1   13.1
// (over 1 GB of sets each is 0.1 to 5 us longer, in the same order)
enum class Mx4RowsCut { k16, k32, kLds };
static Mx4RowsCut rows_cut(int64_t m, int64_t n, int64_t k) {
  const int64_t units = (k + kMx4UnitK - 1) / kMx4UnitK, row_tiles = (m + 15) / 16;
  const double turns = (double)((units + 7) / 8), more = units < 2 ? 0.25 : (units < 8 ? (double)units / 8 : turns);
  auto cost = [&](int64_t cols, double start, double turn) {
    const int64_t rounds = (row_tiles * ((n + cols - 1) / cols) + 255) / 256;
    return start + turn * (turns + (double)(rounds - 1) * more);
  };
  const int64_t tiles = (n + 127) / 128, shares = wide_splits(n, k);
  const double steps = (double)((units + shares - 1) / shares * ((tiles * shares + 255) / 256));
  const bool few = m <= 8;
  const double c16 = few ? cost(16, 2.6, 1.35) : cost(16, 2.9, 2.2);
  const double c32 = few ? cost(32, 2.6, 1.9) : cost(32, 3.2, 2.6);
  const double lds = (few ? 1.15 : 1.0) * (4.6 + 0.8 * (double)row_tiles + (0.8 + 0.1 * (double)row_tiles) * steps +
                                           (shares > 1 ? 2.2 : 0.0));
  if (lds < c16 && lds < c32) return Mx4RowsCut::kLds;
  return c16 <= c32 ? Mx4RowsCut::k16 : Mx4RowsCut::k32;
}
size_t mx4_linear_workspace(int64_t m, int64_t n, int64_t k) {
  if (m <= 4 || rows_cut(m, n, k) != Mx4RowsCut::kLds) return 0;
  const int s = wide_splits(n, k);
  return s > 1 ? (size_t)s * m * n * sizeof(float) : 0;
}

hipError_t launch_mx4_linear(const uint8_t* codes, const uint8_t* scales, int64_t n, int64_t k, const uint16_t* bias,
                             const uint16_t* x, int64_t m, int64_t ldx, void* y, int64_t ldy, bool y_f32, void* ws,
                             hipStream_t s) {
  const int kb = (int)(k / kMx4Block);
  const Mx4RowsArgs q{x, nullptr, ldx, codes, scales, bias, y, ldy, m, n, kb, y_f32, 0, 0, 1, nullptr};
  // up to 4 rows: four pieces (exl3_mx4_rows.hpp) where k is long enough for the fewer
  // loads to show, else two; 32 columns a workgroup where those fill half the chip and
  // x has more than a row to fetch (us: one row 5120 -> 17408 four pieces 11.4, two
  // 12.3; 2048 -> 2048 3.6 / 3.5; 16 / 32 columns: 4 rows 17408 -> 5120 20.3 / 16.1,
  // 5120 -> 2048 5.7 / 7.1, one row 5120 -> 17408 11.4 / 13.0, 17408 -> 5120, where the
  // rule takes the slower, 14.6 / 13.0)
  if (m <= 4) {
    const bool cols32 = m > 1 && n >= 4096;
    if (k >= 4096) return cols32 ? launch_rows<false, 1, 4, 2, 8>(q, s) : launch_rows<false, 1, 4, 1, 8>(q, s);
    return cols32 ? launch_rows<false, 1, 2, 2, 8>(q, s) : launch_rows<false, 1, 2, 1, 8>(q, s);
  }
  const Mx4RowsCut cut = rows_cut(m, n, k);
  // rows too far apart for 32-bit offsets are taken here, 16 at a time
  if (cut == Mx4RowsCut::kLds && ldx <= kMx4WideMaxStride) return launch_mx4_wide(q, wide_splits(n, k), ws, s);
  if (m <= 8)
    return cut == Mx4RowsCut::k32 ? launch_rows<false, 1, 2, 2, 8>(q, s) : launch_rows<false, 1, 2, 1, 8>(q, s);
  return cut == Mx4RowsCut::k32 ? launch_rows<false, 1, 1, 2, 8>(q, s) : launch_rows<false, 1, 1, 1, 8>(q, s);
}

// How a product of more than 16 rows and columns is cut: tiles of 16 x 16, 32 x 32
// or 64 x 32 by eight waves that share k here, or tiles through LDS
// (exl3_mx4_gemm.hip).  Small tiles load more for a product and are more; the
// estimates, in us, count the launch, a wave's turns over k and what further
// rounds of the CUs add, which is less where k is too short for all waves.  As
// measured (us, 16 / 32 / 64 x 32 / LDS):
//   100 rows 17408 ->   50   10.7   19.2   27.3   14.2
//   333 rows  2080 -> 1111    8.5    7.8    6.7   15.1
//   500 rows  5120 ->  500   13.0    8.5   11.3   14.6
//   500 rows  2048 -> 1000   11.8    7.4    6.4   10.9
//    32 rows 17408 -> 5120   27.9   21.0   23.9   20.1
//  1000 rows  1024 -> 4000   34.2   21.8   19.0    9.8
//  4000 rows    96 -> 5000  124     74.8   74.5   21.0
enum class Mx4Cut { k16, k32, k64x32, kLds };
static Mx4Cut matmul_cut(int64_t m, int64_t n, int64_t k) {
  const double units = (double)((k + kMx4UnitK - 1) / kMx4UnitK), eighth = units / 8;
  const double turns = __builtin_ceil(eighth), more = eighth < 0.35 ? 0.35 : (eighth < 1 ? eighth : turns);
  auto cost = [&](int64_t rows, int64_t cols, double turn) {
    const int64_t tiles = ((m + rows - 1) / rows) * ((n + cols - 1) / cols), rounds = (tiles + 255) / 256;
    return 2.2 + turn * (turns + (double)(rounds - 1) * more);
  };
  Mx4Cut best = Mx4Cut::k16;
  double least = cost(16, 16, 0.95);
  const double others[3] = {cost(32, 32, 1.95), cost(64, 32, 2.9), mx4_gemm_cost(m, n, k)};
  const Mx4Cut cuts[3] = {Mx4Cut::k32, Mx4Cut::k64x32, Mx4Cut::kLds};
  for (int i = 0; i < 3; ++i)
    if (others[i] < least) least = others[i], best = cuts[i];
  return best;
}
// The tiles in LDS, and few rows or columns, always do.  The others' 512 threads a
// tile pass a grid's 2^32 where the scales are too many for LDS tiles.
bool mx4_matmul_fits(int64_t m, int64_t n, int64_t k) {
  constexpr int64_t kMost = (int64_t)1 << 23;
  auto tiles = [&](int64_t rows, int64_t cols) { return ((m + rows - 1) / rows) * ((n + cols - 1) / cols); };
  if (m <= 16 || n <= 16 || tiles(16, 16) < kMost) return true;
  switch (matmul_cut(m, n, k)) {
    case Mx4Cut::k16: return false;
    case Mx4Cut::k32: return tiles(32, 32) < kMost;
    case Mx4Cut::k64x32: return tiles(64, 32) < kMost;
    default: return true;
  }
}
static bool use_gemm(int64_t m, int64_t n, int64_t k) {
  return m > 16 && n > 16 && matmul_cut(m, n, k) == Mx4Cut::kLds;
}
size_t mx4_matmul_workspace(int64_t m, int64_t n, int64_t k) {
  return use_gemm(m, n, k) ? mx4_gemm_workspace(m, n, k) : 0;
}

hipError_t launch_mx4_matmul(const uint8_t* a, const uint8_t* a_scales, int64_t m, const uint8_t* b,
                             const uint8_t* b_scales, int64_t n, int64_t k, const uint16_t* bias, void* y, int64_t ldy,
                             bool y_f32, void* ws, hipStream_t s) {
  if (use_gemm(m, n, k)) return launch_mx4_gemm(a, a_scales, m, b, b_scales, n, k, bias, y, ldy, y_f32, ws, s);
  Mx4RowsArgs q{a, a_scales, 0, b, b_scales, bias, y, ldy, m, n, (int)(k / kMx4Block), y_f32, 0, 0, 1, nullptr};
  if (m > 16 && n > 16) {
    const Mx4Cut cut = matmul_cut(m, n, k);
    if (cut == Mx4Cut::k16) return launch_rows<true, 1, 1, 1, 8>(q, s);
    if (cut == Mx4Cut::k32) return launch_rows<true, 2, 1, 2, 8>(q, s);
    return launch_rows<true, 4, 1, 2, 8>(q, s);
  }
  if (m > 16 && m > n) {  // few columns: as few rows, the operands' places changed
    q.a = b, q.a_scales = b_scales, q.m = n;
    q.b = a, q.b_scales = a_scales, q.n = m;
    q.swapped = 1;
  }
  // 16 rows or fewer in 32 columns a workgroup where the chip stays full, for
  // fewer loads of a; not for a row or two, whose a comes from cache, over very many
  // columns, where the two are near each other and whole rounds of the CUs decide (us,
  // 16 / 32 columns: 16 rows 17408 -> 5120 19.3 / 15.9, 17408 -> 2048 11.2 / 15.7, 2048 ->
  // 8192 4.8 / 4.2; one row 17408 -> 5120 14.3 / 12.4, 5120 -> 15000 9.4 / 8.8, 5120 ->
  // 17408 11.1 / 11.6, 5120 -> 20480 11.1 / 11.7, 4 rows 5120 -> 17408 12.2 / 12.5; the
  // rule takes the slower for one row 5120 -> 12288, 7.8 / 8.7, and 2048 -> 32768, 8.6 /
  // 8.3)
  return q.n >= 4096 && (q.m > 4 || q.n < 16384) ? launch_rows<true, 1, 1, 2, 8>(q, s)
                                                 : launch_rows<true, 1, 1, 1, 8>(q, s);
}

}  // namespace exl3
