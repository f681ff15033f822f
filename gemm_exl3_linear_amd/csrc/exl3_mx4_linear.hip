// exl3_mx4_linear and exl3_mx4_matmul: the kernels whose waves split k.
#include "exl3_internal.hpp"
#include "exl3_mx4_rows.hpp"

namespace exl3 {

struct Mx4RowsArgs {
  const void* a;          // fp16 [m][lda], or codes [m][k/2]
  const uint8_t* a_scales;
  int64_t lda;            // elements (fp16 rows only)
  const uint8_t* b;       // codes [n][k/2]
  const uint8_t* b_scales;
  const uint16_t* bias;
  void* y;
  int64_t ldy;
  int64_t m, n;
  int kb;                 // blocks of 32 in a row
  int y_f32;
  uint32_t col_tiles;     // tiles of 16 NG columns
};

// Output tiles that fit the LDS of one combine round, at a kilobyte a wave.
constexpr int kMx4CombineTiles = 64;

template <bool A4, int MG, int NG, int NW>
__global__ __launch_bounds__(NW * 64) void mx4_rows_kernel(Mx4RowsArgs q) {
  constexpr int T = MG * NG;
  constexpr int R = T * NW <= kMx4CombineTiles ? T : kMx4CombineTiles / NW;  // tiles a round
  static_assert(T % R == 0, "combine rounds are whole");
  __shared__ float4_t part[NW * R * 64];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int g = lane >> 4, r = lane & 15;
  const uint32_t tm = blockIdx.x / q.col_tiles, tn = blockIdx.x - tm * q.col_tiles;
  const int64_t m0 = (int64_t)tm * (16 * MG), n0 = (int64_t)tn * (16 * NG);
  const int kb = q.kb;
  const int64_t pitch = (int64_t)kb * 16;

  const uint8_t* bc[NG];
  const uint8_t* bs[NG];
#pragma unroll
  for (int ng = 0; ng < NG; ++ng) {
    int64_t row = n0 + 16 * ng + r;
    row = row < q.n ? row : q.n - 1;  // columns past n are computed and not stored
    bc[ng] = q.b + row * pitch;
    bs[ng] = q.b_scales + row * kb;
  }
  const uint8_t* ac[MG];
  const uint8_t* as[MG];
  bool there[MG];
#pragma unroll
  for (int mg = 0; mg < MG; ++mg) {
    int64_t row = m0 + 16 * mg + r;
    there[mg] = row < q.m;
    row = there[mg] ? row : q.m - 1;
    if constexpr (A4) {
      ac[mg] = static_cast<const uint8_t*>(q.a) + row * pitch;
      as[mg] = q.a_scales + row * kb;
    } else {
      ac[mg] = reinterpret_cast<const uint8_t*>(static_cast<const uint16_t*>(q.a) + row * q.lda);
      as[mg] = nullptr;
    }
  }

  float4_t acc[NG][MG];
#pragma unroll
  for (int ng = 0; ng < NG; ++ng)
#pragma unroll
    for (int mg = 0; mg < MG; ++mg) acc[ng][mg] = float4_t{0.f, 0.f, 0.f, 0.f};

  const int units = (kb + kMx4UnitBlocks - 1) / kMx4UnitBlocks;
  for (int u = wave; u < units; u += NW) {
    Mx4Unit w[NG];
#pragma unroll
    for (int ng = 0; ng < NG; ++ng) mx4_load_unit(bc[ng], bs[ng], kb, u, g, w[ng]);
    if constexpr (A4) {
      Mx4Unit x[MG];
#pragma unroll
      for (int mg = 0; mg < MG; ++mg) mx4_load_unit(ac[mg], as[mg], kb, u, g, x[mg]);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int ng = 0; ng < NG; ++ng)
#pragma unroll
          for (int mg = 0; mg < MG; ++mg)
            acc[ng][mg] = mfma_mx4(x[mg].half[h], mx4_own_scale(x[mg], h, g), w[ng].half[h],
                                   mx4_own_scale(w[ng], h, g), acc[ng][mg]);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        f16x8_t x[MG][4];
#pragma unroll
        for (int mg = 0; mg < MG; ++mg)
          mx4_load_x(reinterpret_cast<const uint16_t*>(ac[mg]), there[mg], kb, u, h, g, x[mg]);
#pragma unroll
        for (int ng = 0; ng < NG; ++ng) mx4_mma_f16<MG>(x, w[ng], h, acc[ng]);
      }
    }
  }

  // Sum over the waves in wave order, R output tiles a round; lane l of a tile
  // holds rows 4 (l / 16) .. + 3 of column l % 16.
#pragma unroll
  for (int t0 = 0; t0 < T; t0 += R) {
    if (t0) __syncthreads();
#pragma unroll
    for (int i = 0; i < R; ++i) part[(wave * R + i) * 64 + lane] = acc[(t0 + i) / MG][(t0 + i) % MG];
    __syncthreads();
    for (int e = threadIdx.x; e < R * 64; e += NW * 64) {
      float4_t v = part[e];
#pragma unroll
      for (int w = 1; w < NW; ++w) v += part[w * R * 64 + e];
      const int t = t0 + (e >> 6), l = e & 63;
      const int64_t col = n0 + 16 * (t / MG) + (l & 15);
      if (col >= q.n) continue;
      const int64_t row = m0 + 16 * (t % MG) + 4 * (l >> 4);
      const float bias = q.bias ? h2f(q.bias[col]) : 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (row + i >= q.m) break;
        const int64_t at = (row + i) * q.ldy + col;
        if (q.y_f32)
          static_cast<float*>(q.y)[at] = v[i] + bias;
        else
          static_cast<uint16_t*>(q.y)[at] = f2h(v[i] + bias);
      }
    }
  }
}

template <bool A4, int MG, int NG, int NW>
static hipError_t launch_rows(Mx4RowsArgs q, hipStream_t s) {
  q.col_tiles = (uint32_t)((q.n + 16 * NG - 1) / (16 * NG));
  const uint32_t row_tiles = (uint32_t)((q.m + 16 * MG - 1) / (16 * MG));
  hipLaunchKernelGGL((mx4_rows_kernel<A4, MG, NG, NW>), dim3(q.col_tiles * row_tiles), dim3(NW * 64), 0, s, q);
  return hipGetLastError();
}

size_t mx4_matmul_workspace(int64_t, int64_t, int64_t) { return 0; }
size_t mx4_linear_workspace(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_mx4_linear(const uint8_t* codes, const uint8_t* scales, int64_t n, int64_t k, const uint16_t* bias,
                             const uint16_t* x, int64_t m, int64_t ldx, void* y, int64_t ldy, bool y_f32, void*,
                             hipStream_t s) {
  const Mx4RowsArgs q{x, nullptr, ldx, codes, scales, bias, y, ldy, m, n, (int)(k / kMx4Block), y_f32, 0};
  if (m <= 16) return launch_rows<false, 1, 1, 8>(q, s);
  if (m <= 32) return launch_rows<false, 2, 1, 8>(q, s);
  return launch_rows<false, 4, 1, 8>(q, s);
}

hipError_t launch_mx4_matmul(const uint8_t* a, const uint8_t* a_scales, int64_t m, const uint8_t* b,
                             const uint8_t* b_scales, int64_t n, int64_t k, const uint16_t* bias, void* y, int64_t ldy,
                             bool y_f32, void*, hipStream_t s) {
  const Mx4RowsArgs q{a, a_scales, 0, b, b_scales, bias, y, ldy, m, n, (int)(k / kMx4Block), y_f32, 0};
  if (m <= 16) return launch_rows<true, 1, 1, 8>(q, s);
  return launch_rows<true, 4, 4, 4>(q, s);
}

}  // namespace exl3
