// What the kernels of exl3_mx4_linear and of exl3_mx4_matmul's few rows share.
#pragma once

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
  int swapped;            // y is [n][ldy], bias [m]: the product's operands changed places
  uint32_t col_tiles;     // tiles of 16 NG columns
  int splits;             // workgroups that share a tile's k
  float* part;            // their sums [split][m][n], where there are several
};

__device__ __forceinline__ void mx4_store(const Mx4RowsArgs& q, int64_t row, int64_t col, float v) {
  const float y = v + (q.bias ? h2f(q.bias[q.swapped ? row : col]) : 0.f);
  const int64_t at = q.swapped ? col * q.ldy + row : row * q.ldy + col;
  if (q.y_f32)
    static_cast<float*>(q.y)[at] = y;
  else
    static_cast<uint16_t*>(q.y)[at] = f2h(y);
}

// y = sum of the splits in order (+ bias).
void launch_mx4_rows_finish(const Mx4RowsArgs& q, hipStream_t s);
// Up to 64 fp16 rows, at most kMx4WideMaxStride elements apart;
// splits > 1: partial sums fp32 [splits][m][n] in ws
constexpr int64_t kMx4WideMaxStride = (int64_t)1 << 24;
hipError_t launch_mx4_wide(Mx4RowsArgs q, int splits, void* ws, hipStream_t s);

}  // namespace exl3
