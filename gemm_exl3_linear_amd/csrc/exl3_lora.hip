// exl3_lora: y_i = base_i + scale_a B_a (A_a x_i), a row's own adapter a.
//
//   1. lora_plan    one workgroup sorts the rows by adapter and cuts each adapter's
//      into segments of up to 16 rows.
//   2. lora_shrink  workgroup (segment, k share): h = A x, fp16 matrix instructions,
//      fp32 sums over the waves' and the workgroups' shares of k.
//   3. lora_expand  workgroup (segment, 256 columns): h as two fp16 pieces against B.
//
// h is kept to 24 bits: a row's h is scaled by a power of two to below 2^15 and split
// into fp16 pieces hi + lo (hi holds 11 bits, lo the next 11 and, down to 2^-40 of the
// row's largest, at least 13 bits of what is left), which share the contraction with
// one load of B.
#include "exl3_internal.hpp"
#include "exl3_mx4.hpp"

namespace exl3 {

constexpr int kLoraSeg = 16;
constexpr int kLoraPlanThreads = 1024;
constexpr int kLoraWaves = 4;
constexpr int kLoraCols = 64 * kLoraWaves;

struct LoraSeg {
  int adapter;  // -1: none, y is base
  int first;    // of its rows in the order of adapters
  int count;
  int pad;
};

struct LoraArgs {
  LoraDesc d;
  const uint16_t* x;
  int64_t m, ldx;
  const int32_t* rows;
  const void* base;
  int64_t ldb;
  void* y;
  int64_t ldy;
  int f32;
  int copy;  // rows without an adapter are copied (base is not y)
  int splits;
  int rpad;  // floats of a row of h
  // workspace
  int* count;     // segments
  LoraSeg* segs;
  int* order;     // [m] rows in the order of adapters
  float* h;       // [splits][m][rpad] in that order
};

// ---------------------------------------------------------------------------
// plan
// ---------------------------------------------------------------------------
__device__ __forceinline__ int lora_bucket(const LoraArgs& q, int64_t i) {
  const int a = q.rows[i];
  return (unsigned)a < (unsigned)q.d.adapters ? a : q.d.adapters;
}

__global__ __launch_bounds__(kLoraPlanThreads) void lora_plan(LoraArgs q) {
  extern __shared__ int lds[];  // [buckets + 1] rows, then first row; [buckets + 1] first segment
  __shared__ int sum_rows[16], sum_segs[16];
  const int buckets = q.d.adapters + 1, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int* rows = lds;
  int* segs = lds + buckets + 1;
  for (int b = tid; b < buckets; b += kLoraPlanThreads) rows[b] = 0;
  __syncthreads();
  for (int64_t i = tid; i < q.m; i += kLoraPlanThreads) atomicAdd(&rows[lora_bucket(q, i)], 1);
  __syncthreads();
  // exclusive sums over the buckets, per consecutive ones a thread
  const int per = (buckets + kLoraPlanThreads - 1) / kLoraPlanThreads;
  int my_rows = 0, my_segs = 0;
  const auto segments = [&](int b, int n) { return b == q.d.adapters && !q.copy ? 0 : (n + kLoraSeg - 1) / kLoraSeg; };
  for (int b = tid * per; b < buckets && b < (tid + 1) * per; ++b) {
    my_rows += rows[b];
    my_segs += segments(b, rows[b]);
  }
  int at_row = my_rows, at_seg = my_segs;  // inclusive
  for (int d = 1; d < 64; d *= 2) {
    const int r = __shfl_up(at_row, d), s = __shfl_up(at_seg, d);
    if (lane >= d) {
      at_row += r;
      at_seg += s;
    }
  }
  if (lane == 63) {
    sum_rows[wave] = at_row;
    sum_segs[wave] = at_seg;
  }
  __syncthreads();
  at_row -= my_rows;
  at_seg -= my_segs;
  int all = 0;
  for (int w = 0; w < 16; ++w) {
    at_row += w < wave ? sum_rows[w] : 0;
    at_seg += w < wave ? sum_segs[w] : 0;
    all += sum_segs[w];
  }
  for (int b = tid * per; b < buckets && b < (tid + 1) * per; ++b) {
    const int n = rows[b];
    rows[b] = at_row;
    segs[b] = at_seg;
    at_row += n;
    at_seg += segments(b, n);
  }
  if (tid == 0) {
    rows[buckets] = (int)q.m;
    segs[buckets] = all;
    q.count[0] = all;
  }
  __syncthreads();
  for (int z = tid; z < all; z += kLoraPlanThreads) {
    int lo = 0, hi = buckets;  // the last bucket whose first segment is not past z
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (segs[mid] <= z) lo = mid;
      else hi = mid;
    }
    const int first = rows[lo] + (z - segs[lo]) * kLoraSeg;
    const int left = rows[lo + 1] - first;
    q.segs[z] = LoraSeg{lo == q.d.adapters ? -1 : lo, first, left < kLoraSeg ? left : kLoraSeg, 0};
  }
  __syncthreads();
  for (int64_t i = tid; i < q.m; i += kLoraPlanThreads) q.order[atomicAdd(&rows[lora_bucket(q, i)], 1)] = (int)i;
}

__device__ __forceinline__ int lora_rank(const LoraArgs& q, int adapter) {
  if (!q.d.ranks) return q.d.rank;
  const int r = q.d.ranks[adapter];
  return r < 0 ? 0 : r < q.d.rank ? r : q.d.rank;
}

// ---------------------------------------------------------------------------
// shrink
// ---------------------------------------------------------------------------
template <int RT>  // 16 RT >= rank
__global__ __launch_bounds__(kLoraWaves * 64) void lora_shrink(LoraArgs q) {
  __shared__ float4_t part[kLoraWaves][RT][64];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int g = lane >> 4, r = lane & 15;
  const int split = blockIdx.y, segs = q.count[0];
  const int64_t k = q.d.k;
  for (int z = blockIdx.x; z < segs; z += gridDim.x) {
    const LoraSeg sg = q.segs[z];
    if (sg.adapter < 0) continue;
    const int rank = lora_rank(q, sg.adapter);
    const uint16_t* x = q.x + (int64_t)q.order[sg.first + (r < sg.count ? r : 0)] * q.ldx;
    const uint16_t* a = q.d.a + (int64_t)sg.adapter * q.d.rank * k;
    float4_t acc[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[i] = float4_t{0.f, 0.f, 0.f, 0.f};
    for (int64_t at = 32 * (int64_t)(split * kLoraWaves + wave) + 8 * g; at - 8 * g < k;
         at += 32 * kLoraWaves * q.splits) {
      u32x4_t xv = {0u, 0u, 0u, 0u};
      if (at < k) xv = load16(x + at);
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        u32x4_t av = {0u, 0u, 0u, 0u};
        if (at < k && 16 * i + r < rank) av = load16(a + (16 * i + r) * k + at);
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, xv), __builtin_bit_cast(f16x8_t, av),
                                                        acc[i], 0, 0, 0);
      }
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) part[wave][i][lane] = acc[i];
    __syncthreads();
    for (int i = wave; 16 * i < q.rpad; i += kLoraWaves) {
      float4_t sum = part[0][i][lane];
#pragma unroll
      for (int w = 1; w < kLoraWaves; ++w) sum += part[w][i][lane];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (4 * g + j < sg.count) q.h[((int64_t)split * q.m + sg.first + 4 * g + j) * q.rpad + 16 * i + r] = sum[j];
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// expand
// ---------------------------------------------------------------------------
// h[.] of ranks 16 c + 8 (g & 1) .. + 7 as the operand's k places 8 g .. 8 g + 7: hi
// for g < 2, lo behind.
template <int RT>
__device__ __forceinline__ int lora_pieces(const LoraArgs& q, const LoraSeg& sg, int rank, int g, int r,
                                           f16x8_t (&piece)[RT]) {
  float h[RT][8];
  float top = 0.f;
#pragma unroll
  for (int c = 0; c < RT; ++c) {
    const int at = 16 * c + 8 * (g & 1);
#pragma unroll
    for (int j = 0; j < 8; ++j) h[c][j] = 0.f;
    if (r < sg.count && at < rank) {
      for (int s = 0; s < q.splits; ++s) {
        const float* p = q.h + ((int64_t)s * q.m + sg.first + r) * q.rpad + at;
#pragma unroll
        for (int j = 0; j < 8; ++j) h[c][j] += p[j];
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      h[c][j] = at + j < rank ? h[c][j] : 0.f;
      const float size = __builtin_fabsf(h[c][j]);
      top = size < __builtin_huge_valf() && size > top ? size : top;
    }
  }
  top = __builtin_fmaxf(top, __shfl_xor(top, 16));
  const int e = top > 0.f ? 15 - (__builtin_amdgcn_frexp_expf(top)) : 0;
#pragma unroll
  for (int c = 0; c < RT; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float v = __builtin_ldexpf(h[c][j], e);
      const _Float16 hi = (_Float16)v;
      const float rest = __builtin_isfinite(v) ? v - (float)hi : 0.f;
      piece[c][j] = g < 2 ? hi : (_Float16)rest;
    }
  return -e;
}

// Column n's sum for the row at `at` in the order of adapters, in fp32 and without
// pieces: an infinity of B times hi and lo of one h may be NaN (hi and lo of two signs,
// or lo 0) where the sum is infinite.
__device__ __noinline__ float lora_dot(const float* h, int64_t step, int splits, const uint16_t* b, int rank) {
  float sum = 0.f;
  for (int j = 0; j < rank; ++j) {
    float v = 0.f;
    for (int s = 0; s < splits; ++s) v += h[s * step + j];
    sum = __builtin_fmaf(v, (float)__builtin_bit_cast(_Float16, b[j]), sum);
  }
  return sum;
}

template <int RT, class T>
__global__ __launch_bounds__(kLoraWaves * 64) void lora_expand(LoraArgs q) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int g = lane >> 4, r = lane & 15;
  const int segs = q.count[0];
  const int64_t n0 = (int64_t)blockIdx.y * kLoraCols + 64 * wave;
  if (n0 >= q.d.n) return;
  for (int z = blockIdx.x; z < segs; z += gridDim.x) {
    const LoraSeg sg = q.segs[z];
    const int64_t row = q.order[sg.first + (r < sg.count ? r : 0)];
    float4_t acc[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[t] = float4_t{0.f, 0.f, 0.f, 0.f};
    float scale = 1.f;
    int e = 0;
    if (sg.adapter >= 0) {
      const int rank = lora_rank(q, sg.adapter);
      if (q.d.scales) scale = q.d.scales[sg.adapter];
      f16x8_t piece[RT];
      e = lora_pieces<RT>(q, sg, rank, g, r, piece);
      const uint16_t* b = q.d.b + (int64_t)sg.adapter * q.d.n * q.d.rank;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        // tile t's row i is column n0 + 16 (i / 4) + 4 t + i % 4, so that a lane ends
        // with 16 columns one after the other
        const int64_t n = n0 + 16 * (r >> 2) + 4 * t + (r & 3);
#pragma unroll
        for (int c = 0; c < RT; ++c) {
          const int at = 16 * c + 8 * (g & 1);
          f16x8_t w = {0, 0, 0, 0, 0, 0, 0, 0};
          if (n < q.d.n && at < rank) w = __builtin_bit_cast(f16x8_t, load16(b + n * q.d.rank + at));
#pragma unroll
          for (int j = 0; j < 8; ++j) w[j] = at + j < rank ? w[j] : (_Float16)0;
          acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w, piece[c], acc[t], 0, 0, 0);
        }
      }
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t n = n0 + 16 * g + 4 * t + j;
          const bool odd = !__builtin_isfinite(acc[t][j]);
          acc[t][j] = __builtin_ldexpf(acc[t][j], e);
          if (odd && r < sg.count && n < q.d.n)
            acc[t][j] = lora_dot(q.h + (int64_t)(sg.first + r) * q.rpad, q.m * q.rpad, q.splits, b + n * q.d.rank, rank);
        }
    }
    if (r >= sg.count) continue;
    const T* from = static_cast<const T*>(q.base) + row * q.ldb;
    T* to = static_cast<T*>(q.y) + row * q.ldy;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t n = n0 + 16 * g + 4 * t + j;
        if (n >= q.d.n) continue;
        const float delta = scale * acc[t][j];
        if (!q.base) to[n] = (T)(sg.adapter >= 0 ? delta : 0.f);
        else to[n] = sg.adapter >= 0 ? (T)((float)from[n] + delta) : from[n];
      }
  }
}

namespace {

constexpr int kLoraGrid = 4096;  // workgroups of segments at most: each takes every gridDim.x-th

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

int64_t lora_most_segs(const LoraDesc& d, int64_t m) {
  const int64_t most = (m + kLoraSeg - 1) / kLoraSeg + d.adapters;
  return most < m ? most : m;
}

int lora_splits(const LoraDesc& d, int64_t m) {
  const int64_t most = (d.k + 32 * kLoraWaves * 4 - 1) / (32 * kLoraWaves * 4);
  const int64_t want = 512 / lora_most_segs(d, m);
  return (int)(want < 1 ? 1 : want < most ? want : most);
}

struct LoraLayout {
  size_t segs, order, h, total;
};
LoraLayout lora_layout(const LoraDesc& d, int64_t m) {
  LoraLayout L;
  size_t off = 256;
  L.segs = off;
  off += align256((size_t)lora_most_segs(d, m) * sizeof(LoraSeg));
  L.order = off;
  off += align256((size_t)m * 4);
  L.h = off;
  off += align256((size_t)lora_splits(d, m) * m * ((d.rank + 15) / 16 * 16) * 4);
  L.total = off;
  return L;
}

template <int RT>
void launch_rt(const LoraArgs& q, hipStream_t s) {
  const int64_t segs = lora_most_segs(q.d, q.m);
  const uint32_t gx = (uint32_t)(segs < kLoraGrid ? segs : kLoraGrid);
  hipLaunchKernelGGL((lora_shrink<RT>), dim3(gx, q.splits), dim3(kLoraWaves * 64), 0, s, q);
  const dim3 grid(gx, (uint32_t)((q.d.n + kLoraCols - 1) / kLoraCols));
  if (q.f32) hipLaunchKernelGGL((lora_expand<RT, float>), grid, dim3(kLoraWaves * 64), 0, s, q);
  else hipLaunchKernelGGL((lora_expand<RT, _Float16>), grid, dim3(kLoraWaves * 64), 0, s, q);
}

}  // namespace

size_t lora_workspace(const LoraDesc& d, int64_t m) { return lora_layout(d, m).total; }

hipError_t launch_lora(const LoraDesc& d, const uint16_t* x, int64_t m, int64_t ldx, const int32_t* rows,
                       const void* base, int64_t ldb, void* y, int64_t ldy, bool f32, void* ws, hipStream_t s) {
  const LoraLayout L = lora_layout(d, m);
  unsigned char* w = static_cast<unsigned char*>(ws);
  LoraArgs q{};
  q.d = d;
  q.x = x;
  q.m = m;
  q.ldx = ldx;
  q.rows = rows;
  q.base = base;
  q.ldb = ldb;
  q.y = y;
  q.ldy = ldy;
  q.f32 = f32;
  q.copy = base != y;
  q.splits = lora_splits(d, m);
  q.rpad = (d.rank + 15) / 16 * 16;
  q.count = reinterpret_cast<int*>(w);
  q.segs = reinterpret_cast<LoraSeg*>(w + L.segs);
  q.order = reinterpret_cast<int*>(w + L.order);
  q.h = reinterpret_cast<float*>(w + L.h);
  hipLaunchKernelGGL(lora_plan, dim3(1), dim3(kLoraPlanThreads), 2 * (size_t)(d.adapters + 2) * 4, s, q);
  if (d.rank <= 16) launch_rt<1>(q, s);
  else if (d.rank <= 32) launch_rt<2>(q, s);
  else if (d.rank <= 64) launch_rt<4>(q, s);
  else if (d.rank <= 128) launch_rt<8>(q, s);
  else launch_rt<16>(q, s);
  return hipGetLastError();
}

}  // namespace exl3
