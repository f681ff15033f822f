// exl3_lora: y_i = base_i + scale_a B_a (A_a x_i), a row's own adapter a.
//
// One or a few rows and a small adapter: one launch (lora_few). Else two:
//   1. lora_shrink  workgroup (segment, k share, 64 ranks): h = A x, fp16 matrix
//      instructions, fp32 sums over the waves' and the workgroups' shares of k.
//   2. lora_expand  workgroup (segment, columns): h as two fp16 pieces against B, added
//      to base.
// A segment is up to 16 or 64 rows of one adapter, so that an adapter is read once for
// as many rows.  Up to kLoraPlanRows rows every workgroup finds its own segment (two
// passes over the rows' adapters in LDS, about a microsecond: less than a launch); more
// are sorted into segments by a launch of one workgroup before (lora_plan).
//
// h is kept to 24 bits: a row's h is scaled by a power of two to below 2^15 and split
// into fp16 pieces hi + lo (hi holds 11 bits, lo the next 11 and, down to 2^-40 of the
// row's largest, at least 13 bits of what is left); both meet one load of B.
#include "exl3_internal.hpp"
#include "exl3_mx4.hpp"

namespace exl3 {

constexpr int kLoraPlanRows = 1024;
constexpr int kLoraPlanThreads = 1024;
constexpr int kLoraThreads = 256;
constexpr int kLoraMaxSeg = 64;

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
  int copy;    // rows without an adapter are copied (base is not y)
  int splits;  // shares of k
  int rpad;    // floats of a row of h
  int tiles;   // 64-column tiles of a workgroup of lora_expand
  // workspace
  int* count;     // segments; null where workgroups find their own
  LoraSeg* segs;
  int* order;     // [m] rows in the order of adapters
  float* h;       // [splits][m][rpad]
};

// The segment of a workgroup.
struct LoraTask {
  int adapter;  // -1: none
  int count;
  int row[kLoraMaxSeg];  // past count: one of the rows
};

__device__ __forceinline__ int lora_bucket(const LoraArgs& q, int64_t i) {
  const int a = q.rows[i];
  return (unsigned)a < (unsigned)q.d.adapters ? a : q.d.adapters;
}

// Counts a row in its bucket; the rows of a wave are mostly of one request, and 64
// additions to one place would take their turns.
__device__ __forceinline__ void lora_count(int* rows, int bucket) {
  const int first = __builtin_amdgcn_readfirstlane(bucket);
  if (__all(bucket == first)) {
    const uint64_t here = __ballot(true);
    if (__ffsll((unsigned long long)here) - 1 == (int)(threadIdx.x & 63)) atomicAdd(&rows[bucket], (int)__popcll(here));
  } else {
    atomicAdd(&rows[bucket], 1);
  }
}

template <int S>
__device__ __forceinline__ int lora_segments(const LoraArgs& q, int bucket, int rows) {
  return bucket == q.d.adapters && !q.copy ? 0 : (rows + S - 1) / S;
}

// Inclusive sums over the threads of a workgroup of 64 W.
template <int W>
__device__ __forceinline__ int block_sum(int v, int* waves, int& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(v, d);
    v += lane >= d ? o : 0;
  }
  if (lane == 63) waves[wave] = v;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    v += w < wave ? waves[w] : 0;
    total += waves[w];
  }
  __syncthreads();
  return v;
}

// ---------------------------------------------------------------------------
// plan
// ---------------------------------------------------------------------------
template <int S>
__global__ __launch_bounds__(kLoraPlanThreads) void lora_plan(LoraArgs q) {
  extern __shared__ int lds[];  // [buckets + 1] rows, then first row; [buckets + 1] first segment
  __shared__ int waves[16];
  const int buckets = q.d.adapters + 1, tid = threadIdx.x;
  int* rows = lds;
  int* segs = lds + buckets + 1;
  for (int b = tid; b < buckets; b += kLoraPlanThreads) rows[b] = 0;
  __syncthreads();
  for (int64_t i = tid; i < q.m; i += kLoraPlanThreads) lora_count(rows, lora_bucket(q, i));
  __syncthreads();
  // exclusive sums over the buckets, consecutive ones a thread
  const int per = (buckets + kLoraPlanThreads - 1) / kLoraPlanThreads;
  int my_rows = 0, my_segs = 0, total, all;
  for (int b = tid * per; b < buckets && b < (tid + 1) * per; ++b) {
    my_rows += rows[b];
    my_segs += lora_segments<S>(q, b, rows[b]);
  }
  int at_row = block_sum<16>(my_rows, waves, total) - my_rows;
  int at_seg = block_sum<16>(my_segs, waves, all) - my_segs;
  for (int b = tid * per; b < buckets && b < (tid + 1) * per; ++b) {
    const int n = rows[b];
    rows[b] = at_row;
    segs[b] = at_seg;
    at_row += n;
    at_seg += lora_segments<S>(q, b, n);
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
    const int first = rows[lo] + (z - segs[lo]) * S;
    const int left = rows[lo + 1] - first;
    q.segs[z] = LoraSeg{lo == q.d.adapters ? -1 : lo, first, left < S ? left : S, 0};
  }
  __syncthreads();
  // places in a bucket by its count; their order has no say in any row's result
  for (int64_t i = tid; i < q.m; i += kLoraPlanThreads) {
    const int b = lora_bucket(q, i), lane = tid & 63;
    const int first = __builtin_amdgcn_readfirstlane(b);
    int at;
    if (__all(b == first)) {
      const uint64_t here = __ballot(true);
      int start = 0;
      if (__ffsll((unsigned long long)here) - 1 == lane) start = atomicAdd(&rows[b], (int)__popcll(here));
      at = __builtin_amdgcn_readfirstlane(start) + __popcll(here & ((1ull << lane) - 1));
    } else {
      at = atomicAdd(&rows[b], 1);
    }
    q.order[at] = (int)i;
  }
}

// Segment z as the workgroup's task; false past the last.  lds: [adapters + 1].
template <int S>
__device__ __forceinline__ bool lora_task(const LoraArgs& q, int z, int* lds, LoraTask& task) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (q.count) {
    if (z >= q.count[0]) return false;
    const LoraSeg sg = q.segs[z];
    if (tid < S) task.row[tid] = q.order[sg.first + (tid < sg.count ? tid : 0)];
    if (tid == 0) {
      task.adapter = sg.adapter;
      task.count = sg.count;
    }
    __syncthreads();
    return true;
  }
  constexpr int kEach = kLoraPlanRows / kLoraThreads;
  __shared__ int waves[4], found[2], chunk[kEach * 4];
  const int buckets = q.d.adapters + 1;
  int bucket[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int row = i * kLoraThreads + tid;
    bucket[i] = row < q.m ? lora_bucket(q, row) : -1;
  }
  for (int b = tid; b < buckets; b += kLoraThreads) lds[b] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    if (bucket[i] >= 0) lora_count(lds, bucket[i]);
  __syncthreads();
  const int per = (buckets + kLoraThreads - 1) / kLoraThreads;
  int mine = 0, total;
  for (int b = tid * per; b < buckets && b < (tid + 1) * per; ++b) mine += lora_segments<S>(q, b, lds[b]);
  int at = block_sum<4>(mine, waves, total) - mine;
  if (z >= total) return false;
  if (z >= at && z < at + mine) {
    int b = tid * per;
    for (;; ++b) {
      const int n = lora_segments<S>(q, b, lds[b]);
      if (z < at + n) break;
      at += n;
    }
    found[0] = b;
    found[1] = z - at;
  }
  // a row's place among its adapter's: those of the chunks of 64 rows before, and of the
  // lanes before
  __syncthreads();
  const int b = found[0], first = found[1] * S;
  uint64_t same[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    same[i] = __ballot(bucket[i] == b);
    if (lane == 0) chunk[i * 4 + wave] = (int)__popcll(same[i]);
  }
  __syncthreads();
  const int left = lds[b] - first, count = left < S ? left : S;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    if (bucket[i] != b) continue;
    int place = (int)__popcll(same[i] & ((1ull << lane) - 1)) - first;
    for (int c = 0; c < i * 4 + wave; ++c) place += chunk[c];
    if (place >= 0 && place < S) task.row[place] = i * kLoraThreads + tid;
    if (place == 0)
      for (int p = count; p < S; ++p) task.row[p] = i * kLoraThreads + tid;
  }
  if (tid == 0) {
    task.adapter = b == q.d.adapters ? -1 : b;
    task.count = count;
  }
  __syncthreads();
  return true;
}

__device__ __forceinline__ int lora_rank(const LoraArgs& q, int adapter) {
  if (!q.d.ranks) return q.d.rank;
  const int r = q.d.ranks[adapter];
  return r < 0 ? 0 : r < q.d.rank ? r : q.d.rank;
}

// ---------------------------------------------------------------------------
// shrink
// ---------------------------------------------------------------------------
// 16 MT rows against 16 RT ranks (from 64 blockIdx.z on); a wave takes whole lines of 64
// k one after the other, lane (row or rank r, g) their places 16 g .. 16 g + 15.
template <int MT, int RT>
__global__ __launch_bounds__(kLoraThreads) void lora_shrink(LoraArgs q) {
  constexpr int U = MT + RT <= 2 ? 4 : MT + RT <= 3 ? 2 : 1;  // lines whose loads go out together
  extern __shared__ int lds[];
  __shared__ float4_t part[4][MT * RT][64];
  __shared__ LoraTask task;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int g = lane >> 4, r = lane & 15;
  const int split = blockIdx.y, r0 = 64 * blockIdx.z;
  const int64_t k = q.d.k;
  for (int z = blockIdx.x; lora_task<16 * MT>(q, z, lds, task); z += gridDim.x) {
    const int rank = task.adapter < 0 ? 0 : lora_rank(q, task.adapter);
    if (rank > r0) {
      const uint16_t* x[MT];
      const uint16_t* a[RT];
#pragma unroll
      for (int i = 0; i < MT; ++i) x[i] = q.x + (int64_t)task.row[16 * i + r] * q.ldx;
#pragma unroll
      for (int j = 0; j < RT; ++j) {  // past the rank: the last rank's, whose sums are not used
        const int of = r0 + 16 * j + r;
        a[j] = q.d.a + ((int64_t)task.adapter * q.d.rank + (of < rank ? of : rank - 1)) * k;
      }
      float4_t acc[MT][RT];
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < RT; ++j) acc[i][j] = float4_t{0.f, 0.f, 0.f, 0.f};
      const int lines = (int)((k + 63) / 64);
      const int first = (int)((int64_t)lines * split / q.splits), end = (int)((int64_t)lines * (split + 1) / q.splits);
      for (int u0 = first + wave; u0 < end; u0 += 4 * U) {
        u32x4_t xv[U][2][MT], av[U][2][RT];
#pragma unroll
        for (int v = 0; v < U; ++v)
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const int u = u0 + 4 * v;
            const int64_t at = 64 * (int64_t)u + 16 * g + 8 * s;
            const int64_t from = u < end && at < k ? at : 0;
#pragma unroll
            for (int i = 0; i < MT; ++i) xv[v][s][i] = load16(x[i] + from);
#pragma unroll
            for (int j = 0; j < RT; ++j) av[v][s][j] = load16(a[j] + from);
          }
        if (64 * (int64_t)(u0 + 4 * (U - 1) + 1) > k || u0 + 4 * (U - 1) >= end) {  // what is not there is 0
#pragma unroll
          for (int v = 0; v < U; ++v)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              const int u = u0 + 4 * v;
              const bool there = u < end && 64 * (int64_t)u + 16 * g + 8 * s < k;
              const u32x4_t zero = {0u, 0u, 0u, 0u};
#pragma unroll
              for (int i = 0; i < MT; ++i) xv[v][s][i] = there ? xv[v][s][i] : zero;
#pragma unroll
              for (int j = 0; j < RT; ++j) av[v][s][j] = there ? av[v][s][j] : zero;
            }
        }
#pragma unroll
        for (int v = 0; v < U; ++v)
#pragma unroll
          for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
              for (int j = 0; j < RT; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, xv[v][s][i]),
                                                                   __builtin_bit_cast(f16x8_t, av[v][s][j]), acc[i][j],
                                                                   0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < RT; ++j) part[wave][i * RT + j][lane] = acc[i][j];
    }
    __syncthreads();
    if (rank > r0) {
      for (int t = wave; t < MT * RT; t += 4) {
        const int col = r0 + 16 * (t % RT) + r;
        float4_t sum = part[0][t][lane];
#pragma unroll
        for (int w = 1; w < 4; ++w) sum += part[w][t][lane];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = 16 * (t / RT) + 4 * g + j;
          if (i < task.count && col < q.rpad) q.h[((int64_t)split * q.m + task.row[i]) * q.rpad + col] = sum[j];
        }
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// expand
// ---------------------------------------------------------------------------
__device__ __forceinline__ void wave_lds_sync() {  // LDS of other lanes of this wave
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Sums that are not finite, again in fp32 and without pieces, for 16 of the task's rows
// from row0 on and 64 columns: an infinity of B times hi and lo of one h may be NaN (hi
// and lo of two signs, or lo 0) where the sum is infinite.
constexpr int kLoraOutStride = 68;  // floats of a row of a wave's 64 columns in LDS

__device__ __forceinline__ void lora_mend(const LoraArgs& q, const LoraTask& task, int row0, int64_t n0, int rank,
                                       float scale, const uint16_t* b, float* out) {
  const int64_t n = n0 + (threadIdx.x & 63);
  for (int i = 0; i < 16 && row0 + i < task.count; ++i) {
    float* at = out + i * kLoraOutStride + (threadIdx.x & 63);
    if (n >= q.d.n || __builtin_isfinite(*at)) continue;
    const float* h = q.h + (int64_t)task.row[row0 + i] * q.rpad;
    float sum = 0.f;
    for (int j = 0; j < rank; ++j) {
      float v = 0.f;
      for (int s = 0; s < q.splits; ++s) v += h[(int64_t)s * q.m * q.rpad + j];
      sum = __builtin_fmaf(v, (float)__builtin_bit_cast(_Float16, b[n * q.d.rank + j]), sum);
    }
    *at = scale * sum;
  }
  wave_lds_sync();
}

// Zeroes the elements of w past `left`.
__device__ __forceinline__ f16x8_t lora_keep(f16x8_t w, int left) {
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = j < left ? w[j] : (_Float16)0;
  return w;
}

template <int MT>
struct LoraExpandLds {
  // pieces: [hi, lo][row][32 chunks ranks], rows 16 bytes apart beyond that: the 16 rows
  // of an operand lie in different banks
  static __host__ __device__ int row_bytes(int chunks) { return 64 * chunks + 16; }
  static __host__ __device__ int pieces(int chunks) { return 2 * 16 * MT * row_bytes(chunks); }
  static __host__ __device__ int out() { return 4 * 16 * kLoraOutStride * 4; }  // 16 rows a wave
};

// The task's h as pieces in LDS, and each row's exponent.
template <int MT>
__device__ __forceinline__ void lora_pieces(const LoraArgs& q, const LoraTask& task, int rank, int chunks, uint8_t* lds,
                                            int* exponent) {
  constexpr int kEach = kLoraThreads / (16 * MT);  // threads of a row
  constexpr int kMost = 256 / 4 / kEach;
  const int row = threadIdx.x / kEach, part = threadIdx.x % kEach;
  float4_t h[kMost];
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    const int at = 4 * (part + i * kEach);
    h[i] = float4_t{0.f, 0.f, 0.f, 0.f};
    if (row < task.count && at < rank) {
      const float* p = q.h + (int64_t)task.row[row] * q.rpad + at;
      for (int s = 0; s < q.splits; ++s) h[i] += *reinterpret_cast<const float4_t*>(p + (int64_t)s * q.m * q.rpad);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      h[i][j] = at + j < rank ? h[i][j] : 0.f;
      const float size = __builtin_fabsf(h[i][j]);
      top = size < __builtin_huge_valf() && size > top ? size : top;
    }
  }
#pragma unroll
  for (int d = 1; d < kEach; d *= 2) top = __builtin_fmaxf(top, __shfl_xor(top, d));
  const int e = top > 0.f ? 15 - __builtin_amdgcn_frexp_expf(top) : 0;
  if (part == 0) exponent[row] = -e;
  const int stride = LoraExpandLds<MT>::row_bytes(chunks);
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    const int at = 4 * (part + i * kEach);
    if (at >= 32 * chunks) continue;
    half4_t hi, lo;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float v = __builtin_ldexpf(h[i][j], e);
      hi[j] = (_Float16)v;
      lo[j] = (_Float16)(__builtin_isfinite(v) ? v - (float)hi[j] : 0.f);
    }
    *reinterpret_cast<half4_t*>(lds + row * stride + 2 * at) = hi;
    *reinterpret_cast<half4_t*>(lds + (16 * MT + row) * stride + 2 * at) = lo;
  }
}

// Bits of V bytes a lane, of base and of y.
template <class T, bool VEC>
struct LoraIo {
  static constexpr int kElems = VEC ? 16 / (int)sizeof(T) : 1;  // of a lane
  static constexpr int kLanes = 64 / kElems;                    // of a row of 64 columns
  static constexpr int kRows = 64 / kLanes;                     // of an instruction
  typedef T vec __attribute__((ext_vector_type(kElems)));
};
template <class T>
struct LoraIo<T, false> {
  static constexpr int kElems = 1, kLanes = 64, kRows = 1;
  struct vec {
    T v;
    __device__ T& operator[](int) { return v; }
  };
};

// 16 MT rows; a wave takes tiles of 64 columns: matrix row i of tile t is column 16 t + i,
// a matrix column is a row of the task.  PAIR (ranks up to 16): an operand's upper half of
// k holds another 16 columns, met by pieces that are zero in the other half.
// VEC: base and y have rows of whole 16 bytes.
template <int MT, bool PAIR, class T, bool VEC>
__global__ __launch_bounds__(kLoraThreads, MT == 4 ? 2 : 4) void lora_expand(LoraArgs q) {
  using L = LoraExpandLds<MT>;
  using Io = LoraIo<T, VEC>;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ LoraTask task;
  __shared__ int exponent[16 * MT];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int g = lane >> 4, r = lane & 15;
  const int64_t N = q.d.n;
  const int64_t tile0 = (int64_t)blockIdx.y * 4 * q.tiles;
  for (int z = blockIdx.x; lora_task<16 * MT>(q, z, reinterpret_cast<int*>(smem), task); z += gridDim.x) {
    const int adapter = __builtin_amdgcn_readfirstlane(task.adapter);
    const int count = __builtin_amdgcn_readfirstlane(task.count);
    const int rank = adapter < 0 ? 0 : lora_rank(q, adapter);
    const int chunks = (rank + 31) / 32;
    const float scale = adapter >= 0 && q.d.scales ? q.d.scales[adapter] : 1.f;
    lora_pieces<MT>(q, task, rank, chunks, smem, exponent);
    __syncthreads();
    const int stride = L::row_bytes(chunks);
    float* out = reinterpret_cast<float*>(smem + L::pieces(chunks)) + wave * (16 * kLoraOutStride);
    const uint16_t* b = q.d.b + (int64_t)(adapter < 0 ? 0 : adapter) * N * q.d.rank;
    for (int it = 0; it < q.tiles; ++it) {
      const int64_t n0 = 64 * (tile0 + wave + 4 * it);
      if (n0 >= N) break;
      // base ahead of the products; of rows past count another row's, of columns past n
      // the first's
      const int col = lane % Io::kLanes * Io::kElems, sub = lane / Io::kLanes;
      const bool col_there = n0 + col < N;
      constexpr int kIo = 16 / Io::kRows;  // instructions of 16 rows
      typename Io::vec from[MT][kIo];
      if (q.base) {
        const T* at = static_cast<const T*>(q.base) + (col_there ? n0 + col : 0);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int o = 0; o < kIo; ++o)
            from[i][o] = *reinterpret_cast<const typename Io::vec*>(at + task.row[16 * i + Io::kRows * o + sub] * q.ldb);
      }
      float4_t acc[MT][4];
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[i][t] = float4_t{0.f, 0.f, 0.f, 0.f};
      if constexpr (PAIR) {
        if (rank > 0) {
          f16x8_t w[2];
          const int at = 8 * (g & 1);
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const int64_t n = n0 + 32 * p + 16 * (g >> 1) + r;
            w[p] = __builtin_bit_cast(f16x8_t, load16(b + (n < N ? n : N - 1) * q.d.rank + (at < rank ? at : 0)));
          }
          if (rank < 16)
            for (int p = 0; p < 2; ++p) w[p] = lora_keep(w[p], rank - at);
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              const f16x8_t h = *reinterpret_cast<const f16x8_t*>(smem + (p * 16 * MT + 16 * i + r) * stride + 2 * at);
#pragma unroll
              for (int o = 0; o < 2; ++o) {
                const f16x8_t part = lora_keep(h, (g >> 1) == o ? 8 : 0);
#pragma unroll
                for (int v = 0; v < 2; ++v)
                  acc[i][2 * v + o] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[v], part, acc[i][2 * v + o], 0, 0, 0);
              }
            }
        }
      } else {
        const uint16_t* of[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int64_t n = n0 + 16 * t + r;
          of[t] = b + (n < N ? n : N - 1) * q.d.rank;
        }
        for (int c = 0; c < chunks; ++c) {
          const int at = 32 * c + 8 * g;
          f16x8_t w[4];
#pragma unroll
          for (int t = 0; t < 4; ++t) w[t] = __builtin_bit_cast(f16x8_t, load16(of[t] + (at < rank ? at : 0)));
          if (32 * c + 32 > rank) {
#pragma unroll
            for (int t = 0; t < 4; ++t) w[t] = lora_keep(w[t], rank - at);
          }
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              const f16x8_t h = *reinterpret_cast<const f16x8_t*>(smem + (p * 16 * MT + 16 * i + r) * stride + 2 * at);
#pragma unroll
              for (int t = 0; t < 4; ++t) acc[i][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[t], h, acc[i][t], 0, 0, 0);
            }
        }
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        if (16 * i >= count) break;
        const int e = exponent[16 * i + r];
        bool odd = false;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          float4_t v;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            odd = odd || !__builtin_isfinite(acc[i][t][j]);
            v[j] = scale * __builtin_ldexpf(acc[i][t][j], e);
          }
          *reinterpret_cast<float4_t*>(out + r * kLoraOutStride + 16 * t + 4 * g) = v;
        }
        wave_lds_sync();
        if (__builtin_expect(__any(odd), 0)) lora_mend(q, task, 16 * i, n0, rank, scale, b, out);
#pragma unroll
        for (int o = 0; o < kIo; ++o) {
          const int row = 16 * i + Io::kRows * o + sub;
          const float* p = out + (Io::kRows * o + sub) * kLoraOutStride + col;
          typename Io::vec to;
#pragma unroll
          for (int j = 0; j < Io::kElems; ++j)
            to[j] = !q.base ? (T)(adapter < 0 ? 0.f : p[j])
                            : adapter < 0 ? from[i][o][j] : (T)((float)from[i][o][j] + p[j]);
          if (row < count && col_there)
            *reinterpret_cast<typename Io::vec*>(static_cast<T*>(q.y) + task.row[row] * q.ldy + n0 + col) = to;
        }
        wave_lds_sync();
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// few rows
// ---------------------------------------------------------------------------
// A workgroup takes a row (blockIdx.y) and 4096 / RJ columns: it makes the row's whole h
// itself (A from L2, which costs less than a launch) and then its columns, RJ / 8 threads
// a column.  RJ: a power of two >= rank.
constexpr int kLoraFewThreads = 512;

template <int RJ, class T>
__global__ __launch_bounds__(kLoraFewThreads) void lora_few(LoraArgs q) {
  constexpr int NW = kLoraFewThreads / 64, kEach = RJ / 8, kCols = kLoraFewThreads / kEach;
  __shared__ float part[NW][RJ];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t row = blockIdx.y, k = q.d.k;
  const int bucket = lora_bucket(q, row);
  const bool none = bucket == q.d.adapters;
  if (none && !q.copy) return;
  const int64_t n = (int64_t)blockIdx.x * kCols + threadIdx.x / kEach;
  const int j0 = 8 * (threadIdx.x % kEach);
  const int rank = none ? 0 : lora_rank(q, bucket);
  f16x8_t w = {0, 0, 0, 0, 0, 0, 0, 0};
  if (n < q.d.n && j0 < rank)
    w = __builtin_bit_cast(f16x8_t, load16(q.d.b + ((int64_t)bucket * q.d.n + n) * q.d.rank + j0));
  float acc[RJ];
#pragma unroll
  for (int j = 0; j < RJ; ++j) acc[j] = 0.f;
  if (rank > 0) {
    const uint16_t* x = q.x + row * q.ldx;
    const uint16_t* a = q.d.a + (int64_t)bucket * q.d.rank * k;
    for (int64_t at = 512 * wave + 8 * lane; at < k; at += 512 * NW) {
      const f16x8_t xv = __builtin_bit_cast(f16x8_t, load16(x + at));
#pragma unroll
      for (int j = 0; j < RJ; ++j) {
        const f16x8_t av = __builtin_bit_cast(f16x8_t, load16(a + (j < rank ? j : 0) * k + at));
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[j] = __builtin_fmaf((float)av[i], (float)xv[i], acc[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < RJ; ++j) {
      float v = acc[j];
#pragma unroll
      for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
      if (lane == 0) part[wave][j] = v;
    }
  }
  __syncthreads();
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (j0 + i < rank) {
      float h = 0.f;
#pragma unroll
      for (int o = 0; o < NW; ++o) h += part[o][j0 + i];
      sum = __builtin_fmaf(h, (float)w[i], sum);
    }
  }
#pragma unroll
  for (int d = 1; d < kEach; d *= 2) sum += __shfl_xor(sum, d);
  if (j0 || n >= q.d.n) return;
  const float delta = none ? 0.f : (q.d.scales ? q.d.scales[bucket] : 1.f) * sum;
  T* to = static_cast<T*>(q.y) + row * q.ldy + n;
  if (!q.base) *to = (T)delta;
  else {
    const T from = static_cast<const T*>(q.base)[row * q.ldb + n];
    *to = none ? from : (T)((float)from + delta);
  }
}

namespace {

constexpr int kLoraGrid = 8192;  // segments' workgroups at most: each takes every gridDim.x-th
constexpr int kLoraFewRows = 4, kLoraFewRank = 64;

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

bool lora_is_few(const LoraDesc& d, int64_t m) {
  return m <= kLoraFewRows && d.rank <= kLoraFewRank && d.rank * d.k <= (int64_t)1 << 17;
}

// 64 rows a segment where adapters have more than 16 each on average.
bool lora_long(const LoraDesc& d, int64_t m) { return m > 16 * (int64_t)(d.adapters > 1 ? d.adapters : 1); }

int64_t lora_most_segs(const LoraDesc& d, int64_t m) {
  const int s = lora_long(d, m) ? 64 : 16;
  const int64_t most = m / s + d.adapters + 1;  // a bucket's last may be short, that of none too
  return most < m ? most : m;
}

int lora_splits(const LoraDesc& d, int64_t m) {
  const int64_t lines = (d.k + 63) / 64;
  const int64_t groups = lora_most_segs(d, m) * ((d.rank + 63) / 64);
  const int64_t want = 512 / groups, most = lines / 8;  // two lines a wave
  const int64_t s = want < most ? want : most;
  return (int)(s < 1 ? 1 : s > 16 ? 16 : s);
}

struct LoraLayout {
  size_t segs, order, h, total;
};
LoraLayout lora_layout(const LoraDesc& d, int64_t m) {
  LoraLayout L;
  size_t off = 256;
  L.segs = off;
  if (m > kLoraPlanRows) off += align256((size_t)lora_most_segs(d, m) * sizeof(LoraSeg));
  L.order = off;
  if (m > kLoraPlanRows) off += align256((size_t)m * 4);
  L.h = off;
  off += align256((size_t)lora_splits(d, m) * m * ((d.rank + 15) / 16 * 16) * 4);
  L.total = off;
  return L;
}

template <class T>
void launch_few(const LoraArgs& q, hipStream_t s) {
  const int rj = q.d.rank <= 8 ? 8 : q.d.rank <= 16 ? 16 : q.d.rank <= 32 ? 32 : 64;
  const int cols = kLoraFewThreads * 8 / rj;
  const dim3 grid((uint32_t)((q.d.n + cols - 1) / cols), (uint32_t)q.m), block(kLoraFewThreads);
  if (rj == 8) hipLaunchKernelGGL((lora_few<8, T>), grid, block, 0, s, q);
  else if (rj == 16) hipLaunchKernelGGL((lora_few<16, T>), grid, block, 0, s, q);
  else if (rj == 32) hipLaunchKernelGGL((lora_few<32, T>), grid, block, 0, s, q);
  else hipLaunchKernelGGL((lora_few<64, T>), grid, block, 0, s, q);
}

template <int MT, class T, bool VEC>
void launch_expand(const LoraArgs& q, dim3 grid, size_t lds, hipStream_t s) {
  if (q.d.rank <= 16) hipLaunchKernelGGL((lora_expand<MT, true, T, VEC>), grid, dim3(kLoraThreads), lds, s, q);
  else hipLaunchKernelGGL((lora_expand<MT, false, T, VEC>), grid, dim3(kLoraThreads), lds, s, q);
}

template <int MT>
void launch_mt(LoraArgs q, bool f32, hipStream_t s) {
  const int64_t segs = lora_most_segs(q.d, q.m);
  const uint32_t gx = (uint32_t)(segs < kLoraGrid ? segs : kLoraGrid);
  const size_t plan = (size_t)(q.d.adapters + 1) * 4;
  const dim3 shrink(gx, (uint32_t)q.splits, (uint32_t)((q.d.rank + 63) / 64)), block(kLoraThreads);
  if (q.d.rank <= 16) hipLaunchKernelGGL((lora_shrink<MT, 1>), shrink, block, plan, s, q);
  else if (q.d.rank <= 32) hipLaunchKernelGGL((lora_shrink<MT, 2>), shrink, block, plan, s, q);
  else hipLaunchKernelGGL((lora_shrink<MT, 4>), shrink, block, plan, s, q);
  const int64_t tiles = (q.d.n + 63) / 64;
  // more tiles a workgroup where there are workgroups enough
  int each = 4;
  while (each > 1 && (int64_t)gx * ((tiles + 4 * each - 1) / (4 * each)) < 1024) each /= 2;
  q.tiles = each;
  const dim3 grid(gx, (uint32_t)((tiles + 4 * each - 1) / (4 * each)));
  const size_t need = LoraExpandLds<MT>::pieces((q.d.rank + 31) / 32) + LoraExpandLds<MT>::out();
  const size_t lds = need > plan ? need : plan;
  const uintptr_t at = reinterpret_cast<uintptr_t>(q.base) | reinterpret_cast<uintptr_t>(q.y);
  const int64_t elems = f32 ? 4 : 8;
  const bool vec = at % 16 == 0 && q.d.n % elems == 0 && q.ldy % elems == 0 && (!q.base || q.ldb % elems == 0);
  if (f32 && vec) launch_expand<MT, float, true>(q, grid, lds, s);
  else if (f32) launch_expand<MT, float, false>(q, grid, lds, s);
  else if (vec) launch_expand<MT, _Float16, true>(q, grid, lds, s);
  else launch_expand<MT, _Float16, false>(q, grid, lds, s);
}

}  // namespace

size_t lora_workspace(const LoraDesc& d, int64_t m) { return lora_is_few(d, m) ? 0 : lora_layout(d, m).total; }

hipError_t launch_lora(const LoraDesc& d, const uint16_t* x, int64_t m, int64_t ldx, const int32_t* rows,
                       const void* base, int64_t ldb, void* y, int64_t ldy, bool f32, void* ws, hipStream_t s) {
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
  q.copy = base != y;
  if (lora_is_few(d, m)) {
    if (f32) launch_few<float>(q, s);
    else launch_few<_Float16>(q, s);
    return hipGetLastError();
  }
  const LoraLayout L = lora_layout(d, m);
  unsigned char* w = static_cast<unsigned char*>(ws);
  q.splits = lora_splits(d, m);
  q.rpad = (d.rank + 15) / 16 * 16;
  q.h = reinterpret_cast<float*>(w + L.h);
  const bool longer = lora_long(d, m);
  if (m > kLoraPlanRows) {
    q.count = reinterpret_cast<int*>(w);
    q.segs = reinterpret_cast<LoraSeg*>(w + L.segs);
    q.order = reinterpret_cast<int*>(w + L.order);
    const size_t lds = 2 * (size_t)(d.adapters + 2) * 4;
    if (longer) hipLaunchKernelGGL((lora_plan<64>), dim3(1), dim3(kLoraPlanThreads), lds, s, q);
    else hipLaunchKernelGGL((lora_plan<16>), dim3(1), dim3(kLoraPlanThreads), lds, s, q);
  }
  if (longer) launch_mt<4>(q, f32, s);
  else launch_mt<1>(q, f32, s);
  return hipGetLastError();
}

}  // namespace exl3
