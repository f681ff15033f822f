// exl3_lora: y_i = base_i + scale_a B_a (A_a x_i), a row's own adapter a.
//
// One or a few rows and a small adapter: one launch (lora_few). Else two:
//   1. lora_shrink  workgroup (segment, k share, 64 ranks): h = A x, fp16 matrix
//      instructions, fp32 sums over the waves' and the workgroups' shares of k.
//   2. lora_expand  workgroup (segment, columns): h as two fp16 pieces against B, added
//      to base.
// A segment is up to 16 or 64 rows of one adapter, so that an adapter is read once for
// as many rows.  Up to kLoraPlanRows rows lora_shrink's workgroups find their own segments
// (two passes over the rows' adapters in LDS, about a microsecond) and leave them to
// lora_expand; more are sorted by a launch of one workgroup before (lora_plan, 6 us).
//
// h is kept to 23 bits: a row's h is scaled by a power of two to below 2^15 and split
// into fp16 pieces hi + 2^-12 lo, both of which meet one load of B.  hi is off by at most
// 2^-12 of the value, and lo, of the same size, by as much of that: hi + 2^-12 lo is off
// by at most 2^-23 of the value down to 2^-29 of the row's largest, where hi leaves fp16's
// normals, and by at most 2^-51 of the largest below.  (fp32 sums of a thousand products
// are off by more.)
#include "exl3_internal.hpp"
#include "exl3_tile64.hpp"

namespace exl3 {

// By workgroups / by lora_plan, us of a call 5120 -> 5120: 1024 rows 20.6 / 26, 2048 rows
// 33.5 / 34.7 of 8 adapters and 38 to 46 / 40.5 of 256, 4096 rows 58.5 / 57.
constexpr int kLoraPlanRows = 1024;
constexpr int kLoraPlanThreads = 1024;
constexpr int kLoraThreads = 256;
constexpr int kLoraMaxSeg = 64;

struct LoraSeg {
  int adapter;  // -1: none, y is base
  int count;    // of its rows; 0: no such segment
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
  int tiles;   // 64-column tiles of a wave (lora_expand) or a workgroup (lora_expand_long)
  // workspace
  int planned;    // segments are in the workspace before lora_shrink, not from it
  LoraSeg* segs;  // [segments at most]
  int* order;     // [segments at most][rows of a segment]
  int* place;     // [m] a row's place among its adapter's, where registers do not hold it
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

// Counts a row in its bucket and gives its place there.  The rows of a wave are mostly of
// one request, and 64 additions to one place would take their turns.
__device__ __forceinline__ int lora_count(int* rows, int bucket) {
  const int first = __builtin_amdgcn_readfirstlane(bucket), lane = threadIdx.x & 63;
  if (!__all(bucket == first)) return atomicAdd(&rows[bucket], 1);
  const uint64_t here = __ballot(true);
  int start = 0;
  if (__ffsll((unsigned long long)here) - 1 == lane) start = atomicAdd(&rows[bucket], (int)__popcll(here));
  return __builtin_amdgcn_readfirstlane(start) + (int)__popcll(here & ((1ull << lane) - 1));
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
// One workgroup.  Rows of an adapter get places in the order of their counting, which is
// not the same in every run; a row's result does not depend on its place.
template <int S>
__global__ __launch_bounds__(kLoraPlanThreads) void lora_plan(LoraArgs q, int most) {
  extern __shared__ int lds[];  // [buckets] rows; [buckets] first segment
  __shared__ int waves[kLoraPlanThreads / 64];
  constexpr int kHeld = 8;  // rows a thread whose buckets and places stay in registers
  const int buckets = q.d.adapters + 1, tid = threadIdx.x;
  const bool held = q.m <= kHeld * kLoraPlanThreads;
  int* rows = lds;
  int* segs = lds + buckets;
  int bucket[kHeld], place[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int64_t row = (int64_t)i * kLoraPlanThreads + tid;
    bucket[i] = held && row < q.m ? lora_bucket(q, row) : -1;
  }
  for (int b = tid; b < buckets; b += kLoraPlanThreads) rows[b] = 0;
  __syncthreads();
  if (held) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (bucket[i] >= 0) place[i] = lora_count(rows, bucket[i]);
  } else {
    for (int64_t i = tid; i < q.m; i += kLoraPlanThreads) q.place[i] = lora_count(rows, lora_bucket(q, i));
  }
  __syncthreads();
  // first segments: exclusive sums over the buckets, consecutive ones a thread
  const int per = (buckets + kLoraPlanThreads - 1) / kLoraPlanThreads;
  int mine = 0, all;
  for (int b = tid * per; b < buckets && b < (tid + 1) * per; ++b) mine += lora_segments<S>(q, b, rows[b]);
  int at = block_sum<kLoraPlanThreads / 64>(mine, waves, all) - mine;
  for (int b = tid * per; b < buckets && b < (tid + 1) * per; ++b) {
    segs[b] = at;
    at += lora_segments<S>(q, b, rows[b]);
  }
  for (int z = all + tid; z < most; z += kLoraPlanThreads) q.segs[z] = LoraSeg{0, 0};
  __syncthreads();
  const auto put = [&](int64_t row, int b, int p) {
    const bool none = b == q.d.adapters;
    if (none && !q.copy) return;
    if ((uint32_t)p >= (uint32_t)rows[b]) return;  // as in lora_read
    const int z = segs[b] + p / S, left = rows[b] - p;
    q.order[(int64_t)z * S + p % S] = (int)row;
    if (p % S == 0) q.segs[z] = LoraSeg{none ? -1 : b, left < S ? left : S};
  };
  if (held) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (bucket[i] >= 0) put((int64_t)i * kLoraPlanThreads + tid, bucket[i], place[i]);
  } else {
    for (int64_t i = tid; i < q.m; i += kLoraPlanThreads) put(i, lora_bucket(q, i), q.place[i]);
  }
}

// Segment z from the workspace; false past the last.  What is read there is held to the
// rows and adapters that exist: a workspace that another stream writes meanwhile gives
// wrong results, but leads nowhere else.
template <int S>
__device__ __forceinline__ bool lora_read(const LoraArgs& q, int z, LoraTask& task) {
  const int tid = threadIdx.x;
  if (tid < S) {  // one wave: past count its first row
    const uint32_t at = (uint32_t)q.order[(int64_t)z * S + tid];
    const LoraSeg sg = q.segs[z];
    const int row = at < (uint32_t)q.m ? (int)at : 0;
    const int count = (uint32_t)sg.count <= (uint32_t)S ? sg.count : S;
    const int first = __builtin_amdgcn_readfirstlane(row);
    task.row[tid] = tid < count ? row : first;
    if (tid == 0) {
      task.adapter = (uint32_t)sg.adapter < (uint32_t)q.d.adapters ? sg.adapter : -1;
      task.count = count;
    }
  }
  __syncthreads();
  return task.count != 0;
}

// Segment z of up to 64 rows, found by every wave by itself, a row a lane.
template <int S>
__device__ __forceinline__ bool lora_ballots(const LoraArgs& q, int z, LoraTask& task) {
  const int lane = threadIdx.x & 63;
  const int bucket = lane < q.m ? lora_bucket(q, lane) : 0;
  uint64_t same = lane < q.m ? ~0ull : 0ull;  // lanes of this lane's adapter
  for (int bit = 0; (q.d.adapters >> bit) != 0; ++bit) {
    const uint64_t set = __ballot(bucket >> bit & 1);
    same &= bucket >> bit & 1 ? set : ~set;
  }
  same &= q.m == 64 ? ~0ull : (1ull << q.m) - 1;
  const uint64_t before = (1ull << lane) - 1;
  const int place = (int)__popcll(same & before);
  const bool leads = lane < q.m && place % S == 0 && (bucket != q.d.adapters || q.copy);
  const uint64_t leaders = __ballot(leads);
  const uint64_t mine = __ballot(leads && (int)__popcll(leaders & before) == z);
  if (mine == 0) return false;
  const int lead = __ffsll((unsigned long long)mine) - 1;
  const int b = __builtin_amdgcn_readlane(bucket, lead), first = __builtin_amdgcn_readlane(place, lead);
  const uint64_t members = __ballot(lane < q.m && bucket == b);
  const int left = (int)__popcll(members) - first, count = left < S ? left : S;
  if ((members >> lane & 1) && place >= first && place < first + S) task.row[place - first] = lane;
  if (lane >= count && lane < S) task.row[lane] = lead;
  if (lane == 0) {
    task.adapter = b == q.d.adapters ? -1 : b;
    task.count = count;
  }
  __syncthreads();
  return true;
}

// Segment z of up to kLoraPlanRows rows, found by the workgroup's W waves.  lds:
// [adapters + 1].
template <int S, int W>
__device__ __forceinline__ bool lora_search(const LoraArgs& q, int z, int* lds, LoraTask& task) {
  constexpr int kThreads = 64 * W, kEach = kLoraPlanRows / kThreads, kChunks = kLoraPlanRows / 64;
  static_assert(kChunks <= 64, "a chunk of rows a lane");
  __shared__ int waves[W], found[2], chunk[kChunks];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int buckets = q.d.adapters + 1;
  int bucket[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int row = i * kThreads + tid;
    bucket[i] = row < q.m ? lora_bucket(q, row) : -1;
  }
  for (int b = tid; b < buckets; b += kThreads) lds[b] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    if (bucket[i] >= 0) lora_count(lds, bucket[i]);
  __syncthreads();
  const int per = (buckets + kThreads - 1) / kThreads;
  int mine = 0, total;
  for (int b = tid * per; b < buckets && b < (tid + 1) * per; ++b) mine += lora_segments<S>(q, b, lds[b]);
  int at = block_sum<W>(mine, waves, total) - mine;
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
  // a row's place among its adapter's, the same in every workgroup: those of the chunks of
  // 64 rows before, and of the lanes before
  __syncthreads();
  const int b = found[0], first = found[1] * S;
  uint64_t same[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    same[i] = __ballot(bucket[i] == b);
    if (lane == 0) chunk[i * W + wave] = (int)__popcll(same[i]);
  }
  __syncthreads();
  const int here = lane < kChunks ? chunk[lane] : 0;
  int before = here;
  for (int d = 1; d < kChunks; d *= 2) {
    const int o = __shfl_up(before, d);
    before += lane >= d ? o : 0;
  }
  before -= here;
  const int left = lds[b] - first, count = left < S ? left : S;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int place =
        __builtin_amdgcn_readlane(before, i * W + wave) + (int)__popcll(same[i] & ((1ull << lane) - 1)) - first;
    if (bucket[i] != b) continue;
    if (place >= 0 && place < S) task.row[place] = i * kThreads + tid;
    if (place == 0)
      for (int p = count; p < S; ++p) task.row[p] = i * kThreads + tid;
  }
  if (tid == 0) {
    task.adapter = b == q.d.adapters ? -1 : b;
    task.count = count;
  }
  __syncthreads();
  return true;
}

// Segment z as the workgroup's task; false past the last.  Found here, it is left in the
// workspace for lora_expand by one of the segment's workgroups.  lds: [adapters + 1].
template <int S, int W>
__device__ __forceinline__ bool lora_task(const LoraArgs& q, int z, int* lds, LoraTask& task) {
  if (q.planned) return lora_read<S>(q, z, task);
  bool there;
  if (S < kLoraMaxSeg && q.m <= 64) there = lora_ballots<S>(q, z, task);  // long segments have 512 rows at least
  else there = lora_search<S, W>(q, z, lds, task);
  if (blockIdx.y == 0 && blockIdx.z == 0) {
    if (there && threadIdx.x < S) q.order[(int64_t)z * S + threadIdx.x] = task.row[threadIdx.x];
    if (threadIdx.x == 0) q.segs[z] = there ? LoraSeg{task.adapter, task.count} : LoraSeg{0, 0};
  }
  return there;
}

__device__ __forceinline__ int lora_rank(const LoraArgs& q, int adapter) {
  if (!q.d.ranks) return q.d.rank;
  const int r = q.d.ranks[adapter];
  return r < 0 ? 0 : r < q.d.rank ? r : q.d.rank;
}

// ---------------------------------------------------------------------------
// shrink
// ---------------------------------------------------------------------------
// 16 rows against 16 RT ranks (from 64 blockIdx.z on); a wave takes whole lines of 64
// k one after the other, lane (row or rank r, g) their places 16 g .. 16 g + 15.  64 rows
// of 5120 and 64 adapters of rank 16, 11 MB, in 6.6 us: start, loads' latency and end.
template <int RT>
__global__ __launch_bounds__(kLoraThreads) void lora_shrink(LoraArgs q) {
  constexpr int U = 4 / RT;  // lines whose loads go out together
  extern __shared__ int lds[];
  __shared__ float4_t part[4][RT][64];
  __shared__ LoraTask task;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int g = lane >> 4, r = lane & 15;
  const int split = blockIdx.y, r0 = 64 * blockIdx.z;
  const int64_t k = q.d.k;
  if (!lora_task<16, 4>(q, blockIdx.x, lds, task)) return;
  const int rank = task.adapter < 0 ? 0 : lora_rank(q, task.adapter);
  if (rank > r0) {
    const uint16_t* x = q.x + (int64_t)task.row[r] * q.ldx;
    const uint16_t* a[RT];
#pragma unroll
    for (int j = 0; j < RT; ++j) {  // past the rank: the last rank's, whose sums are not used
      const int of = r0 + 16 * j + r;
      a[j] = q.d.a + ((int64_t)task.adapter * q.d.rank + (of < rank ? of : rank - 1)) * k;
    }
    float4_t acc[RT];
#pragma unroll
    for (int j = 0; j < RT; ++j) acc[j] = float4_t{0.f, 0.f, 0.f, 0.f};
    const int lines = (int)((k + 63) / 64);
    const int first = (int)((int64_t)lines * split / q.splits), end = (int)((int64_t)lines * (split + 1) / q.splits);
    for (int u0 = first + wave; u0 < end; u0 += 4 * U) {
      u32x4_t xv[U][2], av[U][2][RT];
#pragma unroll
      for (int v = 0; v < U; ++v)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int u = u0 + 4 * v;
          const int64_t at = 64 * (int64_t)u + 16 * g + 8 * s;
          const int64_t from = u < end && at < k ? at : 0;
          xv[v][s] = load16(x + from);
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
            xv[v][s] = there ? xv[v][s] : zero;
#pragma unroll
            for (int j = 0; j < RT; ++j) av[v][s][j] = there ? av[v][s][j] : zero;
          }
      }
#pragma unroll
      for (int v = 0; v < U; ++v)
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int j = 0; j < RT; ++j)
            acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, xv[v][s]),
                                                            __builtin_bit_cast(f16x8_t, av[v][s][j]), acc[j], 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < RT; ++j) part[wave][j][lane] = acc[j];
  }
  __syncthreads();
  if (rank > r0) {
    for (int t = wave; t < RT; t += 4) {
      const int col = r0 + 16 * t + r;
      float4_t sum = part[0][t][lane];
#pragma unroll
      for (int w = 1; w < 4; ++w) sum += part[w][t][lane];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = 4 * g + j;
        if (i < task.count && col < q.rpad) q.h[((int64_t)split * q.m + task.row[i]) * q.rpad + col] = sum[j];
      }
    }
  }
}

// 64 rows against 64 ranks (from 64 blockIdx.z on), for rows that 32-bit offsets reach.
// 4096 x 5120 of rank 64 in 19 us: 84 MB to LDS, 42 of them from memory, behind 4 us of
// start and end.
__global__ __launch_bounds__(kTile64Waves * 64) void lora_shrink_tiled(LoraArgs q) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kTile64Lds];
  __shared__ LoraTask task;
  const int split = blockIdx.y, r0 = 64 * blockIdx.z;
  const uint32_t k = (uint32_t)q.d.k;
  if (!lora_task<64, kTile64Waves>(q, blockIdx.x, reinterpret_cast<int*>(lds), task)) return;
  const int rank = task.adapter < 0 ? 0 : lora_rank(q, task.adapter);
  if (rank > r0) {
    const int ranks = rank - r0 < 64 ? rank - r0 : 64;
    const uint16_t* a = q.d.a + ((int64_t)task.adapter * q.d.rank + r0) * q.d.k;
    const u32x4_t rsrc[2] = {buffer_words(reinterpret_cast<const uint8_t*>(q.x), ((q.m - 1) * q.ldx + k) * 2),
                             buffer_words(reinterpret_cast<const uint8_t*>(a), (uint64_t)ranks * k * 2)};
    uint32_t row[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t of = tile64_row(i);
      row[0][i] = (int)of < task.count ? (uint32_t)task.row[of] * (uint32_t)q.ldx * 2 : kPastEnd;
      row[1][i] = of * k * 2;  // past the ranks: past the buffer's end
    }
    const int stages = (int)((k + kTile64K - 1) / kTile64K);
    __syncthreads();  // the segment's search is done with lds
    const float* sums = tile64_sums(rsrc, row, k, (int)((int64_t)stages * split / q.splits),
                                    (int)((int64_t)stages * (split + 1) / q.splits), lds);
    const int col = threadIdx.x & 63;
    if (col < ranks)
      for (int i = threadIdx.x >> 6; i < task.count; i += kTile64Waves)
        q.h[((int64_t)split * q.m + task.row[i]) * q.rpad + r0 + col] = tile64_sum(sums, i, col);
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
#pragma clang loop unroll(disable)
  for (int i = 0; i < 16 && row0 + i < task.count; ++i) {
    float* at = out + i * kLoraOutStride + (threadIdx.x & 63);
    if (n >= q.d.n || __builtin_isfinite(*at)) continue;
    const float* h = q.h + (int64_t)task.row[row0 + i] * q.rpad;
    float sum = 0.f;
#pragma clang loop unroll(disable)
    for (int j = 0; j < rank; ++j) {
      float v = 0.f;
#pragma clang loop unroll(disable)
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

// Pieces in LDS: [hi, lo][row][32 chunks ranks], a row 16 bytes longer than that, so that
// the 16 rows of an operand lie in different banks.
__host__ __device__ constexpr int lora_piece_row(int chunks) { return 64 * chunks + 16; }

constexpr float kLoraLow = 1.f / 4096;  // of lo

// The task's h as pieces in LDS, and each row's factor of the sums, 2^-e.  (h is a sum of
// at most 2^20 products of fp16 and a multiple of 2^-48, so e lies between -37 and 62 and
// the sums, freed of it, well inside fp32: the adapter's scale, which may be any, is a
// factor of its own.)
template <int S, int CHUNKS>
__device__ __forceinline__ void lora_pieces(const LoraArgs& q, const LoraTask& task, int rank, uint8_t* lds,
                                            float* factor) {
  constexpr int kEach = kLoraThreads / S;  // threads of a row
  constexpr int kMost = (8 * CHUNKS + kEach - 1) / kEach;
  constexpr int kAtOnce = kMost == 1 ? 8 : 4;  // shares whose loads go out together
  constexpr int stride = lora_piece_row(CHUNKS);
  const int row = threadIdx.x / kEach, part = threadIdx.x % kEach;
  float4_t h[kMost];
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    const int at = 4 * (part + i * kEach);
    h[i] = float4_t{0.f, 0.f, 0.f, 0.f};
    if (row < task.count && at < q.rpad) {
      const float* p = q.h + (int64_t)task.row[row] * q.rpad + at;
      for (int s = 0; s < q.splits; s += kAtOnce) {
        float4_t v[kAtOnce];
#pragma unroll
        for (int o = 0; o < kAtOnce; ++o)
          v[o] = *reinterpret_cast<const float4_t*>(p + (int64_t)(s + o < q.splits ? s + o : s) * q.m * q.rpad);
#pragma unroll
        for (int o = 0; o < kAtOnce; ++o)
          if (s + o < q.splits) h[i] += v[o];
      }
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
  if (part == 0) factor[row] = __builtin_ldexpf(1.f, -e);
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    const int at = 4 * (part + i * kEach);
    if (at >= 32 * CHUNKS) continue;
    half4_t hi, lo;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float v = __builtin_ldexpf(h[i][j], e);
      hi[j] = (_Float16)v;
      lo[j] = (_Float16)(__builtin_isfinite(v) ? (v - (float)hi[j]) * (1 / kLoraLow) : 0.f);
    }
    *reinterpret_cast<half4_t*>(lds + row * stride + 2 * at) = hi;
    *reinterpret_cast<half4_t*>(lds + (S + row) * stride + 2 * at) = lo;
  }
}

// The sums of h from those of hi and of lo, made apart: a matrix instruction adds its
// products and its operand C as if no factor were subnormal, to about 24 bits below such a
// product's exponent, so that lo's sums, brought in by C, would be cut where weights are
// subnormal (at 2^-16 of the result for weights of 2^-22).
__device__ __forceinline__ void lora_join(float4_t (&hi)[4], const float4_t (&low)[4]) {
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int j = 0; j < 4; ++j) hi[t][j] = __builtin_fmaf(low[t][j], kLoraLow, hi[t][j]);
}

// How a wave's lanes take 16 rows of 64 columns of base and of y: 16 bytes a lane, of any
// alignment.  Where a tile has fewer than 64 columns, the last lanes' pieces end with it and
// overlap their neighbours', or begin in the tile before, and what lies there is not stored.
// TINY: rows of less than 16 bytes, by elements.
template <class T, bool TINY>
struct LoraIo {
  static constexpr int kElems = 16 / (int)sizeof(T);  // of a lane
  static constexpr int kLanes = 64 / kElems;          // of a row
  static constexpr int kRows = 64 / kLanes;           // of an instruction
  static constexpr int kInstr = 16 / kRows;           // of 16 rows
  typedef T vec __attribute__((ext_vector_type(kElems)));
  typedef vec any __attribute__((aligned(sizeof(T))));

  // A lane's first column in a tile with `left` columns, maybe negative; whether the lane
  // has any.
  static __device__ __forceinline__ int column(int lane, int left) {
    const int col = lane % kLanes * kElems;
    return TINY || col < left - kElems ? col : left - kElems;
  }
  static __device__ __forceinline__ bool takes(int lane, int left) { return lane % kLanes * kElems < left; }

  static __device__ __forceinline__ vec load(const T* p, int col, int left) {
    if constexpr (!TINY) return *reinterpret_cast<const any*>(p + col);
    vec v{};
#pragma unroll
    for (int j = 0; j < kElems; ++j)
      if (col + j < left) v[j] = p[col + j];
    return v;
  }
  // once: without a place in the caches.
  static __device__ __forceinline__ void store(T* p, int col, int left, vec v, bool once = false) {
    if (!TINY && __builtin_expect(col >= 0, 1)) {
      if (once) __builtin_nontemporal_store(v, reinterpret_cast<any*>(p + col));
      else *reinterpret_cast<any*>(p + col) = v;
      return;
    }
#pragma unroll
    for (int j = 0; j < kElems; ++j)
      if (col + j >= 0 && col + j < left) p[col + j] = v[j];
  }
  // base and the sums of a lane's columns, which a wave holds in LDS.
  static __device__ __forceinline__ vec add(const vec& from, bool with, const float* sums, int col, int left) {
    vec to;
    if (left >= 64) {
      const float* p = static_cast<const float*>(__builtin_assume_aligned(sums + col, 16));
#pragma unroll
      for (int j = 0; j < kElems; ++j) to[j] = (T)((with ? (float)from[j] : 0.f) + p[j]);
    } else {
#pragma unroll
      for (int j = 0; j < kElems; ++j) {
        const int at = col + j < 0 ? 0 : col + j < 64 ? col + j : 63;
        to[j] = (T)((with ? (float)from[j] : 0.f) + sums[at]);
      }
    }
    return to;
  }
};

// Up to 16 rows; a wave takes every fourth tile of 64 columns from its first on: matrix row
// i of a tile's product t is column 16 t + i, matrix columns are rows of the task.  The
// loads of a wave's next tile go out before it waits for this one's.
// CH: chunks of 32 ranks; 0: up to 16 ranks, where an operand's upper half of k holds
// another 16 columns, met by pieces that are zero in the other half.
// What bounds it is base, y and B: 64 rows 5120 -> 17408 of 64 adapters of rank 16, 40 MB
// in 12.5 to 13.6 us (3 TB/s) where a workgroup's start, 4 us, counts.
//
// Workgroups a CU:
__host__ __device__ constexpr int lora_expand_groups(int ch) { return ch == 0 ? 5 : ch == 1 ? 4 : ch == 2 ? 3 : 2; }

template <int CH, class T, bool TINY>
__global__ __launch_bounds__(kLoraThreads, lora_expand_groups(CH)) void lora_expand(LoraArgs q) {
  constexpr int S = 16;
  constexpr bool PAIR = CH == 0;
  constexpr int kChunks = PAIR ? 1 : CH;   // of the pieces
  constexpr int kB = PAIR ? 2 : 4 * CH;    // registers' worth of B
  using Io = LoraIo<T, TINY>;
  constexpr int kIo = Io::kInstr;
  constexpr int kRow = lora_piece_row(kChunks);
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ LoraTask task;
  __shared__ float factor[S];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int g = lane >> 4, r = lane & 15;
  const int sub = lane / Io::kLanes;  // a lane's row of an instruction's
  const int N = (int)q.d.n, R = q.d.rank;
  const int first_tile = blockIdx.y * 4 * q.tiles + wave;
  const T* base = static_cast<const T*>(q.base);
  T* y = static_cast<T*>(q.y);
  if (!lora_read<S>(q, blockIdx.x, task)) return;
  const int adapter = __builtin_amdgcn_readfirstlane(task.adapter);
  const int count = __builtin_amdgcn_readfirstlane(task.count);
  const int tiles = (N + 63) / 64;
  if (adapter < 0) {  // only where y is not base
    for (int tile = first_tile; tile < tiles && tile < first_tile + 4 * q.tiles; tile += 4) {
      const int n0 = 64 * tile, left = N - n0, col = Io::column(lane, left);
#pragma clang loop unroll(disable)
      for (int row = sub; row < count; row += Io::kRows)
        if (Io::takes(lane, left)) {
          const int64_t i = task.row[row];
          typename Io::vec v{};
          if (q.base) v = Io::load(base + i * q.ldb + n0, col, left);
          Io::store(y + i * q.ldy + n0, col, left, v);
        }
    }
    return;
  }
  const int rank = lora_rank(q, adapter);
  const float scale = q.d.scales ? q.d.scales[adapter] : 1.f;
  const uint16_t* b = q.d.b + (int64_t)adapter * N * R;
  // Of columns past n and ranks past the adapter's, others': neither has a say.  So it is
  // with tiles past the last, so that every load is made and none waited for early.
  const auto load_b = [&](int tile, f16x8_t* w) {
#pragma unroll
    for (int i = 0; i < kB; ++i) {
      const int n = 64 * tile + (PAIR ? 32 * i + 16 * (g >> 1) + r : 16 * (i & 3) + r);
      const int at = PAIR ? 8 * (g & 1) : 32 * (i >> 2) + 8 * g;
      w[i] = __builtin_bit_cast(f16x8_t, load16(b + (int64_t)(n < N ? n : N - 1) * R + (at < rank ? at : 0)));
    }
  };
  const T* from_where = q.base ? base : y;  // without a base what is loaded is dropped
  const int64_t from_ld = q.base ? q.ldb : q.ldy;
  const auto load_base = [&](int tile, typename Io::vec (&v)[kIo]) {
    const int n0 = 64 * (tile < tiles ? tile : tiles - 1), left = N - n0, col = Io::column(lane, left);
#pragma unroll
    for (int o = 0; o < kIo; ++o)
      v[o] = Io::load(from_where + task.row[Io::kRows * o + sub] * from_ld + n0, col, left);
  };
  struct Tile {
    f16x8_t w[kB];
    typename Io::vec from[kIo];
  } even, odd;
  const auto load = [&](int tile, Tile& to) {
    load_b(tile, to.w);
    load_base(tile, to.from);
  };
  load(first_tile, even);
  lora_pieces<S, kChunks>(q, task, rank, smem, factor);
  __syncthreads();
  float* out = reinterpret_cast<float*>(smem + 2 * S * kRow) + wave * (16 * kLoraOutStride);
  const auto take = [&](int tile, Tile& now) {
    if (rank < (PAIR ? 16 : 32 * CH)) {
#pragma unroll
      for (int i = 0; i < kB; ++i)
        now.w[i] = lora_keep(now.w[i], rank - (PAIR ? 8 * (g & 1) : 32 * (i >> 2) + 8 * g));
    }
    float4_t acc[4], low[4];  // sums of hi and of lo
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[t] = low[t] = float4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        float4_t* to = p ? low : acc;
        const f16x8_t h =
            *reinterpret_cast<const f16x8_t*>(smem + (p * S + r) * kRow + 64 * c + 16 * (PAIR ? g & 1 : g));
        if constexpr (PAIR) {
#pragma unroll
          for (int o = 0; o < 2; ++o) {
            const f16x8_t part = lora_keep(h, (g >> 1) == o ? 8 : 0);
#pragma unroll
            for (int v = 0; v < 2; ++v)
              to[2 * v + o] = __builtin_amdgcn_mfma_f32_16x16x32_f16(now.w[v], part, to[2 * v + o], 0, 0, 0);
          }
        } else {
#pragma unroll
          for (int t = 0; t < 4; ++t) to[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(now.w[4 * c + t], h, to[t], 0, 0, 0);
        }
      }
    lora_join(acc, low);
    const float f = factor[r];
    float odd = 0.f;  // NaN if a sum is not finite
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
      for (int j = 0; j < 4; ++j) odd = __builtin_fmaf(acc[t][j], 0.f, odd);
      *reinterpret_cast<float4_t*>(out + r * kLoraOutStride + 16 * t + 4 * g) = acc[t] * f * scale;
    }
    wave_lds_sync();
    if (__builtin_expect(__any(odd != 0.f), 0)) lora_mend(q, task, 0, 64 * tile, rank, scale, b, out);
    const int left = N - 64 * tile, col = Io::column(lane, left);
#pragma unroll
    for (int o = 0; o < kIo; ++o) {
      const int row = Io::kRows * o + sub;
      const typename Io::vec to = Io::add(now.from[o], q.base != nullptr, out + row * kLoraOutStride, col, left);
      if (row < count && Io::takes(lane, left)) Io::store(y + task.row[row] * q.ldy + 64 * tile, col, left, to);
    }
    wave_lds_sync();
  };
  const int end_tile = first_tile + 4 * q.tiles < tiles ? first_tile + 4 * q.tiles : tiles;
  int tile = first_tile;
  if (tile >= end_tile) return;
  if constexpr (CH <= 2) {
    for (; tile + 8 < end_tile; tile += 8) {
      load(tile + 4, odd);
      take(tile, even);
      load(tile + 8, even);
      take(tile + 4, odd);
    }
    if (tile + 4 < end_tile) {
      load(tile + 4, odd);
      take(tile, even);
      take(tile + 4, odd);
    } else {
      take(tile, even);
    }
  } else {  // no room for another tile's
    for (; tile + 4 < end_tile; tile += 4) {
      take(tile, even);
      load(tile + 4, even);
    }
    take(tile, even);
  }
}

// Up to 64 rows, 16 a wave, whose pieces stay in registers while tiles of 64 columns pass:
// a tile's B goes from memory straight to LDS, sent two tiles ahead, and serves the four
// waves.  (Loaded by the lanes that multiply it, 16 rows an instruction, it comes at 16
// bytes a clock and CU, which for 64 ranks is as long as base and y take.)  4096 rows, n
// 17408, rank 64, four adapters, 294 MB in 69 to 71 us (4.1 to 4.3 TB/s).  Bound by base
// and y and by waits: the compiler, which does not count the copies, waits for all vector
// memory at the top of every second tile, and before the stores for all but the newest
// two or three accesses, so that B and y are waited for once in two tiles at least.
//
// LDS: a tile holds a row of 4 CH 16-byte pieces for each column; piece c of row n lies at
// place c ^ turn(n), so that sixteen rows' pieces c cover all 64 banks.
constexpr int kLoraRing = 3;

template <int CH>
__device__ __forceinline__ uint32_t lora_turn(uint32_t n) {
  return CH == 1 ? n >> 2 & 3 : CH == 2 ? n >> 1 & 7 : n & 15;
}

template <int CH, class T>
__global__ __launch_bounds__(kLoraThreads) void lora_expand_long(LoraArgs q) {
  using Io = LoraIo<T, false>;
  constexpr int S = 64, kIo = Io::kInstr;
  constexpr int kRow = lora_piece_row(CH);
  constexpr int kPieces = 4 * CH, kTile = 64 * 16 * kPieces;  // of a row; bytes of a tile
  constexpr int kCopies = kTile / 1024 / 4;                   // a wave's
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  __shared__ LoraTask task;
  __shared__ float factor[S];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int g = lane >> 4, r = lane & 15;
  const int sub = lane / Io::kLanes;  // a lane's row of an instruction's
  const int N = (int)q.d.n, R = q.d.rank;
  const int first_tile = blockIdx.y * q.tiles, tiles = (N + 63) / 64;
  const int end_tile = first_tile + q.tiles < tiles ? first_tile + q.tiles : tiles;
  const T* base = static_cast<const T*>(q.base);
  T* y = static_cast<T*>(q.y);
  if (!lora_read<S>(q, blockIdx.x, task)) return;
  const int adapter = __builtin_amdgcn_readfirstlane(task.adapter);
  const int count = __builtin_amdgcn_readfirstlane(task.count);
  const int i0 = 16 * wave;
  if (adapter < 0) {  // only where y is not base
    for (int tile = first_tile; tile < end_tile; ++tile) {
      const int n0 = 64 * tile, left = N - n0, col = Io::column(lane, left);
#pragma clang loop unroll(disable)
      for (int row = i0 + sub; row < count && row < i0 + 16; row += Io::kRows)
        if (Io::takes(lane, left)) {
          const int64_t i = task.row[row];
          typename Io::vec v{};
          if (q.base) v = Io::load(base + i * q.ldb + n0, col, left);
          Io::store(y + i * q.ldy + n0, col, left, v);
        }
    }
    return;
  }
  const int rank = lora_rank(q, adapter);
  const float scale = q.d.scales ? q.d.scales[adapter] : 1.f;
  const uint16_t* b = q.d.b + (int64_t)adapter * N * R;
  lora_pieces<S, CH>(q, task, rank, smem, factor);
  __syncthreads();
  f16x8_t h[CH][2];
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int p = 0; p < 2; ++p)
      h[c][p] = *reinterpret_cast<const f16x8_t*>(smem + (p * S + i0 + r) * kRow + 64 * c + 16 * g);
  __syncthreads();
  const float f = factor[i0 + r];
  float* out = reinterpret_cast<float*>(smem + kLoraRing * kTile) + wave * (16 * kLoraOutStride);
  const uint32_t ring = (uint32_t)(uintptr_t)(lds_u8*)smem;
  const u32x4_t rsrc = buffer_words(reinterpret_cast<const uint8_t*>(b), (uint64_t)N * R * 2);
  uint32_t off[kCopies];  // a lane's piece of a copy: ranks past the adapter's are zeros
#pragma unroll
  for (int i = 0; i < kCopies; ++i) {
    const uint32_t at = 64 * (kCopies * wave + i) + lane, n = at / kPieces;
    const uint32_t piece = (at % kPieces) ^ lora_turn<CH>(n);
    off[i] = 8 * piece < (uint32_t)rank ? n * R * 2 + 16 * piece : kPastEnd;
  }
  const auto fetch = [&](int tile, int place) {  // past the last tile: zeros
#pragma unroll
    for (int i = 0; i < kCopies; ++i)
      lds_copy16(rsrc, ring + (uint32_t)place * kTile + (uint32_t)(kCopies * wave + i) * 1024,
                 tile < end_tile ? off[i] : kPastEnd, (uint32_t)(tile < end_tile ? tile : 0) * (128u * R));
  };
  // Without a base what is loaded is dropped.  Of rows past count and columns past n,
  // others'.
  const T* from_row[kIo];
  T* to_row[kIo];
#pragma unroll
  for (int o = 0; o < kIo; ++o) {
    const int64_t i = task.row[i0 + Io::kRows * o + sub];
    to_row[o] = y + i * q.ldy;
    from_row[o] = q.base ? base + i * q.ldb : to_row[o];
  }
  const auto load_base = [&](int tile, typename Io::vec (&v)[kIo]) {
    const int n0 = 64 * (tile < end_tile ? tile : end_tile - 1), left = N - n0, col = Io::column(lane, left);
#pragma unroll
    for (int o = 0; o < kIo; ++o) v[o] = Io::load(from_row[o] + n0, col, left);
  };
  int place = 0;  // of the ring
  const auto step = [&](int tile, typename Io::vec (&from)[kIo], typename Io::vec (&next)[kIo]) {
    // The tile's copies, made two steps ago, have landed here when at most those of the
    // next tile, and the base loaded with either, are open; behind the barrier they have
    // everywhere, and the tile before has been read.
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kCopies + 2 * kIo) : "memory");
    fetch(tile + 2, (place + 2) % kLoraRing);
    load_base(tile + 1, next);
    float4_t acc[4], low[4];  // sums of hi and of lo
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[t] = low[t] = float4_t{0.f, 0.f, 0.f, 0.f};
    const uint32_t at = ring + (uint32_t)place * kTile;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      f16x8_t w[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint32_t n = 16 * t + r;
        w[t] = __builtin_bit_cast(f16x8_t, lds_read16(at + 16 * (n * kPieces + ((4 * c + g) ^ lora_turn<CH>(n)))));
      }
      if (rank % 8) {
#pragma unroll
        for (int t = 0; t < 4; ++t) w[t] = lora_keep(w[t], rank - 32 * c - 8 * g);
      }
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          float4_t* to = p ? low : acc;
          to[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[t], h[c][p], to[t], 0, 0, 0);
        }
    }
    lora_join(acc, low);
    place = place == kLoraRing - 1 ? 0 : place + 1;
    if (i0 >= count) return;
    float odd = 0.f;  // NaN if a sum is not finite
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
      for (int j = 0; j < 4; ++j) odd = __builtin_fmaf(acc[t][j], 0.f, odd);
      *reinterpret_cast<float4_t*>(out + r * kLoraOutStride + 16 * t + 4 * g) = acc[t] * f * scale;
    }
    wave_lds_sync();
    if (__builtin_expect(__any(odd != 0.f), 0)) lora_mend(q, task, i0, 64 * tile, rank, scale, b, out);
    const int left = N - 64 * tile, col = Io::column(lane, left);
#pragma unroll
    for (int o = 0; o < kIo; ++o) {
      const int row = Io::kRows * o + sub;
      const typename Io::vec to = Io::add(from[o], q.base != nullptr, out + row * kLoraOutStride, col, left);
      if (i0 + row < count && Io::takes(lane, left)) Io::store(to_row[o] + 64 * tile, col, left, to, true);
    }
    wave_lds_sync();
  };
  typename Io::vec even[kIo], odd[kIo];
  fetch(first_tile, 0);
  fetch(first_tile + 1, 1);
  load_base(first_tile, even);
  // the first tile's copies have nothing else behind them
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kCopies + kIo) : "memory");
  for (int tile = first_tile; tile < end_tile; tile += 2) {
    step(tile, even, odd);
    if (tile + 1 < end_tile) step(tile + 1, odd, even);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // copies to LDS
}

// ---------------------------------------------------------------------------
// few rows
// ---------------------------------------------------------------------------
// A workgroup takes a row (blockIdx.y) and 8192 / RJ columns: it makes the row's whole h
// itself (A from L2, which costs less than a launch) and then its columns, RJ / 8 threads
// a column.  RJ: a power of two >= rank.  A wave takes 8 ranks of every 512 k from its
// place on.  One row 5120 -> 17408 of rank 16, 0.8 MB, in 6.6 us: latency, first of A and
// x, then of the sums' way through LDS.
constexpr int kLoraFewThreads = 1024;

template <int RJ, class T>
__global__ __launch_bounds__(kLoraFewThreads) void lora_few(LoraArgs q) {
  constexpr int NW = kLoraFewThreads / 64, G = RJ / 8, kCols = kLoraFewThreads / G;
  __shared__ float part[NW][8];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int64_t row = blockIdx.y, k = q.d.k;
  const int bucket = __builtin_amdgcn_readfirstlane(lora_bucket(q, row));
  const bool none = bucket == q.d.adapters;
  if (none && !q.copy) return;
  const int64_t n = (int64_t)blockIdx.x * kCols + threadIdx.x / G;
  const int j0 = 8 * (threadIdx.x % G);
  const bool writes = j0 == 0 && n < q.d.n;
  T from = (T)0;
  if (writes && q.base) from = static_cast<const T*>(q.base)[row * q.ldb + n];
  const int rank = none ? 0 : lora_rank(q, bucket);
  const float scale = none ? 0.f : q.d.scales ? q.d.scales[bucket] : 1.f;
  f16x8_t w = {0, 0, 0, 0, 0, 0, 0, 0};
  if (n < q.d.n && j0 < rank)
    w = __builtin_bit_cast(f16x8_t, load16(q.d.b + ((int64_t)bucket * q.d.n + n) * q.d.rank + j0));
  float acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = 0.f;
  const int a0 = 8 * (wave % G);  // this wave's ranks
  if (a0 < rank) {
    const uint16_t* x = q.x + row * q.ldx;
    const uint16_t* a = q.d.a + ((int64_t)bucket * q.d.rank + a0) * k;
    for (int64_t at = 512 * (wave / G) + 8 * lane; at < k; at += 512 * (NW / G)) {
      const f16x8_t xv = __builtin_bit_cast(f16x8_t, load16(x + at));
      f16x8_t av[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) av[j] = __builtin_bit_cast(f16x8_t, load16(a + (a0 + j < rank ? j : 0) * k + at));
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[j] = __builtin_fmaf((float)av[j][i], (float)xv[i], acc[j]);
    }
    // over the lanes: halves exchange what the other half sums up, so that eight sums take
    // 4 + 2 + 1 + 3 exchanges; lane 8 j ends with sum j
#pragma unroll
    for (int d = 4; d >= 1; d /= 2)
#pragma unroll
      for (int j = 0; j < d; ++j) {
        const bool upper = lane & (8 * d);
        const float mine = upper ? acc[j + d] : acc[j], other = upper ? acc[j] : acc[j + d];
        acc[j] = mine + __shfl_xor(other, 8 * d);
      }
#pragma unroll
    for (int d = 4; d >= 1; d /= 2) acc[0] += __shfl_xor(acc[0], d);
  }
  if ((lane & 7) == 0) part[wave][lane >> 3] = acc[0];
  __syncthreads();
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (j0 + i < rank) {
      float h = 0.f;
#pragma unroll
      for (int o = 0; o < NW / G; ++o) h += part[o * G + threadIdx.x % G][i];
      sum = __builtin_fmaf(h, (float)w[i], sum);
    }
  }
#pragma unroll
  for (int d = 1; d < G; d *= 2) sum += __shfl_xor(sum, d);
  if (!writes) return;
  T* to = static_cast<T*>(q.y) + row * q.ldy + n;
  *to = !q.base ? (T)(none ? 0.f : scale * sum) : none ? from : (T)((float)from + scale * sum);
}

namespace {

constexpr int kLoraFewRank = 64;

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

int lora_few_rank(int rank) { return rank <= 8 ? 8 : rank <= 16 ? 16 : rank <= 32 ? 32 : 64; }

// One launch while a round of workgroups holds it and the A that each reads is short (us,
// one launch / two, 16 adapters): 5120 -> 17408 of rank 16, 1 row 6.1 / 8.5, 4 6.4 / 8.6, 8
// (272 workgroups) 11.4 / 9.2; of rank 32, 1 row 6.9 / 8.5; of rank 64 (655 KB) 9.7 / 9.9;
// 17408 -> 5120 of rank 16 (557 KB), 8 rows 11.9 / 9.4; 2048 -> 512, 64 rows 5.2 / 9.4.
bool lora_is_few(const LoraDesc& d, int64_t m) {
  if (d.rank > kLoraFewRank || m > 256) return false;
  const int64_t cols = kLoraFewThreads * 8 / lora_few_rank(d.rank);
  const int64_t groups = m * ((d.n + cols - 1) / cols), each = d.rank * d.k * 2;
  return groups <= 256 && each <= 384 << 10 && groups * each <= 64 << 20;
}

// 64 rows a segment where adapters have more than 16 each on average, enough of them for
// the chip and 32-bit offsets for the copies to LDS.  Segments of 64 / of 16 rows, us,
// 5120 -> 17408 of rank 64: 256 rows of one adapter 23.4 / 20.4, 512 27.1 / 29.8, 1024 rows
// of 16 adapters 45 / 59, of 63 83 / 87, of 128 134 / 118, 4096 rows of 64 129 / 193, of 200
// 271 / 246; 5120 -> 5120 of rank 16: 512 rows of 8 19.1 / 17.4, 4096 of 64 47 / 53.
bool lora_long(const LoraDesc& d, int64_t m, int64_t ldx) {
  return m >= 512 && d.n >= 8 && m > 16 * (int64_t)d.adapters && m * ldx < (int64_t)1 << 31;
}

int64_t lora_most_segs(const LoraDesc& d, int64_t m, bool longer) {
  const int s = longer ? 64 : 16;
  const int64_t most = m / s + d.adapters + 1;  // a bucket's last may be short, that of none too
  return most < m ? most : m;
}

// Segments of 64 rows that may be expected: of each adapter the last is half full.
int64_t lora_long_segs(const LoraDesc& d, int64_t m) { return (m + 63) / 64 + d.adapters / 2; }

// Shares of k: workgroups for the chip against what each share costs lora_expand, which
// adds them, the more the longer h is.  Over 432 shapes of 8 to 2048 rows, rank 8 to 256,
// k 2048 to 17408 and 1 to 64 adapters, 2.9 % from each shape's best on average and 19 % at
// most (us, shares in brackets, 5120 -> 5120: 333 rows of 8 adapters of rank 16 15.3 (4),
// 13.9 (8), 16.6 (16); 64 rows of 8 adapters of rank 256 27 (2), 22 (4), 28 (16); 17408 ->
// 5120 of one adapter, 600 rows of rank 8 26 (4), 21 (8), of rank 256 45 (4), 56 (8)).
int lora_splits(const LoraDesc& d, int64_t m, bool longer) {
  const int64_t ranks = (d.rank + 63) / 64;
  int64_t s, most, cap;
  if (longer) {
    // a workgroup fills a CU, and a second round costs more than longer shares (4096 x 5120
    // of four adapters of rank 64: 19 us in 3 shares, 22 in 2, 23 in 7)
    s = 256 / (lora_long_segs(d, m) * ranks);
    most = ranks == 1 ? (d.k < 8192 ? 4 : d.k / 2048) : (d.k < 8192 ? 2 : d.k / 4096);
    cap = ranks == 1 ? 8 : 4;
  } else {
    s = (ranks == 1 ? 1024 : 2048) / (lora_most_segs(d, m, false) * ranks);
    most = ranks == 1 ? (d.k + 639) / 640 : (d.k + 511) / 512;
    cap = ranks == 1 ? 16 : 8;
  }
  most = most < cap ? most : cap;
  return (int)(s < 1 ? 1 : s < most ? s : most);
}

struct LoraLayout {
  size_t segs, order, place, h, total;
};
LoraLayout lora_layout(const LoraDesc& d, int64_t m, bool longer) {
  LoraLayout L;
  size_t off = 0;
  const bool planned = m > kLoraPlanRows;
  const size_t most = (size_t)lora_most_segs(d, m, longer);
  L.segs = off;
  off += align256(most * sizeof(LoraSeg));
  L.order = off;
  off += align256(most * (longer ? 64 : 16) * 4);
  L.place = off;
  off += align256(planned ? (size_t)m * 4 : 0);
  L.h = off;
  off += align256((size_t)lora_splits(d, m, longer) * m * ((d.rank + 15) / 16 * 16) * 4);
  L.total = off;
  return L;
}

template <class T>
void launch_few(const LoraArgs& q, hipStream_t s) {
  const int rj = lora_few_rank(q.d.rank);
  const int cols = kLoraFewThreads * 8 / rj;
  const dim3 grid((uint32_t)((q.d.n + cols - 1) / cols), (uint32_t)q.m), block(kLoraFewThreads);
  if (rj == 8) hipLaunchKernelGGL((lora_few<8, T>), grid, block, 0, s, q);
  else if (rj == 16) hipLaunchKernelGGL((lora_few<16, T>), grid, block, 0, s, q);
  else if (rj == 32) hipLaunchKernelGGL((lora_few<32, T>), grid, block, 0, s, q);
  else hipLaunchKernelGGL((lora_few<64, T>), grid, block, 0, s, q);
}

template <int CH, bool TINY = false>
void launch_expand(LoraArgs q, bool f32, hipStream_t s) {
  const size_t lds = 2 * 16 * lora_piece_row(CH ? CH : 1) + 4 * 16 * kLoraOutStride * 4;
  const int64_t segs = lora_most_segs(q.d, q.m, false), tiles = (q.d.n + 63) / 64;
  // one round of workgroups: each begins with its segment and its h, 4 us
  const int64_t slots = 256 * lora_expand_groups(CH);
  q.tiles = 1;
  while (segs * ((tiles + 4 * q.tiles - 1) / (4 * q.tiles)) > slots && 4 * q.tiles < tiles && q.tiles < 16) ++q.tiles;
  const dim3 grid((uint32_t)segs, (uint32_t)((tiles + 4 * q.tiles - 1) / (4 * q.tiles)));
  if (f32) hipLaunchKernelGGL((lora_expand<CH, float, TINY>), grid, dim3(kLoraThreads), lds, s, q);
  else hipLaunchKernelGGL((lora_expand<CH, _Float16, TINY>), grid, dim3(kLoraThreads), lds, s, q);
}

template <int CH>
void launch_expand_long(const LoraArgs& q, bool f32, dim3 grid, hipStream_t s) {
  size_t lds = kLoraRing * 4096 * CH + 4 * 16 * kLoraOutStride * 4;
  if (const size_t pieces = 2 * 64 * lora_piece_row(CH); lds < pieces) lds = pieces;
  if (f32) hipLaunchKernelGGL((lora_expand_long<CH, float>), grid, dim3(kLoraThreads), lds, s, q);
  else hipLaunchKernelGGL((lora_expand_long<CH, _Float16>), grid, dim3(kLoraThreads), lds, s, q);
}

void launch_segments(LoraArgs q, bool longer, bool f32, hipStream_t s) {
  const uint32_t gx = (uint32_t)lora_most_segs(q.d, q.m, longer);
  const size_t plan = (size_t)(q.d.adapters + 1) * 4;
  const dim3 shrink(gx, (uint32_t)q.splits, (uint32_t)((q.d.rank + 63) / 64)), block(kLoraThreads);
  if (longer) hipLaunchKernelGGL(lora_shrink_tiled, shrink, dim3(kTile64Waves * 64), 0, s, q);
  else if (q.d.rank <= 16) hipLaunchKernelGGL((lora_shrink<1>), shrink, block, plan, s, q);
  else if (q.d.rank <= 32) hipLaunchKernelGGL((lora_shrink<2>), shrink, block, plan, s, q);
  else hipLaunchKernelGGL((lora_shrink<4>), shrink, block, plan, s, q);
  const int64_t tiles = (q.d.n + 63) / 64;
  if (longer) {
    // a round of workgroups, as many as LDS holds: shorter ones begin, with their h, too
    // often (4096 rows 5120 -> 17408 of rank 64 of four adapters 93 us, of half as many
    // tiles a workgroup 97, of a quarter 108)
    const int64_t slots = 256 * (q.d.rank <= 32 ? 5 : q.d.rank <= 64 ? 3 : q.d.rank <= 128 ? 2 : 1);
    const int64_t segs = lora_long_segs(q.d, q.m), groups = slots > segs ? slots / segs : 1;
    const int64_t each = (tiles + groups - 1) / groups;
    q.tiles = (int)(each < 4 ? 4 : each);
    const dim3 grid(gx, (uint32_t)((tiles + q.tiles - 1) / q.tiles));
    if (q.d.rank <= 32) launch_expand_long<1>(q, f32, grid, s);
    else if (q.d.rank <= 64) launch_expand_long<2>(q, f32, grid, s);
    else if (q.d.rank <= 128) launch_expand_long<4>(q, f32, grid, s);
    else launch_expand_long<8>(q, f32, grid, s);
    return;
  }
  if (q.d.n < (f32 ? 4 : 8)) launch_expand<8, true>(q, f32, s);
  else if (q.d.rank <= 16) launch_expand<0>(q, f32, s);
  else if (q.d.rank <= 32) launch_expand<1>(q, f32, s);
  else if (q.d.rank <= 64) launch_expand<2>(q, f32, s);
  else if (q.d.rank <= 128) launch_expand<4>(q, f32, s);
  else launch_expand<8>(q, f32, s);
}

}  // namespace

// Of any ldx.
size_t lora_workspace(const LoraDesc& d, int64_t m) {
  if (lora_is_few(d, m)) return 0;
  const size_t a = lora_layout(d, m, false).total, b = lora_layout(d, m, lora_long(d, m, d.k)).total;
  return a > b ? a : b;
}

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
  const bool longer = lora_long(d, m, ldx);
  const LoraLayout L = lora_layout(d, m, longer);
  unsigned char* w = static_cast<unsigned char*>(ws);
  q.splits = lora_splits(d, m, longer);
  q.rpad = (d.rank + 15) / 16 * 16;
  q.h = reinterpret_cast<float*>(w + L.h);
  q.segs = reinterpret_cast<LoraSeg*>(w + L.segs);
  q.order = reinterpret_cast<int*>(w + L.order);
  q.place = reinterpret_cast<int*>(w + L.place);
  q.planned = m > kLoraPlanRows;
  if (q.planned) {
    const size_t lds = 2 * (size_t)(d.adapters + 1) * 4;
    const int most = (int)lora_most_segs(d, m, longer);
    if (longer) hipLaunchKernelGGL((lora_plan<64>), dim3(1), dim3(kLoraPlanThreads), lds, s, q, most);
    else hipLaunchKernelGGL((lora_plan<16>), dim3(1), dim3(kLoraPlanThreads), lds, s, q, most);
  }
  launch_segments(q, longer, f32, s);
  return hipGetLastError();
}

}  // namespace exl3
