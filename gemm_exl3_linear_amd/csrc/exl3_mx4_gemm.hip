// exl3_mx4_matmul for large products: tiles through LDS on the scaled 4-bit
// matrix cores, y = sum over blocks of 2^(sa + sb - 254) sum of a b.
//
// A workgroup computes a TM x TN tile over all of k, or over its share of k.  A
// stage is 256 k: one 128-byte line of codes of every row of both operands (half
// lines, for stages of 128 k, copied 1.6 times as long) and their scale bytes,
// copied straight from memory to LDS while the other stage is multiplied.  The
// instruction applies the scales itself, so a wave only reads and multiplies:
// 128 x 64 a wave of 256 x 256 is as large as its registers allow.
//
// What bounds it: 4096 rows 5120 -> 17408, 181 to 198 us from card to card, 4.0 to 3.7
// PFLOP/s.  Where it takes 184 (192 over 1.6 GB of tensors), a trace of the launches,
// each by itself with its start and end, gives 175 for four rounds of 256 x 256 tiles,
// with the matrix cores busy nearly half of the time, 19 for the small tiles of the rest
// and 5 for the scales.  A loop of these instructions from
// registers alone runs at 7.0 to 7.2 PFLOP/s with random codes and at 9.5 with zeros:
// the clock falls with what the matrix cores switch, and this kernel, too, is a fifth
// faster a step on zeros (1.49 against 1.83 us).
// Without the copies a step takes 1.52 us, with all tiles the same (nothing but L2
// hits) still 1.83.  Reading operands one fragment ahead of the products across
// the barrier (4 % slower), and copies through registers (9 % slower), did not pay.
// A round's output, 128 KB a CU, is not overlapped.
#include "exl3_internal.hpp"
#include "exl3_mx4_lds.hpp"
#include "exl3_mx4_linear.hpp"

namespace exl3 {

constexpr int kStageK = 256;
constexpr int kStageLine = kStageK / 2;             // bytes of codes of a row
constexpr int kStageBlocks = kStageK / kMx4Block;   // scale bytes of a row
constexpr int kStages = 2;
constexpr int kScaleTile = 64;                      // rows of one staged group of scales (256 bytes)

// LDS place of 16-byte chunk c of a row's line: a wave's 16-byte reads take
// one chunk of sixteen rows for every lane group, and the lanes that are served
// together then fall on different banks.
__device__ __forceinline__ int stage_place(int row, int c) { return c ^ (row & 7); }

struct Mx4GemmArgs {
  const uint8_t* a;         // codes [m][k/2]
  const uint8_t* b;         // codes [n][k/2]
  const uint8_t* a_scales;  // staged, see mx4_stage_scales
  const uint8_t* b_scales;
  uint32_t a_step, b_step;  // bytes of one step of staged scales
  const uint16_t* bias;
  void* y;
  int64_t ldy;
  int64_t m, n;
  int kb;
  int steps;
  int y_f32;
  int wide;                 // 16-byte stores of y fit its alignment
  uint32_t tiles_m, tiles_n;
  int splits;               // workgroups that share a tile's steps: y is [split][m][n] then
};

// Scales as the matrix instructions take them: per step and group of 64 rows
// two dwords for each lane (r = l % 16, g = l / 16); byte j of dword h is the
// scale of block 4 h + g of row 16 j + r, so one LDS read serves eight
// operands.  127 past a row's end and past the last row.
struct StageScales {
  const uint8_t* s;
  uint32_t* out;
  int64_t rows;
  uint32_t groups;  // of 64 rows
};
__global__ __launch_bounds__(256) void mx4_stage_scales(StageScales a, StageScales b, int kb, int steps) {
  const bool second = blockIdx.x >= a.groups;
  const StageScales& q = second ? b : a;
  const uint32_t group = blockIdx.x - (second ? a.groups : 0);
  const int r = threadIdx.x & 15, half = blockIdx.y * 16 + (threadIdx.x >> 4);  // 128 k
  if (half >= steps * 2) return;
  const int left = kb - half * 4;
  uint32_t v[4];  // blocks of row j
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t row = (int64_t)group * kScaleTile + 16 * j + r;
    v[j] = 0x7F7F7F7Fu;
    if (row < q.rows) {
      const uint8_t* p = q.s + row * kb + half * 4;
      if (left >= 4) {
        __builtin_memcpy(&v[j], p, 4);
      } else {
        v[j] = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) v[j] |= (c < left ? (uint32_t)p[c] : kMx4One) << (8 * c);
      }
    }
  }
  uint32_t* o = q.out + ((int64_t)(half >> 1) * q.groups + group) * 128 + 2 * r + (half & 1);
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) w |= ((v[j] >> (8 * g)) & 0xFFu) << (8 * j);
    o[32 * g] = w;
  }
}

// acc += b a^T with byte JB, JA of the scale dwords.
template <int JB, int JA>
__device__ __forceinline__ float4_t mfma_mx4_sel(u32x4_t b, uint32_t sb, u32x4_t a, uint32_t sa, float4_t c) {
  const i32x8_t B = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  const i32x8_t A = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(B, A, c, kMfmaFp4, kMfmaFp4, JB, (int)sb, JA, (int)sa);
}

template <int I, int N, class F>
__device__ __forceinline__ void unrolled(F&& f) {
  if constexpr (I < N) {
    f(PowC<I>{});
    unrolled<I + 1, N>(f);
  }
}

// STREAM: y is whole lines past what the caches keep (launch_mx4_gemm).
template <int TM, int TN, int WM, int WN, bool STREAM>
__global__ __launch_bounds__(WM* WN * 64, 2) void mx4_gemm_kernel(Mx4GemmArgs q) {
  constexpr int NW = WM * WN;
  constexpr int MI = TM / WM / 16, NI = TN / WN / 16;  // 16 x 16 tiles of a wave
  static_assert(MI % 4 == 0 && NI % 4 == 0, "a scale dword serves four operands");
  constexpr uint32_t kA = 0, kB = kA + TM * kStageLine, kSA = kB + TN * kStageLine, kSB = kSA + TM * kStageBlocks,
                     kBytes = kSB + TN * kStageBlocks;
  constexpr int CA = TM / 8 / NW, CB = TN / 8 / NW;  // code copies of a wave and stage, 8 rows each
  static_assert(CA * NW * 8 == TM && CB * NW * 8 == TN && (TM + TN) / 64 == NW, "copies are even");
  constexpr int kOutBytes = TM / WM * 128;             // a wave's region when it writes y
  static_assert(kOutBytes * NW <= kBytes * kStages, "output regions fit");
  __shared__ __align__(128) uint8_t smem[kStages * kBytes];
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_u8*)smem;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int g = lane >> 4, r = lane & 15;
  // tiles in XCD order: workgroups b, b + 8, ... share an XCD and its L2
  const uint32_t total = gridDim.x;
  const uint32_t x = blockIdx.x & 7, per = total >> 3, rest = total & 7;
  const uint32_t at = x * per + (x < rest ? x : rest) + (blockIdx.x >> 3);
  const uint32_t split = at / (q.tiles_m * q.tiles_n), tile = at - split * (q.tiles_m * q.tiles_n);
  const int begin = (int)((uint32_t)q.steps * split / (uint32_t)q.splits);
  const int end = (int)((uint32_t)q.steps * (split + 1) / (uint32_t)q.splits);
  constexpr uint32_t kGroup = 8;  // row tiles walked together
  const uint32_t group = tile / (kGroup * q.tiles_n);
  const uint32_t gm = q.tiles_m - group * kGroup < kGroup ? q.tiles_m - group * kGroup : kGroup;
  const uint32_t in = tile - group * kGroup * q.tiles_n;
  const uint32_t tn = in / gm, tm = group * kGroup + (in - tn * gm);
  const int64_t m0 = (int64_t)tm * TM, n0 = (int64_t)tn * TN;
  const int wm = wave % WM, wn = wave / WM;
  const uint32_t pitch = (uint32_t)q.kb * 16;

  // rows past the end read as zeros, with staged scales of 1
  auto buffer = [&](const uint8_t* p, int64_t row0, int64_t rows, int most) {
    const int64_t left = rows - row0 < most ? rows - row0 : most;
    return buffer_words(p + row0 * pitch, (uint64_t)left * pitch);
  };
  const u32x4_t ra = buffer(q.a, m0, q.m, TM), rb = buffer(q.b, n0, q.n, TN);
  const u32x4_t rsa = buffer_words(q.a_scales, (uint64_t)q.steps * q.a_step);
  const u32x4_t rsb = buffer_words(q.b_scales, (uint64_t)q.steps * q.b_step);
  const int lane_chunk = stage_place(lane >> 3, lane & 7);
  const uint32_t lane_off = pitch * (lane >> 3) + 16 * lane_chunk;
  const bool scales_of_b = wave >= TM / 64;
  const u32x4_t rss = scales_of_b ? rsb : rsa;
  const uint32_t s_step = scales_of_b ? q.b_step : q.a_step;
  const uint32_t s_off = scales_of_b ? (uint32_t)(n0 * kStageBlocks) + (wave - TM / 64) * 512
                                     : (uint32_t)(m0 * kStageBlocks) + wave * 512;
  auto copy = [&](uint32_t stage, int step) {
    // chunks past a row's end, and steps past the last, read past the buffer: zeros
    const uint32_t at_lane = step < end && step * kStageBlocks + lane_chunk < q.kb ? lane_off : kPastEnd;
    const uint32_t k_off = (uint32_t)step * kStageLine;
#pragma unroll
    for (int c = 0; c < CA; ++c)
      lds_copy16(ra, stage + kA + (wave * CA + c) * 1024, at_lane, pitch * 8 * (wave * CA + c) + k_off);
#pragma unroll
    for (int c = 0; c < CB; ++c)
      lds_copy16(rb, stage + kB + (wave * CB + c) * 1024, at_lane, pitch * 8 * (wave * CB + c) + k_off);
#pragma unroll
    for (int c = 0; c < 2; ++c)
      lds_copy4(rss, stage + kSA + wave * 512 + c * 256, step < end ? lane * 4 : kPastEnd,
                s_off + (uint32_t)step * s_step + c * 256);
  };

  float4_t acc[NI][MI];
#pragma unroll
  for (int j = 0; j < NI; ++j)
#pragma unroll
    for (int k = 0; k < MI; ++k) acc[j][k] = float4_t{0.f, 0.f, 0.f, 0.f};

  // LDS addresses of this lane's operands in a stage: 16 rows on is 2048 bytes
  uint32_t va[2], vb[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    va[h] = lds0 + kA + (wm * MI * 16 + r) * kStageLine + 16 * stage_place(r, 4 * h + g);
    vb[h] = lds0 + kB + (wn * NI * 16 + r) * kStageLine + 16 * stage_place(r, 4 * h + g);
  }
  const uint32_t vsa = lds0 + kSA + wm * (MI / 4) * 512 + lane * 8, vsb = lds0 + kSB + wn * (NI / 4) * 512 + lane * 8;
  auto compute = [&](uint32_t stage) {
    u32x2_t sa[MI / 4], sb[NI / 4];
#pragma unroll
    for (int j = 0; j < NI / 4; ++j) sb[j] = lds_read8(vsb + stage + j * 512);
#pragma unroll
    for (int j = 0; j < MI / 4; ++j) sa[j] = lds_read8(vsa + stage + j * 512);
    unrolled<0, 2>([&](auto hc) {
      constexpr int h = decltype(hc)::value;
      u32x4_t fa[MI], fb[NI];
#pragma unroll
      for (int j = 0; j < NI; ++j) fb[j] = lds_read16(vb[h] + stage + j * 16 * kStageLine);
#pragma unroll
      for (int j = 0; j < MI; ++j) fa[j] = lds_read16(va[h] + stage + j * 16 * kStageLine);
      unrolled<0, MI>([&](auto kc) {
        constexpr int k = decltype(kc)::value;
        unrolled<0, NI>([&](auto jc) {
          constexpr int j = decltype(jc)::value;
          acc[j][k] = mfma_mx4_sel<j % 4, k % 4>(fb[j], sb[j / 4][h], fa[k], sa[k / 4][h], acc[j][k]);
        });
      });
    });
  };

  copy(lds0, begin);
  uint32_t stage = 0;
  for (int s = begin; s < end; ++s) {
    // this wave's copies of stage s are in, its LDS reads of the stage before
    // are done; then everybody's
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    copy(lds0 + (kBytes - stage), s + 1);  // the stage that was read last
    compute(stage);
    stage = kBytes - stage;
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");

  // A lane holds row l % 16, columns 4 (l / 16) .. + 3 of a 16 x 16 tile.
  // Whole rows of a wave's columns go through its own piece of LDS, so that
  // stores cover whole lines (in place, eight bytes a lane, they were four times
  // as long); chunks of 16 bytes are spread over the banks by the row.
  const int64_t wave_m = m0 + wm * MI * 16, wave_n = n0 + wn * NI * 16;
  if (q.bias) {
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int64_t col = wave_n + 16 * j + 4 * g + c;
        const float b = col < q.n ? h2f(q.bias[col]) : 0.f;
#pragma unroll
        for (int k = 0; k < MI; ++k) acc[j][k][c] += b;
      }
  }
  uint8_t* out = smem + wave * kOutBytes;
  if (q.wide && !q.y_f32) {
    static_assert(NI == 4, "a row of a wave's columns is 128 bytes of fp16");
#pragma unroll
    for (int k = 0; k < MI; ++k)
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const float4_t v = acc[j][k];
        const uint2 h = make_uint2((uint32_t)f2h(v[0]) | ((uint32_t)f2h(v[1]) << 16),
                                   (uint32_t)f2h(v[2]) | ((uint32_t)f2h(v[3]) << 16));
        *reinterpret_cast<uint2*>(out + (16 * k + r) * 128 + (((2 * j + (g >> 1)) ^ (r & 7)) * 16) + 8 * (g & 1)) = h;
      }
    uint16_t* y = static_cast<uint16_t*>(q.y);
    const int c = lane & 7;
    const int64_t col = wave_n + 8 * c;
#pragma unroll 4
    for (int i = 0; i < MI * 2; ++i) {
      const int row = 8 * i + (lane >> 3);
      const u32x4_t v = *reinterpret_cast<const u32x4_t*>(out + row * 128 + ((c ^ (row & 7)) * 16));
      if (wave_m + row >= q.m) continue;
      uint16_t* o = y + (wave_m + row) * q.ldy + col;
      if (col + 8 <= q.n) {
        u32x4_t* to = reinterpret_cast<u32x4_t*>(o);
        if constexpr (STREAM) __builtin_nontemporal_store(v, to);
        else *to = v;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (col + e < q.n) o[e] = (uint16_t)(v[e / 2] >> (16 * (e % 2)));
      }
    }
  } else if (q.wide) {
    float* y = static_cast<float*>(q.y) + split * q.m * q.n;
#pragma unroll
    for (int half = 0; half < 2; ++half) {  // 32 columns: 128 bytes a row
#pragma unroll
      for (int k = 0; k < MI; ++k)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          *reinterpret_cast<float4_t*>(out + (16 * k + r) * 128 + (((4 * j + g) ^ (r & 7)) * 16)) =
              acc[2 * half + j][k];
      const int c = lane & 7;
      const int64_t col = wave_n + 32 * half + 4 * c;
#pragma unroll 4
      for (int i = 0; i < MI * 2; ++i) {
        const int row = 8 * i + (lane >> 3);
        const float4_t v = *reinterpret_cast<const float4_t*>(out + row * 128 + ((c ^ (row & 7)) * 16));
        if (wave_m + row >= q.m) continue;
        float* o = y + (wave_m + row) * q.ldy + col;
        if (col + 4 <= q.n) {
          float4_t* to = reinterpret_cast<float4_t*>(o);
          if constexpr (STREAM) __builtin_nontemporal_store(v, to);
          else *to = v;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (col + e < q.n) o[e] = v[e];
        }
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < MI; ++k) {
      const int64_t row = wave_m + 16 * k + r;
      if (row >= q.m) continue;
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int64_t col = wave_n + 16 * j + 4 * g + c;
          if (col >= q.n) continue;
          if (q.y_f32)
            static_cast<float*>(q.y)[split * q.m * q.n + row * q.ldy + col] = acc[j][k][c];
          else
            static_cast<uint16_t*>(q.y)[row * q.ldy + col] = f2h(acc[j][k][c]);
        }
    }
  }
}

static uint32_t scale_groups(int64_t rows) { return (uint32_t)((rows + 255) / 256 * (256 / kScaleTile)); }

// How a product is cut.  A round of the chip is 256 tiles of 256 x 256 or 512 of
// 128 x 128 and takes 1.6 times as long with the large ones (5120 -> 17408, us,
// large / small: 4096 rows 212 / 228, 1024 rows 79 / 74; 1024 rows 5120 -> 5120
// 39 / 27; 4096 rows 2048 -> 4096 27 / 29).  A last round of large tiles that would
// be short is left to small ones, as columns of their own (4096 rows 5120 -> 17408
// 212 without, 201 with; 1024 rows 75 / 68; these figures with y in the caches).  Small tiles that would
// leave CUs empty share k, six steps a workgroup at least (64 rows 17408 -> 5120:
// 48 unshared, 21 shared; eight steps shared by two and added up, 4096 rows 2048 ->
// 512: 12 unshared, 18 shared), and long k by two workgroups a CU where one each
// would leave many without (1500 rows 17408 -> 1500: 55 / 41; ten steps each, 512
// rows 5120 -> 5120: 21 / 27).
struct GemmPlan {
  int64_t large;  // columns of large tiles, the first ones
  int splits;     // of k, of small tiles where there are no large ones
  size_t scales, part;
};
static int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
static int64_t rounds_small(int64_t m, int64_t n) { return cdiv(cdiv(m, 128) * cdiv(n, 128), 512); }
static GemmPlan gemm_plan(int64_t m, int64_t n, int64_t k) {
  const int64_t steps = cdiv(k, kStageK), tiles_m = cdiv(m, 256), all = tiles_m * cdiv(n, 256);
  GemmPlan p{0, 1, (size_t)steps * ((size_t)scale_groups(m) + scale_groups(n)) * 512, 0};
  int64_t best = 5 * rounds_small(m, n);
  if (8 * cdiv(all, 256) <= best) best = 8 * cdiv(all, 256), p.large = n;
  const int64_t cols = all / 256 * 256 / tiles_m * 256;  // of whole rounds
  if (cols > 0 && cols < n && 8 * cdiv(tiles_m * (cols / 256), 256) + 5 * rounds_small(m, n - cols) < best)
    p.large = cols;
  if (p.large == 0) {
    const int64_t small = cdiv(m, 128) * cdiv(n, 128);
    int64_t s = 256 / small < steps / 6 ? 256 / small : steps / 6;
    const int64_t two = 512 / small < steps / 14 ? 512 / small : steps / 14;
    if (s < 3 && two > s) s = two;
    if (s > 1) p.splits = (int)s, p.part = (size_t)s * m * n * sizeof(float);
  }
  return p;
}

// Estimated us: two launches, a step, rounds, a third launch.  Offsets into the
// staged scales are 32-bit: products past them are not for this kernel.
double mx4_gemm_cost(int64_t m, int64_t n, int64_t k) {
  const GemmPlan p = gemm_plan(m, n, k);
  if (p.scales >= ((size_t)1 << 32)) return 1e30;
  const double steps = (double)cdiv(cdiv(k, kStageK), p.splits);
  return 6.8 + 0.55 * steps * (double)rounds_small(m, n) + (p.splits > 1 ? 4.0 : 0.0);
}

size_t mx4_gemm_workspace(int64_t m, int64_t n, int64_t k) {
  const GemmPlan p = gemm_plan(m, n, k);
  return p.scales + p.part;
}

template <int TM, int TN, int WM, int WN>
static void launch_gemm_tiles(Mx4GemmArgs q, bool stream, hipStream_t s) {
  q.tiles_m = (uint32_t)((q.m + TM - 1) / TM);
  q.tiles_n = (uint32_t)((q.n + TN - 1) / TN);
  const dim3 grid(q.tiles_m * q.tiles_n * (uint32_t)q.splits), block(WM * WN * 64);
  if (stream)
    hipLaunchKernelGGL((mx4_gemm_kernel<TM, TN, WM, WN, true>), grid, block, 0, s, q);
  else
    hipLaunchKernelGGL((mx4_gemm_kernel<TM, TN, WM, WN, false>), grid, block, 0, s, q);
}

hipError_t launch_mx4_gemm(const uint8_t* a, const uint8_t* a_scales, int64_t m, const uint8_t* b,
                           const uint8_t* b_scales, int64_t n, int64_t k, const uint16_t* bias, void* y, int64_t ldy,
                           bool y_f32, void* ws, hipStream_t s) {
  const int kb = (int)(k / kMx4Block), steps = (int)((k + kStageK - 1) / kStageK);
  const GemmPlan p = gemm_plan(m, n, k);
  const uint32_t ga = scale_groups(m), gb = scale_groups(n);
  uint8_t* sa = static_cast<uint8_t*>(ws);
  uint8_t* sb = sa + (size_t)steps * ga * 512;
  float* part = reinterpret_cast<float*>(sa + p.scales);
  hipLaunchKernelGGL(mx4_stage_scales, dim3(ga + gb, (2 * steps + 15) / 16), dim3(256), 0, s,
                     StageScales{a_scales, reinterpret_cast<uint32_t*>(sa), m, ga},
                     StageScales{b_scales, reinterpret_cast<uint32_t*>(sb), n, gb}, kb, steps);
  const bool shared = p.splits > 1;
  Mx4GemmArgs q{a, b, sa, sb, ga * 512, gb * 512, shared ? nullptr : bias, y, ldy, m, n, kb, steps, y_f32, 0, 0, 0,
                p.splits};
  if (shared) q.y = part, q.ldy = n, q.y_f32 = 1;
  q.wide = (reinterpret_cast<uintptr_t>(q.y) & 15) == 0 && q.ldy % (q.y_f32 ? 4 : 8) == 0 && (!shared || n % 4 == 0);
  // 32 MB of y (the L2s together) and more, in whole lines, are stored without a place
  // in the caches
  // (us, with / without a place: 4096 rows 5120 -> 17408 199 / 187, 2048 rows 112 / 106;
  // in parts of lines, 4000 rows 96 -> 5000 21 / 29)
  const bool stream = !shared && (int64_t)m * n * (y_f32 ? 4 : 2) >= ((int64_t)32 << 20) &&
                      (reinterpret_cast<uintptr_t>(y) & 127) == 0 && ldy * (y_f32 ? 4 : 2) % 128 == 0;
  if (p.large > 0) {
    q.n = p.large;
    launch_gemm_tiles<256, 256, 2, 4>(q, stream, s);
    q.b += p.large * kb * 16;
    q.b_scales += p.large * kStageBlocks;
    if (q.bias) q.bias += p.large;
    q.y = static_cast<uint8_t*>(q.y) + p.large * (q.y_f32 ? 4 : 2);
    q.n = n - p.large;
  }
  if (q.n > 0) launch_gemm_tiles<128, 128, 2, 2>(q, stream, s);
  if (shared)
    launch_mx4_rows_finish({nullptr, nullptr, 0, nullptr, nullptr, bias, y, ldy, m, n, kb, y_f32, 0, 0, p.splits, part},
                           s);
  return hipGetLastError();
}

}  // namespace exl3
