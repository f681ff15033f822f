// exl3_mx4_moe: a whole mixture-of-experts layer for 1 to 16 tokens, in three
// launches.
//
//   1. mx4_moe_router  logits x W_r^T (the shared expert's gate as one more
//      row): workgroup (16 experts, k share), fp16 matrix instructions.  The last
//      workgroup to arrive takes every token's top-k and weights and lists the
//      chosen experts in ascending order, each with its tokens.
//   2. mx4_moe_gate_up workgroup (16 columns, listed expert): gate and up over
//      the waves' shares of k, a = silu(g) * u.
//   3. mx4_moe_down    workgroup (16 columns): the waves share the (expert, 256
//      k) units, sums are weighted per expert and meet in LDS.
//
// A token chooses an expert at most once, so 16 tokens fill at most one 16-row
// matrix operand per expert and each expert's weights are read once, whatever
// the routing.  The weights' bytes bound the two products.
//
// a is kept as three bf16 pieces (8 + 8 + 8 significand bits, exact to fp32's
// 24), so the down product runs on bf16 matrix instructions against weights
// that are exact in bf16 at any scale byte.
#include "exl3_gemm.hpp"
#include "exl3_internal.hpp"
#include "exl3_mx4_rows.hpp"

namespace exl3 {

constexpr int kMoeTokens = 16;
constexpr int kMoeExperts = 1024;
constexpr int kMoeRouterWaves = 8, kMoeGateUpWaves = 8, kMoeDownWaves = 16;
constexpr int kMoeRouterThreads = kMoeRouterWaves * 64;

// A listed expert: its tokens, in order, and the first of their rows in the
// activations.
struct MoeEntry {
  int e;
  int count;        // tokens
  int row0;
  int pad;
  uint64_t tokens;  // token i in bits 4 i .. 4 i + 3
  uint64_t pad2;
  __device__ int token(int i) const { return (int)(tokens >> (4 * i)) & 15; }
};

struct MoeArgs {
  Mx4MoeDesc d;
  const uint16_t* x;
  int64_t ldx;
  int t, topk;
  void* y;
  int64_t ldy;
  int y_f32;
  int32_t* ids;
  float* weights;
  int most;           // routed entries at most
  int rows[2];        // rows of activations: t * topk routed, t shared
  int splits;         // k shares of the router
  int lstride;        // floats of a token's partial logits
  // workspace
  uint32_t* arrived;  // router workgroups done, 0 between calls
  float* logits;      // [splits][16][lstride] partial sums, the shared gate's after the experts'
  MoeEntry* entries;  // [most + 1]; the last is the shared expert
  int* count;         // routed entries
  float* wtab;        // [most + 1][16]: weight of an entry's i-th token
  uint16_t* act[2];   // bf16 [3][rows][inter]
};

// ---------------------------------------------------------------------------
// router
// ---------------------------------------------------------------------------
// Unsigned key in the order of floats, NaN lowest, both zeros equal.
__device__ __forceinline__ uint32_t order_key(float f) {
  if (f != f) return 0u;
  const uint32_t b = __float_as_uint(f + 0.f);
  return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_ds_bpermute((int)((lane_id() ^ (uint32_t)m) << 2), (int)v);
    v = v > o ? v : o;
  }
  return v;
}
__device__ __forceinline__ float wave_max_f(float v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v = fmaxf(v, shfl_xor_f(v, m));
  return v;
}
__device__ __forceinline__ float wave_sum_f(float v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += shfl_xor_f(v, m);
  return v;
}

// Top-k and weights of one token by one wave, from its logits; lane s ends with
// choice s and its weight.  Expert 64 i + lane is the lane's i-th.
template <int EPL>
__device__ void moe_route_token(const MoeArgs& q, const float* logits, int lane, int& id, float& weight) {
  const int E = q.d.experts;
  float score[EPL];
  uint32_t key[EPL];
  bool open[EPL];  // not yet chosen
  float top = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 64 * i;
    open[i] = e < E;
    score[i] = 0.f;
    key[i] = 0;
    if (open[i]) {
      const float b = q.d.router_bias ? q.d.router_bias[e] : 0.f;
      float choice = logits[e];
      if (q.d.scoring == 0) {
        choice += b;
        score[i] = choice;
        top = fmaxf(top, choice);
      } else {
        score[i] = 1.f / (1.f + expf(-choice));
        choice = q.d.router_bias ? score[i] + b : choice;
      }
      key[i] = order_key(choice);
    }
  }
  if (q.d.scoring == 0) {
    top = wave_max_f(top);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (open[i]) {
        score[i] = expf(score[i] - top);
        sum += score[i];
      }
    sum = wave_sum_f(sum);
#pragma unroll
    for (int i = 0; i < EPL; ++i) score[i] = score[i] / sum;
  }
  id = 0;
  weight = 0.f;
  float total = 0.f;
  for (int s = 0; s < q.topk; ++s) {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) best = open[i] && key[i] > best ? key[i] : best;
    best = wave_max_u32(best);
    // the lowest expert among the equal ones: lowest i, then lowest lane
    int at = -1, from = 0;
    float mine = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const uint64_t equal = __ballot(open[i] && key[i] == best);
      if (at < 0 && equal) {
        at = i;
        from = __ffsll((unsigned long long)equal) - 1;
        mine = score[i];
        if (lane == from) open[i] = false;
      }
    }
    const float w = __shfl(mine, from);
    total += w;
    if (lane == s) {
      id = 64 * at + from;
      weight = w;
    }
  }
  if (q.d.renormalize) weight = weight / total;
  weight *= q.d.scale;
}

struct MoeRouteLds {
  float logits[kMoeTokens * (kMoeExperts + 1)];
  uint32_t masks[kMoeExperts];
  int place[kMoeExperts];
  int chunk_entries[kMoeExperts / 64], chunk_rows[kMoeExperts / 64];
};

// Routing of all tokens by one workgroup, from the partial logits.
template <int EPL>
__device__ void moe_route(const MoeArgs& q, MoeRouteLds& s) {
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int E = q.d.experts, cols = E + 1;
  for (int e = tid; e < kMoeExperts; e += kMoeRouterThreads) s.masks[e] = 0;
  for (int t = 0; t < q.t; ++t)
    for (int e = tid; e < cols; e += kMoeRouterThreads) {
      if (e == E && !q.d.shared_gate) continue;
      const float* p = q.logits + (int64_t)t * q.lstride + e;
      float v = 0.f;
      for (int k = 0; k < q.splits; ++k)
        v += __hip_atomic_load(p + (int64_t)k * kMoeTokens * q.lstride, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      s.logits[t * cols + e] = v;
    }
  __syncthreads();
  constexpr int kTurns = kMoeTokens / kMoeRouterWaves;
  int id[kTurns];
  float weight[kTurns];
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const int t = wave + kMoeRouterWaves * i;
    if (t >= q.t) break;
    moe_route_token<EPL>(q, s.logits + t * cols, lane, id[i], weight[i]);
    if (lane < q.topk) {
      atomicOr(&s.masks[id[i]], 1u << t);
      if (q.ids) q.ids[t * q.topk + lane] = id[i];
      if (q.weights) q.weights[t * q.topk + lane] = weight[i];
    }
  }
  __syncthreads();
  // entries in expert order: 64 experts at a time, then over the chunks before
  constexpr int kChunks = kMoeExperts / 64 / kMoeRouterWaves;
  int before[kChunks], rows[kChunks];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int chunk = wave + kMoeRouterWaves * c;
    const uint32_t mask = s.masks[chunk * 64 + lane];
    const uint64_t chosen = __ballot(mask != 0);
    before[c] = __popcll(chosen & ((1ull << lane) - 1));
    int sum = __popc(mask);
    for (int m = 1; m < 64; m <<= 1) {
      const int o = __shfl_up(sum, m);
      if (lane >= m) sum += o;
    }
    rows[c] = sum - __popc(mask);
    if (lane == 63) {
      s.chunk_entries[chunk] = __popcll(chosen);
      s.chunk_rows[chunk] = sum;
    }
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int chunk = wave + kMoeRouterWaves * c;
    for (int o = 0; o < chunk; ++o) {
      before[c] += s.chunk_entries[o];
      rows[c] += s.chunk_rows[o];
    }
    uint32_t mask = s.masks[chunk * 64 + lane];
    if (mask) {
      MoeEntry en{chunk * 64 + lane, (int)__popc(mask), rows[c], 0, 0, 0};
      for (int i = 0; mask; ++i, mask &= mask - 1) en.tokens |= (uint64_t)(__ffs((int)mask) - 1) << (4 * i);
      q.entries[before[c]] = en;
      s.place[chunk * 64 + lane] = before[c];
    }
    if (chunk == kMoeExperts / 64 - 1 && lane == 63) {
      q.count[0] = before[c] + (s.masks[kMoeExperts - 1] != 0);
      q.entries[q.most] = MoeEntry{-1, q.t, 0, 0, 0xFEDCBA9876543210ull, 0};
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const int t = wave + kMoeRouterWaves * i;
    if (t >= q.t) break;
    if (lane < q.topk) {
      const uint32_t earlier = s.masks[id[i]] & ((1u << t) - 1u);
      q.wtab[s.place[id[i]] * kMoeTokens + __popc(earlier)] = weight[i];
    }
    if (lane == 0) {
      float w = 1.f;
      if (q.d.shared_gate) w = 1.f / (1.f + expf(-s.logits[t * cols + E]));
      q.wtab[q.most * kMoeTokens + t] = w;
    }
  }
}

template <int EPL>
__global__ __launch_bounds__(kMoeRouterThreads) void mx4_moe_router(MoeArgs q) {
  __shared__ union {
    float4_t part[kMoeRouterWaves * 64];
    MoeRouteLds route;
  } s;
  __shared__ uint32_t before;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int g = lane >> 4, r = lane & 15;
  const int E = q.d.experts, H = q.d.hidden;
  const int group = blockIdx.x / q.splits, split = blockIdx.x - group * q.splits;
  const int e = group * 16 + r;
  const uint16_t* w = e < E ? q.d.router + (int64_t)e * H : q.d.shared_gate;
  const bool there = e < E || (e == E && q.d.shared_gate);
  float4_t acc = {0.f, 0.f, 0.f, 0.f};
  const int steps = H / 32;
#pragma unroll 4
  for (int st = split * kMoeRouterWaves + wave; st < steps; st += kMoeRouterWaves * q.splits) {
    u32x4_t a = {0u, 0u, 0u, 0u}, b = {0u, 0u, 0u, 0u};
    if (r < q.t) a = load16(q.x + r * q.ldx + 32 * st + 8 * g);
    if (there) b = load16(w + 32 * st + 8 * g);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), acc, 0, 0, 0);
  }
  s.part[wave * 64 + lane] = acc;
  __syncthreads();
  if (wave == 0) {
#pragma unroll
    for (int o = 1; o < kMoeRouterWaves; ++o) acc += s.part[o * 64 + lane];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (there && 4 * g + i < q.t)
        __hip_atomic_store(q.logits + ((int64_t)split * kMoeTokens + 4 * g + i) * q.lstride + e, acc[i],
                           __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    // device scope: the workgroups run on different XCDs
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "agent");
    if (lane == 0) before = __hip_atomic_fetch_add(q.arrived, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  if (before != gridDim.x - 1) return;
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
  if (threadIdx.x == 0) __hip_atomic_store(q.arrived, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  moe_route<EPL>(q, s.route);
}

// ---------------------------------------------------------------------------
// gate and up
// ---------------------------------------------------------------------------
// v as three bf16 pieces by truncation; their sum is v (24 significant bits).
__device__ __forceinline__ void split_bf16(float v, uint16_t (&p)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const uint32_t b = __float_as_uint(v) & 0xFFFF0000u;
    p[i] = (uint16_t)(b >> 16);
    v -= __uint_as_float(b);
  }
}

// Sums of this wave's share of k for 16 gate and 16 up rows; operand rows are
// the entry's tokens, P pieces at a time (exl3_mx4_rows.hpp).
template <int P>
__device__ void moe_gate_up_wave(const MoeArgs& q, const MoeEntry& en, const uint8_t* codes, const uint8_t* scales,
                                 int64_t row, int64_t up, int wave, int g, int r, float4_t& vg, float4_t& vu) {
  constexpr int kLoads = Mx4X<P>::kLoads;
  const int kb = q.d.hidden / kMx4Block;
  const int i = r % Mx4X<P>::kRows;
  const bool there = i < en.count;
  const uint16_t* x = q.x + (there ? en.token(i) : 0) * q.ldx;
  float4_t ag[1][P], au[1][P];
#pragma unroll
  for (int p = 0; p < P; ++p) ag[0][p] = au[0][p] = float4_t{0.f, 0.f, 0.f, 0.f};
  const int units = (kb + kMx4UnitBlocks - 1) / kMx4UnitBlocks;
  for (int u = wave; u < units; u += kMoeGateUpWaves) {
    Mx4Unit wg, wu;
    mx4_load_unit(codes + row * kb * 16, scales + row * kb, kb, u, g, wg);
    mx4_load_unit(codes + up * kb * 16, scales + up * kb, kb, u, g, wu);
    f16x8_t f[2][1][kLoads];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int l = 0; l < kLoads; ++l) f[h][0][l] = mx4_load_x<P>(x, there, kb, u, h, g, r, l);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      mx4_mma_f16<1, P>(f[h], wg, h, g, ag);
      mx4_mma_f16<1, P>(f[h], wu, h, g, au);
    }
  }
  vg = mx4_pick<P>(ag[0], g);
  vu = mx4_pick<P>(au[0], g);
}

__global__ __launch_bounds__(kMoeGateUpWaves * 64) void mx4_moe_gate_up(MoeArgs q) {
  __shared__ float part[kMoeGateUpWaves][2][16][16];  // [wave][gate, up][operand row][column]
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int g = lane >> 4, r = lane & 15;
  const int entry = blockIdx.y;
  const bool shared = entry == q.most;
  const MoeEntry en = q.entries[entry];
  if (!shared && entry >= q.count[0]) return;
  const int inter = shared ? q.d.shared_inter : q.d.inter;
  const int i0 = blockIdx.x * 16;
  if (i0 >= inter) return;
  const int64_t kb = q.d.hidden / kMx4Block;
  const uint8_t* codes = shared ? q.d.sgu_codes : q.d.gu_codes + (int64_t)en.e * 2 * inter * kb * 16;
  const uint8_t* scales = shared ? q.d.sgu_scales : q.d.gu_scales + (int64_t)en.e * 2 * inter * kb;
  const bool few = en.count <= 4;
  float4_t vg, vu;
  if (few)
    moe_gate_up_wave<4>(q, en, codes, scales, i0 + r, i0 + r + inter, wave, g, r, vg, vu);
  else
    moe_gate_up_wave<1>(q, en, codes, scales, i0 + r, i0 + r + inter, wave, g, r, vg, vu);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    part[wave][0][4 * g + i][r] = vg[i];
    part[wave][1][4 * g + i][r] = vu[i];
  }
  __syncthreads();
  // thread (token i, column c): the waves in order, of each the pieces in order
  const int i = threadIdx.x >> 4, c = threadIdx.x & 15;
  if (i >= en.count) return;
  float sg = 0.f, su = 0.f;
  for (int w = 0; w < kMoeGateUpWaves; ++w)
    for (int row = i; row < 16; row += few ? 4 : 16) {
      sg += part[w][0][row][c];
      su += part[w][1][row][c];
    }
  uint16_t p[3];
  split_bf16(sg / (1.0f + expf(-sg)) * su, p);
  const int64_t plane = (int64_t)q.rows[shared] * inter;
  uint16_t* o = q.act[shared] + (int64_t)(en.row0 + i) * inter + i0 + c;
  o[0] = p[0];
  o[plane] = p[1];
  o[2 * plane] = p[2];
}

// ---------------------------------------------------------------------------
// down
// ---------------------------------------------------------------------------
constexpr int kMoeDownWide = 5;  // tokens whose three pieces fit one operand

// A wave's task: unit u of an entry's k, for this workgroup's 16 columns.
struct MoeDownTask {
  MoeEntry en;
  const uint16_t* a;     // the entry's activations, plane 0
  const uint8_t* codes;  // this lane's weight row
  const uint8_t* scales;
  const float* weights;
  int64_t plane;
  int inter, kb, u;
};

__global__ __launch_bounds__(kMoeDownWaves * 64) void mx4_moe_down(MoeArgs q) {
  __shared__ float tiles[kMoeDownWaves][kMoeTokens][16];  // weighted sums [token][column]
  __shared__ float dump[kMoeDownWaves][16][16];           // one unit's sums [operand row][column]
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int g = lane >> 4, r = lane & 15;
  const int64_t h0 = (int64_t)blockIdx.x * 16, H = q.d.hidden;
  const int routed = q.count[0];
  const int units = (q.d.inter / kMx4Block + kMx4UnitBlocks - 1) / kMx4UnitBlocks;
  const int tasks = routed * units + (q.d.shared_inter / kMx4Block + kMx4UnitBlocks - 1) / kMx4UnitBlocks;
  auto task = [&](int id) {
    MoeDownTask t;
    const bool shared = id >= routed * units;
    const int entry = shared ? q.most : id / units;
    t.u = shared ? id - routed * units : id - entry * units;
    t.en = q.entries[entry];
    t.inter = shared ? q.d.shared_inter : q.d.inter;
    t.kb = t.inter / kMx4Block;
    t.plane = (int64_t)q.rows[shared] * t.inter;
    t.a = q.act[shared] + (int64_t)t.en.row0 * t.inter;
    t.weights = q.wtab + entry * kMoeTokens;
    const int64_t row = (shared ? 0 : (int64_t)t.en.e * H) + h0 + r;
    t.codes = (shared ? q.d.sdn_codes : q.d.dn_codes) + row * t.kb * 16;
    t.scales = (shared ? q.d.sdn_scales : q.d.dn_scales) + row * t.kb;
    return t;
  };
#pragma unroll
  for (int i = 0; i < 4; ++i) tiles[wave][4 * g + i][r] = 0.f;
  // the weights of the next task are fetched before this one's product
  MoeDownTask now, next;
  Mx4Unit w, wn;
  if (wave < tasks) {
    now = task(wave);
    mx4_load_unit(now.codes, now.scales, now.kb, now.u, g, w);
  }
  for (int id = wave; id < tasks; id += kMoeDownWaves) {
    const bool more = id + kMoeDownWaves < tasks;
    if (more) {
      next = task(id + kMoeDownWaves);
      mx4_load_unit(next.codes, next.scales, next.kb, next.u, g, wn);
    }
    const int n = now.en.count;
    // 8 elements of this lane's block of half h, piece j, of plane p of token row i
    auto act = [&](bool there, int i, int p, int h, int j) {
      const int b = now.u * kMx4UnitBlocks + 4 * h + g;
      u32x4_t v = {0u, 0u, 0u, 0u};
      if (there && b < now.kb) v = load16(now.a + p * now.plane + (int64_t)i * now.inter + b * kMx4Block + 8 * j);
      return __builtin_bit_cast(bf16x8_t, v);
    };
    if (n == 1) {
      // operand row 3 j + p: piece j of plane p; the sums of piece j are wanted
      // in rows 3 j .. 3 j + 2
      bf16x8_t f[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) f[h] = act(r < 12, 0, r % 3, h, r / 3);
      float4_t acc[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] = float4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float s = mx4_scale(mx4_own_scale(w, h, g) & 0xFFu);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[h], mx4_to_bf16(w.half[h][j], s), acc[j], 0, 0, 0);
      }
      // rows 4 g .. 4 g + 3 of this lane: smallest plane first
      float v = 0.f;
      if (g == 0) v = (acc[0][2] + acc[0][1]) + acc[0][0] + acc[1][3];
      if (g == 1) v = (acc[1][1] + acc[1][0]) + (acc[2][3] + acc[2][2]);
      if (g == 2) v = acc[2][0] + ((acc[3][3] + acc[3][2]) + acc[3][1]);
      v += shfl_xor_f(v, 16);
      v += shfl_xor_f(v, 32);
      if (g == 0) tiles[wave][now.en.token(0)][r] += now.weights[0] * v;
    } else {
      float4_t acc = {0.f, 0.f, 0.f, 0.f};
      const bool wide = n <= kMoeDownWide;  // operand row 3 i + p, else row i and one plane after the other
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float s = mx4_scale(mx4_own_scale(w, h, g) & 0xFFu);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bf16x8_t c = mx4_to_bf16(w.half[h][j], s);
          if (wide) {
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(act(r < 3 * n, r / 3, r % 3, h, j), c, acc, 0, 0, 0);
          } else {
#pragma unroll
            for (int p = 2; p >= 0; --p)
              acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(act(r < n, r, p, h, j), c, acc, 0, 0, 0);
          }
        }
      }
      if (wide) {
#pragma unroll
        for (int i = 0; i < 4; ++i) dump[wave][4 * g + i][r] = acc[i];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        for (int i = g; i < n; i += 4) {
          const float v = dump[wave][3 * i + 2][r] + dump[wave][3 * i + 1][r] + dump[wave][3 * i][r];
          tiles[wave][now.en.token(i)][r] += now.weights[i] * v;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (4 * g + i < n) tiles[wave][now.en.token(4 * g + i)][r] += now.weights[4 * g + i] * acc[i];
      }
    }
    now = next;
    w = wn;
  }
  __syncthreads();
  const int t = threadIdx.x >> 4, c = threadIdx.x & 15;
  if (t >= q.t) return;
  float v = 0.f;
#pragma unroll
  for (int o = 0; o < kMoeDownWaves; ++o) v += tiles[o][t][c];
  const int64_t at = t * q.ldy + h0 + c;
  if (q.y_f32)
    static_cast<float*>(q.y)[at] = v;
  else
    static_cast<uint16_t*>(q.y)[at] = f2h(v);
}

// ---------------------------------------------------------------------------
namespace {
size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

int moe_most(const Mx4MoeDesc& d, int64_t t, int topk) { return (int)(t * topk < d.experts ? t * topk : d.experts); }

// k shares of the router: a wave takes about two matrix instructions, the
// chip's 256 CUs at most one workgroup each.
int moe_splits(const Mx4MoeDesc& d) {
  const int groups = d.experts / 16 + 1, steps = d.hidden / 32;
  int s = steps / (2 * kMoeRouterWaves);
  if (s > 256 / groups) s = 256 / groups;
  return s < 1 ? 1 : (s > 8 ? 8 : s);
}

struct MoeLayout {
  size_t arrived, logits, entries, count, wtab, act[2], total;
  int lstride;
};
MoeLayout moe_layout(const Mx4MoeDesc& d, int64_t t, int topk) {
  const size_t most = (size_t)moe_most(d, t, topk) + 1;
  MoeLayout L;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += align256(bytes);
    return at;
  };
  L.lstride = (d.experts + 16) / 16 * 16;
  L.arrived = take(4);  // first in every layout: a workspace serves all sizes
  L.logits = take((size_t)moe_splits(d) * kMoeTokens * L.lstride * 4);
  L.entries = take(most * sizeof(MoeEntry));
  L.count = take(4);
  L.wtab = take(most * kMoeTokens * 4);
  L.act[0] = take((size_t)t * topk * d.inter * 6);
  L.act[1] = take((size_t)t * d.shared_inter * 6);
  L.total = off;
  return L;
}
}  // namespace

size_t mx4_moe_workspace(const Mx4MoeDesc& d, int64_t t, int topk) { return moe_layout(d, t, topk).total; }

hipError_t launch_mx4_moe(const Mx4MoeDesc& d, const uint16_t* x, int64_t t, int64_t ldx, int topk, void* y,
                          int64_t ldy, bool y_f32, int32_t* ids, float* weights, void* ws, hipStream_t s) {
  const MoeLayout L = moe_layout(d, t, topk);
  unsigned char* w = static_cast<unsigned char*>(ws);
  const int most = moe_most(d, t, topk), splits = moe_splits(d);
  const MoeArgs q{d, x, ldx, (int)t, topk, y, ldy, y_f32, ids, weights, most, {(int)t * topk, (int)t}, splits, L.lstride,
                  reinterpret_cast<uint32_t*>(w + L.arrived), reinterpret_cast<float*>(w + L.logits),
                  reinterpret_cast<MoeEntry*>(w + L.entries), reinterpret_cast<int*>(w + L.count),
                  reinterpret_cast<float*>(w + L.wtab),
                  {reinterpret_cast<uint16_t*>(w + L.act[0]), reinterpret_cast<uint16_t*>(w + L.act[1])}};
  const dim3 rgrid((uint32_t)((d.experts / 16 + 1) * splits)), rblock(kMoeRouterThreads);
  if (d.experts <= 64) hipLaunchKernelGGL(mx4_moe_router<1>, rgrid, rblock, 0, s, q);
  else if (d.experts <= 128) hipLaunchKernelGGL(mx4_moe_router<2>, rgrid, rblock, 0, s, q);
  else if (d.experts <= 256) hipLaunchKernelGGL(mx4_moe_router<4>, rgrid, rblock, 0, s, q);
  else hipLaunchKernelGGL(mx4_moe_router<16>, rgrid, rblock, 0, s, q);
  const int wide = d.inter > d.shared_inter ? d.inter : d.shared_inter;
  hipLaunchKernelGGL(mx4_moe_gate_up, dim3(wide / 16, most + (d.shared_inter ? 1 : 0)), dim3(kMoeGateUpWaves * 64), 0, s, q);
  hipLaunchKernelGGL(mx4_moe_down, dim3(d.hidden / 16), dim3(kMoeDownWaves * 64), 0, s, q);
  return hipGetLastError();
}

}  // namespace exl3
