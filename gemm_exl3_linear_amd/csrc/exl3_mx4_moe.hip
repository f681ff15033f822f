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
//      k) units, sums are weighted per expert and meet in LDS; many experts are
//      shared among workgroups, the last of which adds their sums.
//
// A token chooses an expert at most once, so 16 tokens fill at most one 16-row
// matrix operand per expert and each expert's weights are read once, whatever
// the routing.  The weights' bytes bound the two products.
//
// Measured (us, router / gate and up / down, of kernels; a call, and one over 1.4 GB
// of weights in turn): 1 token, 8 of 256 experts 2048 x 512 7.4 / 6.5 / 4.9, 17.2, 19.7;
// 16 tokens, about 101 experts of them and a shared one 11 / 30 / 22, 62, 63 (116 and 58
// MB: 3.9 and 2.6 TB/s); 5 tokens, 4 of 60 experts 1440 x 352 6.6 / 7.6 / 7.9, 21, 24.5.
// Few tokens are bound by the three launches, each with its loads, sums and routing
// one after the other; many experts by what eight waves a SIMD have in flight: more
// loads a wave at the price of waves were slower (two units at a time 67 us, six
// waves 74).
//
// a is kept as three bf16 pieces (8 + 8 + 8 significand bits, exact to fp32's
// 24), so the down product runs on bf16 matrix instructions against weights
// that are exact in bf16 up to scale byte 252 (6 2^125); units with a block past
// that are taken block by block (moe_down_far).
#include "exl3_gemm.hpp"
#include "exl3_internal.hpp"
#include "exl3_mx4_rows.hpp"

namespace exl3 {

constexpr int kMoeTokens = 16;
constexpr int kMoeMaxDim = 65536;  // of hidden and of an expert
constexpr int kMoeDownWaves = 16;

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
  uint32_t* arrived;  // workgroups done, 0 between calls: the router's, then those of each 16 columns of down
  float* logits;      // [splits][16][lstride] partial sums, the shared gate's after the experts'
  MoeEntry* entries;  // [most + 1]; the last is the shared expert
  int* count;         // routed entries
  float* wtab;        // [most + 1][16]: weight of an entry's i-th token
  uint16_t* act[2];   // bf16 [3][rows][inter]
  int down_splits;    // workgroups that share the entries of 16 columns
  float* down;        // their sums [split][t][hidden], where there are several
};

// Sums that the last workgroup to arrive takes from the others, which run on
// other XCDs, pass by stores and loads of device scope: those do not stay in an
// XCD's L2, so a wave that has waited for its stores may count itself in.  (Fences
// of device scope write the L2 back and drop it: 1 to 2 us.)
__device__ __forceinline__ void store_shared(float* p, float v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float load_shared(const float* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void wait_stores() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
// Counts one of n in; true for the last, which leaves 0.
__device__ __forceinline__ bool last_in(uint32_t* count, uint32_t n) {
  const bool last = __hip_atomic_fetch_add(count, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == n - 1;
  if (last) __hip_atomic_store(count, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return last;
}

// ---------------------------------------------------------------------------
// router
// ---------------------------------------------------------------------------
// Unsigned key in the order of floats, NaN lowest, both zeros equal; never 0.
__device__ __forceinline__ uint32_t order_key(float f) {
  if (f != f) return 1u;
  const uint32_t b = __float_as_uint(f + 0.f);
  return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

// Reductions over a wave on the vector unit alone: shifts by 1, 2, 4, 8 inside
// the rows of 16 lanes, then row ends to the next row and to the upper half; lane
// 63 ends with the result.  (Six LDS permutes took 6 x 100 cycles a choice.)
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_or_zero(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, ROWS == 0xF);
}
template <class Op>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t v, Op op) {  // 0 is neutral
  v = op(v, dpp_or_zero<0x111, 0xF>(v));
  v = op(v, dpp_or_zero<0x112, 0xF>(v));
  v = op(v, dpp_or_zero<0x114, 0xF>(v));
  v = op(v, dpp_or_zero<0x118, 0xF>(v));
  v = op(v, dpp_or_zero<0x142, 0xA>(v));
  v = op(v, dpp_or_zero<0x143, 0xC>(v));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  return wave_reduce(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
__device__ __forceinline__ float wave_sum_f(float v) {
  return __uint_as_float(wave_reduce(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

// e^x in few instructions: x log2 e with the product's own rounding error, and log2
// e's, put back after the power.  To about an ulp for 2^-125 < e^x < 2^126; past that, where
// a correction could meet an infinity or a subnormal, without it: off by up to 2^-17 of
// the value.  (The routing runs once
// a call, so its instructions come from memory: their number is its time.)
__device__ __forceinline__ float exp_f(float x) {
  constexpr float kLog2e = 1.44269502162933349609375f, kLog2eRest = 1.925963033500e-8f, kLn2 = 0.693147180559945309f;
  const float t = x * kLog2e;
  const float rest = __builtin_fmaf(x, kLog2eRest, __builtin_fmaf(x, kLog2e, -t));
  const float p = __builtin_amdgcn_exp2f(t);
  return t > 126.f || t < -125.f ? p : __builtin_fmaf(p, rest * kLn2, p);
}

// Top-k and weights of one token by one wave, from its keys (in the order of
// its choices, 0 where there is no expert) and its scores, before the softmax;
// lane s ends with choice s and its weight.  Expert 64 i + lane is the lane's i-th.
// A choice takes the highest key of the wave and then the lowest expert that
// holds it; its key becomes 0.
template <int EPL>
__device__ __forceinline__ void moe_route_token(const MoeArgs& q, const uint32_t* keys, const float* scores, int lane,
                                                int& id, float& weight) {
  uint32_t key[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) key[i] = keys[lane + 64 * i];
  id = 0;
  uint32_t top = 0;
  for (int s = 0; s < q.topk; ++s) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) best = best > key[i] ? best : key[i];
    best = wave_max_u32(best);
    top = s ? top : best;
    int e = 0;
#pragma unroll
    for (int i = EPL - 1; i >= 0; --i) {
      const uint64_t equal = __ballot(key[i] == best);
      e = equal ? 64 * i + __ffsll((unsigned long long)equal) - 1 : e;
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = lane + 64 * i == e ? 0u : key[i];
    id = lane == s ? e : id;
  }
  weight = scores[id];
  if (q.d.scoring == 0) {
    // the highest l + b (NaN if every one is)
    const float high = __uint_as_float(top >> 31 ? top ^ 0x80000000u : ~top);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) sum += lane + 64 * i < q.d.experts ? exp_f(scores[lane + 64 * i] - high) : 0.f;
    weight = exp_f(weight - high) / wave_sum_f(sum);
  }
  if (q.d.renormalize) weight = weight / wave_sum_f(lane < q.topk ? weight : 0.f);
  weight *= q.d.scale;
}

template <int EPL>
struct MoeRouteLds {
  static constexpr int kCols = 64 * EPL;
  float scores[kMoeTokens * kCols];   // l + b (softmax), or sigmoid(l)
  uint32_t keys[kMoeTokens * kCols];
  float gates[kMoeTokens];            // the shared expert's logits
  uint32_t masks[kCols];
  int place[kCols];
  int chunk_entries[EPL], chunk_rows[EPL];
};

// Routing of all tokens by one workgroup of NW waves, at least as many as tokens,
// from the partial logits.
template <int EPL, int NW>
__device__ __forceinline__ void moe_route(const MoeArgs& q, MoeRouteLds<EPL>& s) {
  constexpr int cols = MoeRouteLds<EPL>::kCols;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int E = q.d.experts;
  for (int e = tid; e < cols; e += NW * 64) s.masks[e] = 0;
#pragma unroll 2
  for (int i = tid; i < q.t * cols; i += NW * 64) {
    const int t = i / cols, e = i - t * cols;
    uint32_t key = 0;
    if (e < E) {
      const float* p = q.logits + (int64_t)t * q.lstride + e;
      float l = 0.f;
#pragma unroll 4
      for (int k = 0; k < q.splits; ++k) l += load_shared(p + (int64_t)k * kMoeTokens * q.lstride);
      const float b = q.d.router_bias ? q.d.router_bias[e] : 0.f;
      const float score = q.d.scoring == 0 ? l + b : 1.f / (1.f + exp_f(-l));
      // without a bias the sigmoid's order is the logit's, where it has not saturated
      key = order_key(q.d.scoring == 0 ? score : (q.d.router_bias ? score + b : l));
      s.scores[i] = score;
    }
    s.keys[i] = key;
  }
  if (q.d.shared_gate && tid < q.t) {
    float l = 0.f;
    for (int k = 0; k < q.splits; ++k) l += load_shared(q.logits + ((int64_t)k * kMoeTokens + tid) * q.lstride + E);
    s.gates[tid] = l;
  }
  __syncthreads();
  const int t = wave;  // a token a wave
  int id = 0;
  float weight = 0.f;
  if (t < q.t) {
    moe_route_token<EPL>(q, s.keys + t * cols, s.scores + t * cols, lane, id, weight);
    if (lane < q.topk) {
      atomicOr(&s.masks[id], 1u << t);
      if (q.ids) q.ids[t * q.topk + lane] = id;
      if (q.weights) q.weights[t * q.topk + lane] = weight;
    }
  }
  __syncthreads();
  // entries in expert order: 64 experts a wave, then over the chunks before
  constexpr int kChunks = (EPL + NW - 1) / NW;
  int before[kChunks], rows[kChunks];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int chunk = wave + NW * c;
    if (chunk >= EPL) break;
    const uint32_t mask = s.masks[chunk * 64 + lane];
    const uint64_t chosen = __ballot(mask != 0);
    before[c] = __popcll(chosen & ((1ull << lane) - 1));
    // pairs of the lanes before: bit by bit of their counts (at most 16)
    const int n = __popc(mask);
    int sum = 0, all = 0;
#pragma unroll
    for (int bit = 0; bit < 5; ++bit) {
      const uint64_t b = __ballot((n >> bit) & 1);
      sum += __popcll(b & ((1ull << lane) - 1)) << bit;
      all += __popcll(b) << bit;
    }
    rows[c] = sum;
    if (lane == 0) {
      s.chunk_entries[chunk] = __popcll(chosen);
      s.chunk_rows[chunk] = all;
    }
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int chunk = wave + NW * c;
    if (chunk >= EPL) break;
#pragma unroll
    for (int o = 0; o < EPL; ++o) {
      before[c] += o < chunk ? s.chunk_entries[o] : 0;
      rows[c] += o < chunk ? s.chunk_rows[o] : 0;
    }
    uint32_t mask = s.masks[chunk * 64 + lane];
    if (mask) {
      MoeEntry en{chunk * 64 + lane, (int)__popc(mask), rows[c], 0, 0, 0};
      for (int i = 0; mask; ++i, mask &= mask - 1) en.tokens |= (uint64_t)(__ffs((int)mask) - 1) << (4 * i);
      q.entries[before[c]] = en;
      s.place[chunk * 64 + lane] = before[c];
    }
    if (chunk == EPL - 1 && lane == 63) {
      q.count[0] = before[c] + (s.masks[64 * EPL - 1] != 0);
      q.entries[q.most] = MoeEntry{-1, q.t, 0, 0, 0xFEDCBA9876543210ull, 0};
    }
  }
  __syncthreads();
  if (t >= q.t) return;
  if (lane < q.topk) {
    const uint32_t earlier = s.masks[id] & ((1u << t) - 1u);
    q.wtab[s.place[id] * kMoeTokens + __popc(earlier)] = weight;
  }
  if (lane == 0) {
    float w = 1.f;
    if (q.d.shared_gate) w = 1.f / (1.f + exp_f(-s.gates[t]));
    q.wtab[q.most * kMoeTokens + t] = w;
  }
}

// NW waves: 16 where there are more than 8 tokens to route, else the quicker 8.
template <int EPL, int NW>
__global__ __launch_bounds__(NW * 64) void mx4_moe_router(MoeArgs q) {
  __shared__ union {
    float4_t part[NW * 64];
    MoeRouteLds<EPL> route;
  } s;
  __shared__ int last;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int g = lane >> 4, r = lane & 15;
  const int E = q.d.experts, H = q.d.hidden;
  const int group = blockIdx.x / q.splits, split = blockIdx.x - group * q.splits;
  const int e = group * 16 + r;
  const uint16_t* w = e < E ? q.d.router + (int64_t)e * H : q.d.shared_gate;
  const bool there = e < E || (e == E && q.d.shared_gate);
  float4_t acc = {0.f, 0.f, 0.f, 0.f};
  const int steps = H / 32, stride = NW * q.splits;
  for (int st = split * NW + wave; st < steps; st += 4 * stride) {
    u32x4_t a[4], b[4];  // four steps' loads at a time
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = st + i * stride;
      a[i] = b[i] = u32x4_t{0u, 0u, 0u, 0u};
      if (r < q.t && at < steps) a[i] = load16(q.x + r * q.ldx + 32 * at + 8 * g);
      if (there && at < steps) b[i] = load16(w + 32 * at + 8 * g);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a[i]), __builtin_bit_cast(f16x8_t, b[i]),
                                                   acc, 0, 0, 0);
  }
  s.part[wave * 64 + lane] = acc;
  __syncthreads();
  if (wave == 0) {
#pragma unroll
    for (int o = 1; o < NW; ++o) acc += s.part[o * 64 + lane];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (there && 4 * g + i < q.t)
        store_shared(q.logits + ((int64_t)split * kMoeTokens + 4 * g + i) * q.lstride + e, acc[i]);
    wait_stores();
    if (lane == 0) last = last_in(q.arrived, gridDim.x);
  }
  __syncthreads();
  if (!last) return;
  moe_route<EPL, NW>(q, s.route);
}

// ---------------------------------------------------------------------------
// gate and up
// ---------------------------------------------------------------------------
// v as three bf16 pieces by truncation; their sum is v (24 significant bits; an
// infinity or a NaN is all in the first).
__device__ __forceinline__ void split_bf16(float v, uint16_t (&p)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const uint32_t b = __float_as_uint(v) & 0xFFFF0000u;
    p[i] = (uint16_t)(b >> 16);
    v = __builtin_isfinite(v) ? v - __uint_as_float(b) : 0.f;
  }
}

// An entry by a uniform index, through scalar loads.
__device__ __forceinline__ MoeEntry load_entry(const MoeEntry* p, int i) {
  typedef __attribute__((address_space(4))) const uint64_t* words;
  const words w = (words)(uintptr_t)(p + i);
  uint64_t v[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = w[k];
  static_assert(sizeof(MoeEntry) == 32, "four words");
  return MoeEntry{(int)(uint32_t)v[0], (int)(v[0] >> 32), (int)(uint32_t)v[1], 0, v[2], 0};
}
__device__ __forceinline__ int load_uniform(const int* p) {
  return *(__attribute__((address_space(4))) const int*)(uintptr_t)p;
}

// Sums of 16 weight rows over every SHARES-th unit of k from `first`, fetched GU at a
// time; operand rows are the entry's tokens, P pieces at a time (exl3_mx4_rows.hpp).
template <int P, int SHARES, int GU>
__device__ __forceinline__ float4_t moe_gate_up_wave(const MoeArgs& q, const MoeEntry& en, const Mx4Row& row,
                                                     int first, int g, int r) {
  constexpr int kLoads = Mx4X<P>::kLoads;
  const int kb = q.d.hidden / kMx4Block;
  const int i = r % Mx4X<P>::kRows;
  const bool there = i < en.count;
  const uint16_t* x = q.x + (there ? en.token(i) : 0) * q.ldx;
  float4_t acc[1][1][P];
#pragma unroll
  for (int p = 0; p < P; ++p) acc[0][0][p] = float4_t{0.f, 0.f, 0.f, 0.f};
  const int units = (kb + kMx4UnitBlocks - 1) / kMx4UnitBlocks;
  bool exact = true;
  for (int u = first; u < units; u += GU * SHARES) {
    Mx4Unit w[GU][1];
    f16x8_t f[GU][2][1][kLoads];
#pragma unroll
    for (int i = 0; i < GU; ++i) mx4_load_unit(row, kb, u + i * SHARES, g, w[i][0]);
#pragma unroll
    for (int i = 0; i < GU * 2 * kLoads; ++i) {
      const int k = i / (2 * kLoads), h = i / kLoads % 2, l = i % kLoads;
      f[k][h][0][l] = mx4_load_x<P>(x, there, kb, u + k * SHARES, h, g, r, l);
    }
#pragma unroll
    for (int i = 0; i < GU * 2; ++i) exact = mx4_mma_f16<1, P, 1>(f[i / 2][i % 2], w[i / 2], i % 2, g, acc) && exact;
  }
  if (__builtin_expect(!__all(exact), 0))
    mx4_sum_blocks<1, P, 1>({x}, {there}, {row}, kb, first, units, SHARES, 0, 2, g, r, acc);
  return mx4_pick<P>(acc[0][0], g);
}

// NW waves: half gate, half up.
// ROOMY: a workgroup a CU at most, whose waves may have twice the registers and fetch
// two units at a time.
template <int NW, bool ROOMY>
__global__ __launch_bounds__(NW * 64, ROOMY ? 4 : 8) void mx4_moe_gate_up(MoeArgs q) {
  constexpr int GU = ROOMY ? 2 : 1;
  constexpr int kShares = NW / 2;
  __shared__ float part[NW][16][16];  // [wave][operand row][column]; the first half of the waves: gate
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int g = lane >> 4, r = lane & 15;
  const int entry = blockIdx.y;
  const bool shared = entry == q.most;
  const MoeEntry en = load_entry(q.entries, entry);
  if (!shared && entry >= load_uniform(q.count)) return;
  const int inter = shared ? q.d.shared_inter : q.d.inter;
  const int i0 = blockIdx.x * 16;
  if (i0 >= inter) return;
  const int64_t top = (shared ? 0 : (int64_t)en.e * 2 * inter) + (wave >= kShares ? inter : 0) + i0;
  const Mx4Row row = mx4_row(shared ? q.d.sgu_codes : q.d.gu_codes, shared ? q.d.sgu_scales : q.d.gu_scales, top, r,
                             q.d.hidden / kMx4Block);
  const int first = wave % kShares;
  const bool few = en.count <= 4;
  const float4_t v = few ? moe_gate_up_wave<4, kShares, GU>(q, en, row, first, g, r)
                         : moe_gate_up_wave<1, kShares, GU>(q, en, row, first, g, r);
#pragma unroll
  for (int i = 0; i < 4; ++i) part[wave][4 * g + i][r] = v[i];
  __syncthreads();
  // thread (token i, column c): the waves in order, of each the pieces in order
  const int i = threadIdx.x >> 4, c = threadIdx.x & 15;
  if (i >= en.count) return;
  float sg = 0.f, su = 0.f;
#pragma unroll
  for (int w = 0; w < kShares; ++w)
    for (int o = i; o < 16; o += few ? 4 : 16) {
      sg += part[w][o][c];
      su += part[kShares + w][o][c];
    }
  uint16_t p[3];
  split_bf16(sg / (1.0f + exp_f(-sg)) * su, p);
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

__device__ __forceinline__ void moe_store(const MoeArgs& q, int t, int64_t h, float v) {
  if (q.y_f32)
    static_cast<float*>(q.y)[t * q.ldy + h] = v;
  else
    static_cast<uint16_t*>(q.y)[t * q.ldy + h] = f2h(v);
}

// A wave's task: unit u of an entry's k, for this workgroup's 16 columns.
struct MoeDownTask {
  MoeEntry en;
  const uint16_t* a;     // the entry's activations, plane 0
  Mx4Row row;            // this lane's weight row
  const float* weights;
  int64_t plane;
  int inter, kb, u;
};

// The sums of a unit with blocks at scale bytes 253 and 254, whose larger values
// pass bf16's range: block by block, those blocks at 2^-4 of their scale and
// their sums by 2^4.  The other blocks are taken out of both operands: an infinite
// activation times their zeros would be NaN.  Operand row i is token i, one plane
// after the other.
__device__ __forceinline__ bool moe_down_is_far(uint32_t s) { return s - 253u <= 1u; }
__device__ __forceinline__ bool moe_down_any_far(const Mx4Unit& w, int g) {
  return __any(moe_down_is_far(mx4_own_scale(w, 0, g) & 0xFFu) || moe_down_is_far(mx4_own_scale(w, 1, g) & 0xFFu));
}
__device__ __forceinline__ float4_t moe_down_far(const MoeDownTask& t, const Mx4Unit& w, int g, int r) {
  float4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int b = 0; b < kMx4UnitBlocks; ++b) {
    const u32x4_t codes = b < 4 ? w.half[0] : w.half[1];
    const uint32_t s = ((b < 4 ? w.sc[0] : w.sc[1]) >> (8 * (b & 3))) & 0xFFu;  // of this lane's column
    const bool far = moe_down_is_far(s), own = g == (b & 3);
    const float scale = mx4_scale(own ? (far ? s - 4u : s) : kMx4One), back = far ? 16.f : 1.f;
    const int at = t.u * kMx4UnitBlocks + b;
    const bool there = own && r < t.en.count && at < t.kb;
    const uint16_t* a = t.a + (int64_t)(there ? r : 0) * t.inter + at * kMx4Block;
    float4_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bf16x8_t c = mx4_to_bf16(own ? codes[j] : 0u, scale);
#pragma unroll
      for (int p = 2; p >= 0; --p) {  // smallest plane first
        u32x4_t f = {0u, 0u, 0u, 0u};
        if (there) f = load16(a + p * t.plane + 8 * j);
        v = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, f), c, v, 0, 0, 0);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(v[i], back, acc[i]);
  }
  return acc;
}

// ROOMY: a workgroup a CU at most, whose waves may have twice the registers and
// fetch the activations of several tokens together.
template <bool ROOMY>
__global__ __launch_bounds__(kMoeDownWaves * 64, ROOMY ? 4 : 8) void mx4_moe_down(MoeArgs q) {
  __shared__ float tiles[kMoeDownWaves][kMoeTokens][16];  // weighted sums [token][column]
  __shared__ float dump[kMoeDownWaves][16][16];           // one unit's sums [operand row][column]
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int g = lane >> 4, r = lane & 15;
  const int64_t h0 = (int64_t)blockIdx.x * 16, H = q.d.hidden;
  const int routed = load_uniform(q.count);
  const int units = (q.d.inter / kMx4Block + kMx4UnitBlocks - 1) / kMx4UnitBlocks;
  const int tasks = routed * units + (q.d.shared_inter / kMx4Block + kMx4UnitBlocks - 1) / kMx4UnitBlocks;
  auto task = [&](int id, int r) {
    MoeDownTask t;
    const bool shared = id >= routed * units;
    const int entry = shared ? q.most : id / units;
    t.u = shared ? id - routed * units : id - entry * units;
    t.en = load_entry(q.entries, entry);
    t.inter = shared ? q.d.shared_inter : q.d.inter;
    t.kb = t.inter / kMx4Block;
    t.plane = (int64_t)q.rows[shared] * t.inter;
    t.a = q.act[shared] + (int64_t)t.en.row0 * t.inter;
    t.weights = q.wtab + entry * kMoeTokens;
    t.row = mx4_row(shared ? q.d.sdn_codes : q.d.dn_codes, shared ? q.d.sdn_scales : q.d.dn_scales,
                    (shared ? 0 : (int64_t)t.en.e * H) + h0, r, t.kb);
    return t;
  };
#pragma unroll
  for (int i = 0; i < 4; ++i) tiles[wave][4 * g + i][r] = 0.f;
  // the weights of the next task are fetched before this one's product, and (ROOMY)
  // a single token's activations, operand row 3 j + p piece j of plane p: loads return
  // in order, so one for this task would wait for the next one's weights.  (Its
  // routing weight comes by a scalar load for the same reason.  Two tasks in turn,
  // without the moves at the end, were slower for their longer code.)
  // the sums of operand rows 4 g .. 4 g + 3, by their tokens' weights
  auto add_rows = [&](const MoeDownTask& t, const float4_t& acc, int g, int r) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (4 * g + i < t.en.count) tiles[wave][t.en.token(4 * g + i)][r] += t.weights[4 * g + i] * acc[i];
  };
  bool met_far = false;  // a unit left for the second way
  MoeDownTask now, next;
  Mx4Unit w, wn;
  bf16x8_t one[2], one_n[2];
  auto load_one = [&](const MoeDownTask& t, bf16x8_t (&f)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int b = t.u * kMx4UnitBlocks + 4 * h + g;
      u32x4_t v = {0u, 0u, 0u, 0u};
      if (r < 12 && b < t.kb) v = load16(t.a + (r % 3) * t.plane + b * kMx4Block + 8 * (r / 3));
      f[h] = __builtin_bit_cast(bf16x8_t, v);
    }
  };
  const int first = (int)blockIdx.y * kMoeDownWaves + wave, stride = kMoeDownWaves * q.down_splits;
  if (first < tasks) {
    now = task(first, r);
    mx4_load_unit(now.row, now.kb, now.u, g, w);
    if (ROOMY && now.en.count == 1) load_one(now, one);
  }
  for (int id = first; id < tasks; id += stride) {
    const bool more = id + stride < tasks;
    if (more) {
      next = task(id + stride, r);
      mx4_load_unit(next.row, next.kb, next.u, g, wn);
      if (ROOMY && next.en.count == 1) load_one(next, one_n);
    }
    const int n = now.en.count;
    // 8 elements of this lane's block of half h, piece j, of plane p of token row i
    auto act = [&](bool there, int i, int p, int h, int j) {
      const int b = now.u * kMx4UnitBlocks + 4 * h + g;
      u32x4_t v = {0u, 0u, 0u, 0u};
      if (there && b < now.kb) v = load16(now.a + p * now.plane + (int64_t)i * now.inter + b * kMx4Block + 8 * j);
      return __builtin_bit_cast(bf16x8_t, v);
    };
    // asked after the products (and the loads before them), which then go nowhere
    auto is_far = [&] {
      const bool far = moe_down_any_far(w, g);
      met_far = met_far || far;
      return far;
    };
    if (n == 1) {
      // the sums of piece j are wanted in rows 3 j .. 3 j + 2
      if (!ROOMY) load_one(now, one);
      const float weight = __int_as_float(load_uniform(reinterpret_cast<const int*>(now.weights)));
      float4_t acc[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] = float4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float s = mx4_scale(mx4_own_scale(w, h, g) & 0xFFu);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(one[h], mx4_to_bf16(w.half[h][j], s), acc[j], 0, 0, 0);
      }
      // rows 4 g .. 4 g + 3 of this lane: smallest plane first
      float v = 0.f;
      if (g == 0) v = (acc[0][2] + acc[0][1]) + acc[0][0] + acc[1][3];
      if (g == 1) v = (acc[1][1] + acc[1][0]) + (acc[2][3] + acc[2][2]);
      if (g == 2) v = acc[2][0] + ((acc[3][3] + acc[3][2]) + acc[3][1]);
      v += shfl_xor_f(v, 16);
      v += shfl_xor_f(v, 32);
      if (!is_far() && g == 0) tiles[wave][now.en.token(0)][r] += weight * v;
    } else {
      float4_t acc = {0.f, 0.f, 0.f, 0.f};
      const bool wide = n <= kMoeDownWide;  // operand row 3 i + p, else row i and one plane after the other
      if constexpr (ROOMY) {
        // PL planes of this lane's row, from `from` on, both halves of the unit
        auto rows = [&](auto planes, bool there, const uint16_t* from) {
          constexpr int PL = decltype(planes)::value;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float s = mx4_scale(mx4_own_scale(w, h, g) & 0xFFu);
            const int b = now.u * kMx4UnitBlocks + 4 * h + g;
            u32x4_t f[PL][4];
#pragma unroll
            for (int i = 0; i < PL * 4; ++i) f[i / 4][i % 4] = u32x4_t{0u, 0u, 0u, 0u};
            if (there && b < now.kb) {
#pragma unroll
              for (int i = 0; i < PL * 4; ++i)
                f[i / 4][i % 4] = load16(from + (i / 4) * now.plane + b * kMx4Block + 8 * (i % 4));
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const bf16x8_t c = mx4_to_bf16(w.half[h][j], s);
#pragma unroll
              for (int p = PL - 1; p >= 0; --p)  // smallest plane first
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, f[p][j]), c, acc, 0, 0, 0);
            }
          }
        };
        if (wide)
          rows(PowC<1>{}, r < 3 * n, now.a + (r % 3) * now.plane + (int64_t)(r < 3 * n ? r / 3 : 0) * now.inter);
        else
          rows(PowC<3>{}, r < n, now.a + (int64_t)(r < n ? r : 0) * now.inter);
      } else {
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
      }
      if (is_far()) {
        // left for the second way
      } else if (wide) {
#pragma unroll
        for (int i = 0; i < 4; ++i) dump[wave][4 * g + i][r] = acc[i];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        for (int i = g; i < n; i += 4) {
          const float v = dump[wave][3 * i + 2][r] + dump[wave][3 * i + 1][r] + dump[wave][3 * i][r];
          tiles[wave][now.en.token(i)][r] += now.weights[i] * v;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      } else {
        add_rows(now, acc, g, r);
      }
    }
    now = next;
    w = wn;
#pragma unroll
    for (int h = 0; h < 2; ++h) one[h] = one_n[h];
  }
  // in a loop of its own, with a lane that the compiler takes for another: inside the
  // first loop, or sharing its addresses, it cost that one registers
  if (__builtin_expect(met_far, 0)) {
    int l = lane;
    asm volatile("" : "+v"(l));
    const int fg = l >> 4, fr = l & 15;
#pragma unroll 1
    for (int id = first; id < tasks; id += stride) {
      const MoeDownTask t = task(id, fr);
      Mx4Unit v;
      mx4_load_unit(t.row, t.kb, t.u, fg, v);
      if (moe_down_any_far(v, fg)) add_rows(t, moe_down_far(t, v, fg, fr), fg, fr);
    }
  }
  __syncthreads();
  const int t = threadIdx.x >> 4, c = threadIdx.x & 15;
  float v = 0.f;
  if (t < q.t) {
#pragma unroll
    for (int o = 0; o < kMoeDownWaves; ++o) v += tiles[o][t][c];
  }
  if (q.down_splits > 1) {
    __shared__ int last;
    const int64_t plane = (int64_t)q.t * H;
    float* p = q.down + t * H + h0 + c;
    if (t < q.t) store_shared(p + blockIdx.y * plane, v);
    wait_stores();
    __syncthreads();
    if (threadIdx.x == 0) last = last_in(q.arrived + 1 + blockIdx.x, (uint32_t)q.down_splits);
    __syncthreads();
    if (!last) return;
    v = 0.f;
    if (t < q.t)
      for (int i = 0; i < q.down_splits; ++i) v += load_shared(p + i * plane);
  }
  if (t < q.t) moe_store(q, t, h0 + c, v);
}

// ---------------------------------------------------------------------------
namespace {
size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

int moe_most(const Mx4MoeDesc& d, int64_t t, int topk) { return (int)(t * topk < d.experts ? t * topk : d.experts); }

// k shares of the router: a wave takes about two matrix instructions, the
// chip's 256 CUs at most one workgroup each.
int moe_splits(const Mx4MoeDesc& d) {
  const int groups = d.experts / 16 + 1, steps = d.hidden / 32;
  int s = steps / 16;
  if (s > 256 / groups) s = 256 / groups;
  return s < 1 ? 1 : (s > 8 ? 8 : s);
}

// Shares of the down product's entries: about a task a wave, where there
// may be so many, and no more than one workgroup a CU (us a call, one / two: 16 tokens,
// 128 entries of 512, hidden 2048 64.2 / 65.6; 14 tokens, 52 of 1248, hidden 608 30.6 /
// 34.8; 5 tokens, 20 of 352, hidden 1440 21.1 / 22.4).
int moe_down_splits(const Mx4MoeDesc& d, int64_t t, int topk) {
  const int units = (d.inter + kMx4UnitK - 1) / kMx4UnitK, tasks = moe_most(d, t, topk) * units;
  const int room = 256 / (d.hidden / 16);
  int s = (tasks + kMoeDownWaves / 2) / kMoeDownWaves;
  if (s > room) s = room;
  return s < 1 ? 1 : s;
}

struct MoeLayout {
  size_t arrived, logits, entries, count, wtab, act[2], down, total;
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
  L.arrived = take((1 + kMoeMaxDim / 16) * 4);  // first and as long in every layout: a workspace serves all sizes
  L.logits = take((size_t)moe_splits(d) * kMoeTokens * L.lstride * 4);
  L.entries = take(most * sizeof(MoeEntry));
  L.count = take(4);
  L.wtab = take(most * kMoeTokens * 4);
  L.act[0] = take((size_t)t * topk * d.inter * 6);
  L.act[1] = take((size_t)t * d.shared_inter * 6);
  const size_t splits = moe_down_splits(d, t, topk);
  L.down = take(splits > 1 ? splits * t * d.hidden * 4 : 0);
  L.total = off;
  return L;
}
}  // namespace

template <int EPL>
static void launch_router(const MoeArgs& q, hipStream_t s) {
  const dim3 grid((uint32_t)((q.d.experts / 16 + 1) * q.splits));
  if (q.t > 8)
    hipLaunchKernelGGL((mx4_moe_router<EPL, 16>), grid, dim3(1024), 0, s, q);
  else
    hipLaunchKernelGGL((mx4_moe_router<EPL, 8>), grid, dim3(512), 0, s, q);
}

size_t mx4_moe_workspace(const Mx4MoeDesc& d, int64_t t, int topk) { return moe_layout(d, t, topk).total; }

hipError_t launch_mx4_moe(const Mx4MoeDesc& d, const uint16_t* x, int64_t t, int64_t ldx, int topk, void* y,
                          int64_t ldy, bool y_f32, int32_t* ids, float* weights, void* ws, hipStream_t s) {
  const MoeLayout L = moe_layout(d, t, topk);
  unsigned char* w = static_cast<unsigned char*>(ws);
  const int most = moe_most(d, t, topk), splits = moe_splits(d);
  const MoeArgs q{d, x, ldx, (int)t, topk, y, ldy, y_f32, ids, weights, most, {(int)t * topk, (int)t}, splits,
                  L.lstride,
                  reinterpret_cast<uint32_t*>(w + L.arrived), reinterpret_cast<float*>(w + L.logits),
                  reinterpret_cast<MoeEntry*>(w + L.entries), reinterpret_cast<int*>(w + L.count),
                  reinterpret_cast<float*>(w + L.wtab),
                  {reinterpret_cast<uint16_t*>(w + L.act[0]), reinterpret_cast<uint16_t*>(w + L.act[1])},
                  moe_down_splits(d, t, topk), reinterpret_cast<float*>(w + L.down)};
  if (d.experts <= 64) launch_router<1>(q, s);
  else if (d.experts <= 128) launch_router<2>(q, s);
  else if (d.experts <= 256) launch_router<4>(q, s);
  else if (d.experts <= 512) launch_router<8>(q, s);
  else launch_router<16>(q, s);
  const int wide = d.inter > d.shared_inter ? d.inter : d.shared_inter;
  // four waves where workgroups are many or k is short, else eight, for fewer turns
  // over k (us a call, four / eight: 16 tokens, 128 entries of 512, hidden 2048 65.6 /
  // 68.7; 1 token, 7 of 256, hidden 576 13.9 / 14.8; 1 token, 8 of 512, hidden 2048 18.5
  // / 17.7, 17.2 with twice the registers; 13 tokens, 13 of 160, hidden 2976 22.9 /
  // 21.6; 16 tokens, 80 of 128, hidden 1440, more than a workgroup a CU, 26.8 with eight,
  // 28.4 with twice the registers)
  const dim3 grid(wide / 16, most + (d.shared_inter ? 1 : 0));
  const int groups = (int)(grid.x * grid.y);
  if (groups >= 1536 || d.hidden <= 1280)
    hipLaunchKernelGGL((mx4_moe_gate_up<4, false>), grid, dim3(256), 0, s, q);
  else if (groups > 256)
    hipLaunchKernelGGL((mx4_moe_gate_up<8, false>), grid, dim3(512), 0, s, q);
  else
    hipLaunchKernelGGL((mx4_moe_gate_up<8, true>), grid, dim3(512), 0, s, q);
  // the same for down (us a call, with twice the registers / without: 14 tokens, 8
  // experts of 704, hidden 128 19.9 / 22.0; 10 tokens, 28 of 96, hidden 480 16.8 / 18.0;
  // 15 tokens, 51 of 128, hidden 4320, more than a workgroup a CU, 40 / 37)
  const dim3 down(d.hidden / 16, q.down_splits);
  if (down.x * down.y <= 256)
    hipLaunchKernelGGL(mx4_moe_down<true>, down, dim3(kMoeDownWaves * 64), 0, s, q);
  else
    hipLaunchKernelGGL(mx4_moe_down<false>, down, dim3(kMoeDownWaves * 64), 0, s, q);
  return hipGetLastError();
}

}  // namespace exl3
