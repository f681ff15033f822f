// exl3_mx4_moe: a whole mixture-of-experts layer for 1 to 16 tokens.
//
//   1. mx4_moe_router  logits x W_r^T, one wave per expert (and the shared
//      expert's gate as one more row)
//   2. mx4_moe_route   one workgroup: a wave per token takes its top-k and
//      weights, then the chosen experts are listed in ascending order, each
//      with the mask of its tokens (an expert is chosen by a token at most
//      once, so 16 tokens fill at most one 16-row matrix operand per expert and
//      every expert's weights are read once)
//   3. mx4_moe_gate_up workgroup (16 columns, listed expert): gate and up over
//      the waves' shares of k, a = silu(g) * u
//   4. mx4_moe_down    workgroup (16 columns): the waves share the listed
//      experts, sums are weighted per expert and meet in LDS in expert order
//
// a is kept as three bf16 pieces (8 + 8 + 8 significand bits, exact to fp32's
// 24), so the down product runs on bf16 matrix instructions against weights
// that are exact in bf16 at any scale byte.
#include "exl3_gemm.hpp"
#include "exl3_internal.hpp"
#include "exl3_mx4_rows.hpp"

namespace exl3 {

constexpr int kMoeTokens = 16;
constexpr int kMoeWaves = 8;
constexpr int kMoeRouteThreads = 1024;
constexpr int kMoeExperts = 1024;
constexpr int kMoeExpertsPerLane = kMoeExperts / 64;

// A chosen expert: its tokens, and the first of their rows in the activations.
struct MoeEntry {
  int e;
  uint32_t mask;
  int row0;
  int pad;
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
  // workspace
  float* logits;      // [16][experts + 1], the last column the shared gate's
  MoeEntry* entries;  // [max_entries + 1]; the routed ones, then the shared expert
  int* count;         // entries in use
  float* wtab;        // [max_entries + 1][16]: weight of (entry, token)
  uint16_t* act[2];   // bf16 [3][rows][inter]: routed pairs, shared expert's tokens
  int rows[2];        // t * topk, t
};

__global__ __launch_bounds__(256) void mx4_moe_router(MoeArgs q) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int E = q.d.experts, H = q.d.hidden;
  const int e = blockIdx.x * 4 + wave;
  if (e > E || (e == E && !q.d.shared_gate)) return;
  const uint16_t* w = e < E ? q.d.router + (int64_t)e * H : q.d.shared_gate;
  float acc[kMoeTokens];
#pragma unroll
  for (int t = 0; t < kMoeTokens; ++t) acc[t] = 0.f;
  for (int k = 8 * lane; k < H; k += 512) {
    const f16x8_t a = __builtin_bit_cast(f16x8_t, load16(w + k));
#pragma unroll
    for (int t = 0; t < kMoeTokens; ++t) {
      if (t < q.t) {
        const f16x8_t b = __builtin_bit_cast(f16x8_t, load16(q.x + t * q.ldx + k));
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[t] = __builtin_fmaf((float)a[i], (float)b[i], acc[t]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < kMoeTokens; ++t) {
    if (t < q.t) {
      float v = acc[t];
      for (int m = 1; m < 64; m <<= 1) v += shfl_xor_f(v, m);
      if (lane == 0) q.logits[t * (E + 1) + e] = v;
    }
  }
}

// Unsigned key in the order of floats, NaN lowest, both zeros equal.
__device__ __forceinline__ uint32_t order_key(float f) {
  if (f != f) return 0u;
  const uint32_t b = __float_as_uint(f + 0.f);
  return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v) {
  for (int m = 1; m < 64; m <<= 1) {
    const uint64_t o = __shfl_xor(v, m);
    v = v > o ? v : o;
  }
  return v;
}
__device__ __forceinline__ float wave_max_f(float v) {
  for (int m = 1; m < 64; m <<= 1) v = fmaxf(v, shfl_xor_f(v, m));
  return v;
}
__device__ __forceinline__ float wave_sum_f(float v) {
  for (int m = 1; m < 64; m <<= 1) v += shfl_xor_f(v, m);
  return v;
}

// Top-k and weights of one token by one wave: slot s ends in lane s (id, w).
__device__ void moe_route_token(const MoeArgs& q, int t, int lane, int& id, float& weight) {
  const int E = q.d.experts;
  const float* l = q.logits + t * (E + 1);
  float score[kMoeExpertsPerLane];
  uint64_t key[kMoeExpertsPerLane];
  float top = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < kMoeExpertsPerLane; ++i) {
    const int e = lane + 64 * i;
    score[i] = 0.f;
    key[i] = 0;
    if (e < E) {
      const float b = q.d.router_bias ? q.d.router_bias[e] : 0.f;
      float choice = l[e];
      if (q.d.scoring == 0) {
        choice += b;
        score[i] = choice;
        top = fmaxf(top, choice);
      } else {
        score[i] = 1.f / (1.f + expf(-choice));
        choice = q.d.router_bias ? score[i] + b : choice;
      }
      key[i] = ((uint64_t)order_key(choice) << 32) | (0xFFFFFFFFu - (uint32_t)e);
    }
  }
  if (q.d.scoring == 0) {
    top = wave_max_f(top);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kMoeExpertsPerLane; ++i)
      if (lane + 64 * i < E) {
        score[i] = expf(score[i] - top);
        sum += score[i];
      }
    sum = wave_sum_f(sum);
#pragma unroll
    for (int i = 0; i < kMoeExpertsPerLane; ++i) score[i] = score[i] / sum;
  }
  id = 0;
  weight = 0.f;
  float total = 0.f;
  for (int s = 0; s < q.topk; ++s) {
    uint64_t best = 0;
#pragma unroll
    for (int i = 0; i < kMoeExpertsPerLane; ++i) best = best > key[i] ? best : key[i];
    best = wave_max_u64(best);
    const int e = (int)(0xFFFFFFFFu - (uint32_t)best);
    float w = 0.f;
#pragma unroll
    for (int i = 0; i < kMoeExpertsPerLane; ++i)
      if (e == lane + 64 * i) {
        w = score[i];
        key[i] = 0;
      }
    w = __shfl(w, e & 63);
    total += w;
    if (lane == s) {
      id = e;
      weight = w;
    }
  }
  if (q.d.renormalize) weight = weight / total;
  weight *= q.d.scale;
}

__global__ __launch_bounds__(kMoeRouteThreads) void mx4_moe_route(MoeArgs q) {
  __shared__ uint32_t masks[kMoeExperts];
  __shared__ int place[kMoeExperts];
  __shared__ int sums[2][kMoeRouteThreads / 64];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  masks[tid] = 0;
  __syncthreads();
  int id = 0;
  float weight = 0.f;
  if (wave < q.t) {
    moe_route_token(q, wave, lane, id, weight);
    if (lane < q.topk) {
      atomicOr(&masks[id], 1u << wave);
      if (q.ids) q.ids[wave * q.topk + lane] = id;
      if (q.weights) q.weights[wave * q.topk + lane] = weight;
    }
  }
  __syncthreads();
  // entries in expert order: thread e counts the chosen experts and the pairs before it
  const uint32_t mask = masks[tid];
  const int pairs = __popc(mask);
  const uint64_t chosen = __ballot(mask != 0);
  int before = __popcll(chosen & ((1ull << lane) - 1));
  int rows = pairs;
  for (int m = 1; m < 64; m <<= 1) {
    const int o = __shfl_up(rows, m);
    if (lane >= m) rows += o;
  }
  if (lane == 63) {
    sums[0][wave] = __popcll(chosen);
    sums[1][wave] = rows;
  }
  __syncthreads();
  int total = 0;
  rows -= pairs;
  for (int w = 0; w < kMoeRouteThreads / 64; ++w) {
    if (w < wave) {
      before += sums[0][w];
      rows += sums[1][w];
    }
    total += sums[0][w];
  }
  if (mask) {
    q.entries[before] = MoeEntry{tid, mask, rows, 0};
    place[tid] = before;
  }
  if (tid == 0) {
    q.count[0] = total;
    q.entries[total] = MoeEntry{-1, (1u << q.t) - 1u, 0, 0};
  }
  __syncthreads();
  if (wave < q.t) {
    if (lane < q.topk) q.wtab[place[id] * kMoeTokens + wave] = weight;
    if (lane == 0) {
      float w = 1.f;
      if (q.d.shared_gate) w = 1.f / (1.f + expf(-q.logits[wave * (q.d.experts + 1) + q.d.experts]));
      q.wtab[total * kMoeTokens + wave] = w;
    }
  }
}

// v as three bf16 pieces by truncation; their sum is v (24 significant bits).
__device__ __forceinline__ void split_bf16(float v, uint16_t (&p)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const uint32_t b = __float_as_uint(v) & 0xFFFF0000u;
    p[i] = (uint16_t)(b >> 16);
    v -= __uint_as_float(b);
  }
}

__global__ __launch_bounds__(kMoeWaves * 64) void mx4_moe_gate_up(MoeArgs q) {
  __shared__ float4_t part[kMoeWaves * 2 * 64];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int g = lane >> 4, r = lane & 15;
  const int count = q.count[0];
  const int entry = blockIdx.y;
  if (entry > count || (entry == count && !q.d.shared_inter)) return;
  const bool shared = entry == count;
  const MoeEntry en = q.entries[entry];
  const int inter = shared ? q.d.shared_inter : q.d.inter;
  const int i0 = blockIdx.x * 16;
  if (i0 >= inter) return;
  const int kb = q.d.hidden / kMx4Block;
  const uint8_t* codes = shared ? q.d.sgu_codes : q.d.gu_codes + (int64_t)en.e * 2 * inter * kb * 16;
  const uint8_t* scales = shared ? q.d.sgu_scales : q.d.gu_scales + (int64_t)en.e * 2 * inter * kb;
  const int64_t row = i0 + r, up = row + inter;
  const bool there = (en.mask >> r) & 1u;
  const uint16_t* x = q.x + (there ? r : 0) * q.ldx;
  float4_t ag[1] = {{0.f, 0.f, 0.f, 0.f}}, au[1] = {{0.f, 0.f, 0.f, 0.f}};
  const int units = (kb + kMx4UnitBlocks - 1) / kMx4UnitBlocks;
  for (int u = wave; u < units; u += kMoeWaves) {
    Mx4Unit wg, wu;
    mx4_load_unit(codes + row * kb * 16, scales + row * kb, kb, u, g, wg);
    mx4_load_unit(codes + up * kb * 16, scales + up * kb, kb, u, g, wu);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      f16x8_t xf[1][4];
      mx4_load_x(x, there, kb, u, h, g, xf[0]);
      mx4_mma_f16<1>(xf, wg, h, ag);
      mx4_mma_f16<1>(xf, wu, h, au);
    }
  }
  part[(wave * 2 + 0) * 64 + lane] = ag[0];
  part[(wave * 2 + 1) * 64 + lane] = au[0];
  __syncthreads();
  if (wave != 0) return;
  float4_t vg = part[lane], vu = part[64 + lane];
#pragma unroll
  for (int w = 1; w < kMoeWaves; ++w) {
    vg += part[w * 128 + lane];
    vu += part[w * 128 + 64 + lane];
  }
  uint16_t* act = q.act[shared];
  const int64_t plane = (int64_t)q.rows[shared] * inter;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = 4 * g + i;
    if (!((en.mask >> t) & 1u)) continue;
    uint16_t p[3];
    split_bf16(vg[i] / (1.0f + expf(-vg[i])) * vu[i], p);
    uint16_t* o = act + (int64_t)(en.row0 + __popc(en.mask & ((1u << t) - 1u))) * inter + i0 + r;
    o[0] = p[0];
    o[plane] = p[1];
    o[2 * plane] = p[2];
  }
}

__global__ __launch_bounds__(kMoeWaves * 64) void mx4_moe_down(MoeArgs q) {
  __shared__ float4_t part[kMoeWaves * 64];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int g = lane >> 4, r = lane & 15;
  const int h0 = blockIdx.x * 16, H = q.d.hidden;
  const int count = q.count[0] + (q.d.shared_inter ? 1 : 0);
  const int routed = q.count[0];
  float4_t total = {0.f, 0.f, 0.f, 0.f};
  for (int entry = wave; entry < count; entry += kMoeWaves) {
    const bool shared = entry == routed;
    const MoeEntry en = q.entries[entry];
    const int inter = shared ? q.d.shared_inter : q.d.inter;
    const int kb = inter / kMx4Block;
    const int64_t row = (shared ? 0 : (int64_t)en.e * H) + h0 + r;
    const uint8_t* codes = (shared ? q.d.sdn_codes : q.d.dn_codes) + row * kb * 16;
    const uint8_t* scales = (shared ? q.d.sdn_scales : q.d.dn_scales) + row * kb;
    const bool there = (en.mask >> r) & 1u;
    const uint16_t* a = q.act[shared] +
                        (int64_t)(en.row0 + (there ? __popc(en.mask & ((1u << r) - 1u)) : 0)) * inter;
    const int64_t plane = (int64_t)q.rows[shared] * inter;
    float4_t acc = {0.f, 0.f, 0.f, 0.f};
    const int units = (kb + kMx4UnitBlocks - 1) / kMx4UnitBlocks;
    for (int u = 0; u < units; ++u) {
      Mx4Unit w;
      mx4_load_unit(codes, scales, kb, u, g, w);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int b = u * kMx4UnitBlocks + 4 * h + g;  // this lane's block
        const float s = mx4_scale(mx4_own_scale(w, h, g) & 0xFFu);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bf16x8_t wf = mx4_to_bf16(w.half[h][j], s);
#pragma unroll
          for (int p = 0; p < 3; ++p) {
            u32x4_t v = {0u, 0u, 0u, 0u};
            if (there && b < kb) v = load16(a + p * plane + b * kMx4Block + 8 * j);
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, v), wf, acc, 0, 0, 0);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 4 * g + i;
      if ((en.mask >> t) & 1u) total[i] = __builtin_fmaf(q.wtab[entry * kMoeTokens + t], acc[i], total[i]);
    }
  }
  part[wave * 64 + lane] = total;
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int w = 1; w < kMoeWaves; ++w) total += part[w * 64 + lane];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = 4 * g + i;
    if (t >= q.t) break;
    const int64_t at = t * q.ldy + h0 + r;
    if (q.y_f32)
      static_cast<float*>(q.y)[at] = total[i];
    else
      static_cast<uint16_t*>(q.y)[at] = f2h(total[i]);
  }
}

namespace {
size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }
struct MoeLayout {
  size_t logits, entries, count, wtab, act[2], total;
};
MoeLayout moe_layout(const Mx4MoeDesc& d, int64_t t, int topk) {
  const size_t most = (size_t)(t * topk < d.experts ? t * topk : d.experts) + 1;
  MoeLayout L;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += align256(bytes);
    return at;
  };
  L.logits = take((size_t)kMoeTokens * (d.experts + 1) * 4);
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
  MoeArgs q{d, x, ldx, (int)t, topk, y, ldy, y_f32, ids, weights,
            reinterpret_cast<float*>(w + L.logits), reinterpret_cast<MoeEntry*>(w + L.entries),
            reinterpret_cast<int*>(w + L.count), reinterpret_cast<float*>(w + L.wtab),
            {reinterpret_cast<uint16_t*>(w + L.act[0]), reinterpret_cast<uint16_t*>(w + L.act[1])},
            {(int)t * topk, (int)t}};
  const int most = (int)(t * topk < d.experts ? t * topk : d.experts) + (d.shared_inter ? 1 : 0);
  const int wide = d.inter > d.shared_inter ? d.inter : d.shared_inter;
  hipLaunchKernelGGL(mx4_moe_router, dim3(d.experts / 4 + 1), dim3(256), 0, s, q);
  hipLaunchKernelGGL(mx4_moe_route, dim3(1), dim3(kMoeRouteThreads), 0, s, q);
  hipLaunchKernelGGL(mx4_moe_gate_up, dim3(wide / 16, most), dim3(kMoeWaves * 64), 0, s, q);
  hipLaunchKernelGGL(mx4_moe_down, dim3(d.hidden / 16), dim3(kMoeWaves * 64), 0, s, q);
  return hipGetLastError();
}

}  // namespace exl3
