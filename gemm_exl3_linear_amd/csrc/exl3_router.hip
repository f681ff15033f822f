// exl3_router_linear and exl3_router: a router's logits l = x W^T (+ c), fp16 matrix
// instructions with fp32 sums, and for few tokens their routing in the same launch.
#include "exl3_mx4.hpp"
#include "exl3_route.hpp"

namespace exl3 {

constexpr int kRouterRows = 16;           // of an operand
constexpr int kRouterCounts = 128;        // arrival counts at the head of a workspace: one a group of 16 experts,
                                          // and the routing's
constexpr int kRouterWaves = 8;

struct RouterArgs {
  RouterDesc d;
  const uint16_t* x;
  int64_t t, ldx;
  float* logits;  // may be null where the routing takes the sums
  int64_t ldl;
  int splits;
  uint32_t* arrived;  // 0 between calls
  float* part;        // [splits][t][estride], with several splits or the routing
  int estride;
  RouteRule rule;
  int32_t* ids;
  float* weights;
};

// Sums of 16 experts (blockIdx.x / splits) for 16 tokens (from blockIdx.y on) over a
// share of hidden.  VPL > 0: the last workgroup to arrive routes every token, expert 64 i +
// lane at a lane's i-th place.
template <int VPL, int K>
__global__ __launch_bounds__(kRouterWaves * 64) void router_rows_kernel(RouterArgs q) {
  constexpr bool kRoutes = VPL > 0;
  constexpr int kV = kRoutes ? VPL : 1;
  __shared__ float4_t sums[kRouterWaves * 64];
  __shared__ RouteLds<64, kV> lds[kRoutes ? kRouterWaves : 1];
  __shared__ int last;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int g = lane >> 4, r = lane & 15;
  const int group = blockIdx.x / q.splits, split = blockIdx.x - group * q.splits;
  const int e = group * 16 + r;
  for (int64_t row0 = (int64_t)blockIdx.y * kRouterRows; row0 < q.t; row0 += (int64_t)gridDim.y * kRouterRows) {
    const bool row_there = row0 + r < q.t, e_there = e < q.d.experts;
    const uint16_t* x = q.x + (row_there ? (row0 + r) * q.ldx : 0);
    const uint16_t* w = q.d.weight + (e_there ? (int64_t)e * q.d.hidden : 0);
    float4_t acc = {0.f, 0.f, 0.f, 0.f};
    const int stride = kRouterWaves * q.splits;
    for (int st = split * kRouterWaves + wave; 32 * st < q.d.hidden; st += 4 * stride) {
      u32x4_t a[4], b[4];  // four steps' loads at a time
  #pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = 32 * (st + i * stride) + 8 * g;
        a[i] = b[i] = u32x4_t{0u, 0u, 0u, 0u};
        if (row_there && at < q.d.hidden) a[i] = load16(x + at);
        if (e_there && at < q.d.hidden) b[i] = load16(w + at);
      }
  #pragma unroll
      for (int i = 0; i < 4; ++i)
        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a[i]), __builtin_bit_cast(f16x8_t, b[i]),
                                                     acc, 0, 0, 0);
    }
    sums[wave * 64 + lane] = acc;
    __syncthreads();
    if (wave == 0) {
  #pragma unroll
      for (int o = 1; o < kRouterWaves; ++o) acc += sums[o * 64 + lane];
      const bool whole = q.splits == 1 && !kRoutes;
      const float c = whole && q.d.bias && e_there ? q.d.bias[e] : 0.f;
  #pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t row = row0 + 4 * g + i;
        if (!e_there || row >= q.t) continue;
        if (whole) q.logits[row * q.ldl + e] = acc[i] + c;
        else store_shared(q.part + ((int64_t)split * q.t + row) * q.estride + e, acc[i]);
      }
      if (!whole) {
        wait_stores();
        if (lane == 0) last = kRoutes ? last_in(q.arrived, gridDim.x) : last_in(q.arrived + 1 + group, q.splits);
      }
    }
    if (kRoutes || q.splits > 1) break;  // all tokens are in one tile
    __syncthreads();
  }
  if (q.splits == 1 && !kRoutes) return;
  __syncthreads();
  if (!last) return;
  const auto sum = [&](int64_t row, int expert) {
    const float* p = q.part + row * q.estride + expert;
    float l = 0.f;
#pragma unroll 4
    for (int k = 0; k < q.splits; ++k) l += load_shared(p + (int64_t)k * q.t * q.estride);
    return q.d.bias ? l + q.d.bias[expert] : l;
  };
  if constexpr (!kRoutes) {
    for (int i = threadIdx.x; i < (int)q.t * 16; i += kRouterWaves * 64)
      if (const int o = group * 16 + (i & 15); o < q.d.experts) q.logits[(i >> 4) * q.ldl + o] = sum(i >> 4, o);
  } else {
    for (int row = wave; row < (int)q.t; row += kRouterWaves) {
      float l[kV];
#pragma unroll
      for (int i = 0; i < kV; ++i) l[i] = 64 * i + lane < q.d.experts ? sum(row, 64 * i + lane) : 0.f;
      if (q.logits)
#pragma unroll
        for (int i = 0; i < kV; ++i)
          if (64 * i + lane < q.d.experts) q.logits[row * q.ldl + 64 * i + lane] = l[i];
      int id;
      float weight;
      route_token<64, kV, K>(q.rule, l, lane, lds + wave, id, weight);
      if (lane < q.rule.topk) {
        q.ids[(int64_t)row * q.rule.topk + lane] = id;
        q.weights[(int64_t)row * q.rule.topk + lane] = weight;
      }
    }
  }
}

namespace {

constexpr int kFewTokens = 16;  // of which one launch makes the logits and routes them

int router_splits(const RouterDesc& d, int64_t t) {
  if (t > kFewTokens) return 1;
  const int groups = (d.experts + 15) / 16;
  const int most = (d.hidden + 32 * kRouterWaves * 4 - 1) / (32 * kRouterWaves * 4);
  const int want = (256 + groups - 1) / groups;
  return want < most ? want : most;
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }
int router_estride(const RouterDesc& d) { return (d.experts + 15) / 16 * 16; }
size_t router_parts(const RouterDesc& d, int64_t t, int splits) {
  return align256((size_t)splits * t * router_estride(d) * 4);
}

RouterArgs router_args(const RouterDesc& d, const uint16_t* x, int64_t t, int64_t ldx, float* logits, int64_t ldl,
                       void* ws) {
  RouterArgs q{};
  q.d = d;
  q.x = x;
  q.t = t;
  q.ldx = ldx;
  q.logits = logits;
  q.ldl = ldl;
  q.splits = router_splits(d, t);
  q.arrived = static_cast<uint32_t*>(ws);
  q.part = reinterpret_cast<float*>(static_cast<unsigned char*>(ws) + kRouterCounts * 4);
  q.estride = router_estride(d);
  return q;
}

dim3 router_grid(const RouterArgs& q) {
  const int64_t tiles = (q.t + kRouterRows - 1) / kRouterRows;
  return dim3((uint32_t)((q.d.experts + 15) / 16 * q.splits), (uint32_t)(tiles < 65535 ? tiles : 65535));
}

template <int VPL>
void launch_fused(const RouterArgs& q, hipStream_t s) {
  const dim3 grid = router_grid(q), block(kRouterWaves * 64);
  if (q.rule.topk <= 4) hipLaunchKernelGGL((router_rows_kernel<VPL, 4>), grid, block, 0, s, q);
  else if (q.rule.topk <= 8) hipLaunchKernelGGL((router_rows_kernel<VPL, 8>), grid, block, 0, s, q);
  else hipLaunchKernelGGL((router_rows_kernel<VPL, 16>), grid, block, 0, s, q);
}

}  // namespace

size_t router_linear_workspace(const RouterDesc& d, int64_t t) {
  const int splits = router_splits(d, t);
  return splits > 1 ? kRouterCounts * 4 + router_parts(d, t, splits) : 0;
}

// Bytes ahead of what else a workspace holds: the counts are never written over.
static size_t router_head(const RouterDesc& d, int64_t t) {
  const size_t linear = router_linear_workspace(d, t);
  return linear ? linear : kRouterCounts * 4;
}

hipError_t launch_router_linear(const RouterDesc& d, const uint16_t* x, int64_t t, int64_t ldx, float* logits,
                                int64_t ldl, void* ws, hipStream_t s) {
  const RouterArgs q = router_args(d, x, t, ldx, logits, ldl, ws);
  hipLaunchKernelGGL((router_rows_kernel<0, 1>), router_grid(q), dim3(kRouterWaves * 64), 0, s, q);
  return hipGetLastError();
}

size_t router_workspace(const RouterDesc& d, int64_t t, bool logits) {
  if (t <= kFewTokens) return kRouterCounts * 4 + router_parts(d, t, router_splits(d, t));
  return logits ? router_linear_workspace(d, t) : router_head(d, t) + router_parts(d, t, 1);
}

hipError_t launch_router(const RouterDesc& d, const RouteRule& rule, const uint16_t* x, int64_t t, int64_t ldx,
                         float* logits, int64_t ldl, int32_t* ids, float* weights, void* ws, hipStream_t s) {
  if (t > kFewTokens) {
    if (!logits) {
      logits = reinterpret_cast<float*>(static_cast<unsigned char*>(ws) + router_head(d, t));
      ldl = router_estride(d);
    }
    const hipError_t e = launch_router_linear(d, x, t, ldx, logits, ldl, ws, s);
    return e != hipSuccess ? e : launch_route_topk(rule, logits, true, t, ldl, ids, weights, s);
  }
  RouterArgs q = router_args(d, x, t, ldx, logits, ldl, ws);
  q.rule = rule;
  q.ids = ids;
  q.weights = weights;
  if (d.experts <= 64) launch_fused<1>(q, s);
  else if (d.experts <= 128) launch_fused<2>(q, s);
  else if (d.experts <= 256) launch_fused<4>(q, s);
  else if (d.experts <= 512) launch_fused<8>(q, s);
  else launch_fused<16>(q, s);
  return hipGetLastError();
}

}  // namespace exl3
