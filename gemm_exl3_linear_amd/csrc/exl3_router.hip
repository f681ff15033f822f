// exl3_router_linear and exl3_router: a router's logits l = x W^T (+ c), fp16 matrix
// instructions with fp32 sums, and their routing: in the same launch for a token or a few,
// else in a second one, which also adds the shares of k.
#include "exl3_route.hpp"
#include "exl3_tile64.hpp"

namespace exl3 {

constexpr int kRouterRows = 16;     // of an operand
constexpr int kRouterCounts = 128;  // arrival counts at the head of a workspace: one a group of 16 experts, and the
                                    // routing's
constexpr int kRouterWaves = 8;
constexpr int kRouterShares = 16;  // of k at most

struct RouterArgs {
  RouterDesc d;
  const uint16_t* x;
  int64_t t, ldx;
  float* logits;  // may be null where the routing takes the sums
  int64_t ldl;
  int splits;         // shares of hidden
  uint32_t* arrived;  // 0 between calls
  float* part;        // [splits][t][estride], with several splits or the routing
  int estride;
  RouteRule rule;
  int32_t* ids;
  float* weights;
};

// What becomes of the sums: logits, or shares of k in `part` for another launch; shares
// that the last workgroup of their experts adds (one tile of tokens); shares that the last
// workgroup of all adds and routes.
enum class RouterEnd { kStore, kAdd, kRoute };

// Sums of 16 experts (blockIdx.x / splits) for 16 tokens (from blockIdx.y on) over a
// share of hidden.  END == kRoute: at most 64 VPL experts, topk <= K.  kAdd and kRoute: one
// tile of tokens (gridDim.y is 1).  Small calls, bound by a chain of latencies: 333 x 1440
// x 60 in 4.9 us; one token's 2048 x 256 with its routing in 7.6, of which the way of the
// sums to the last workgroup takes 2 and the routing 1.5.
template <RouterEnd END, int VPL, int K>
__global__ __launch_bounds__(kRouterWaves * 64) void router_rows_kernel(RouterArgs q) {
  constexpr bool kRoutes = END == RouterEnd::kRoute;
  __shared__ float4_t sums[kRouterWaves * 64];
  __shared__ RouteLds<64, VPL> lds[kRoutes ? kRouterWaves : 1];
  __shared__ int last;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int g = lane >> 4, r = lane & 15;
  const int group = blockIdx.x / q.splits, split = blockIdx.x - group * q.splits;
  const int e = group * 16 + r;
  const bool e_there = e < q.d.experts;
  const uint16_t* w = q.d.weight + (e_there ? (int64_t)e * q.d.hidden : 0);
  const int stride = kRouterWaves * q.splits;
  for (int64_t row0 = (int64_t)blockIdx.y * kRouterRows; row0 < q.t; row0 += (int64_t)gridDim.y * kRouterRows) {
    const bool row_there = row0 + r < q.t;
    const uint16_t* x = q.x + (row_there ? (row0 + r) * q.ldx : 0);
    float4_t acc = {0.f, 0.f, 0.f, 0.f};
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
        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a[i]),
                                                     __builtin_bit_cast(f16x8_t, b[i]), acc, 0, 0, 0);
    }
    sums[wave * 64 + lane] = acc;
    __syncthreads();
    if (wave == 0) {
#pragma unroll
      for (int o = 1; o < kRouterWaves; ++o) acc += sums[o * 64 + lane];
      const bool whole = END == RouterEnd::kStore && q.splits == 1;
      const float c = whole && q.d.bias && e_there ? q.d.bias[e] : 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t row = row0 + 4 * g + i;
        if (!e_there || row >= q.t) continue;
        float* part = q.part + ((int64_t)split * q.t + row) * q.estride + e;
        if (whole) q.logits[row * q.ldl + e] = acc[i] + c;
        else if (END == RouterEnd::kStore) *part = acc[i];
        else store_shared(part, acc[i]);
      }
      if (END != RouterEnd::kStore) {
        wait_stores();
        if (lane == 0) last = kRoutes ? last_in(q.arrived, gridDim.x) : last_in(q.arrived + 1 + group, q.splits);
      }
    }
    __syncthreads();
  }
  if (END == RouterEnd::kStore || !last) return;
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
      float l[VPL];
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int o = route_expert<64, VPL>(i, lane);
        l[i] = o < q.d.experts ? sum(row, o) : 0.f;
      }
      if (q.logits)
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if (const int o = route_expert<64, VPL>(i, lane); o < q.d.experts) q.logits[row * q.ldl + o] = l[i];
      int id;
      float weight;
      route_token<64, VPL, K>(q.rule, l, lane, lds + wave, [&](int e) { return route_held<VPL>(l, e); }, id, weight);
      if (lane < q.rule.topk) {
        q.ids[(int64_t)row * q.rule.topk + lane] = id;
        q.weights[(int64_t)row * q.rule.topk + lane] = weight;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// many tokens
// ---------------------------------------------------------------------------
// 64 tokens x 64 experts over a share of k (blockIdx.y): exl3_tile64.hpp.  4096 x 5120 x
// 256 in 20 to 22 us (0.5 PFLOP/s), of which the 335 MB that 256 CUs copy to LDS take 17
// by themselves, and as long to registers.  (Larger tiles halve them; 128 x 128 makes 64
// workgroups of that product, so that three CUs of four are idle or shares of k are to be
// added.)
__global__ __launch_bounds__(kTile64Waves * 64) void router_gemm_kernel(RouterArgs q) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kTile64Lds];
  // a row tile's workgroups run on one XCD (workgroup i on XCD i % 8), one behind the
  // other, so that x comes from memory once; those of the last down % 8 row tiles as they
  // come, with no empty one between (which would hold a CU's LDS for a microsecond)
  const uint32_t across = (q.d.experts + kTile64 - 1) / kTile64, down = gridDim.x / across, whole8 = down / 8 * 8;
  const uint32_t rest = blockIdx.x - whole8 * across;  // wraps before them
  const bool last = blockIdx.x >= whole8 * across;
  const uint32_t j = blockIdx.x >> 3;
  const int64_t row0 = (int64_t)(last ? whole8 + rest % (down - whole8) : j / across * 8 + (blockIdx.x & 7)) * kTile64;
  const int e0 = (int)(last ? rest / (down - whole8) : j % across) * kTile64;
  const int rows = (int)(q.t - row0 < kTile64 ? q.t - row0 : kTile64);
  const int cols = q.d.experts - e0 < kTile64 ? q.d.experts - e0 : kTile64;
  const uint32_t hidden = (uint32_t)q.d.hidden;
  const u32x4_t rsrc[2] = {buffer_words(reinterpret_cast<const uint8_t*>(q.x + row0 * q.ldx),
                                        ((uint64_t)(rows - 1) * q.ldx + hidden) * 2),
                           buffer_words(reinterpret_cast<const uint8_t*>(q.d.weight + (int64_t)e0 * hidden),
                                        (uint64_t)cols * hidden * 2)};
  uint32_t row[2][2];  // past the last: past the buffer's end
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    row[0][i] = tile64_row(i) * (uint32_t)q.ldx * 2;
    row[1][i] = tile64_row(i) * hidden * 2;
  }
  const int stages = (int)((hidden + kTile64K - 1) / kTile64K);
  const float* sums = tile64_sums(rsrc, row, hidden, (int)((int64_t)stages * blockIdx.y / q.splits),
                                  (int)((int64_t)stages * (blockIdx.y + 1) / q.splits), lds);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  if (lane >= cols) return;
  const bool whole = q.splits == 1;
  const float bias = whole && q.d.bias ? q.d.bias[e0 + lane] : 0.f;
  float* out = whole ? q.logits + row0 * q.ldl : q.part + ((int64_t)blockIdx.y * q.t + row0) * q.estride;
  const int64_t ld = whole ? q.ldl : q.estride;
#pragma unroll 4
  for (int i = wave; i < rows; i += kTile64Waves) out[i * ld + e0 + lane] = tile64_sum(sums, i, lane) + bias;
}

// The logits of shares of k: a thread takes four experts of a token.
__global__ __launch_bounds__(256) void router_sum_kernel(RouterArgs q) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int across = q.estride / 4;
  const int64_t row = i / across;
  const int e = (int)(i - row * across) * 4;
  if (row >= q.t) return;
  const float* p = q.part + row * q.estride + e;
  float4_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int k = 0; k < q.splits; ++k) v += *reinterpret_cast<const float4_t*>(p + (int64_t)k * q.t * q.estride);
#pragma unroll
  for (int o = 0; o < 4; ++o)
    if (e + o < q.d.experts) q.logits[row * q.ldl + e + o] = v[o] + (q.d.bias ? q.d.bias[e + o] : 0.f);
}

namespace {

// Who adds shares of k: a launch of its own, or, for a tile of tokens, their last workgroup
// (exl3_router_linear); the routing's launch (exl3_router); the routing in the same launch.
enum class RouterJoin { kLinear, kRouted, kFused };

// A product's cut: shares of k, 16 x 16 by router_rows_kernel or 64 x 64 by
// router_gemm_kernel.
struct RouterCut {
  bool tiled;
  int splits;
};

// Routed by the launch that makes the logits: the last workgroup's waves route a token
// after the other (us of 2048 hidden, calls one behind the other, fused / in two launches,
// which the host bounds: 256 experts, 1 token 7.1 / 9.5, 4 7.5 / 9.1, 8 9.2 / 9.5, 16 12.9 /
// 9.4; 64 experts, 16 tokens 9.2 / 9.5.  In a graph, where the host has no part, 7.2 / 6.1,
// 7.6 / 6.7, 9.4 / 6.8, 13.1 / 6.9 and 9.3 / 6.5).  One tile of tokens: the arrivals that
// make a workgroup the last are counted over the experts and shares of one.
bool router_fused(const RouterDesc& d, int64_t t) {
  return t <= kRouterRows && d.experts <= 256 && t * d.experts <= 1024;
}

// The cut by estimates in us, fitted to kernels alone, and measured where they meet
// (tokens x hidden x experts, by rows / tiled, shares in brackets): 64 x 5120 x 256 8.1
// (8) / 8.8 (8), 256 13.0 (1) / 9.6 (8), 1000 38 (1) / 14.0 (4); 17 x 5120 x 1000 9.3 (4) /
// 8.5 (8), 512 75 (1) / 21 (2); 1000 x 2048 x 60 7.2 (1) / 9.0 (8), 2000 10.6 (1) / 9.3 (1).
// Over 203 shapes of 17 to 8000 tokens 1.1 % from each shape's best on average, 15 % at
// most; routed, 293 shapes from one token on, 0.6 and 18 %.
RouterCut router_cut(const RouterDesc& d, int64_t t, int64_t ldx, RouterJoin join) {
  const int64_t groups = (d.experts + 15) / 16, rows = (t + kRouterRows - 1) / kRouterRows;
  const auto joined = [&](int splits) {
    if (splits == 1) return 0.0;
    if (join == RouterJoin::kFused) return 0.3 * splits;
    const double moved = splits * (double)t * d.experts * 8 / 4.5e6;
    if (join == RouterJoin::kRouted)  // many tokens are else routed by 16 lanes each
      return 0.3 + 0.15 * splits + 0.002 * d.experts + moved + (t > kRouteFew ? 1e-3 * t : 0.0);
    return t <= kRouterRows ? 1.0 + 0.1 * splits : 4.5 + moved;
  };
  RouterCut best{false, 1};
  double cost = 1e30;
  // by rows: 16 bytes a clock and CU of operands that are loaded as they are multiplied,
  // 9.6 TB/s of all; shares of 256 k at least, a load a wave
  const double all = groups * rows * 64.0 * d.hidden / 9.6e6;
  for (int splits = 1; splits <= kRouterShares && (splits == 1 || splits * 256 <= d.hidden); splits *= 2) {
    const double lone = 1.7 / 1024 * d.hidden / splits;
    const double c = 2.5 + (lone > all ? lone : all) + joined(splits);
    if (c < cost) {
      cost = c;
      best = {false, splits};
    }
  }
  if (ldx >= (1 << 24) || t <= kRouterRows) return best;  // offsets into 64 rows have 32 bits
  // tiled: 0.36 a stage and round of a workgroup a CU; of fewer stages than the ring's a
  // share is all latency
  const int64_t tiles = (t + kTile64 - 1) / kTile64 * ((d.experts + kTile64 - 1) / kTile64);
  const int stages = (d.hidden + kTile64K - 1) / kTile64K;
  for (int splits = 1; splits <= kRouterShares && (splits == 1 || splits * kTile64Ring <= stages); splits *= 2) {
    const double rounds = (double)((tiles * splits + 255) / 256);
    const double c = 3.0 + 0.36 * ((stages + splits - 1) / splits) * rounds + joined(splits);
    if (c < cost) {
      cost = c;
      best = {true, splits};
    }
  }
  return best;
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }
int router_estride(const RouterDesc& d) { return (d.experts + 15) / 16 * 16; }
size_t router_parts(const RouterDesc& d, int64_t t, int splits) {
  return align256((size_t)splits * t * router_estride(d) * 4);
}

// Bytes of a call of any ldx: far rows are cut by rows, in as many shares or fewer.
size_t router_bytes(const RouterDesc& d, int64_t t, RouterJoin join) {
  const int near = router_cut(d, t, 0, join).splits, far = router_cut(d, t, 1 << 24, join).splits;
  const int splits = near > far ? near : far;
  return splits == 1 && join != RouterJoin::kFused ? 0 : kRouterCounts * 4 + router_parts(d, t, splits);
}

// The counts at a workspace's head are never written over.
RouterArgs router_args(const RouterDesc& d, const uint16_t* x, int64_t t, int64_t ldx, float* logits, int64_t ldl,
                       void* ws) {
  RouterArgs q{};
  q.d = d;
  q.x = x;
  q.t = t;
  q.ldx = ldx;
  q.logits = logits;
  q.ldl = ldl;
  q.arrived = static_cast<uint32_t*>(ws);
  q.part = reinterpret_cast<float*>(static_cast<unsigned char*>(ws) + kRouterCounts * 4);
  q.estride = router_estride(d);
  return q;
}

dim3 router_grid(const RouterArgs& q) {
  const int64_t tiles = (q.t + kRouterRows - 1) / kRouterRows;
  return dim3((uint32_t)((q.d.experts + 15) / 16 * q.splits), (uint32_t)(tiles < 65535 ? tiles : 65535));
}

// The logits, or shares of them in q.part; true if those are left to be added.
bool launch_product(RouterArgs& q, RouterJoin join, hipStream_t s) {
  const RouterCut cut = router_cut(q.d, q.t, q.ldx, join);
  q.splits = cut.splits;
  if (cut.tiled) {
    const int64_t down = (q.t + kTile64 - 1) / kTile64, across = (q.d.experts + kTile64 - 1) / kTile64;
    const dim3 grid((uint32_t)(down * across), (uint32_t)q.splits);
    hipLaunchKernelGGL(router_gemm_kernel, grid, dim3(kTile64Waves * 64), 0, s, q);
    return q.splits > 1;
  }
  const dim3 block(kRouterWaves * 64);
  if (q.splits > 1 && join == RouterJoin::kLinear && q.t <= kRouterRows) {
    hipLaunchKernelGGL((router_rows_kernel<RouterEnd::kAdd, 1, 1>), router_grid(q), block, 0, s, q);
    return false;
  }
  hipLaunchKernelGGL((router_rows_kernel<RouterEnd::kStore, 1, 1>), router_grid(q), block, 0, s, q);
  return q.splits > 1;
}

template <int VPL>
void launch_fused(RouterArgs& q, hipStream_t s) {
  q.splits = router_cut(q.d, q.t, q.ldx, RouterJoin::kFused).splits;
  const dim3 grid = router_grid(q), block(kRouterWaves * 64);
  if (q.rule.topk <= 4) hipLaunchKernelGGL((router_rows_kernel<RouterEnd::kRoute, VPL, 4>), grid, block, 0, s, q);
  else if (q.rule.topk <= 8) hipLaunchKernelGGL((router_rows_kernel<RouterEnd::kRoute, VPL, 8>), grid, block, 0, s, q);
  else hipLaunchKernelGGL((router_rows_kernel<RouterEnd::kRoute, VPL, 16>), grid, block, 0, s, q);
}

}  // namespace

size_t router_linear_workspace(const RouterDesc& d, int64_t t) { return router_bytes(d, t, RouterJoin::kLinear); }

hipError_t launch_router_linear(const RouterDesc& d, const uint16_t* x, int64_t t, int64_t ldx, float* logits,
                                int64_t ldl, void* ws, hipStream_t s) {
  RouterArgs q = router_args(d, x, t, ldx, logits, ldl, ws);
  if (launch_product(q, RouterJoin::kLinear, s))
    hipLaunchKernelGGL(router_sum_kernel, dim3((uint32_t)((t * (q.estride / 4) + 255) / 256)), dim3(256), 0, s, q);
  return hipGetLastError();
}

size_t router_workspace(const RouterDesc& d, int64_t t, bool logits) {
  if (router_fused(d, t)) return router_bytes(d, t, RouterJoin::kFused);
  const size_t shares = router_bytes(d, t, RouterJoin::kRouted);
  const size_t whole = logits ? 0 : kRouterCounts * 4 + router_parts(d, t, 1);  // logits of its own
  return shares > whole ? shares : whole;
}

hipError_t launch_router(const RouterDesc& d, const RouteRule& rule, const uint16_t* x, int64_t t, int64_t ldx,
                         float* logits, int64_t ldl, int32_t* ids, float* weights, void* ws, hipStream_t s) {
  RouterArgs q = router_args(d, x, t, ldx, logits, ldl, ws);
  if (router_fused(d, t)) {
    q.rule = rule;
    q.ids = ids;
    q.weights = weights;
    if (d.experts <= 64) launch_fused<1>(q, s);
    else if (d.experts <= 128) launch_fused<2>(q, s);
    else launch_fused<4>(q, s);
    return hipGetLastError();
  }
  if (!logits) {  // where they are not left as shares
    q.logits = q.part;
    q.ldl = q.estride;
  }
  if (launch_product(q, RouterJoin::kRouted, s)) {
    const RouteParts parts{q.part, q.splits, q.estride, d.bias, logits, ldl};
    return launch_route_parts(rule, parts, t, ids, weights, s);
  }
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? e : launch_route_topk(rule, q.logits, true, t, q.ldl, ids, weights, s);
}

}  // namespace exl3
