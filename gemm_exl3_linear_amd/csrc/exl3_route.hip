// exl3_route_topk: choices and weights of every token from its logits.
//
// Many tokens of up to 256 experts take 16 lanes each: a wave's instructions are what
// they cost (a merge of two lists of eight is 56 of them), and four tokens share them.
// Few tokens wait for one wave's instructions, and for their way from memory: they take
// a wave each, whose lanes hold a quarter of the values.
// Measured (us of a call in a graph of 20, a wave / 16 lanes a token, 8 of 256 experts):
// softmax, 1 token 2.8 / 3.3, 2048 4.2 / 3.8, 4096 6.2 / 3.8, 16384 18.5 / 7.5; balanced
// sigmoids in 8 groups 4.5 / 6.6, 6.0 / 7.1, 8.8 / 7.2, 24.8 / 14.6; 4 of 60 experts, 2048
// tokens 3.1 / 2.7, 16384 9.8 / 3.9.
#include "exl3_mx4.hpp"
#include "exl3_route.hpp"

namespace exl3 {

constexpr int kRouteWaves = 4;

template <int LANES, int VPL, int K, class T>
__global__ __launch_bounds__(kRouteWaves * 64) void route_topk_kernel(RouteRule q, const T* logits, int vec, int64_t t,
                                                                      int64_t ldl, int32_t* ids, float* weights) {
  constexpr int kTokens = kRouteWaves * 64 / LANES;  // of a workgroup
  constexpr int V = VPL < 4 ? VPL : 4;
  typedef T four __attribute__((ext_vector_type(V)));
  __shared__ RouteLds<LANES, VPL> lds[kTokens];
  const int token = threadIdx.x / LANES, lane = threadIdx.x % LANES;
  const int64_t row = (int64_t)blockIdx.x * kTokens + token;
  const T* p = logits + (row < t ? row : t - 1) * ldl;  // past the last: it again, and nothing is stored
  float l[VPL];
#pragma unroll
  for (int i = 0; i < VPL; i += V) {
    const int e = route_expert<LANES, VPL>(i, lane);
    if (vec) {  // experts and rows are whole fours, so that one holds all or none
      const four f = *reinterpret_cast<const four*>(p + (e < q.experts ? e : 0));
#pragma unroll
      for (int j = 0; j < V; ++j) l[i + j] = (float)f[j];
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) l[i + j] = (float)p[e + j < q.experts ? e + j : 0];
    }
  }
  int id;
  float weight;
  route_token<LANES, VPL, K>(q, l, lane, lds + token, [&](int e) { return (float)p[e]; }, id, weight);
  if (lane < q.topk && row < t) {
    ids[row * q.topk + lane] = id;
    weights[row * q.topk + lane] = weight;
  }
}

// The same from sums of shares of k, a wave a token.
template <int VPL, int K>
__global__ __launch_bounds__(kRouteWaves * 64) void route_parts_kernel(RouteRule q, RouteParts parts, int64_t t,
                                                                       int32_t* ids, float* weights) {
  constexpr int V = VPL < 4 ? VPL : 4;
  typedef float four __attribute__((ext_vector_type(V)));
  __shared__ RouteLds<64, VPL> lds[kRouteWaves];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * kRouteWaves + wave;
  if (row >= t) return;
  const float* p = parts.part + row * parts.stride;
  const int64_t step = t * parts.stride;
  float l[VPL];
#pragma unroll
  for (int i = 0; i < VPL; i += V) {
    const int e = route_expert<64, VPL>(i, lane);
    four sum = {};
    if (e < q.experts) {
#pragma unroll 4
      for (int k = 0; k < parts.splits; ++k) sum += *reinterpret_cast<const four*>(p + k * step + e);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const bool there = e + j < q.experts;
      l[i + j] = there ? parts.bias ? sum[j] + parts.bias[e + j] : sum[j] : 0.f;
      if (there && parts.logits) parts.logits[row * parts.ldl + e + j] = l[i + j];
    }
  }
  int id;
  float weight;
  route_token<64, VPL, K>(q, l, lane, lds + wave, [&](int e) { return route_held<VPL>(l, e); }, id, weight);
  if (lane < q.topk) {
    ids[row * q.topk + lane] = id;
    weights[row * q.topk + lane] = weight;
  }
}

namespace {

template <int VPL>
void launch_parts(const RouteRule& q, const RouteParts& parts, int64_t t, int32_t* ids, float* weights,
                  hipStream_t s) {
  const dim3 grid((uint32_t)((t + kRouteWaves - 1) / kRouteWaves)), block(kRouteWaves * 64);
  if (q.topk <= 4) hipLaunchKernelGGL((route_parts_kernel<VPL, 4>), grid, block, 0, s, q, parts, t, ids, weights);
  else if (q.topk <= 8) hipLaunchKernelGGL((route_parts_kernel<VPL, 8>), grid, block, 0, s, q, parts, t, ids, weights);
  else hipLaunchKernelGGL((route_parts_kernel<VPL, 16>), grid, block, 0, s, q, parts, t, ids, weights);
}

template <int LANES, int VPL, class T>
void launch_vpl(const RouteRule& q, const T* logits, int64_t t, int64_t ldl, int32_t* ids, float* weights,
                hipStream_t s) {
  constexpr int kTokens = kRouteWaves * 64 / LANES, V = VPL < 4 ? VPL : 4;
  const dim3 grid((uint32_t)((t + kTokens - 1) / kTokens)), block(kRouteWaves * 64);
  const int vec = q.experts % V == 0 && ldl % V == 0 && reinterpret_cast<uintptr_t>(logits) % (V * sizeof(T)) == 0;
  if (q.topk <= 4)
    hipLaunchKernelGGL((route_topk_kernel<LANES, VPL, 4, T>), grid, block, 0, s, q, logits, vec, t, ldl, ids, weights);
  else if (q.topk <= 8)
    hipLaunchKernelGGL((route_topk_kernel<LANES, VPL, 8, T>), grid, block, 0, s, q, logits, vec, t, ldl, ids, weights);
  else
    hipLaunchKernelGGL((route_topk_kernel<LANES, VPL, 16, T>), grid, block, 0, s, q, logits, vec, t, ldl, ids, weights);
}

template <class T>
void launch_type(const RouteRule& q, const T* logits, int64_t t, int64_t ldl, int32_t* ids, float* weights,
                 hipStream_t s) {
  if (q.experts > 256 || t <= kRouteFew) {
    if (q.experts <= 64) launch_vpl<64, 1>(q, logits, t, ldl, ids, weights, s);
    else if (q.experts <= 128) launch_vpl<64, 2>(q, logits, t, ldl, ids, weights, s);
    else if (q.experts <= 256) launch_vpl<64, 4>(q, logits, t, ldl, ids, weights, s);
    else if (q.experts <= 512) launch_vpl<64, 8>(q, logits, t, ldl, ids, weights, s);
    else launch_vpl<64, 16>(q, logits, t, ldl, ids, weights, s);
  } else {
    if (q.experts <= 64) launch_vpl<16, 4>(q, logits, t, ldl, ids, weights, s);
    else if (q.experts <= 128) launch_vpl<16, 8>(q, logits, t, ldl, ids, weights, s);
    else launch_vpl<16, 16>(q, logits, t, ldl, ids, weights, s);
  }
}

}  // namespace

hipError_t launch_route_topk(const RouteRule& q, const void* logits, bool f32, int64_t t, int64_t ldl, int32_t* ids,
                             float* weights, hipStream_t s) {
  if (f32) launch_type(q, static_cast<const float*>(logits), t, ldl, ids, weights, s);
  else launch_type(q, static_cast<const _Float16*>(logits), t, ldl, ids, weights, s);
  return hipGetLastError();
}

hipError_t launch_route_parts(const RouteRule& q, const RouteParts& parts, int64_t t, int32_t* ids, float* weights,
                              hipStream_t s) {
  if (q.experts <= 64) launch_parts<1>(q, parts, t, ids, weights, s);
  else if (q.experts <= 128) launch_parts<2>(q, parts, t, ids, weights, s);
  else if (q.experts <= 256) launch_parts<4>(q, parts, t, ids, weights, s);
  else if (q.experts <= 512) launch_parts<8>(q, parts, t, ids, weights, s);
  else launch_parts<16>(q, parts, t, ids, weights, s);
  return hipGetLastError();
}

}  // namespace exl3
