// exl3_route_topk: choices and weights of every token from its logits.
#include "exl3_route.hpp"

namespace exl3 {

constexpr int kRouteWaves = 4;

template <int VPL, int K>
__global__ __launch_bounds__(kRouteWaves * 64) void route_topk_kernel(RouteRule q, const void* logits, int f32,
                                                                      int64_t t, int64_t ldl, int32_t* ids,
                                                                      float* weights) {
  __shared__ RouteLds<64, VPL> lds[kRouteWaves];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * kRouteWaves + wave;
  if (row >= t) return;
  float l[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = 64 * i + lane;
    l[i] = 0.f;
    if (e < q.experts)
      l[i] = f32 ? static_cast<const float*>(logits)[row * ldl + e]
                 : (float)static_cast<const _Float16*>(logits)[row * ldl + e];
  }
  int id;
  float weight;
  route_token<64, VPL, K>(q, l, lane, lds + wave, id, weight);
  if (lane < q.topk) {
    ids[row * q.topk + lane] = id;
    weights[row * q.topk + lane] = weight;
  }
}

template <int VPL>
static void launch_vpl(const RouteRule& q, const void* logits, bool f32, int64_t t, int64_t ldl, int32_t* ids,
                       float* weights, hipStream_t s) {
  const dim3 grid((uint32_t)((t + kRouteWaves - 1) / kRouteWaves)), block(kRouteWaves * 64);
  if (q.topk <= 4)
    hipLaunchKernelGGL((route_topk_kernel<VPL, 4>), grid, block, 0, s, q, logits, (int)f32, t, ldl, ids, weights);
  else if (q.topk <= 8)
    hipLaunchKernelGGL((route_topk_kernel<VPL, 8>), grid, block, 0, s, q, logits, (int)f32, t, ldl, ids, weights);
  else
    hipLaunchKernelGGL((route_topk_kernel<VPL, 16>), grid, block, 0, s, q, logits, (int)f32, t, ldl, ids, weights);
}

hipError_t launch_route_topk(const RouteRule& q, const void* logits, bool f32, int64_t t, int64_t ldl, int32_t* ids,
                             float* weights, hipStream_t s) {
  if (q.experts <= 64) launch_vpl<1>(q, logits, f32, t, ldl, ids, weights, s);
  else if (q.experts <= 128) launch_vpl<2>(q, logits, f32, t, ldl, ids, weights, s);
  else if (q.experts <= 256) launch_vpl<4>(q, logits, f32, t, ldl, ids, weights, s);
  else if (q.experts <= 512) launch_vpl<8>(q, logits, f32, t, ldl, ids, weights, s);
  else launch_vpl<16>(q, logits, f32, t, ldl, ids, weights, s);
  return hipGetLastError();
}

}  // namespace exl3
