// C ABI of the MXFP4 operators (declared in include/exl3.h): host-side
// validation, then dispatch; nothing is enqueued when validation fails and
// nothing is allocated.
#include <stdio.h>
#include <stdlib.h>

#include "exl3.h"
#include "exl3_internal.hpp"

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 24;
constexpr int64_t kMaxK = (int64_t)1 << 24;
// Launch sizes: a grid holds less than 2^32 threads.  Quantizing, a thread takes
// eight elements, of 256 a workgroup.
constexpr int64_t kMaxElements = (int64_t)1 << 35;
constexpr int64_t kMaxQuantized = kMaxElements - 2048;
constexpr int64_t kMaxTiles = (int64_t)1 << 26;     // 16 x 16 output tiles
constexpr int kMaxExpertDim = 65536;

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

void trace(const char* what, long long a, long long b, long long c, long long d) {
  static const bool on = [] {
    const char* v = getenv("EXL3_TRACE");
    return v && v[0] && v[0] != '0';
  }();
  if (on) fprintf(stderr, "[exl3] %s %lld %lld %lld %lld\n", what, a, b, c, d);
}

exl3_status from_hip(hipError_t e) { return e == hipSuccess ? EXL3_OK : EXL3_E_HIP; }

bool valid_dtype(int32_t t) { return t == EXL3_F16 || t == EXL3_F32; }

// Bytes of one element of y: the alignment its rows need.
uintptr_t dtype_bytes(int32_t t) { return t == EXL3_F32 ? 4 : 2; }

bool valid_shape(int64_t rows, int64_t k) {
  return rows >= 0 && rows <= kMaxRows && k > 0 && k < kMaxK && k % EXL3_MX4_BLOCK == 0;
}

exl3_status check_matrix(const exl3_mx4* w) {
  if (!w || !valid_shape(w->rows, w->k)) return EXL3_E_INVALID;
  if (w->rows == 0) return EXL3_OK;
  if (!w->codes || !w->scales || !aligned(w->codes, 16) || !aligned(w->scales, 16)) return EXL3_E_INVALID;
  return EXL3_OK;
}

int64_t tiles16(int64_t m, int64_t n) { return ((m + 15) / 16) * ((n + 15) / 16); }

// y [m][ldy] and the bias of a product, m and n not 0.
exl3_status check_product(const uint16_t* bias, const void* y, int64_t m, int64_t n, int64_t ldy, int32_t y_dtype) {
  if (!valid_dtype(y_dtype) || ldy < n) return EXL3_E_INVALID;
  if (tiles16(m, n) >= kMaxTiles) return EXL3_E_INVALID;
  if (m == 0 || n == 0) return EXL3_OK;
  if (!y || !aligned(y, dtype_bytes(y_dtype)) || (bias && !aligned(bias, 2))) return EXL3_E_INVALID;
  return EXL3_OK;
}

bool have_workspace(const void* ws, size_t bytes, size_t need) {
  return need == 0 || (ws && bytes >= need && aligned(ws, 16));
}

exl3_status check_experts(const exl3_mx4_experts& a, int slots) {
  if (!a.codes || !a.scales || !aligned(a.codes, 16) || !aligned(a.scales, 16)) return EXL3_E_INVALID;
  if (a.experts <= 0 || a.slots != slots) return EXL3_E_INVALID;
  for (int32_t v : {a.n, a.k})
    if (v <= 0 || v > kMaxExpertDim || v % EXL3_MX4_BLOCK) return EXL3_E_INVALID;
  return EXL3_OK;
}

exl3_status check_layer(const exl3_mx4_moe_layer* l, int64_t t, int32_t topk) {
  if (!l || t < 0 || t > EXL3_MX4_MOE_MAX_TOKENS) return EXL3_E_INVALID;
  exl3_status st = check_experts(l->gate_up, 2);
  if (st != EXL3_OK || (st = check_experts(l->down, 1)) != EXL3_OK) return st;
  const int32_t e = l->gate_up.experts;
  if (e > EXL3_MX4_MOE_MAX_EXPERTS || l->down.experts != e) return EXL3_E_INVALID;
  if (l->down.k != l->gate_up.n || l->down.n != l->gate_up.k) return EXL3_E_INVALID;
  if (topk < 1 || topk > EXL3_MAX_TOPK || topk > e) return EXL3_E_INVALID;
  if (l->scoring != EXL3_ROUTE_SOFTMAX && l->scoring != EXL3_ROUTE_SIGMOID) return EXL3_E_INVALID;
  if (!l->router || !aligned(l->router, 16)) return EXL3_E_INVALID;
  if (l->router_bias && !aligned(l->router_bias, 4)) return EXL3_E_INVALID;
  const bool has_gu = l->shared_gate_up.codes != nullptr, has_dn = l->shared_down.codes != nullptr;
  if (has_gu != has_dn) return EXL3_E_INVALID;
  if (has_gu) {
    if ((st = check_experts(l->shared_gate_up, 2)) != EXL3_OK) return st;
    if ((st = check_experts(l->shared_down, 1)) != EXL3_OK) return st;
    if (l->shared_gate_up.experts != 1 || l->shared_down.experts != 1) return EXL3_E_INVALID;
    if (l->shared_gate_up.k != l->gate_up.k || l->shared_down.n != l->gate_up.k) return EXL3_E_INVALID;
    if (l->shared_down.k != l->shared_gate_up.n) return EXL3_E_INVALID;
    if (l->shared_gate && !aligned(l->shared_gate, 16)) return EXL3_E_INVALID;
  } else if (l->shared_gate) {
    return EXL3_E_INVALID;
  }
  return EXL3_OK;
}

exl3::Mx4MoeDesc moe_desc(const exl3_mx4_moe_layer* l) {
  exl3::Mx4MoeDesc d{};
  d.router = l->router;
  d.router_bias = l->router_bias;
  d.scoring = l->scoring;
  d.renormalize = l->renormalize;
  d.scale = l->scale;
  d.experts = l->gate_up.experts;
  d.hidden = l->gate_up.k;
  d.inter = l->gate_up.n;
  d.gu_codes = l->gate_up.codes;
  d.gu_scales = l->gate_up.scales;
  d.dn_codes = l->down.codes;
  d.dn_scales = l->down.scales;
  if (l->shared_gate_up.codes) {
    d.shared_inter = l->shared_gate_up.n;
    d.sgu_codes = l->shared_gate_up.codes;
    d.sgu_scales = l->shared_gate_up.scales;
    d.sdn_codes = l->shared_down.codes;
    d.sdn_scales = l->shared_down.scales;
    d.shared_gate = l->shared_gate;
  }
  return d;
}

}  // namespace

extern "C" {

exl3_status exl3_mx4_quantize(const void* x, int32_t dtype, int64_t rows, int64_t k, int64_t ldx, uint8_t* codes,
                              uint8_t* scales, exl3_stream_t stream) {
  if (!valid_dtype(dtype) || !valid_shape(rows, k) || rows * k > kMaxQuantized) return EXL3_E_INVALID;
  if (ldx < k || ldx % 8) return EXL3_E_INVALID;
  if (rows == 0) return EXL3_OK;
  if (!x || !codes || !scales || !aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 16))
    return EXL3_E_INVALID;
  trace("mx4_quantize rows k dtype", rows, k, dtype, 0);
  return from_hip(exl3::launch_mx4_quantize(x, dtype == EXL3_F32, rows, k, ldx, codes, scales,
                                            reinterpret_cast<hipStream_t>(stream)));
}

exl3_status exl3_mx4_reconstruct(const exl3_mx4* w, void* out, int32_t dtype, int64_t ld_out, exl3_stream_t stream) {
  const exl3_status st = check_matrix(w);
  if (st != EXL3_OK) return st;
  if (!valid_dtype(dtype) || w->rows * w->k >= kMaxElements) return EXL3_E_INVALID;
  if (ld_out < w->k || ld_out % 8) return EXL3_E_INVALID;
  if (w->rows == 0) return EXL3_OK;
  if (!out || !aligned(out, 16)) return EXL3_E_INVALID;
  trace("mx4_reconstruct rows k dtype", w->rows, w->k, dtype, 0);
  return from_hip(exl3::launch_mx4_reconstruct(w->codes, w->scales, w->rows, w->k, out, dtype == EXL3_F32, ld_out,
                                               reinterpret_cast<hipStream_t>(stream)));
}

size_t exl3_mx4_matmul_workspace_size(const exl3_mx4* a, const exl3_mx4* b) {
  if (check_matrix(a) != EXL3_OK || check_matrix(b) != EXL3_OK || a->k != b->k) return 0;
  if (a->rows == 0 || b->rows == 0 || tiles16(a->rows, b->rows) >= kMaxTiles) return 0;
  if (!exl3::mx4_matmul_fits(a->rows, b->rows, a->k)) return 0;
  return exl3::mx4_matmul_workspace(a->rows, b->rows, a->k);
}

exl3_status exl3_mx4_matmul(const exl3_mx4* a, const exl3_mx4* b, const uint16_t* bias, void* y, int64_t ldy,
                            int32_t y_dtype, void* ws, size_t ws_bytes, exl3_stream_t stream) {
  exl3_status st = check_matrix(a);
  if (st != EXL3_OK || (st = check_matrix(b)) != EXL3_OK) return st;
  if (a->k != b->k) return EXL3_E_INVALID;
  if ((st = check_product(bias, y, a->rows, b->rows, ldy, y_dtype)) != EXL3_OK) return st;
  if (a->rows == 0 || b->rows == 0) return EXL3_OK;
  if (!exl3::mx4_matmul_fits(a->rows, b->rows, a->k)) return EXL3_E_INVALID;
  if (!have_workspace(ws, ws_bytes, exl3::mx4_matmul_workspace(a->rows, b->rows, a->k))) return EXL3_E_WORKSPACE;
  trace("mx4_matmul m k n", a->rows, a->k, b->rows, 0);
  return from_hip(exl3::launch_mx4_matmul(a->codes, a->scales, a->rows, b->codes, b->scales, b->rows, a->k, bias, y,
                                          ldy, y_dtype == EXL3_F32, ws, reinterpret_cast<hipStream_t>(stream)));
}

size_t exl3_mx4_linear_workspace_size(const exl3_mx4* w, int64_t m) {
  if (check_matrix(w) != EXL3_OK || w->rows == 0 || m <= 0 || m > EXL3_MX4_LINEAR_MAX_ROWS) return 0;
  return exl3::mx4_linear_workspace(m, w->rows, w->k);
}

exl3_status exl3_mx4_linear(const exl3_mx4* w, const uint16_t* bias, const void* x, int64_t m, int64_t ldx, void* y,
                            int64_t ldy, int32_t y_dtype, void* ws, size_t ws_bytes, exl3_stream_t stream) {
  exl3_status st = check_matrix(w);
  if (st != EXL3_OK) return st;
  if (m < 0 || m > EXL3_MX4_LINEAR_MAX_ROWS || ldx < w->k || ldx % 8) return EXL3_E_INVALID;
  if ((st = check_product(bias, y, m, w->rows, ldy, y_dtype)) != EXL3_OK) return st;
  if (m == 0 || w->rows == 0) return EXL3_OK;
  if (!x || !aligned(x, 16)) return EXL3_E_INVALID;
  if (!have_workspace(ws, ws_bytes, exl3::mx4_linear_workspace(m, w->rows, w->k))) return EXL3_E_WORKSPACE;
  trace("mx4_linear m k n", m, w->k, w->rows, 0);
  return from_hip(exl3::launch_mx4_linear(w->codes, w->scales, w->rows, w->k, bias, static_cast<const uint16_t*>(x), m,
                                          ldx, y, ldy, y_dtype == EXL3_F32, ws, reinterpret_cast<hipStream_t>(stream)));
}

size_t exl3_mx4_moe_workspace_size(const exl3_mx4_moe_layer* layer, int64_t t, int32_t topk) {
  if (check_layer(layer, t, topk) != EXL3_OK || t == 0) return 0;
  return exl3::mx4_moe_workspace(moe_desc(layer), t, topk);
}

exl3_status exl3_mx4_moe(const exl3_mx4_moe_layer* layer, const void* x, int64_t t, int64_t ldx, int32_t topk, void* y,
                         int64_t ldy, int32_t y_dtype, int32_t* topk_ids, float* topk_weights, void* ws,
                         size_t ws_bytes, exl3_stream_t stream) {
  const exl3_status st = check_layer(layer, t, topk);
  if (st != EXL3_OK) return st;
  const int32_t hidden = layer->gate_up.k;
  if (!valid_dtype(y_dtype) || ldx < hidden || ldx % 8 || ldy < hidden) return EXL3_E_INVALID;
  if (t == 0) return EXL3_OK;
  if (!x || !y || !aligned(x, 16) || !aligned(y, dtype_bytes(y_dtype))) return EXL3_E_INVALID;
  if (!aligned(topk_ids, 4) || !aligned(topk_weights, 4)) return EXL3_E_INVALID;
  const exl3::Mx4MoeDesc d = moe_desc(layer);
  if (!have_workspace(ws, ws_bytes, exl3::mx4_moe_workspace(d, t, topk))) return EXL3_E_WORKSPACE;
  trace("mx4_moe t topk experts hidden", t, topk, d.experts, d.hidden);
  return from_hip(exl3::launch_mx4_moe(d, static_cast<const uint16_t*>(x), t, ldx, topk, y, ldy, y_dtype == EXL3_F32,
                                       topk_ids, topk_weights, ws, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
