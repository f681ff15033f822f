// C ABI of the routing and of the low-rank adapters (declared in include/exl3.h):
// host-side validation, then dispatch; nothing is enqueued when validation fails and
// nothing is allocated.
#include <stdio.h>
#include <stdlib.h>

#include "exl3.h"
#include "exl3_internal.hpp"

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 24;
constexpr int32_t kMaxHidden = 65536;
constexpr int64_t kMaxDim = (int64_t)1 << 20;  // of an adapter

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
uintptr_t dtype_bytes(int32_t t) { return t == EXL3_F32 ? 4 : 2; }

bool have_workspace(const void* ws, size_t bytes, size_t need) {
  return need == 0 || (ws && bytes >= need && aligned(ws, 16));
}

exl3_status check_rule(const exl3_route_rule* r) {
  if (!r || r->experts < 1 || r->experts > EXL3_ROUTE_MAX_EXPERTS) return EXL3_E_INVALID;
  if (r->scoring != EXL3_ROUTE_SOFTMAX && r->scoring != EXL3_ROUTE_SIGMOID) return EXL3_E_INVALID;
  if (r->group_score != EXL3_GROUP_MAX && r->group_score != EXL3_GROUP_TOP2) return EXL3_E_INVALID;
  if (r->groups < 1 || r->groups > EXL3_ROUTE_MAX_GROUPS || r->experts % r->groups) return EXL3_E_INVALID;
  if (r->topk_groups < 1 || r->topk_groups > r->groups) return EXL3_E_INVALID;
  const int32_t size = r->experts / r->groups;
  if (r->groups > 1 && r->group_score == EXL3_GROUP_TOP2 && size < 2) return EXL3_E_INVALID;
  if (r->topk < 1 || r->topk > EXL3_MAX_TOPK || r->topk > r->topk_groups * size) return EXL3_E_INVALID;
  if (r->balance && !aligned(r->balance, 4)) return EXL3_E_INVALID;
  return EXL3_OK;
}

exl3::RouteRule rule_desc(const exl3_route_rule* r) {
  exl3::RouteRule q{};
  q.balance = r->balance;
  q.experts = r->experts;
  q.topk = r->topk;
  q.scoring = r->scoring;
  q.groups = r->topk_groups == r->groups ? 1 : r->groups;  // all groups kept: none
  q.group_size = r->experts / q.groups;
  q.topk_groups = q.groups == 1 ? 1 : r->topk_groups;
  q.top2 = r->group_score == EXL3_GROUP_TOP2;
  q.group_inverse = (uint32_t)(((1 << 20) + q.group_size - 1) / q.group_size);
  q.renormalize = r->renormalize;
  q.scale = r->scale;
  return q;
}

exl3_status check_router(const exl3_router_weight* w) {
  if (!w || w->experts < 1 || w->experts > EXL3_ROUTE_MAX_EXPERTS) return EXL3_E_INVALID;
  if (w->hidden <= 0 || w->hidden > kMaxHidden || w->hidden % 8) return EXL3_E_INVALID;
  if (!w->weight || !aligned(w->weight, 16) || (w->bias && !aligned(w->bias, 4))) return EXL3_E_INVALID;
  return EXL3_OK;
}

exl3::RouterDesc router_desc(const exl3_router_weight* w) {
  return exl3::RouterDesc{w->weight, w->bias, w->experts, w->hidden};
}

exl3_status check_choices(const int32_t* ids, const float* weights) {
  return ids && weights && aligned(ids, 4) && aligned(weights, 4) ? EXL3_OK : EXL3_E_INVALID;
}

exl3_status check_lora(const exl3_lora_stack* l) {
  if (!l || l->adapters < 0 || l->adapters > EXL3_LORA_MAX_ADAPTERS) return EXL3_E_INVALID;
  if (l->rank <= 0 || l->rank > EXL3_LORA_MAX_RANK || l->rank % 8) return EXL3_E_INVALID;
  if (l->k <= 0 || l->k > kMaxDim || l->k % 8 || l->n <= 0 || l->n > kMaxDim) return EXL3_E_INVALID;
  if (l->adapters == 0) return EXL3_OK;
  if (!l->a || !l->b || !aligned(l->a, 16) || !aligned(l->b, 16)) return EXL3_E_INVALID;
  if (!aligned(l->scales, 4) || !aligned(l->ranks, 4)) return EXL3_E_INVALID;
  return EXL3_OK;
}

exl3::LoraDesc lora_desc(const exl3_lora_stack* l) {
  return exl3::LoraDesc{l->a, l->b, l->scales, l->ranks, l->adapters, l->rank, l->k, l->n};
}

}  // namespace

extern "C" {

exl3_status exl3_route_topk(const exl3_route_rule* rule, const void* logits, int32_t dtype, int64_t t, int64_t ldl,
                            int32_t* topk_ids, float* topk_weights, exl3_stream_t stream) {
  exl3_status st = check_rule(rule);
  if (st != EXL3_OK) return st;
  if (!valid_dtype(dtype) || t < 0 || t > kMaxRows || ldl < rule->experts) return EXL3_E_INVALID;
  if (t == 0) return EXL3_OK;
  if (!logits || !aligned(logits, dtype_bytes(dtype))) return EXL3_E_INVALID;
  if ((st = check_choices(topk_ids, topk_weights)) != EXL3_OK) return st;
  trace("route_topk t experts topk groups", t, rule->experts, rule->topk, rule->groups);
  return from_hip(exl3::launch_route_topk(rule_desc(rule), logits, dtype == EXL3_F32, t, ldl, topk_ids, topk_weights,
                                          reinterpret_cast<hipStream_t>(stream)));
}

size_t exl3_router_linear_workspace_size(const exl3_router_weight* w, int64_t t) {
  if (check_router(w) != EXL3_OK || t <= 0 || t > kMaxRows) return 0;
  return exl3::router_linear_workspace(router_desc(w), t);
}

exl3_status exl3_router_linear(const exl3_router_weight* w, const void* x, int64_t t, int64_t ldx, float* logits,
                               int64_t ldl, void* ws, size_t ws_bytes, exl3_stream_t stream) {
  const exl3_status st = check_router(w);
  if (st != EXL3_OK) return st;
  if (t < 0 || t > kMaxRows || ldx < w->hidden || ldx % 8 || ldl < w->experts) return EXL3_E_INVALID;
  if (t == 0) return EXL3_OK;
  if (!x || !aligned(x, 16) || !logits || !aligned(logits, 4)) return EXL3_E_INVALID;
  const exl3::RouterDesc d = router_desc(w);
  if (!have_workspace(ws, ws_bytes, exl3::router_linear_workspace(d, t))) return EXL3_E_WORKSPACE;
  trace("router_linear t hidden experts", t, d.hidden, d.experts, 0);
  return from_hip(exl3::launch_router_linear(d, static_cast<const uint16_t*>(x), t, ldx, logits, ldl, ws,
                                             reinterpret_cast<hipStream_t>(stream)));
}

size_t exl3_router_workspace_size(const exl3_router_weight* w, int64_t t, int32_t logits) {
  if (check_router(w) != EXL3_OK || t <= 0 || t > kMaxRows) return 0;
  return exl3::router_workspace(router_desc(w), t, logits != 0);
}

exl3_status exl3_router(const exl3_router_weight* w, const exl3_route_rule* rule, const void* x, int64_t t,
                        int64_t ldx, float* logits, int64_t ldl, int32_t* topk_ids, float* topk_weights, void* ws,
                        size_t ws_bytes, exl3_stream_t stream) {
  exl3_status st = check_router(w);
  if (st != EXL3_OK || (st = check_rule(rule)) != EXL3_OK) return st;
  if (rule->experts != w->experts) return EXL3_E_INVALID;
  if (t < 0 || t > kMaxRows || ldx < w->hidden || ldx % 8) return EXL3_E_INVALID;
  if (t == 0) return EXL3_OK;
  if (!x || !aligned(x, 16)) return EXL3_E_INVALID;
  if (logits && (ldl < w->experts || !aligned(logits, 4))) return EXL3_E_INVALID;
  if ((st = check_choices(topk_ids, topk_weights)) != EXL3_OK) return st;
  const exl3::RouterDesc d = router_desc(w);
  if (!have_workspace(ws, ws_bytes, exl3::router_workspace(d, t, logits != nullptr))) return EXL3_E_WORKSPACE;
  trace("router t hidden experts topk", t, d.hidden, d.experts, rule->topk);
  return from_hip(exl3::launch_router(d, rule_desc(rule), static_cast<const uint16_t*>(x), t, ldx, logits, ldl,
                                      topk_ids, topk_weights, ws, reinterpret_cast<hipStream_t>(stream)));
}

size_t exl3_lora_workspace_size(const exl3_lora_stack* l, int64_t m) {
  if (check_lora(l) != EXL3_OK || m <= 0 || m > kMaxRows) return 0;
  return exl3::lora_workspace(lora_desc(l), m);
}

exl3_status exl3_lora(const exl3_lora_stack* l, const void* x, int64_t m, int64_t ldx, const int32_t* rows,
                      const void* base, int64_t ldb, void* y, int64_t ldy, int32_t y_dtype, void* ws, size_t ws_bytes,
                      exl3_stream_t stream) {
  const exl3_status st = check_lora(l);
  if (st != EXL3_OK) return st;
  if (!valid_dtype(y_dtype) || m < 0 || m > kMaxRows || ldx < l->k || ldx % 8 || ldy < l->n) return EXL3_E_INVALID;
  if (base && ldb < l->n) return EXL3_E_INVALID;
  if (base && base == y && m > 1 && ldb != ldy) return EXL3_E_INVALID;
  if (m == 0) return EXL3_OK;
  if (!x || !aligned(x, 16) || !rows || !aligned(rows, 4)) return EXL3_E_INVALID;
  if (!y || !aligned(y, dtype_bytes(y_dtype)) || !aligned(base, dtype_bytes(y_dtype))) return EXL3_E_INVALID;
  const exl3::LoraDesc d = lora_desc(l);
  if (!have_workspace(ws, ws_bytes, exl3::lora_workspace(d, m))) return EXL3_E_WORKSPACE;
  trace("lora m k n rank", m, d.k, d.n, d.rank);
  return from_hip(exl3::launch_lora(d, static_cast<const uint16_t*>(x), m, ldx, rows, base, ldb, y, ldy,
                                    y_dtype == EXL3_F32, ws, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
