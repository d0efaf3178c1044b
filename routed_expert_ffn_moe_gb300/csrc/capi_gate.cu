// The C ABI of scored routing (include/moe.h): host-side validation and dispatch.
#include <cmath>

#include "capi.h"
#include "router_gate.h"

namespace moe {
namespace {

moe_status check_gate(const moe_shape* s, const moe_gate* g) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  if (!g) return fail(MOE_ERR_INVALID_ARG, "gate is NULL");
  if (g->score != MOE_SCORE_SOFTMAX && g->score != MOE_SCORE_SIGMOID)
    return fail(MOE_ERR_INVALID_ARG, "score=%d unknown", g->score);
  if (g->n_group < 1 || g->n_group > 32 || s->E % g->n_group)
    return fail(MOE_ERR_INVALID_ARG, "n_group=%d not in [1, 32] or E=%d not a multiple",
                g->n_group, s->E);
  if (g->topk_group < 1 || g->topk_group > g->n_group)
    return fail(MOE_ERR_INVALID_ARG, "topk_group=%d not in [1, n_group]", g->topk_group);
  const int per = s->E / g->n_group;
  if (s->k > g->topk_group * per)
    return fail(MOE_ERR_INVALID_ARG, "k=%d experts of topk_group=%d groups of %d", s->k,
                g->topk_group, per);
  if (g->group_top < 1 || g->group_top > 2 || g->group_top > per)
    return fail(MOE_ERR_INVALID_ARG, "group_top=%d not 1 or 2, or over the %d of a group",
                g->group_top, per);
  if (!std::isfinite(g->scale)) return fail(MOE_ERR_INVALID_ARG, "scale is not finite");
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_route_select(const moe_shape* shape, const moe_gate* gate, const float* logits,
                            const float* sel_bias, int32_t* topk_idx, float* topk_w,
                            void* stream) {
  moe_status st = check_gate(shape, gate);
  if (st != MOE_OK) return st;
  if (shape->T > 0) {
    REQUIRE_PTR(logits, 16);
    REQUIRE_PTR(topk_idx, 16);
    REQUIRE_PTR(topk_w, 16);
  }
  if (!aligned(sel_bias, 16)) return fail(MOE_ERR_INVALID_ARG, "sel_bias not 16-byte aligned");
  cudaError_t e = launch_route_select(*shape, *gate, logits, sel_bias, topk_idx, topk_w,
                                      static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : cuda_fail(e, "moe_route_select launch");
}

moe_status moe_route_gate(const moe_shape* shape, const moe_gate* gate, const void* x,
                          const void* wg, const float* bias, const float* sel_bias,
                          int32_t* topk_idx, float* topk_w, void* ws, size_t ws_bytes,
                          void* stream) {
  moe_status st = check_gate(shape, gate);
  if (st != MOE_OK) return st;
  if (shape->T > 0) {
    REQUIRE_PTR(x, 16);
    REQUIRE_PTR(topk_idx, 16);
    REQUIRE_PTR(topk_w, 16);
  }
  REQUIRE_PTR(wg, 16);
  if (!aligned(bias, 16)) return fail(MOE_ERR_INVALID_ARG, "bias not 16-byte aligned");
  if (!aligned(sel_bias, 16)) return fail(MOE_ERR_INVALID_ARG, "sel_bias not 16-byte aligned");
  WsLayout L;
  if ((st = check_ws(shape, ws, ws_bytes, &L)) != MOE_OK) return st;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  char* w = static_cast<char*>(ws);
  cudaError_t e = cudaMemsetAsync(w + L.status, 0, sizeof(int), cs);
  if (e != cudaSuccess) return cuda_fail(e, "moe_route_gate status reset");
  if (shape->T == 0) return MOE_OK;
  float* logits = reinterpret_cast<float*>(w + L.logits);
  const uint16_t* xb = static_cast<const uint16_t*>(x);
  const uint16_t* wb = static_cast<const uint16_t*>(wg);
  const bool groups = gate->topk_group < gate->n_group;
  // softmax scores depend on every logit: where they count, all are formed
  const bool by_logits = gate->score == MOE_SCORE_SIGMOID ||
                         (!sel_bias && gate->renorm && (!groups || gate->group_top == 1));
  if (by_logits && router_settles(*shape)) {
    const SettleRule rule{groups ? gate->n_group : 1, groups ? shape->E / gate->n_group : shape->E,
                          groups ? gate->topk_group : 1, gate->group_top};
    e = launch_settled_logits(*shape, xb, wb, bias, sel_bias, rule, w, L, cs);
  } else {
    e = launch_router_logits(*shape, xb, wb, bias, logits, cs);
  }
  if (e == cudaSuccess)
    e = launch_route_select(*shape, *gate, logits, sel_bias, topk_idx, topk_w, cs);
  return e == cudaSuccess ? MOE_OK : cuda_fail(e, "moe_route_gate launch");
}

}  // extern "C"
