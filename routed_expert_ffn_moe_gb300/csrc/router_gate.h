// Interface of the scored routing kernels (router_gate.cu).
#pragma once

#include "internal.h"

namespace moe {

struct GateParams {
  const float* logits;
  const float* bias;
  int32_t* idx;
  float* w;
  int T, E, k;
  int G, per, keep, group_top;  // groups (1 if all are kept), experts of one, groups kept
  int P;                        // lanes of a group
  int sigmoid, renorm;
  float scale;
};

cudaError_t launch_route_select(const moe_shape& s, const moe_gate& gate, const float* logits,
                                const float* bias, int32_t* idx, float* w, cudaStream_t st);

}  // namespace moe
