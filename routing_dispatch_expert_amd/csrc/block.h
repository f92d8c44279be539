// What a transformer block has around the experts: the gate with its gradient,
// the norm in front of the layer, 8-bit matrices and the experts' products with
// them (gate.hip, norm.hip, mx8.hip, mx8_experts.hip). Apart from common.h, so that
// the counters of the kernels which only share that one stay current.
#pragma once

#include "common.h"

namespace moe {

// ---- the gate (gate.hip) ----
constexpr int kGateMaxGroups = 64;
// As moe_gate_t.
struct GateRule {
  bool sigmoid, renormalize;
  int groups, top_groups, best;  // groups = 1: no limit
  float scale;
};
hipError_t launch_gate(const float* logits, const float* bias, const GateRule& g, int64_t T, int E, int k, int32_t* idx,
                       float* w, hipStream_t s);
hipError_t launch_gate_backward(const float* logits, const int32_t* idx, const float* dw, const float* dscores,
                                const GateRule& g, int64_t T, int E, int k, float* dlogits, hipStream_t s);

}  // namespace moe
