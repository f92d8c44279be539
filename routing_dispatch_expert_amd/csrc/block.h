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

// ---- 8-bit matrices (mx8.hip): codes [E][N][K], scale dwords [E][ceil(K/128)][N] ----
int64_t mx8_units(int64_t E, int64_t N, int64_t K, bool bf16);  // waves of a launch
hipError_t launch_mx8_quantize(const void* W, bool bf16, int64_t E, int64_t N, int64_t K, uint8_t* codes, uint32_t* scale,
                               hipStream_t s);
hipError_t launch_mx8_dequantize(const uint8_t* codes, const uint32_t* scale, int64_t E, int64_t N, int64_t K, bool bf16,
                                 void* W, hipStream_t s);

// ---- the norm (norm.hip) ----
// residual, h, y, codes (with scale), rstd and dres may be NULL; h is written with a residual only.
int64_t rmsnorm_max_width(bool bf16);
hipError_t launch_rmsnorm(const void* x, const void* residual, const void* weight, float eps, int64_t R, int64_t d,
                          bool bf16, void* h, void* y, uint8_t* codes, uint32_t* scale, float* rstd, hipStream_t s);
// parts: fp32 [rmsnorm_shares()][d].
int64_t rmsnorm_shares(int64_t R, int64_t d, bool bf16);
hipError_t launch_rmsnorm_backward(const void* dy, const void* h, const void* weight, const float* rstd,
                                   const void* dres, int64_t R, int64_t d, bool bf16, void* dh, void* dweight,
                                   float* parts, hipStream_t s);

// ---- the experts with 8-bit rows and weights (mx8_experts.hip) ----
struct Mx8Ptr {
  uint8_t* codes;
  uint32_t* scale;
};
// The kept copies by expert, in token order: row off[e] + i is copy (flat t k + j)
// copy[off[e] + i]; act [n_act]: the experts that have rows; tile: prefix of the
// experts' row tiles.
struct ExpertLists {
  int32_t *off, *tile, *n_act, *act, *copy;  // [E + 1], [E + 1], [1], [min(E, T k)], [T k]
};
struct ExpertsMx8 {
  Mx8Ptr x, gate, up, down;
  const void* residual;
  const int32_t* idx;
  const float* w;
  int64_t T, d, f, C;
  int E, k;
  bool bf16;       // residual and out
  void* out;
  int32_t *slot, *routed, *kept;
  // workspace
  ExpertLists ls;
  int32_t *tile_cnt, *tile_off;  // [ceil(T / kTileTokens)][E]
  Mx8Ptr h;        // rows [T k][f]
  float* y;        // [T k][d]
  float* parts;    // mx8_parts_bytes(T k, min(E, T k), f), or NULL
};
// Sums of down's split tiles (mx8_tiles.hip); 0 where none can be.
int64_t mx8_parts_bytes(int64_t copies, int64_t experts, int64_t K);
hipError_t launch_experts_mx8(const ExpertsMx8& L, hipStream_t s);

// ---- the layer with a given routing (routed.hip) ----
// The weights that dy = first dout is formed with: w, and 1 for weights of 0 and of unusual size.
hipError_t launch_split_weights(const float* w, int64_t n, float* first, hipStream_t s);
// dw = <dh, h> / first, 0 for a dropped copy; after it dh and dy have the whole weight.
hipError_t launch_weight_grad(void* dh, const void* h, void* dy, const int32_t* idx, const float* w, const int32_t* slot,
                              int64_t T, int64_t d, int64_t F, int k, int64_t C, bool bf16, float* dw, hipStream_t s);
// dx[t] = sum_j [slot >= 0] dX[idx, slot].
hipError_t launch_gather_copies(const void* dX, const int32_t* idx, const int32_t* slot, int64_t T, int64_t d, int k,
                                int64_t C, bool bf16, void* dx, hipStream_t s);

}  // namespace moe
