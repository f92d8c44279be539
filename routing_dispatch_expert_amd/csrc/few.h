// The layer for a few tokens and the 4-bit weights (few.hip, q4.hip). Apart from
// common.h, so that the counters of the kernels which only share that one stay
// current.
#pragma once

#include "common.h"

namespace moe {

constexpr int kFewMaxT = 64, kFewMaxE = 1024, kFewMaxCopies = kFewMaxT * 32;
constexpr int kFewMaxSplits = 8;  // slices of d of the router scores
constexpr int kFewMaxShares = 8;  // work-groups that share a strip of out
constexpr int64_t kFewMaxWidth = 1 << 22;  // of d, d_ff and K
enum { kQ4U4 = 0, kQ4E2m1 = 1 };  // MOE_Q4_U4, MOE_Q4_E2M1
// Expert weights: kind < 0 dense (bf16 or fp32 rows), else 4-bit (q4.h).
struct FewWeights {
  int kind, group;
  const void *w[3], *scale[3], *zero[3];
};
// The kept copies by expert: experts with copies act_e[n_act], copies
// act_off[i] .. act_off[i + 1] - 1 of the i-th, and each copy's token and gate.
// done [strips]: counters of the down kernel's work-groups, zeroed by the
// routing kernel where the strips are split (n_done of them, else 0).
struct FewLists {
  int32_t *n_act, *act_e, *act_off, *token;
  float* gate;
  int32_t* done;
  int n_done;
};
struct FewLayer {
  const void *x, *wr;
  const float* bias;
  FewWeights wt;  // gate, up, down
  int T, E, k, P, M;
  int64_t d, f, C;
  bool bf16;
  void* out;
  int32_t *idx, *slot, *routed, *kept, *send;  // slot, routed, kept, send, totals may be NULL
  float* w;
  int64_t* totals;
  // workspace
  double* part;     // [splits][T][E]
  bf16_t* xparts;   // [3][T][d]: fp32 x beside 4-bit weights, else NULL
  FewLists ls;
  void* h;          // [parts][T k][few_ld_h(f)], bf16 (fp32 beside fp32 weights)
  float* sums;      // [strips][splits][T][16] where the down strips are split
  int splits;
};
int few_router_splits(int64_t T, int64_t d, int E);
// Work-groups that share 16 columns of out; columns of W_down that one of its
// units has (64 bf16, 32 fp32, 128 4-bit).
int few_down_splits(int64_t T, int64_t d, int64_t f, int E, int k, int unit_cols);
// Row length of h: whole 128-byte lines.
inline int64_t few_ld_h(int64_t f) { return ceil_div(f, 64) * 64; }
hipError_t launch_few_layer(const FewLayer& L, hipStream_t s);
// out[r] = W[expert[r]] x[r] for R <= 64 rows, W (w.w[0]) 4-bit [E, N, K];
// expert NULL: matrix 0; a row whose expert is outside [0, E) is left as it
// was. fp32 x: parts [3][R][K] is scratch.
hipError_t launch_q4_matvec(const void* x, bool bf16, const int32_t* expert, const FewWeights& w, int R, int E,
                            int64_t N, int64_t K, bf16_t* parts, void* out, hipStream_t s);
hipError_t launch_q4_quantize(const void* W, bool bf16, int E, int64_t N, int64_t K, int kind, int group, void* codes,
                              bf16_t* scale, uint8_t* zero, hipStream_t s);
hipError_t launch_q4_dequantize(const void* codes, const bf16_t* scale, const uint8_t* zero, int E, int64_t N,
                                int64_t K, int kind, int group, bool bf16, void* W, hipStream_t s);

}  // namespace moe
