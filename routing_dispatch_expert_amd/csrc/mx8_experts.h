// What the kernels of the experts with 8-bit rows and weights share.
#pragma once

#include "mx8.h"

namespace moe {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// g / (1 + e^-g) by the hardware's 2^x and reciprocal (a step each), in nine
// instructions: off by less than 2^-21 of itself down to g = -87. The product -g
// log2(e) is taken with its rounding, which alone would be off by 2^-24 |g| of the
// power. Past +-126 the power is 0 or infinite and the result g or -0; -g is held
// there, so that the rounding stays a number. Below -87 the reciprocal leaves the
// normal numbers and may come as 0: off by less than 1.1e-36.
// (expf and a division instead took a third of the gate and up products' time with
// d = 4096.)
__device__ inline float silu(float g) {
  const float c = __builtin_amdgcn_fmed3f(-g, -126.f, 126.f), l = 1.44269502162933349609375f;  // log2(e) less 1.92596299e-8
  const float t = c * l, rest = fmaf(c, 1.92596299e-8f, fmaf(c, l, -t));
  const float p = __builtin_amdgcn_exp2f(t);
  return g * __builtin_amdgcn_rcpf(fmaf(p, fmaf(rest, 0.693147182f, 1.f), 1.f));
}

struct Mx8 {
  const uint8_t* codes;   // [E][N][K]
  const uint32_t* scale;  // [E][steps][N]
};

// One grouped product: rows x of the experts' lists by their weights.
struct Mx8Gemm {
  Mx8 a0, a1;         // weights: gate and up, or down alone
  int64_t N, K;       // of one matrix
  Mx8 x;              // rows [R][K]
  int64_t R;
  ExpertLists ls;
  int k;
  uint8_t* hcodes;    // GU: h [rows][N], scale [steps][H]
  uint8_t* hscale;
  int64_t H;
  float* y;           // else: [copies][N]
  float* parts;       // or NULL: of down's tiles that are split over K
};

// Many rows an expert (mx8_tiles.hip): row tiles of mx8_tile_rows() rows, by the rows
// that the experts have on average, listed in ls.tile. Grid: at most `tiles` of them.
// parts: as mx8_parts_bytes() says (block.h).
// From 20 rows an expert on: by strips and by tiles of 128 rows, 8 experts of d = 4096,
// d_ff = 14336 take 319 and 380 us with 16 rows each, 522 and 411 - 447 with 32; 256
// of d = 7168, d_ff = 2048 2.52 and 2.40 ms with 16, 3.75 and 2.58 with 32; 64 of d =
// 2048, d_ff = 1408 166 and 163 us with 24, 298 and 186 with 48 (before down's tiles
// were split).
inline bool mx8_many(int64_t copies, int64_t experts) { return copies > 20 * experts; }
int mx8_tile_rows(int64_t copies, int64_t experts);
hipError_t launch_mx8_tiles(const Mx8Gemm& a, bool gate_up, int E, int64_t tiles, int tile_rows, hipStream_t s);

}  // namespace moe
