// What the kernels of the experts with 8-bit rows and weights share.
#pragma once

#include "mx8.h"

namespace moe {

typedef int i32x8 __attribute__((ext_vector_type(8)));

__device__ inline float silu(float g) { return g / (1.0f + expf(-g)); }

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
  void* y;            // else: [copies][N]
  bool y_bf16;
};

// Many rows an expert (mx8_tiles.hip): row tiles of mx8_tile_rows() rows, listed in
// ls.tile. Grid: at most `tiles` of them.
int mx8_tile_rows();
hipError_t launch_mx8_tiles(const Mx8Gemm& a, bool gate_up, int E, int64_t tiles, hipStream_t s);

}  // namespace moe
