// What the layer's backward needs where the routing was given from outside: the
// weights' gradients and the experts' part of dx by itself (gfx950).
//
// Source: "Expert Parallelism & All-to-All" (neelmishra.github.io), "All-to-all: the
// distributed transpose" - the backward of the dispatch adds up the copies.
#include "block.h"

namespace moe {
namespace {

// q_j = <dh_j, h_j> = w_j <dout, y_j> is what the hidden gradients give; with w_j = 0
// they hold nothing of <dout, y_j>, and the gradient is taken as 0 (a gate whose
// score is 0 passes none on).
__global__ __launch_bounds__(256) void weight_grad_kernel(const float* __restrict__ q, const float* __restrict__ w,
                                                          int64_t n, float* __restrict__ dw) {
  const int64_t i = blockIdx.x * 256ll + threadIdx.x;
  if (i < n) dw[i] = w[i] != 0.f ? q[i] / w[i] : 0.f;
}

__global__ __launch_bounds__(256) void zero_kernel(float* p, int64_t n) {
  const int64_t i = blockIdx.x * 256ll + threadIdx.x;
  if (i < n) p[i] = 0.f;
}

// dx[t] = sum over the kept copies of dX[e_j, s_j], j ascending, in fp32, rounded once.
template <bool BF16>
__global__ __launch_bounds__(256) void gather_copies_kernel(const uint4* __restrict__ dX, const int32_t* __restrict__ idx,
                                                            const int32_t* __restrict__ slot, int k, int64_t C, int64_t V,
                                                            int64_t blocks, uint4* __restrict__ dx) {
  constexpr int P = BF16 ? 8 : 4;
  const int64_t t = blockIdx.x / blocks, v = blockIdx.x % blocks * 256 + threadIdx.x;
  if (v >= V) return;
  float acc[P];
#pragma unroll
  for (int i = 0; i < P; ++i) acc[i] = 0.f;
  for (int j = 0; j < k; ++j) {
    const int s = slot[t * k + j];
    if (s < 0) continue;
    const uint4 word = load_stream(dX + (static_cast<int64_t>(idx[t * k + j]) * C + s) * V + v);
    const uint32_t u[4] = {word.x, word.y, word.z, word.w};
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if constexpr (BF16) {
        acc[2 * q] += __uint_as_float(u[q] << 16);
        acc[2 * q + 1] += __uint_as_float(u[q] & 0xffff0000u);
      } else {
        acc[q] += __uint_as_float(u[q]);
      }
  }
  uint32_t u[4];
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if constexpr (BF16)
      u[q] = f32_to_bf16(acc[2 * q]) | static_cast<uint32_t>(f32_to_bf16(acc[2 * q + 1])) << 16;
    else
      u[q] = __float_as_uint(acc[q]);
  store_stream(dx + t * V + v, uint4{u[0], u[1], u[2], u[3]});
}

}  // namespace

hipError_t launch_zero(float* p, int64_t n, hipStream_t s) {
  zero_kernel<<<dim3(static_cast<unsigned>(ceil_div(n, 256))), dim3(256), 0, s>>>(p, n);
  return hipGetLastError();
}

hipError_t launch_weight_grad(const float* q, const float* w, int64_t n, float* dw, hipStream_t s) {
  weight_grad_kernel<<<dim3(static_cast<unsigned>(ceil_div(n, 256))), dim3(256), 0, s>>>(q, w, n, dw);
  return hipGetLastError();
}

hipError_t launch_gather_copies(const void* dX, const int32_t* idx, const int32_t* slot, int64_t T, int64_t d, int k,
                                int64_t C, bool bf16, void* dx, hipStream_t s) {
  const int64_t V = d * (bf16 ? 2 : 4) / 16, blocks = ceil_div(V, 256);
  const dim3 grid(static_cast<unsigned>(T * blocks));
  const auto* in = static_cast<const uint4*>(dX);
  auto* out = static_cast<uint4*>(dx);
  if (bf16)
    gather_copies_kernel<true><<<grid, dim3(256), 0, s>>>(in, idx, slot, k, C, V, blocks, out);
  else
    gather_copies_kernel<false><<<grid, dim3(256), 0, s>>>(in, idx, slot, k, C, V, blocks, out);
  return hipGetLastError();
}

}  // namespace moe
