// What the layer's backward needs where the routing was given from outside: the
// weights' gradients and the experts' part of dx by itself (gfx950).
//
// Source: "Expert Parallelism & All-to-All" (neelmishra.github.io), "All-to-all: the
// distributed transpose" - the backward of the dispatch adds up the copies.
#include "block.h"

namespace moe {
namespace {

// The gradient of a weight is dw_j = <dout, y_j> = <dout Wd, h_j>, whatever the weight
// is. The experts' gradients need dh_j = (w_j dout) Wd, and with a weight of ordinary
// size dw_j = <dh_j, h_j> / w_j comes with it. With a weight of 0 nothing of <dout,
// y_j> is left in dh_j, and with a tiny or huge one w_j dout leaves the type's range:
// such a copy's dy is dout as it is (a weight of 1, split_weights_kernel), and its dy
// and dh are multiplied by the weight after dw_j has been formed. Between 2^-40 and
// 2^40 w dout keeps its bits for every |dout| from 2^-86 to 2^87; a softmax reaches
// 2^-40 where two scores are 28 apart.
constexpr float kLeastWeight = 0x1p-40f, kMostWeight = 0x1p40f;

__device__ inline bool ordinary(float w) { return fabsf(w) >= kLeastWeight && fabsf(w) <= kMostWeight; }

__global__ __launch_bounds__(256) void split_weights_kernel(const float* __restrict__ w, int64_t n,
                                                            float* __restrict__ first) {
  const int64_t i = blockIdx.x * 256ll + threadIdx.x;
  if (i < n) first[i] = ordinary(w[i]) ? w[i] : 1.f;
}

template <bool BF16>
__device__ inline void unpack(uint4 w, float (&v)[BF16 ? 8 : 4]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if constexpr (BF16) {
      v[2 * q] = __uint_as_float(u[q] << 16);
      v[2 * q + 1] = __uint_as_float(u[q] & 0xffff0000u);
    } else {
      v[q] = __uint_as_float(u[q]);
    }
}

template <bool BF16>
__device__ inline uint4 pack(const float (&v)[BF16 ? 8 : 4]) {
  uint32_t u[4];
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if constexpr (BF16)
      u[q] = f32_to_bf16(v[2 * q]) | static_cast<uint32_t>(f32_to_bf16(v[2 * q + 1])) << 16;
    else
      u[q] = __float_as_uint(v[q]);
  return uint4{u[0], u[1], u[2], u[3]};
}

template <bool BF16>
__device__ inline void scale_row(uint4* row, int64_t V, float w, int lane) {
  constexpr int P = BF16 ? 8 : 4;
  for (int64_t v = lane; v < V; v += 64) {
    float f[P];
    unpack<BF16>(row[v], f);
#pragma unroll
    for (int i = 0; i < P; ++i) f[i] *= w;
    row[v] = pack<BF16>(f);
  }
}

// One wave a token. V, VF: words of a row of dy and of dh.
template <bool BF16>
__global__ __launch_bounds__(256) void weight_grad_kernel(uint4* __restrict__ dh, const uint4* __restrict__ h,
                                                          uint4* __restrict__ dy, const int32_t* __restrict__ idx,
                                                          const float* __restrict__ w, const int32_t* __restrict__ slot,
                                                          int64_t T, int k, int64_t C, int64_t V, int64_t VF,
                                                          float* __restrict__ dw) {
  constexpr int P = BF16 ? 8 : 4;
  const int lane = threadIdx.x & 63;
  const int64_t t = blockIdx.x * 4ll + (threadIdx.x >> 6);
  if (t >= T) return;  // whole waves, no barrier below
  for (int j = 0; j < k; ++j) {
    const int s = __builtin_amdgcn_readfirstlane(slot[t * k + j]);
    float g = 0.f;  // of a dropped copy
    if (s >= 0) {
      const int64_t row = static_cast<int64_t>(__builtin_amdgcn_readfirstlane(idx[t * k + j])) * C + s;
      const float wj = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(w[t * k + j])));
      float part = 0.f;
      for (int64_t v = lane; v < VF; v += 64) {
        float a[P], b[P];
        unpack<BF16>(dh[row * VF + v], a);
        unpack<BF16>(h[row * VF + v], b);
#pragma unroll
        for (int i = 0; i < P; ++i) part = fmaf(a[i], b[i], part);
      }
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) part += __shfl_xor(part, off, 64);
      if (ordinary(wj)) {
        g = part / wj;
      } else {
        g = part;
        scale_row<BF16>(dh + row * VF, VF, wj, lane);
        scale_row<BF16>(dy + row * V, V, wj, lane);
      }
    }
    if (lane == 0) dw[t * k + j] = g;
  }
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
    float f[P];
    unpack<BF16>(load_stream(dX + (static_cast<int64_t>(idx[t * k + j]) * C + s) * V + v), f);
#pragma unroll
    for (int i = 0; i < P; ++i) acc[i] += f[i];
  }
  store_stream(dx + t * V + v, pack<BF16>(acc));
}

}  // namespace

hipError_t launch_split_weights(const float* w, int64_t n, float* first, hipStream_t s) {
  split_weights_kernel<<<dim3(static_cast<unsigned>(ceil_div(n, 256))), dim3(256), 0, s>>>(w, n, first);
  return hipGetLastError();
}

hipError_t launch_weight_grad(void* dh, const void* h, void* dy, const int32_t* idx, const float* w, const int32_t* slot,
                              int64_t T, int64_t d, int64_t F, int k, int64_t C, bool bf16, float* dw, hipStream_t s) {
  const int64_t per = bf16 ? 8 : 4;
  const dim3 grid(static_cast<unsigned>(ceil_div(T, 4)));
  auto* a = static_cast<uint4*>(dh);
  const auto* b = static_cast<const uint4*>(h);
  auto* c = static_cast<uint4*>(dy);
  if (bf16)
    weight_grad_kernel<true><<<grid, dim3(256), 0, s>>>(a, b, c, idx, w, slot, T, k, C, d / per, F / per, dw);
  else
    weight_grad_kernel<false><<<grid, dim3(256), 0, s>>>(a, b, c, idx, w, slot, T, k, C, d / per, F / per, dw);
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
