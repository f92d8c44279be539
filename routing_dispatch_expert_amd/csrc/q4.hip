// Making 4-bit weights and reading them back (layout: q4.h). Both are one pass
// over memory: a wave takes a tile of 16 rows by 128 columns, a lane the 32
// columns of one row that its 16 bytes of codes hold, so codes are written and
// read as 1 KiB in a row and the rows in pieces of 64 bytes (bf16) a load. The
// four lanes of a row join their extremes by shuffles.
#include "common.h"
#include "q4.h"

#include <type_traits>

namespace moe {
namespace {

// The lane's eight columns c .. c + 7 of row `row`, 0 past the matrix (K is a
// multiple of 8, so all eight are inside or none).
template <typename T>
__device__ inline void load_cols(const T* row, int64_t c, bool in, float (&v)[8]) {
  if (!in) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
  } else if constexpr (sizeof(T) == 2) {
    const bf16x8 b = *reinterpret_cast<const bf16x8*>(row + c);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = static_cast<float>(b[i]);
  } else {
    const f32x4 a = *reinterpret_cast<const f32x4*>(row + c), b = *reinterpret_cast<const f32x4*>(row + c + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  }
}

// Code of the E2M1 value nearest to r (ties to the even code, 6 for more).
__device__ inline uint32_t e2m1_code(float r) {
  const float a = fabsf(r);
  const uint32_t m = (a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) + (a >= 3.5f) + (a > 5.f);
  return m | (r < 0.f ? 8u : 0u);
}

template <typename T, bool U4>
__global__ __launch_bounds__(256) void quantize_kernel(const T* __restrict__ W, int64_t tiles, int64_t N, int64_t K,
                                                       int group, uint4* __restrict__ codes, bf16_t* __restrict__ scale,
                                                       uint8_t* __restrict__ zero) {
  const int lane = threadIdx.x & 63, quad = lane >> 4;
  const int64_t nt = ceil_div(N, 16), kt = ceil_div(K, 128);
  const int64_t tile = blockIdx.x * 4ll + (threadIdx.x >> 6);
  if (tile >= tiles) return;
  const int64_t strip = tile / kt, j = tile % kt, e = strip / nt, n = (strip % nt) * 16 + (lane & 15);
  const T* row = W + (e * N + n) * K;
  float v[4][8], lo[4], hi[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int64_t c = j * 128 + 32 * s + 8 * quad;
    load_cols(row, c, n < N && c < K, v[s]);
    lo[s] = 0.f;
    hi[s] = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo[s] = fminf(lo[s], v[s][i]);
      hi[s] = fmaxf(hi[s], v[s][i]);
    }
#pragma unroll
    for (int off = 16; off < 64; off <<= 1) {
      lo[s] = fminf(lo[s], __shfl_xor(lo[s], off));
      hi[s] = fmaxf(hi[s], __shfl_xor(hi[s], off));
    }
  }
  if (group > 32) {
#pragma unroll
    for (int s = 0; s < 4; s += 2) {
      lo[s] = lo[s + 1] = fminf(lo[s], lo[s + 1]);
      hi[s] = hi[s + 1] = fmaxf(hi[s], hi[s + 1]);
    }
  }
  if (group > 64) {
    lo[0] = lo[1] = lo[2] = lo[3] = fminf(lo[0], lo[2]);
    hi[0] = hi[1] = hi[2] = hi[3] = fmaxf(hi[0], hi[2]);
  }
  uint32_t word[4];
  const int gs = group / 32;  // words of a group
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const float big = fmaxf(hi[s], -lo[s]);
    // times the constants' fp32 reciprocals, as moe.h defines the scales
    const float span = !U4 ? big * (1.f / 6.f) : zero ? (hi[s] - lo[s]) * (1.f / 15.f) : big * (1.f / 7.f);
    const bf16_t sb = f32_to_bf16(span);
    const float sc = bf16_to_f32(sb);
    float z = zero ? 0.f : 8.f;
    if (U4 && zero && sc > 0.f) z = fminf(fmaxf(rintf(-lo[s] / sc), 0.f), 15.f);
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float r = sc > 0.f ? v[s][i] / sc : 0.f;
      const uint32_t q = U4 ? static_cast<uint32_t>(fminf(fmaxf(rintf(r) + z, 0.f), 15.f)) : e2m1_code(r);
      w |= q << q4_shift(U4, i);
    }
    word[s] = w;
    if (quad == 0 && s % gs == 0) {
      const int64_t at = (tile * (4 / gs) + s / gs) * 16 + lane;
      scale[at] = sb;
      if (U4 && zero) zero[at] = static_cast<uint8_t>(z);
    }
  }
  codes[tile * 64 + lane] = uint4{word[0], word[1], word[2], word[3]};
}

template <typename T, bool U4>
__global__ __launch_bounds__(256) void dequantize_kernel(const uint4* __restrict__ codes,
                                                         const bf16_t* __restrict__ scale,
                                                         const uint8_t* __restrict__ zero, int64_t tiles, int64_t N,
                                                         int64_t K, int group, T* __restrict__ W) {
  const int lane = threadIdx.x & 63, quad = lane >> 4;
  const int64_t nt = ceil_div(N, 16), kt = ceil_div(K, 128);
  const int64_t tile = blockIdx.x * 4ll + (threadIdx.x >> 6);
  if (tile >= tiles) return;
  const int64_t strip = tile / kt, j = tile % kt, e = strip / nt, n = (strip % nt) * 16 + (lane & 15);
  if (n >= N) return;
  const uint4 cw = codes[tile * 64 + lane];
  const uint32_t word[4] = {cw.x, cw.y, cw.z, cw.w};
  T* row = W + (e * N + n) * K;
  const int gs = group / 32;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int64_t c = j * 128 + 32 * s + 8 * quad;
    if (c >= K) break;
    const int64_t at = (tile * (4 / gs) + s / gs) * 16 + (lane & 15);
    const float sc = bf16_to_f32(scale[at]);
    const float z = U4 ? (zero ? static_cast<float>(zero[at]) : 8.f) + 16.f : 0.f;
    const bf16x8 q = q4_decode<U4>(word[s]);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (static_cast<float>(q[i]) - z) * sc;  // exact: 5 bits times 8
    if constexpr (sizeof(T) == 2) {
      bf16x8 o;
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = static_cast<__bf16>(v[i]);
      *reinterpret_cast<bf16x8*>(row + c) = o;
    } else {
      *reinterpret_cast<f32x4*>(row + c) = f32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4*>(row + c + 4) = f32x4{v[4], v[5], v[6], v[7]};
    }
  }
}

// f(element type, is U4) with compile-time arguments.
template <typename F>
void by_type(bool bf16, int kind, F&& f) {
  auto with = [&](auto elem) {
    if (kind == kQ4U4)
      f(elem, std::true_type{});
    else
      f(elem, std::false_type{});
  };
  if (bf16)
    with(bf16_t{});
  else
    with(float{});
}

}  // namespace

hipError_t launch_q4_quantize(const void* W, bool bf16, int E, int64_t N, int64_t K, int kind, int group, void* codes,
                              bf16_t* scale, uint8_t* zero, hipStream_t s) {
  const int64_t tiles = E * ceil_div(N, 16) * ceil_div(K, 128);
  by_type(bf16, kind, [&](auto elem, auto u4) {
    using T = decltype(elem);
    quantize_kernel<T, decltype(u4)::value><<<dim3(static_cast<unsigned>(ceil_div(tiles, 4))), dim3(256), 0, s>>>(
        static_cast<const T*>(W), tiles, N, K, group, static_cast<uint4*>(codes), scale, zero);
  });
  return hipGetLastError();
}

hipError_t launch_q4_dequantize(const void* codes, const bf16_t* scale, const uint8_t* zero, int E, int64_t N,
                                int64_t K, int kind, int group, bool bf16, void* W, hipStream_t s) {
  const int64_t tiles = E * ceil_div(N, 16) * ceil_div(K, 128);
  by_type(bf16, kind, [&](auto elem, auto u4) {
    using T = decltype(elem);
    dequantize_kernel<T, decltype(u4)::value><<<dim3(static_cast<unsigned>(ceil_div(tiles, 4))), dim3(256), 0, s>>>(
        static_cast<const uint4*>(codes), scale, zero, tiles, N, K, group, static_cast<T*>(W));
  });
  return hipGetLastError();
}

}  // namespace moe
