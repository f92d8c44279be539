// Making 4-bit weights and reading them back (layout: q4.h). Both are one pass
// over memory: a wave takes a tile of 16 rows by 128 columns, a lane the 32
// columns of one row that its 16 bytes of codes hold, so codes are written and
// read as 1 KiB in a row and the rows in whole 128-byte lines. The four lanes of
// a row join their extremes by shuffles. Bound by memory: 4 x 14336 x 4096 bf16
// (470 MB, and 120 MB of u4) quantised in 113 - 142 us and read back in 105 - 121,
// 4.2 - 5.6 TB/s, where a plain copy reaches 4.7. With half lines, through the
// caches, these took 176 and 127 us, a division for each weight included.
#include "common.h"
#include "few.h"
#include "q4.h"

#include <type_traits>

namespace moe {
namespace {

// A tile's 16 rows in whole 128-byte lines: lane l has 16-byte piece
// piece_at(l) of row l % 8, and of row 8 + l % 8, of a line; operands() turns
// these into two pieces of row l % 16 and back. Two lines of bf16 (four of fp32)
// make a tile; whole lines can stream past the caches.
template <typename T>
struct Lines {
  static constexpr int kPer = 16 / sizeof(T), kLines = sizeof(T) == 2 ? 2 : 4;  // elements of a piece; lines of a tile
  static __device__ inline int piece_at(int lane) {
    const int quad = lane >> 4, half = (lane >> 3) & 1;
    // bf16: pieces quad and quad + 4, eight columns each, of steps 2 line and
    // 2 line + 1; fp32: 2 quad and 2 quad + 1, the eight columns of step `line`
    return sizeof(T) == 2 ? quad + 4 * half : 2 * quad + half;
  }
};

// The lane's columns of the tile at row n0 and column c0 of matrix W [N, K]: v[s]
// are the columns c0 + 32 s + 8 (l / 16) .. + 7 of row n0 + l % 16, 0 past the
// matrix (K is a multiple of 8).
template <typename T>
__device__ inline void load_tile(const T* W, int64_t n0, int64_t c0, int64_t N, int64_t K, float (&v)[4][8]) {
  using L = Lines<T>;
  const int lane = threadIdx.x & 63, r = lane & 7;
  u32x4 lo[L::kLines], hi[L::kLines];
#pragma unroll
  for (int i = 0; i < L::kLines; ++i) {
    const int64_t c = c0 + i * 8 * L::kPer + L::piece_at(lane) * L::kPer;
    lo[i] = hi[i] = u32x4{0, 0, 0, 0};
    if (c < K && n0 + r < N) lo[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(W + (n0 + r) * K + c));
    if (c < K && n0 + 8 + r < N)
      hi[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(W + (n0 + 8 + r) * K + c));
  }
#pragma unroll
  for (int i = 0; i < L::kLines; ++i) {
    u32x4 a0, a1;
    operands(lo[i], hi[i], a0, a1);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if constexpr (sizeof(T) == 2) {
        v[2 * i][2 * q] = __uint_as_float(a0[q] << 16);
        v[2 * i][2 * q + 1] = __uint_as_float(a0[q] & 0xffff0000u);
        v[2 * i + 1][2 * q] = __uint_as_float(a1[q] << 16);
        v[2 * i + 1][2 * q + 1] = __uint_as_float(a1[q] & 0xffff0000u);
      } else {
        v[i][q] = __uint_as_float(a0[q]);
        v[i][4 + q] = __uint_as_float(a1[q]);
      }
  }
}

// The other way: v rounded to T, into the tile.
template <typename T>
__device__ inline void store_tile(T* W, int64_t n0, int64_t c0, int64_t N, int64_t K, const float (&v)[4][8]) {
  using L = Lines<T>;
  const int lane = threadIdx.x & 63, r = lane & 7;
#pragma unroll
  for (int i = 0; i < L::kLines; ++i) {
    u32x4 a0, a1, lo, hi;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if constexpr (sizeof(T) == 2) {
        a0[q] = f32_to_bf16(v[2 * i][2 * q]) | static_cast<uint32_t>(f32_to_bf16(v[2 * i][2 * q + 1])) << 16;
        a1[q] = f32_to_bf16(v[2 * i + 1][2 * q]) | static_cast<uint32_t>(f32_to_bf16(v[2 * i + 1][2 * q + 1])) << 16;
      } else {
        a0[q] = __float_as_uint(v[i][q]);
        a1[q] = __float_as_uint(v[i][4 + q]);
      }
    operands(a0, a1, lo, hi);
    const int64_t c = c0 + i * 8 * L::kPer + L::piece_at(lane) * L::kPer;
    if (c < K && n0 + r < N) __builtin_nontemporal_store(lo, reinterpret_cast<u32x4*>(W + (n0 + r) * K + c));
    if (c < K && n0 + 8 + r < N) __builtin_nontemporal_store(hi, reinterpret_cast<u32x4*>(W + (n0 + 8 + r) * K + c));
  }
}

// v / sc, rounded as the division rounds it, without a division for each v: inv
// is the rounded 1 / sc, and the product's remainder, exact in an fma, corrects
// it to v / sc (1 + 2^-46) before the last rounding. That rounds the same way, as
// no quotient of a 24-bit by an 8-bit number lies nearer than 2^-33 of its value
// to a midpoint of two floats. Below 1/4, where every code is the nearest one,
// the remainder may underflow. Scales that are tiny, 0 or infinite divide.
struct Quotient {
  float sc, inv;
  bool ordinary;
  __device__ explicit Quotient(float s) : sc(s), ordinary(s >= 0x1p-100f && s < 0x1p127f) {
    inv = 1.f / (ordinary ? s : 1.f);
  }
  __device__ float fast(float v) const {
    const float r = v * inv;
    return fmaf(fmaf(-r, sc, v), inv, r);
  }
  __device__ float operator()(float v) const { return ordinary ? fast(v) : sc > 0.f ? v / sc : 0.f; }
};

// The eight codes of v / sc as a word.
template <bool U4>
__device__ inline uint32_t codes_of(const float (&v)[8], const Quotient& by, float z) {
  float r[8];
  if (by.ordinary) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = by.fast(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = by(v[i]);
  }
  uint32_t w = 0;
  if constexpr (U4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w |= static_cast<uint32_t>(__builtin_amdgcn_fmed3f(rintf(r[i]) + z, 0.f, 15.f)) << q4_shift(true, i);
  } else {  // the conversion rounds ties to the even code and takes 6 for more
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, r[0], r[1], 1.0f, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, r[2], r[3], 1.0f, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, r[4], r[5], 1.0f, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, r[6], r[7], 1.0f, 3);
  }
  return w;
}

template <typename T, bool U4>
__global__ __launch_bounds__(256) void quantize_kernel(const T* __restrict__ W, int64_t tiles, int64_t N, int64_t K,
                                                       int group, uint4* __restrict__ codes, bf16_t* __restrict__ scale,
                                                       uint8_t* __restrict__ zero) {
  const int lane = threadIdx.x & 63, quad = lane >> 4;
  const int64_t nt = ceil_div(N, 16), kt = ceil_div(K, 128);
  const int64_t tile = blockIdx.x * 4ll + (threadIdx.x >> 6);
  if (tile >= tiles) return;
  const int64_t strip = tile / kt, j = tile % kt, e = strip / nt;
  float v[4][8], lo[4], hi[4];
  load_tile(W + e * N * K, (strip % nt) * 16, j * 128, N, K, v);
#pragma unroll
  for (int s = 0; s < 4; ++s) {
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
    const Quotient by(bf16_to_f32(sb));
    const float z = U4 && zero ? fminf(fmaxf(rintf(by(-lo[s])), 0.f), 15.f) : 8.f;
    word[s] = codes_of<U4>(v[s], by, z);
    if (quad == 0 && s % gs == 0) {
      const int64_t at = (tile * (4 / gs) + s / gs) * 16 + lane;
      scale[at] = sb;
      if (U4 && zero) zero[at] = static_cast<uint8_t>(z);
    }
  }
  __builtin_nontemporal_store(u32x4{word[0], word[1], word[2], word[3]}, reinterpret_cast<u32x4*>(codes + tile * 64 + lane));
}

template <typename T, bool U4>
__global__ __launch_bounds__(256) void dequantize_kernel(const uint4* __restrict__ codes,
                                                         const bf16_t* __restrict__ scale,
                                                         const uint8_t* __restrict__ zero, int64_t tiles, int64_t N,
                                                         int64_t K, int group, T* __restrict__ W) {
  const int lane = threadIdx.x & 63;
  const int64_t nt = ceil_div(N, 16), kt = ceil_div(K, 128);
  const int64_t tile = blockIdx.x * 4ll + (threadIdx.x >> 6);
  if (tile >= tiles) return;
  const int64_t strip = tile / kt, j = tile % kt, e = strip / nt;
  const u32x4 word = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(codes + tile * 64 + lane));
  float v[4][8];
  const int gs = group / 32;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int64_t at = (tile * (4 / gs) + s / gs) * 16 + (lane & 15);
    const float sc = bf16_to_f32(scale[at]);
    const float z = U4 ? (zero ? static_cast<float>(zero[at]) : 8.f) + 16.f : 0.f;
    const bf16x8 q = q4_decode<U4>(word[s]);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[s][i] = (static_cast<float>(q[i]) - z) * sc;  // exact: 5 bits times 8
  }
  store_tile(W + e * N * K, (strip % nt) * 16, j * 128, N, K, v);
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
