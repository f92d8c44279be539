// Making 8-bit matrices and reading them back (format: mx8.h). One pass over
// memory: 16 lanes (bf16; 32 in fp32) take a row's 128 columns, so that rows are
// read and codes written in whole 128-byte lines, and a wave's rows' scales stand
// next to each other. Bound by memory.
#include "mx8.h"

namespace moe {
namespace {

template <typename T>
constexpr int kPer = 16 / sizeof(T);  // elements of a lane's 16 bytes
template <typename T>
constexpr int kLanes = 128 / kPer<T>;  // lanes of a row's step
constexpr int kPasses = 4;             // rows a lane takes, one after the other

template <typename T>
__device__ inline void unpack(uint4 w, float (&v)[kPer<T>]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if constexpr (sizeof(T) == 2) {
      v[2 * q] = __uint_as_float(u[q] << 16);
      v[2 * q + 1] = __uint_as_float(u[q] & 0xffff0000u);
    } else {
      v[q] = __uint_as_float(u[q]);
    }
}

// A unit is a step of 128 columns of kPasses * 64 / kLanes rows; a wave takes one.
template <typename T>
__global__ __launch_bounds__(256) void quantize_mx8_kernel(const T* __restrict__ W, int64_t units, int64_t N, int64_t K,
                                                           uint8_t* __restrict__ codes, uint32_t* __restrict__ scale) {
  constexpr int P = kPer<T>, L = kLanes<T>, ROWS = 64 / L;
  const int lane = threadIdx.x & 63, sub = lane % L;
  const int64_t unit = blockIdx.x * 4ll + (threadIdx.x >> 6);
  if (unit >= units) return;
  const int64_t steps = ceil_div(K, 128), blocks = ceil_div(N, ROWS * kPasses);
  const int64_t s = unit % steps, nb = unit / steps % blocks, e = unit / steps / blocks;
  const int64_t c = s * 128 + sub * P;
  uint4 in[kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int64_t n = (nb * kPasses + p) * ROWS + lane / L;
    in[p] = uint4{0, 0, 0, 0};
    if (n < N && c < K) in[p] = load_stream(reinterpret_cast<const uint4*>(W + (e * N + n) * K + c));
  }
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int64_t n = (nb * kPasses + p) * ROWS + lane / L;
    float v[P];
    unpack<T>(in[p], v);
    uint32_t big = 0;
#pragma unroll
    for (int i = 0; i < P; ++i) big = max(big, __float_as_uint(v[i]) & 0x7fffffffu);
#pragma unroll
    for (int off = 1; off < 32 / P; off <<= 1) big = max(big, static_cast<uint32_t>(__shfl_xor(big, off, 64)));
    const uint32_t byte = mx8_scale_byte(big);
    const float inv = mx8_inverse(byte);
    uint32_t word = 0;  // the row's four bytes
#pragma unroll
    for (int b = 0; b < 4; ++b) word |= static_cast<uint32_t>(__shfl(byte, (lane & ~(L - 1)) + b * (L / 4), 64)) << (8 * b);
    if (n >= N) continue;
    if (sub == 0) scale[e * steps * N + mx8_scale_at(s, N, n)] = word;
    if (c >= K) continue;
    uint8_t* to = codes + (e * N + n) * K + c;
    const uint32_t lo = mx8_codes(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    if constexpr (P == 8) {
      *reinterpret_cast<uint2*>(to) = uint2{lo, mx8_codes(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv)};
    } else {
      *reinterpret_cast<uint32_t*>(to) = lo;
    }
  }
}

template <typename T>
__global__ __launch_bounds__(256) void dequantize_mx8_kernel(const uint8_t* __restrict__ codes,
                                                             const uint32_t* __restrict__ scale, int64_t units, int64_t N,
                                                             int64_t K, T* __restrict__ W) {
  constexpr int P = kPer<T>, L = kLanes<T>, ROWS = 64 / L;
  const int lane = threadIdx.x & 63, sub = lane % L;
  const int64_t unit = blockIdx.x * 4ll + (threadIdx.x >> 6);
  if (unit >= units) return;
  const int64_t steps = ceil_div(K, 128), blocks = ceil_div(N, ROWS * kPasses);
  const int64_t s = unit % steps, nb = unit / steps % blocks, e = unit / steps / blocks;
  const int64_t c = s * 128 + sub * P;
  uint32_t in[kPasses][P / 4], sc[kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int64_t n = (nb * kPasses + p) * ROWS + lane / L;
#pragma unroll
    for (int q = 0; q < P / 4; ++q) in[p][q] = 0;
    sc[p] = 0;
    if (n < N && c < K) {
      const uint8_t* from = codes + (e * N + n) * K + c;
#pragma unroll
      for (int q = 0; q < P / 4; ++q) in[p][q] = reinterpret_cast<const uint32_t*>(from)[q];
      sc[p] = scale[e * steps * N + mx8_scale_at(s, N, n)];
    }
  }
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int64_t n = (nb * kPasses + p) * ROWS + lane / L;
    if (n >= N || c >= K) continue;
    const float two = mx8_value(sc[p] >> (8 * (sub * P / 32)) & 255);
    uint32_t out[4];
#pragma unroll
    for (int q = 0; q < P / 4; ++q) {
      const int w = static_cast<int>(in[p][q]);
      const float a = __builtin_amdgcn_cvt_f32_fp8(w, 0) * two, b = __builtin_amdgcn_cvt_f32_fp8(w, 1) * two;
      const float g = __builtin_amdgcn_cvt_f32_fp8(w, 2) * two, d = __builtin_amdgcn_cvt_f32_fp8(w, 3) * two;
      if constexpr (sizeof(T) == 2) {
        out[2 * q] = f32_to_bf16(a) | static_cast<uint32_t>(f32_to_bf16(b)) << 16;
        out[2 * q + 1] = f32_to_bf16(g) | static_cast<uint32_t>(f32_to_bf16(d)) << 16;
      } else {
        out[0] = __float_as_uint(a);
        out[1] = __float_as_uint(b);
        out[2] = __float_as_uint(g);
        out[3] = __float_as_uint(d);
      }
    }
    store_stream(reinterpret_cast<uint4*>(W + (e * N + n) * K + c), uint4{out[0], out[1], out[2], out[3]});
  }
}

}  // namespace

int64_t mx8_units(int64_t E, int64_t N, int64_t K, bool bf16) {
  return E * ceil_div(N, (bf16 ? 64 / kLanes<bf16_t> : 64 / kLanes<float>) * kPasses) * ceil_div(K, 128);
}

hipError_t launch_mx8_quantize(const void* W, bool bf16, int64_t E, int64_t N, int64_t K, uint8_t* codes, uint32_t* scale,
                               hipStream_t s) {
  const int64_t units = mx8_units(E, N, K, bf16);
  const dim3 grid(static_cast<unsigned>(ceil_div(units, 4)));
  if (bf16)
    quantize_mx8_kernel<bf16_t><<<grid, dim3(256), 0, s>>>(static_cast<const bf16_t*>(W), units, N, K, codes, scale);
  else
    quantize_mx8_kernel<float><<<grid, dim3(256), 0, s>>>(static_cast<const float*>(W), units, N, K, codes, scale);
  return hipGetLastError();
}

hipError_t launch_mx8_dequantize(const uint8_t* codes, const uint32_t* scale, int64_t E, int64_t N, int64_t K, bool bf16,
                                 void* W, hipStream_t s) {
  const int64_t units = mx8_units(E, N, K, bf16);
  const dim3 grid(static_cast<unsigned>(ceil_div(units, 4)));
  if (bf16)
    dequantize_mx8_kernel<bf16_t><<<grid, dim3(256), 0, s>>>(codes, scale, units, N, K, static_cast<bf16_t*>(W));
  else
    dequantize_mx8_kernel<float><<<grid, dim3(256), 0, s>>>(codes, scale, units, N, K, static_cast<float*>(W));
  return hipGetLastError();
}

}  // namespace moe
