// The 8-bit format (moe_mx8_t in moe.h): e4m3 codes with a power-of-two scale for
// every 32 columns of a row, as the scaled matrix instructions take them.
#pragma once

#include "block.h"

namespace moe {

// Bits of |v|'s largest (integer order: infinities above numbers, NaN above
// those) -> the group's scale byte: the exponent, biased by 127, of the smallest
// power of two of which 448 times reaches it, at least 2^-126; 127 for zeros; 255
// (NaN) where the group has an infinity or a NaN. 448 = 1.75 2^8: the exponent is
// that of the largest less 8, one more where its mantissa is above 1.75.
__device__ inline uint32_t mx8_scale_byte(uint32_t big) {
  const int b = static_cast<int>((big + 0x1fffffu) >> 23) - 8;
  return big >= 0x7f800000u ? 255u : big == 0 ? 127u : static_cast<uint32_t>(b < 1 ? 1 : b);
}

// 1 / scale as a float (byte 1 .. 247; NaN for 255: every code of the group becomes NaN).
__device__ inline float mx8_inverse(uint32_t byte) {
  return __uint_as_float(byte == 255 ? 0x7fc00000u : (254u - byte) << 23);
}

__device__ inline float mx8_value(uint32_t byte) {
  return __uint_as_float(byte == 255 ? 0x7fc00000u : byte == 0 ? 0x00400000u : byte << 23);
}

// Four codes, rounded to the nearest with ties to even.
__device__ inline uint32_t mx8_codes(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  return static_cast<uint32_t>(w);
}

// The scale dword (bytes b of columns 32 b .. of a 128-column step) of row n of N, step s.
__host__ __device__ inline int64_t mx8_scale_at(int64_t s, int64_t N, int64_t n) { return s * N + n; }

}  // namespace moe
