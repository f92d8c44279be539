// The 4-bit weight layout, its codes in registers, and the split of fp32 into
// bf16 parts, shared by the kernels that make and read such weights.
#pragma once

#include "common.h"

namespace moe {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// The A operands of a line's two steps from the loads of rows 0 - 7 and 8 - 15:
// step 0 wants piece l / 16 of row l % 16, so lanes 8 - 15 of every 16 take
// the other load's lanes 0 - 7; step 1 the other way round.
__device__ inline void operands(u32x4 lo, u32x4 hi, u32x4& a0, u32x4& a1) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    constexpr int kRotate8 = 0x128;
    a0[i] = __builtin_amdgcn_update_dpp(lo[i], hi[i], kRotate8, 0xf, 0xc, false);
    a1[i] = __builtin_amdgcn_update_dpp(hi[i], lo[i], kRotate8, 0xf, 0x3, false);
  }
}

// A matrix stack [E, N, K] in 4 bits (the layout of moe_q4_t in moe.h): tiles
// of 16 rows by 128 columns, 1024 bytes each, [E][ceil(N/16)][ceil(K/128)].
// Lane l of a wave owns 16 bytes of a tile, row l % 16 and, in word s, the
// columns 32 s + 8 (l / 16) .. + 7: its share of the A operand of four
// 16x16x32 matrix instructions, so one 16-byte load a lane, 1 KiB in a row for
// the wave, feeds them.
//
// u4: nibble n of a word holds column 2 n (n < 4) or 2 n - 7. Column pair
// (2 p, 2 p + 1) then sits at bits 4 p and 16 + 4 p, and one shift and one
// and-or make both halves of a bf16 pair: the code goes into the upper four of
// the seven mantissa bits of 16.0, which makes it 16 + q exactly.
// e2m1: nibble n holds column n; the conversion instruction takes a byte at a
// time, two neighbouring columns.
template <bool U4>
__device__ inline bf16x8 q4_decode(uint32_t w) {
  if constexpr (U4) {
    // Opaque constants: of two literals the compiler would split the and-or in two. The instruction itself is the
    // compiler's, which then keeps the wait states between it and the matrix instructions that use the same registers
    // (around an instruction in inline assembly it keeps none).
    uint32_t mask = 0x00780078u, sixteen = 0x41804180u;
    asm("" : "+s"(mask));
    asm("" : "+v"(sixteen));
    u32x4 v;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const uint32_t shifted = p == 0 ? w << 3 : w >> (4 * p - 3);
      v[p] = (shifted & mask) | sixteen;
    }
    return __builtin_bit_cast(bf16x8, v);
  } else {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 0),
                 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 1),
                 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 2),
                 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 3);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
  }
}

// Bit position of column i (0 .. 7) of a lane's eight in its word.
__device__ inline int q4_shift(bool u4, int i) { return u4 ? ((i & 1) ? 16 + 2 * (i - 1) : 2 * i) : 4 * i; }

// v as the exact sum of three bf16 numbers: each takes the leading 8 of the
// bits that are left (24 in all), by cutting off the rest. An infinity is the
// first of them alone.
__device__ inline void split3(float v, bf16_t (&q)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const uint32_t top = __float_as_uint(v) & 0xffff0000u;
    q[i] = static_cast<bf16_t>(top >> 16);
    v = v == __uint_as_float(top) ? 0.f : v - __uint_as_float(top);
  }
}

// The three parts of n floats, parts [3][n]: this thread's share.
__device__ inline void split_rows(const float* x, int64_t n, bf16_t* parts, int64_t first, int64_t stride) {
  for (int64_t i = first; i < n; i += stride) {
    bf16_t q[3];
    split3(x[i], q);
    parts[i] = q[0];
    parts[n + i] = q[1];
    parts[2 * n + i] = q[2];
  }
}

}  // namespace moe
