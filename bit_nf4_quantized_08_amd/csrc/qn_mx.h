// MXFP4 encoding of a unit, eight consecutive elements of a row (gfx950): a quad
// of lanes holds one block of 32.  The block's largest magnitude is an integer
// maximum of the absolute bit patterns, whose exponent field gives the scale
// byte directly; the hardware conversion rounds x 2^-e to E2M1 (nearest even,
// saturating), the format's rule bit for bit, subnormal inputs included.
#pragma once

#include "qn_device.h"

namespace qn {

// dword t of v (a vector of four dwords per register quad).
template <int N>
__device__ __forceinline__ uint32_t dw(const u32x4 (&v)[N], int t) {
  const uint32_t w[4] = {v[t >> 2].x, v[t >> 2].y, v[t >> 2].z, v[t >> 2].w};
  return w[t & 3];
}

// Largest absolute bit pattern of a unit: bf16 pairs packed (result in 16 bits)
// or fp32.
template <bool BF16>
__device__ __forceinline__ uint32_t unit_amax(const u32x4 (&x)[BF16 ? 1 : 2]) {
  if constexpr (BF16) {
    u16x2 m = {0, 0};
#pragma unroll
    for (int t = 0; t < 4; ++t)
      m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, dw(x, t) & 0x7FFF7FFFu));
    return m.x > m.y ? m.x : m.y;
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int t = 0; t < 8; ++t) m = max(m, dw(x, t) & 0x7FFFFFFFu);
    return m;
  }
}

// Scale byte of a block from its largest absolute bit pattern: the exponent
// field less 2, at least 0; 255 for a block that is not finite.
template <bool BF16>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  const uint32_t e = amax >> (BF16 ? 7 : 23);
  return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}

// The unit's eight codes (one dword) under a scale byte.
template <bool BF16>
__device__ __forceinline__ uint32_t unit_codes(const u32x4 (&x)[BF16 ? 1 : 2], uint32_t byte) {
  const float sc = as_f32(byte << 23);   // the conversion reads the exponent field; 0 stands for 2^-127
  uint32_t c = 0;
  if constexpr (BF16) {
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, dw(x, 0)), sc, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, dw(x, 1)), sc, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, dw(x, 2)), sc, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, dw(x, 3)), sc, 3);
  } else {
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, as_f32(dw(x, 0)), as_f32(dw(x, 1)), sc, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, as_f32(dw(x, 2)), as_f32(dw(x, 3)), sc, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, as_f32(dw(x, 4)), as_f32(dw(x, 5)), sc, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, as_f32(dw(x, 6)), as_f32(dw(x, 7)), sc, 3);
  }
  return byte == 255u ? 0u : c;
}

// Largest value of the quad, in all four lanes.
__device__ __forceinline__ uint32_t quad_max(uint32_t m) {
  m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, true));
  return max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, true));
}

}  // namespace qn
