// Device-side coding of the microscaled 4-bit copy (layout and scales: mx4.hip).
#pragma once

#include "w12_device.hpp"

namespace w12 {

constexpr uint32_t kMXLowest = 110;   // scale byte of a block whose largest weight is at the window bottom
constexpr int kTileMX = 1088;    // bytes of a tile: 64 lanes x 16 bytes of codes, 64 block scales

// A block's 32 codes and its scale byte -> the 16 dwords of bfloat16 pairs w' of its columns: each
// product of a code and a power of two is exact.  A scale byte of 0 (padding, loads past a range)
// goes with codes of 0, which convert to 0.
__device__ __forceinline__ void mx4_pairs(u32x4 v, uint32_t s, uint32_t p[16]) {
  const float scale = __uint_as_float(s << 23);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    p[4 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v[i], scale, 0));
    p[4 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v[i], scale, 1));
    p[4 * i + 2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v[i], scale, 2));
    p[4 * i + 3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v[i], scale, 3));
  }
}

// Eight codes -> the four bfloat16 pairs of one operand.
__device__ __forceinline__ u32x4 mx4_quarter(uint32_t v, uint32_t s) {
  const float scale = __uint_as_float(s << 23);
  return (u32x4){__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 0)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 1)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 2)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 3))};
}

// Eight bfloat16 values (four pairs) -> eight codes of value / scale, nearest with ties to even,
// magnitudes above 6 to 6.
__device__ __forceinline__ uint32_t mx4_encode8(const uint32_t p[4], float scale) {
  uint32_t o = 0;
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(bf16x2, p[0]), scale, 0);
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(bf16x2, p[1]), scale, 1);
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(bf16x2, p[2]), scale, 2);
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(bf16x2, p[3]), scale, 3);
  return o;
}

}  // namespace w12
