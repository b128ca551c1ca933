// The 4-bit format of kvx_fp4.h on gfx950: what one group's scale byte is, and the conversions, which the hardware has
// (v_cvt_scalef32_*: a scale's exponent bits alone count; to 4 bits to nearest, ties to even, saturating).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kvx_fp4.h"
#include "kvx_paged.h"

namespace kvx {

constexpr int kGroup = KVX_FP4_GROUP;
constexpr uint32_t kNanScale = 255;

// Scale byte of a group whose largest magnitude has these bits: with the top at 1.75 * 2^k and up, which is 7 * 2^(k-2),
// the exponent one higher; NaN and infinity carry the top exponent.
template <class E>
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  constexpr int32_t most = __is_same(E, Bf16) ? 125 + 127 : 13 + 127;
  const int32_t s = (int32_t)((top + 0x200000u) >> 23) - 2;
  if (top >= 0x7f800000u) return kNanScale;
  return s < 0 ? 0 : s > most ? most : s;
}

// 2^(s - 127) as the conversions take it: the exponent's bits, and one below them so that s = 0 is no zero and s = 255 is NaN.
__device__ __forceinline__ float scale_of(uint32_t s) { return __builtin_bit_cast(float, s << 23 | 0x400000u); }

// Eight elements to their codes, the first in the lowest bits.
__device__ __forceinline__ uint32_t encode(f32x8 v, uint32_t s) {
  const float scale = scale_of(s);
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], scale, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], scale, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], scale, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], scale, 3);
  return s == kNanScale ? 0 : r;
}

// Eight codes to the 16-bit type.
template <class E>
__device__ __forceinline__ u32x4 decode(uint32_t codes, float scale) {
  u32x4 r;
  if constexpr (__is_same(E, Bf16)) {
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1));
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2));
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3));
  } else {
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 0));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 1));
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 2));
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 3));
  }
  return r;
}

// Largest magnitude of eight elements, as bits: of non-negative numbers the order of the bits, with NaN on top.
__device__ __forceinline__ uint32_t top_of(f32x8 v) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = v[i];  // a bit cast of a vector's element itself reads the first one
    const uint32_t b = __builtin_bit_cast(uint32_t, x) & 0x7fffffffu;
    top = b > top ? b : top;
  }
  return top;
}
// Over the four lanes that hold one group.
__device__ __forceinline__ uint32_t top_of_quad(uint32_t x) {
  uint32_t y = __builtin_amdgcn_mov_dpp(x, 0xb1, 0xf, 0xf, true);  // lanes 1 0 3 2
  x = x > y ? x : y;
  y = __builtin_amdgcn_mov_dpp(x, 0x4e, 0xf, 0xf, true);  // lanes 2 3 0 1
  return x > y ? x : y;
}

// What no kernel writes while this one runs and all lanes ask for: a scalar load.
template <class T>
__device__ __forceinline__ T constant(const T* p) {
  return *(const __attribute__((address_space(4))) T*)p;
}

// Division of 32-bit numbers by one that the host knows: a product, a sum and shifts.
struct Divisor {
  uint32_t by, mul, shift;
};
inline Divisor divisor(uint32_t d) {
  uint32_t s = 0;
  while (s < 32 && (1ull << s) < d) ++s;
  return {d, (uint32_t)(((1ull << 32) * ((1ull << s) - d)) / d + 1), s};
}
__device__ __forceinline__ uint32_t operator/(uint32_t n, Divisor d) {
  const uint32_t t = __umulhi(n, d.mul);
  return (uint32_t)(((uint64_t)t + n) >> d.shift);
}

}  // namespace kvx
