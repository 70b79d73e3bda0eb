// Blocks of 4-bit values (E2M1, 32 of them sharing a power-of-two scale byte)
// and their conversions.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ttt_device.h"

namespace tttk {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

// The largest scale byte of finite values; those above stand for NaN, and
// append writes the last.
constexpr uint32_t kScaleMax = 252, kScaleNan = 255;

// The scale byte of a block whose largest |value| is `a` (finite): 127 + e
// with e the least exponent with a <= 7 * 2^e. Values between 6 and 7 units
// saturate at 6, with an error of at most one unit, which is what rounding
// costs in the topmost step (4 to 6) anyway; the next larger scale would
// double the error of every other value. Over Gaussian values the limit 7
// leaves an rms error of 11.2% (6: 11.6%, 8: 11.5%). e stays in [-125, 125]
// so that every value held is a normal bf16 number.
__device__ __forceinline__ uint32_t scale_byte(float a) {
  const uint32_t bits = __float_as_uint(a);
  // a = m 2^E, 1 <= m < 2, in units of 2^(E-2): 4m, which has to be <= 7
  const int e = (int)(bits >> 23) - 2 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return (uint32_t)min(max(e, 2), (int)kScaleMax);
}

__device__ __forceinline__ float scale_value(uint32_t byte) { return __uint_as_float(byte << 23); }

// Byte e of a word as a scale for the conversions below, which read the
// exponent field alone: the byte is shifted there, whatever comes with it.
__device__ __forceinline__ float scale_at(uint32_t w, int e) {
  return __uint_as_float(e == 0 ? w << 23 : e == 1 ? w << 15 : e == 2 ? w << 7 : w >> 1);
}

// Eight values divided by the scale, as codes, the first in the low bits:
// nearest, ties to the even code, saturating (v_cvt_scalef32_pk_fp4_f32).
__device__ __forceinline__ uint32_t encode8(const float (&x)[8], float scale) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], scale, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], scale, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], scale, 3);
  return w;
}

// Codes 2 SEL and 2 SEL + 1 of `w` times the scale, exact in bf16.
template <int SEL>
__device__ __forceinline__ uint32_t decode2(uint32_t w, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, SEL));
}

__device__ __forceinline__ uint32_t decode2(uint32_t w, float scale, int sel) {
  switch (sel) {  // folded where sel is known
    case 0: return decode2<0>(w, scale);
    case 1: return decode2<1>(w, scale);
    case 2: return decode2<2>(w, scale);
    default: return decode2<3>(w, scale);
  }
}

__device__ __forceinline__ void decode8(uint32_t w, float scale, uint32_t (&v)[4]) {
  v[0] = decode2<0>(w, scale);
  v[1] = decode2<1>(w, scale);
  v[2] = decode2<2>(w, scale);
  v[3] = decode2<3>(w, scale);
}

}  // namespace tttk
