// fp4_device.hpp - device-side conversions of the four-bit format (gkdfp4.h).
#pragma once

#include "gkd_device.hpp"

namespace gkd {

// The scale 2^(s - 127) of a scale byte, as the conversions take it: they look at
// the exponent's bits alone, 0 and 255 (NaN) included.
__device__ __forceinline__ float fp4_unit(uint32_t s) { return __uint_as_float(s << 23); }

// Two codes of a word (byte SEL) as a pair of bfloat16 values. Exact over all scale
// bytes: the 32 values of a scale were checked for each of the 256.
template <int SEL>
__device__ __forceinline__ uint32_t fp4_pair(uint32_t codes, float unit) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, unit, SEL));
}

// Eight codes as values, in their order.
__device__ __forceinline__ u32x4 fp4_values(uint32_t codes, float unit) {
  return u32x4{fp4_pair<0>(codes, unit), fp4_pair<1>(codes, unit), fp4_pair<2>(codes, unit),
               fp4_pair<3>(codes, unit)};
}

// The scale byte of a group whose largest magnitude has these bits (as an
// integer; NaN and infinity are the largest): one exponent more where the
// mantissa reaches 1.75.
__device__ __forceinline__ uint32_t fp4_scale(uint32_t bits) {
  if (bits >= 0x7f800000u) return 255u;
  const int s = (int)((bits + 0x200000u) >> 23) - 2;
  return (uint32_t)min(max(s, 2), 252);
}

// Eight values as codes: the conversion rounds ties to the even code and stops at 6.
__device__ __forceinline__ uint32_t fp4_codes(const float (&v)[8], uint32_t scale) {
  if (scale == 255u) return 0u;
  const float unit = fp4_unit(scale);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], unit, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], unit, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], unit, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], unit, 3);
  return w;
}

}  // namespace gkd
