// fp4_device.hpp - device-side conversions of the four-bit format (gkdfp4.h), and what its
// kernels' loads and products have in common.
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

// Eight values as an operand of a product
__device__ __forceinline__ bf16x8 frag(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

typedef __attribute__((address_space(3))) void lds_void;  // where loads straight to LDS go

// All but the last N loads of this wave are here.
template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0f70 | (N & 15) | ((N >> 4) << 14));  // vmcnt(N), the other counters left alone
  asm volatile("" ::: "memory");
}

// What this wave has read of LDS is in its registers.
__device__ __forceinline__ void wait_lds() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0), the other counters left alone
  asm volatile("" ::: "memory");
}

}  // namespace gkd
