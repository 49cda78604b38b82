// epilogue.hpp - bias, activation, residual and the store of a matrix product,
// for the kernels of gkd_linear and gkd_linear_fp4. P is the kernel's parameters:
//   bias [N] bf16 or null; res [M,N] out type or null, row stride ldr; out [M,N],
//   row stride ldo; N; out_f32.
#pragma once

#include "gkd_device.hpp"
#include "gkdtokens.h"

#include <type_traits>

namespace gkd {

// z Phi(z) = max(z, 0) - |z| Phi(-|z|) with Phi(-a) = 2^P(a): log2 Phi(-a) is
// smooth, so a polynomial of degree 8 (minimax on 0..6.5 with P(0) = -1, fitted
// with the error weighted as it enters the result) leaves 9e-8 of error in
// z Phi(z). Evaluated in float32 the result is right to 2^-20 |z| (to 6.6e-7 |z|
// by evaluation, near |z| = 0.1) and, in the tail down to z = -6, to 2^-13 of
// itself; further out P falls on without bound and the tail goes to 0. 12 VALU
// operations and one quarter-rate one.
__device__ __forceinline__ float gelu(float z) {
  const float a = fminf(fabsf(z), 64.f);  // Phi(-64) is 0 in float32
  float y = fmaf(-2.734757629e-07f, a, 4.388933576e-06f);
  y = fmaf(y, a, 5.59604905e-06f);
  y = fmaf(y, a, -0.0006766107981f);
  y = fmaf(y, a, 0.007893478498f);
  y = fmaf(y, a, -0.05318199843f);
  y = fmaf(y, a, -0.458932668f);
  y = fmaf(y, a, -1.151145458f);
  y = fmaf(y, a, -1.f);
  return fmaf(-a, __builtin_amdgcn_exp2f(y), z < 0.f ? 0.f : z);
}

template <int ACT>
__device__ __forceinline__ float activate(float z) {
  if constexpr (ACT == GKD_ACT_RELU) return z < 0.f ? 0.f : z;  // a NaN stays one
  if constexpr (ACT == GKD_ACT_GELU) return gelu(z);
  // z / (1 + exp(-c z)): for z far below 0 exp gives infinity and the quotient 0.
  // The exponent is rounded by 2^-22 of itself, exponential, sum, reciprocal and
  // product by a float32 step or less each
  if constexpr (ACT == GKD_ACT_QUICK_GELU)
    return z * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.702f * 1.4426950408889634f * z));
  if constexpr (ACT == GKD_ACT_SILU)
    return z * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.4426950408889634f * z));
  return z;
}

// Calls f with the activation as a compile-time constant.
template <class F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  switch (act) {
    case GKD_ACT_RELU: f(std::integral_constant<int, GKD_ACT_RELU>{}); break;
    case GKD_ACT_GELU: f(std::integral_constant<int, GKD_ACT_GELU>{}); break;
    case GKD_ACT_QUICK_GELU: f(std::integral_constant<int, GKD_ACT_QUICK_GELU>{}); break;
    case GKD_ACT_SILU: f(std::integral_constant<int, GKD_ACT_SILU>{}); break;
    default: f(std::integral_constant<int, GKD_ACT_NONE>{}); break;
  }
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  const bf16x2 h = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
  return __builtin_bit_cast(uint32_t, h);
}

// bias[n .. n + W), zeros without one and past N
template <int W, class P>
__device__ __forceinline__ void load_bias(const P& p, int n, float (&b)[W]) {
#pragma unroll
  for (int e = 0; e < W; ++e) b[e] = p.bias && n + e < p.N ? bf16_bits_to_f32(p.bias[n + e]) : 0.f;
}

// Rows may start anywhere: pieces are moved with their elements' alignment
// (the hardware takes such accesses; aligned ones cost the same as before).
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));

// The residual and the store of W columns in whole pieces, at elements o
// (out) and r (residual).
template <int W, class P>
__device__ __forceinline__ void finish_pieces(const P& p, long long o, long long r, float (&v)[W]) {
  if (p.out_f32) {
#pragma unroll
    for (int q = 0; q < W / 4; ++q) {
      f32x4 t = {v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
      if (p.res) t += *reinterpret_cast<const f32x4_any*>(static_cast<const float*>(p.res) + r + 4 * q);
      *reinterpret_cast<f32x4_any*>(static_cast<float*>(p.out) + o + 4 * q) = t;
    }
  } else {
    typedef uint32_t words __attribute__((ext_vector_type(W / 2), aligned(2)));
    if (p.res) {
      const words q = *reinterpret_cast<const words*>(static_cast<const uint16_t*>(p.res) + r);
#pragma unroll
      for (int e = 0; e < W / 2; ++e) {
        v[2 * e] += __uint_as_float(q[e] << 16);
        v[2 * e + 1] += __uint_as_float(q[e] & 0xffff0000u);
      }
    }
    words t;
#pragma unroll
    for (int e = 0; e < W / 2; ++e) t[e] = bf16_pair(v[2 * e], v[2 * e + 1]);
    *reinterpret_cast<words*>(static_cast<uint16_t*>(p.out) + o) = t;
  }
}

// Bias, activation, residual and the store of the W (4 or 8) columns from n
// of row m < M: whole pieces, and one by one where the matrix ends.
template <int ACT, int W, class P>
__device__ __forceinline__ void finish(const P& p, int m, int n, float (&v)[W], const float (&b)[W]) {
  if (n >= p.N) return;
  const long long o = (long long)m * p.ldo + n, r = (long long)m * p.ldr + n;
#pragma unroll
  for (int e = 0; e < W; ++e) v[e] = activate<ACT>(v[e] + b[e]);
  if (n + W <= p.N) {
    finish_pieces<W>(p, o, r, v);
    return;
  }
#pragma unroll
  for (int e = 0; e < W; ++e) {
    if (n + e >= p.N) break;
    if (p.out_f32) {
      if (p.res) v[e] += static_cast<const float*>(p.res)[r + e];
      static_cast<float*>(p.out)[o + e] = v[e];
    } else {
      if (p.res) v[e] += bf16_bits_to_f32(static_cast<const uint16_t*>(p.res)[r + e]);
      static_cast<uint16_t*>(p.out)[o + e] = f32_to_bf16_bits(v[e]);
    }
  }
}

}  // namespace gkd
