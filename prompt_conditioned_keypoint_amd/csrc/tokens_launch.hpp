// tokens_launch.hpp - internal interface between the C ABI of the token
// operators (tokens_api.hip) and their kernels (linear.hip, rope.hip,
// prefix_attn.hip). Arguments arrive here already validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gkd {

struct LinearArgs {
  const uint16_t* x;         // [M,K] bf16
  const uint16_t* w;         // [N,K] bf16
  const uint16_t* bias;      // [N] bf16 or null
  const void* residual;      // [M,N] out type or null
  void* out;                 // [M,N]
  long long ldx, ldw, ldr, ldo;
  int M, N, K;
  int act;                   // gkd_activation
  bool out_f32;
  void* ws;
};

size_t linear_workspace_bytes(int M, int N, int K, long long ldx, long long ldw);
hipError_t launch_linear(const LinearArgs& a, hipStream_t stream);

// One operand of heads: base pointer and element strides.
struct Heads {
  void* p;
  long long b, t, h;
};

struct RopeArgs {
  Heads q, k, qo, ko;
  int Hq, Hk, B, T, D;
  const float* pos;
  long long pos_batch;
  int n_axes;
  const float* freqs;
  int rot;
  const void *wq, *wk;
  float eps;
  bool bf16, interleaved;
};

hipError_t launch_rope(const RopeArgs& a, hipStream_t stream);

struct PrefixAttnArgs {
  Heads q, kp, vp, ko, vo, out;
  int P, S;
  const int32_t *own_len, *q_len;  // or null
  const uint8_t* mask;             // or null
  int B, Tq, Hq, Hk, D;
  float scale;
  bool causal;
  void* ws;
};

size_t prefix_attn_workspace_bytes(int B, int Tq, int Hq, int Hk, int D, int P, int S);
hipError_t launch_prefix_attn(const PrefixAttnArgs& a, hipStream_t stream);

}  // namespace gkd
