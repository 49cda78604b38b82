// fp4_launch.hpp - internal interface between the C ABI of the four-bit token
// operators (fp4_api.hip) and their kernels (fp4_linear.hip, fp4_cache.hip,
// fp4_attn.hip). Arguments arrive here already validated.
#pragma once

#include "tokens_launch.hpp"

namespace gkd {

struct QuantizeArgs {
  const void* x;     // [N,K]
  long long ldx;
  int N, K;
  bool bf16;
  uint8_t *codes, *scales;
};

hipError_t launch_quantize_fp4(const QuantizeArgs& a, hipStream_t stream);

struct LinearFp4Args {
  const uint16_t* x;         // [M,K] bf16
  const uint8_t *codes, *scales;
  const uint16_t* bias;      // [N] bf16 or null
  const void* residual;      // [M,N] out type or null
  void* out;                 // [M,N]
  long long ldx, ldr, ldo;
  int M, N, K;
  int act;                   // gkd_activation
  bool out_f32;
  void* ws;
};

size_t linear_fp4_workspace_bytes(int M, int N, int K);
hipError_t launch_linear_fp4(const LinearFp4Args& a, hipStream_t stream);

// A cache and the table of its sequences' pages.
struct Pages {
  uint8_t *codes, *scales;
  int pages, page, Hk, D;
  const int32_t* table;
  int L;
};

struct CacheMoveArgs {
  Heads k, v;                       // read by append, written by read
  Pages c;
  int B, T;
  const int32_t *start, *count;     // or null
  bool bf16;                        // append's k and v
};

hipError_t launch_cache_append(const CacheMoveArgs& a, hipStream_t stream);
hipError_t launch_cache_read(const CacheMoveArgs& a, hipStream_t stream);

struct CacheAttnArgs {
  Heads q, out;
  Pages c;
  const int32_t *length, *q_len;    // or null
  int B, Tq, Hq;
  float scale;
  bool causal;
  void* ws;
};

size_t cache_attn_workspace_bytes(int B, int Tq, int Hq, int Hk, int D, int page, int L);
hipError_t launch_cache_attn(const CacheAttnArgs& a, hipStream_t stream);

}  // namespace gkd
