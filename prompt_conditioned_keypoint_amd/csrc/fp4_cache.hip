// fp4_cache.hip - values into four-bit codes and back: rows of weights
// (gkd_quantize_fp4), tokens into a cache's pages (gkd_cache_append) and out of
// them (gkd_cache_read).
//
// A thread takes 8 neighbouring values, one 16-byte piece of bfloat16; four
// neighbouring lanes hold a group and agree on its largest magnitude.
#include "fp4_device.hpp"
#include "fp4_launch.hpp"

namespace gkd {
namespace {

// Values i .. i + 8 of an array in bfloat16 or float32.
template <bool BF16>
__device__ __forceinline__ void load8(const void* base, long long i, float (&v)[8]) {
  if constexpr (BF16) {
    const u32x4 w = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(base) + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = __uint_as_float(w[e] << 16);
      v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
  } else {
    const f32x4* q = reinterpret_cast<const f32x4*>(static_cast<const float*>(base) + i);
    const f32x4 a = q[0], b = q[1];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = a[e];
      v[4 + e] = b[e];
    }
  }
}

// The group's largest magnitude, as bits (which order like integers, NaN last), of
// its four lanes: quad permutes [1,0,3,2] and [2,3,0,1].
__device__ __forceinline__ uint32_t group_max(const float (&v)[8]) {
  uint32_t a = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) a = max(a, __float_as_uint(v[e]) & 0x7fffffffu);
  a = max(a, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a, 0xB1, 0xf, 0xf, false));
  return max(a, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a, 0x4E, 0xf, 0xf, false));
}

struct QuantParams {
  const void* x;
  long long ldx, pieces;
  int per;  // pieces a row
  uint8_t *codes, *scales;
};

template <bool BF16>
__global__ __launch_bounds__(256) void fp4_quantize_kernel(QuantParams p) {
  for (long long u = (long long)blockIdx.x * 256 + threadIdx.x; u < p.pieces; u += (long long)gridDim.x * 256) {
    const long long r = u / p.per;
    const int c = (int)(u - r * p.per);
    float v[8];
    load8<BF16>(p.x, r * p.ldx + 8 * c, v);
    const uint32_t s = fp4_scale(group_max(v));
    reinterpret_cast<uint32_t*>(p.codes)[u] = fp4_codes(v, s);
    if ((u & 3) == 0) p.scales[u >> 2] = (uint8_t)s;
  }
}

struct MoveParams {
  Heads k, v;
  Pages c;
  int T, per;           // pieces of a token: 2 Hk D / 8
  const int32_t *start, *count;
  long long pieces;
};

// A thread's piece: 8 values of token t of sequence b, of the keys or the values.
struct Piece {
  long long at;   // element offset in k or v
  long long code; // piece of the cache's codes, -1 without a place
  bool value, live;
};

__device__ __forceinline__ Piece piece(const MoveParams& p, long long u) {
  Piece w;
  const long long token = u / p.per;
  int r = (int)(u - token * p.per);
  const int b = (int)(token / p.T), t = (int)(token - (long long)b * p.T);
  const int D8 = p.c.D / 8, half = p.per / 2;
  w.value = r >= half;
  if (w.value) r -= half;
  const int h = r / D8, d = r - h * D8;
  const Heads& x = w.value ? p.v : p.k;
  w.at = b * x.b + t * x.t + h * x.h + 8 * d;
  w.live = !p.count || t < p.count[b];
  w.code = -1;
  const long long pos = (long long)(p.start ? p.start[b] : 0) + t;
  if (pos >= 0 && pos < (long long)p.c.L * p.c.page) {
    const int col = (int)pos / p.c.page, row = (int)pos - col * p.c.page;
    const int page = p.c.table[(long long)b * p.c.L + col];
    if (page >= 0 && page < p.c.pages)
      w.code = ((((long long)page * 2 + (w.value ? 1 : 0)) * p.c.Hk + h) * p.c.page + row) * D8 + d;
  }
  return w;
}

template <bool BF16>
__global__ __launch_bounds__(256) void fp4_append_kernel(MoveParams p) {
  for (long long u = (long long)blockIdx.x * 256 + threadIdx.x; u < p.pieces; u += (long long)gridDim.x * 256) {
    const Piece w = piece(p, u);
    if (!w.live || w.code < 0) continue;  // the four lanes of a group alike
    float v[8];
    load8<BF16>(w.value ? p.v.p : p.k.p, w.at, v);
    const uint32_t s = fp4_scale(group_max(v));
    reinterpret_cast<uint32_t*>(p.c.codes)[w.code] = fp4_codes(v, s);
    if ((w.code & 3) == 0) p.c.scales[w.code >> 2] = (uint8_t)s;
  }
}

__global__ __launch_bounds__(256) void fp4_read_kernel(MoveParams p) {
  for (long long u = (long long)blockIdx.x * 256 + threadIdx.x; u < p.pieces; u += (long long)gridDim.x * 256) {
    const Piece w = piece(p, u);
    if (!w.live) continue;
    u32x4 y = {0u, 0u, 0u, 0u};
    if (w.code >= 0)
      y = fp4_values(reinterpret_cast<const uint32_t*>(p.c.codes)[w.code], fp4_unit(p.c.scales[w.code >> 2]));
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(w.value ? p.v.p : p.k.p) + w.at) = y;
  }
}

unsigned groups_for(long long pieces) {
  const long long n = (pieces + 255) / 256;
  return (unsigned)(n < 8192 ? n : 8192);
}

MoveParams move_params(const CacheMoveArgs& a) {
  MoveParams p{};
  p.k = a.k;
  p.v = a.v;
  p.c = a.c;
  p.T = a.T;
  p.per = 2 * a.c.Hk * (a.c.D / 8);
  p.start = a.start;
  p.count = a.count;
  p.pieces = (long long)a.B * a.T * p.per;
  return p;
}

}  // namespace

hipError_t launch_quantize_fp4(const QuantizeArgs& a, hipStream_t st) {
  QuantParams p{a.x, a.ldx, (long long)a.N * (a.K / 8), a.K / 8, a.codes, a.scales};
  if (a.bf16)
    hipLaunchKernelGGL(fp4_quantize_kernel<true>, dim3(groups_for(p.pieces)), dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL(fp4_quantize_kernel<false>, dim3(groups_for(p.pieces)), dim3(256), 0, st, p);
  return hipGetLastError();
}

hipError_t launch_cache_append(const CacheMoveArgs& a, hipStream_t st) {
  const MoveParams p = move_params(a);
  if (a.bf16)
    hipLaunchKernelGGL(fp4_append_kernel<true>, dim3(groups_for(p.pieces)), dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL(fp4_append_kernel<false>, dim3(groups_for(p.pieces)), dim3(256), 0, st, p);
  return hipGetLastError();
}

hipError_t launch_cache_read(const CacheMoveArgs& a, hipStream_t st) {
  const MoveParams p = move_params(a);
  hipLaunchKernelGGL(fp4_read_kernel, dim3(groups_for(p.pieces)), dim3(256), 0, st, p);
  return hipGetLastError();
}

}  // namespace gkd
