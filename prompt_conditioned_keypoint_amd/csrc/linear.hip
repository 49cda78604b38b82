// linear.hip - matrix product with bias, activation and residual in its
// epilogue (gkd_linear): out = act(x w^T + bias) + residual.
//
// Two kernels, chosen by the row count:
//   linear_tile_kernel   a tile of rows x columns a workgroup, both operands
//                        through LDS: bound by the matrix pipes;
//   linear_few_kernel    up to 64 rows: 16 columns a workgroup, whose waves
//                        share the K axis, operands straight to registers:
//                        bound by reading w once.
// The products run on v_mfma_f32_16x16x32_bf16 with w as the first operand,
// so a lane ends with four adjacent columns of one row.
#include "gkd_device.hpp"
#include "gkdtokens.h"
#include "tokens_launch.hpp"

namespace gkd {
namespace {

struct LinParams {
  const uint16_t* x;
  const uint16_t* w;
  const uint16_t* bias;
  const void* res;
  void* out;
  long long ldr, ldo;
  int ldx, ldw;        // below 2^22
  int M, N, K;         // K a multiple of 8
  int act;
  int out_f32;
  int vec_out, vec_res;  // four adjacent columns are one aligned piece
};

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(1))) void glb_void;

__device__ __forceinline__ bf16x8 frag(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

// s_waitcnt vmcnt(N), the other counters left alone
template <int N>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt(0x0f70 | (N & 15) | ((N >> 4) << 14));
}

// erf to 1.5e-7 (Abramowitz and Stegun, Handbook of Mathematical Functions,
// 7.1.26): below a float32 step of the activations that use it.
__device__ __forceinline__ float erf_as(float x) {
  const float a = fabsf(x);
  const float t = __builtin_amdgcn_rcpf(fmaf(0.3275911f, a, 1.f));
  float y = fmaf(1.061405429f, t, -1.453152027f);
  y = fmaf(y, t, 1.421413741f);
  y = fmaf(y, t, -0.284496736f);
  y = fmaf(y, t, 0.254829592f);
  const float e = 1.f - y * t * __builtin_amdgcn_exp2f(-1.4426950408889634f * a * a);
  return copysignf(e, x);
}

__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case GKD_ACT_RELU: return z < 0.f ? 0.f : z;  // a NaN stays one
    case GKD_ACT_GELU: return 0.5f * z * (1.f + erf_as(z * 0.70710678118654752f));
    // z / (1 + exp(-c z)): for z very negative exp gives infinity and the quotient 0
    case GKD_ACT_QUICK_GELU:
      return z * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.702f * 1.4426950408889634f * z));
    case GKD_ACT_SILU:
      return z * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.4426950408889634f * z));
    default: return z;
  }
}

// Bias, activation, residual and the store of columns n .. n + 3 of row m
// (m < M; columns past N are left out).
__device__ __forceinline__ void finish(const LinParams& p, int m, int n, f32x4 v) {
  if (n >= p.N) return;
  const long long o = (long long)m * p.ldo + n, r = (long long)m * p.ldr + n;
  if (n + 4 <= p.N && p.vec_out && (p.res == nullptr || p.vec_res)) {
    if (p.bias) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += bf16_bits_to_f32(p.bias[n + e]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = activate(v[e], p.act);
    if (p.out_f32) {
      if (p.res) v += *reinterpret_cast<const f32x4*>(static_cast<const float*>(p.res) + r);
      *reinterpret_cast<f32x4*>(static_cast<float*>(p.out) + o) = v;
    } else {
      if (p.res) {
        const u32x2 q = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(p.res) + r);
        v += f32x4{__uint_as_float(q[0] << 16), __uint_as_float(q[0] & 0xffff0000u),
                   __uint_as_float(q[1] << 16), __uint_as_float(q[1] & 0xffff0000u)};
      }
      const bf16x2 lo = {static_cast<__bf16>(v[0]), static_cast<__bf16>(v[1])};
      const bf16x2 hi = {static_cast<__bf16>(v[2]), static_cast<__bf16>(v[3])};
      *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p.out) + o) =
          u32x2{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (n + e >= p.N) break;
    float z = v[e];
    if (p.bias) z += bf16_bits_to_f32(p.bias[n + e]);
    z = activate(z, p.act);
    if (p.out_f32) {
      if (p.res) z += static_cast<const float*>(p.res)[r + e];
      static_cast<float*>(p.out)[o + e] = z;
    } else {
      if (p.res) z += bf16_bits_to_f32(static_cast<const uint16_t*>(p.res)[r + e]);
      static_cast<uint16_t*>(p.out)[o + e] = f32_to_bf16_bits(z);
    }
  }
}

// ---------------------------------------------------------------------------
// Tiles of BM x BN, K in steps of 64 through a ring of two LDS stages, WM x
// WN waves of (BM / WM) x (BN / WN). Both tiles stream straight into LDS
// (16 bytes a lane); 16-byte piece c of tile row r sits at place c ^ (r & 7),
// so the 16 rows of one operand read fall in different banks. Rows past M
// or N repeat the last one and are not stored; pieces past K repeat the
// row's last and enter the product as zeros.
// ---------------------------------------------------------------------------
constexpr int kBK = 64;

template <int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void linear_tile_kernel(LinParams p) {
  constexpr int NW = WM * WN;                  // waves
  constexpr int MT = BM / WM / 16, NT = BN / WN / 16;
  constexpr int NA = BM * 8 / (64 * NW), NB = BN * 8 / (64 * NW);  // loads a wave and step
  constexpr int A_BYTES = BM * kBK * 2, STAGE = (BM + BN) * kBK * 2;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tiles_n = (p.N + BN - 1) / BN;
  const int total = gridDim.x;
  // Workgroups are dealt round-robin over the XCDs: each takes a contiguous
  // run of the tiles, so the column tiles of one row band share an L2.
  const int bid = blockIdx.x, xcd = bid % kXcds, q = total / kXcds, rem = total % kXcds;
  const int lin = xcd * q + min(xcd, rem) + bid / kXcds;
  const int m0 = (lin / tiles_n) * BM, n0 = (lin % tiles_n) * BN;
  const uint16_t* xb = p.x + (long long)m0 * p.ldx;
  const uint16_t* wb = p.w + (long long)n0 * p.ldw;

  uint32_t aoff[NA], woff[NB];
  int acol, wcol;  // this lane's piece of a step is the same for all its rows
#pragma unroll
  for (int i = 0; i < NA; ++i) {
    const int s = (wave + NW * i) * 64 + lane, r = s >> 3;
    acol = (s & 7) ^ (r & 7);
    aoff[i] = (uint32_t)(min(r, p.M - 1 - m0) * p.ldx);
  }
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int s = (wave + NW * i) * 64 + lane, r = s >> 3;
    wcol = (s & 7) ^ (r & 7);
    woff[i] = (uint32_t)(min(r, p.N - 1 - n0) * p.ldw);
  }
  auto issue = [&](int stage, int k0) {
    unsigned char* base = lds + stage * STAGE;
    const int ka = min(k0 + 8 * acol, p.K - 8), kw = min(k0 + 8 * wcol, p.K - 8);
#pragma unroll
    for (int i = 0; i < NA; ++i)
      __builtin_amdgcn_global_load_lds((glb_void*)(xb + aoff[i] + ka),
                                       (lds_void*)(base + (wave + NW * i) * 1024), 16, 0, 0);
#pragma unroll
    for (int i = 0; i < NB; ++i)
      __builtin_amdgcn_global_load_lds((glb_void*)(wb + woff[i] + kw),
                                       (lds_void*)(base + A_BYTES + (wave + NW * i) * 1024), 16, 0, 0);
  };

  const int wm0 = (wave / WN) * (BM / WM), wn0 = (wave % WN) * (BN / WN);
  const int fr = lane & 15, g = lane >> 4;
  f32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int nk = (p.K + kBK - 1) / kBK;
  issue(0, 0);
  for (int kt = 0; kt < nk; ++kt) {
    wait_vm<0>();
    __syncthreads();
    if (kt + 1 < nk) issue((kt + 1) & 1, (kt + 1) * kBK);
    const unsigned char* sa = lds + (kt & 1) * STAGE;
    const unsigned char* sb = sa + A_BYTES;
    const int left = p.K - kt * kBK;  // of this step, in elements
    auto piece = [&](const unsigned char* t, int r, int c) {
      const u32x4 v = *reinterpret_cast<const u32x4*>(t + (r * 8 + (c ^ (r & 7))) * 16);
      return frag(8 * c < left ? v : u32x4{0u, 0u, 0u, 0u});
    };
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      bf16x8 a[MT], b[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) b[j] = piece(sb, wn0 + 16 * j + fr, 4 * h + g);
#pragma unroll
      for (int i = 0; i < MT; ++i) a[i] = piece(sa, wm0 + 16 * i + fr, 4 * h + g);
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j], a[i], acc[i][j], 0, 0, 0);
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int m = m0 + wm0 + 16 * i + fr;
    if (m >= p.M) continue;
#pragma unroll
    for (int j = 0; j < NT; ++j) finish(p, m, n0 + wn0 + 16 * j + 4 * g, acc[i][j]);
  }
}

// ---------------------------------------------------------------------------
// Up to 16 MT rows: a workgroup takes 16 columns (rows of w), its waves take
// every 8th 64-wide piece of K, and their sums meet in LDS in a fixed order.
// ---------------------------------------------------------------------------
constexpr int kFewWaves = 8;

template <int MT>
__global__ __launch_bounds__(64 * kFewWaves) void linear_few_kernel(LinParams p) {
  __shared__ f32x4 part[kFewWaves][MT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int fr = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * 16;
  const uint16_t* wr = p.w + (long long)min(n0 + fr, p.N - 1) * p.ldw;
  const uint16_t* xr[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) xr[i] = p.x + (long long)min(16 * i + fr, p.M - 1) * p.ldx;
  f32x4 acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int k0 = wave * 64; k0 < p.K; k0 += 64 * kFewWaves) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = k0 + 32 * h + 8 * g;
      const bool in = k < p.K;
      const int kc = min(k, p.K - 8);
      const u32x4 z = {0u, 0u, 0u, 0u};
      const u32x4 wv = *reinterpret_cast<const u32x4*>(wr + kc);
      const bf16x8 b = frag(in ? wv : z);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const u32x4 xv = *reinterpret_cast<const u32x4*>(xr[i] + kc);
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, frag(in ? xv : z), acc[i], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) part[wave][i][lane] = acc[i];
  __syncthreads();
  for (int i = wave; i < MT; i += kFewWaves) {
    f32x4 s = part[0][i][lane];
#pragma unroll
    for (int v = 1; v < kFewWaves; ++v) s += part[v][i][lane];
    const int m = 16 * i + fr;
    if (m < p.M) finish(p, m, n0 + 4 * g, s);
  }
}

// Rows of n elements, ld apart, into rows of n8 = n rounded up to 8, the
// rest zero: one 16-byte piece a thread.
__global__ __launch_bounds__(256) void linear_pack_kernel(const uint16_t* src, long long ld,
                                                          int rows, int n, int n8, uint16_t* dst) {
  const int per = n8 / 8;
  for (long long u = (long long)blockIdx.x * 256 + threadIdx.x; u < (long long)rows * per;
       u += (long long)gridDim.x * 256) {
    const long long r = u / per;
    const int c = (int)(u - r * per) * 8;
    uint16_t t[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = c + e < n ? src[r * ld + c + e] : (uint16_t)0;
    u32x4 v;
    __builtin_memcpy(&v, t, 16);
    *reinterpret_cast<u32x4*>(dst + r * n8 + c) = v;
  }
}

size_t al256(size_t n) { return (n + 255) & ~(size_t)255; }
int up8(int n) { return (n + 7) & ~7; }
bool packs(int K, long long ld) { return K % 8 != 0 || ld % 8 != 0; }

template <int BM, int BN, int WM, int WN>
hipError_t run_tiles(const LinParams& p, hipStream_t st) {
  const long long tiles = (long long)((p.M + BM - 1) / BM) * ((p.N + BN - 1) / BN);
  hipLaunchKernelGGL((linear_tile_kernel<BM, BN, WM, WN>), dim3((unsigned)tiles),
                     dim3(64 * WM * WN), 2 * (BM + BN) * kBK * 2, st, p);
  return hipGetLastError();
}

template <int MT>
hipError_t run_few(const LinParams& p, hipStream_t st) {
  hipLaunchKernelGGL((linear_few_kernel<MT>), dim3((p.N + 15) / 16), dim3(64 * kFewWaves), 0, st, p);
  return hipGetLastError();
}

}  // namespace

size_t linear_workspace_bytes(int M, int N, int K, long long ldx, long long ldw) {
  size_t n = 0;
  if (packs(K, ldx)) n += al256((size_t)M * up8(K) * 2);
  if (packs(K, ldw)) n += al256((size_t)N * up8(K) * 2);
  return n;
}

hipError_t launch_linear(const LinearArgs& a, hipStream_t st) {
  LinParams p{};
  p.x = a.x;
  p.w = a.w;
  p.ldx = (int)a.ldx;
  p.ldw = (int)a.ldw;
  p.bias = a.bias;
  p.res = a.residual;
  p.out = a.out;
  p.ldr = a.ldr;
  p.ldo = a.ldo;
  p.M = a.M;
  p.N = a.N;
  p.K = up8(a.K);
  p.act = a.act;
  p.out_f32 = a.out_f32;
  const unsigned mask = a.out_f32 ? 15u : 7u;
  p.vec_out = (reinterpret_cast<uintptr_t>(a.out) & mask) == 0 && a.ldo % 4 == 0;
  p.vec_res = (reinterpret_cast<uintptr_t>(a.residual) & mask) == 0 && a.ldr % 4 == 0;
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  auto pack = [&](const uint16_t*& src, int& ld, int rows) -> hipError_t {
    uint16_t* dst = reinterpret_cast<uint16_t*>(ws);
    const long long pieces = (long long)rows * (p.K / 8);
    const long long wgs = (pieces + 255) / 256;
    hipLaunchKernelGGL(linear_pack_kernel, dim3((unsigned)(wgs < 4096 ? wgs : 4096)), dim3(256), 0,
                       st, src, (long long)ld, rows, a.K, p.K, dst);
    ws += al256((size_t)rows * p.K * 2);
    src = dst;
    ld = p.K;
    return hipGetLastError();
  };
  hipError_t e = hipSuccess;
  if (packs(a.K, a.ldx) && (e = pack(p.x, p.ldx, a.M)) != hipSuccess) return e;
  if (packs(a.K, a.ldw) && (e = pack(p.w, p.ldw, a.N)) != hipSuccess) return e;
  if (p.M <= 16) return run_few<1>(p, st);
  if (p.M <= 32) return run_few<2>(p, st);
  if (p.M <= 64) return run_few<4>(p, st);
  if ((long long)p.M * p.N >= 256LL * 256 * 256) return run_tiles<256, 256, 2, 4>(p, st);
  return run_tiles<128, 128, 2, 2>(p, st);
}

}  // namespace gkd
