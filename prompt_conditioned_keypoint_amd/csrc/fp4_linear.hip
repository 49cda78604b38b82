// fp4_linear.hip - matrix product with four-bit weights (gkd_linear_fp4):
// out = act(x w^T + bias) + residual.
//
// A wave takes 16 rows of w and 128 of K at a time: each lane one group of 32
// codes (16 bytes) and its scale byte, which the conversion instructions turn into
// the first operand of four v_mfma_f32_16x16x32_bf16. Which k a lane's place in the
// instruction stands for is free as long as x is read alike: place (g, i) of
// product t is k = 32 g + 8 t + i. So weights go from memory to the matrix pipe
// through registers alone, and nothing is rounded on the way.
#include "epilogue.hpp"
#include "fp4_device.hpp"
#include "fp4_launch.hpp"

namespace gkd {
namespace {

struct Fp4Params {
  const uint16_t* x;
  const uint8_t *codes, *scales;
  const uint16_t* bias;
  const void* res;
  void* out;
  long long ldr, ldo;
  int ldx;
  int M, N, K;  // K a multiple of 32
  int act;
  int out_f32;
};

__device__ __forceinline__ bf16x8 frag(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

// 16 MT rows of x and 16 rows of w a workgroup; its NW waves take every NW-th
// 128-wide piece of K, and their sums meet in LDS in a fixed order.
template <int MT, int NW>
__global__ __launch_bounds__(64 * NW) void fp4_few_kernel(Fp4Params p) {
  __shared__ f32x4 part[NW][MT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int fr = lane & 15, g = lane >> 4;
  const int tiles_n = (p.N + 15) / 16, tm = blockIdx.x / tiles_n;
  const int n0 = (blockIdx.x - tm * tiles_n) * 16, m0 = tm * 16 * MT;
  const long long row = min(n0 + fr, p.N - 1);
  const uint8_t* cr = p.codes + row * (p.K / 2);
  const uint8_t* sr = p.scales + row * (p.K / 32);
  const uint16_t* xr[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) xr[i] = p.x + (long long)min(m0 + 16 * i + fr, p.M - 1) * p.ldx;
  f32x4 acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int k0 = wave * 128; k0 < p.K; k0 += 128 * NW) {
    const int k = k0 + 32 * g;
    u32x4 c = {0u, 0u, 0u, 0u};
    uint32_t s = 127u;
    u32x4 xv[MT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int t = 0; t < 4; ++t) xv[i][t] = u32x4{0u, 0u, 0u, 0u};
    if (k < p.K) {
      c = *reinterpret_cast<const u32x4*>(cr + k / 2);
      s = sr[k / 32];
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int t = 0; t < 4; ++t) xv[i][t] = *reinterpret_cast<const u32x4*>(xr[i] + k + 8 * t);
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const bf16x8 w = frag(fp4_values(c[t], fp4_unit(s)));
#pragma unroll
      for (int i = 0; i < MT; ++i)
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, frag(xv[i][t]), acc[i], 0, 0, 0);
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) part[wave][i][lane] = acc[i];
  __syncthreads();
  for (int i = wave; i < MT; i += NW) {
    f32x4 s = part[0][i][lane];
#pragma unroll
    for (int v = 1; v < NW; ++v) s += part[v][i][lane];
    const int m = m0 + 16 * i + fr, n = n0 + 4 * g;
    float b[4], v[4] = {s[0], s[1], s[2], s[3]};
    load_bias(p, n, b);
    if (m < p.M) with_act(p.act, [&](auto act) { finish<act, 4>(p, m, n, v, b); });
  }
}

template <int MT, int NW>
hipError_t run_few(const Fp4Params& p, hipStream_t st) {
  const long long tiles = (long long)((p.N + 15) / 16) * ((p.M + 16 * MT - 1) / (16 * MT));
  hipLaunchKernelGGL((fp4_few_kernel<MT, NW>), dim3((unsigned)tiles), dim3(64 * NW), 0, st, p);
  return hipGetLastError();
}

}  // namespace

size_t linear_fp4_workspace_bytes(int, int, int) { return 0; }

hipError_t launch_linear_fp4(const LinearFp4Args& a, hipStream_t st) {
  Fp4Params p{};
  p.x = a.x;
  p.codes = a.codes;
  p.scales = a.scales;
  p.bias = a.bias;
  p.res = a.residual;
  p.out = a.out;
  p.ldr = a.ldr;
  p.ldo = a.ldo;
  p.ldx = (int)a.ldx;
  p.M = a.M;
  p.N = a.N;
  p.K = a.K;
  p.act = a.act;
  p.out_f32 = a.out_f32;
  if (p.M <= 16) return run_few<1, 8>(p, st);
  return run_few<4, 8>(p, st);
}

}  // namespace gkd
