// linear.hip - matrix product with bias, activation and residual in its
// epilogue (gkd_linear): out = act(x w^T + bias) + residual.
//
// Three kernels, chosen by the sizes:
//   linear_turn_kernel   256 x 256 tiles, both operands through LDS, waves that
//                        take turns on the matrix pipe: bound by it;
//   linear_ring_kernel   smaller tiles with a ring of stages in LDS, where there
//                        are too few large ones: bound by the loads' latency;
//   linear_few_kernel    up to 64 rows: 16 columns a workgroup, whose waves
//                        share the K axis, operands straight to registers:
//                        bound by reading w once.
// The products run on v_mfma_f32_16x16x32_bf16 with w as the first operand,
// so a lane ends with four adjacent columns of one row.
//
// Measured (M x K x N; a call, inputs that change from call to call; the card
// copies at 5.08 TB/s; cards differ by 3%):
//   turn  36864 x 1024 x 4096, GELU             275-285 us, 1.1 PFLOP/s
//   turn and ring  19706 x 1024 x 1024, float32 residual  70-72 us, 0.58 PFLOP/s,
//         2.8 TB/s: one round of 256 x 256 tiles and 3322 rows apart; their
//         epilogues, 161 MB of them, come when no products are left to hide them
//   few   37 x 1024 x 4096, GELU 6.8 us on the GPU; 1 x 1024 x 1024 4.1 us
#include "gkd_device.hpp"
#include "gkdtokens.h"
#include "tokens_launch.hpp"

#include <type_traits>

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
};

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(1))) void glb_void;

__device__ __forceinline__ bf16x8 frag(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

// s_waitcnt vmcnt(N), the other counters left alone
template <int N>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt(0x0f70 | (N & 15) | ((N >> 4) << 14));
}

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
template <int W>
__device__ __forceinline__ void load_bias(const LinParams& p, int n, float (&b)[W]) {
#pragma unroll
  for (int e = 0; e < W; ++e) b[e] = p.bias && n + e < p.N ? bf16_bits_to_f32(p.bias[n + e]) : 0.f;
}

// Rows may start anywhere: pieces are moved with their elements' alignment
// (the hardware takes such accesses; aligned ones cost the same as before).
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));

// The residual and the store of W columns in whole pieces, at elements o
// (out) and r (residual).
template <int W>
__device__ __forceinline__ void finish_pieces(const LinParams& p, long long o, long long r, float (&v)[W]) {
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
template <int ACT, int W>
__device__ __forceinline__ void finish(const LinParams& p, int m, int n, float (&v)[W], const float (&b)[W]) {
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

constexpr int kBK = 64;

template <int N>
__device__ __forceinline__ void wait_vm_here() {
  asm volatile("" ::: "memory");
  wait_vm<N>();
  asm volatile("" ::: "memory");
}

// s_waitcnt lgkmcnt(0), the other counters left alone
__device__ __forceinline__ void wait_lds_here() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xc07f);
  asm volatile("" ::: "memory");
}

// Rows `row` .. rows - 1 of a matrix as a buffer: rows past the last one are
// past its end and come out as zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_from(const uint16_t* base, int row, int rows, int ld) {
  const long long bytes = (long long)(rows - row) * ld * 2;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(base + (long long)row * ld), 0,
                                           (int)(uint32_t)min(bytes, 0xffffffffLL), 0x00020000);
}

// This workgroup's place in the order of the tiles: workgroups are dealt
// round-robin over the XCDs, and each XCD takes a contiguous run.
__device__ __forceinline__ int xcd_run(int total) {
  const int xcd = blockIdx.x % kXcds, rem = total % kXcds;
  return xcd * (total / kXcds) + min(xcd, rem) + blockIdx.x / kXcds;
}

// ---------------------------------------------------------------------------
// Tiles of BM x BN for products too small to fill the card with 256 x 256
// ones: WM x WN waves of (BM / WM) x 32, times WK groups of such waves that
// take every WK-th 64-wide step of K and join at the end, through a ring of
// NS stages in LDS. What bounds these is how long a step's loads take, so
// NS - 1 stages are always under way. Places of the pieces in LDS and the
// lanes' columns are those of the 256 x 256 kernel below.
// ---------------------------------------------------------------------------
template <int BM, int BN, int WM, int WN, int WK, int NS>
__global__ __launch_bounds__(64 * WM * WN * WK) void linear_ring_kernel(LinParams p) {
  constexpr int GW = WM * WN;                               // waves of a group
  constexpr int MT = BM / WM / 16, PT = BN / WN / 32;       // row tiles and column pairs of a wave
  constexpr int NA = BM / 8 / GW, NB = BN / 8 / GW;         // loads a wave and step
  constexpr int A_BYTES = BM * kBK * 2, STEP = (BM + BN) * kBK * 2, STAGE = WK * STEP;
  static_assert(NA >= 1 && NB >= 1 && GW % 2 == 0 && (NS - 2) * (NA + NB) < 64, "ring shape");
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int gw = wave % GW, kg = wave / GW;
  const int fr = lane & 15, g = lane >> 4, lr = lane >> 3;
  const int tiles_n = (p.N + BN - 1) / BN, tiles_m = (p.M + BM - 1) / BM;
  const int l = xcd_run(gridDim.x), per = 8 * tiles_n;      // bands of 8 rows of tiles
  const int band = l / per, rr = l - band * per, rows = min(8, tiles_m - band * 8);
  const int m0 = (band * 8 + rr % rows) * BM, n0 = (rr / rows) * BN;
  const auto xb = rows_from(p.x, m0, p.M, p.ldx), wb = rows_from(p.w, n0, p.N, p.ldw);

  const int acol = (lane & 7) ^ lr, bcol = (lane & 7) ^ ((lr & 3) | ((gw & 1) << 2));
  uint32_t aoff[NA], boff[NB];
#pragma unroll
  for (int i = 0; i < NA; ++i) aoff[i] = (uint32_t)((gw + GW * i) * 8 + lr) * (uint32_t)p.ldx * 2u;
#pragma unroll
  for (int i = 0; i < NB; ++i) boff[i] = (uint32_t)((gw + GW * i) * 8 + lr) * (uint32_t)p.ldw * 2u;
  const int nk = (p.K + kBK - 1) / kBK, nit = (nk + WK - 1) / WK;
  auto load = [&](int it) {
    const int k0 = (it * WK + kg) * kBK;
    // pieces past K repeat the row's last one and enter the product as zeros
    const int ka = min(k0 + 8 * acol, p.K - 8) * 2, kw = min(k0 + 8 * bcol, p.K - 8) * 2;
    unsigned char* dst = lds + (it % NS) * STAGE + kg * STEP + gw * 1024;
#pragma unroll
    for (int i = 0; i < NA; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(xb, (lds_void*)(dst + i * GW * 1024), 16, (int)(aoff[i] + ka), 0, 0, 0);
#pragma unroll
    for (int i = 0; i < NB; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(wb, (lds_void*)(dst + A_BYTES + i * GW * 1024), 16, (int)(boff[i] + kw), 0, 0, 0);
  };

  f32x4 acc[MT][PT][2];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < PT; ++j)
#pragma unroll
      for (int t = 0; t < 2; ++t) acc[i][j][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int wm0 = (gw / WN) * (BM / WM), wn0 = (gw % WN) * (BN / WN);
  const int ar = wm0 + fr, br = wn0 + 8 * (fr >> 2) + (fr & 3);
  const int aaddr = ar * 128 + ((g ^ (ar & 7)) << 4);
  const int baddr = A_BYTES + br * 128 + ((g ^ ((br & 3) | ((br & 8) >> 1))) << 4);
  auto step = [&](int it, bool last) {
    const int at = (it % NS) * STAGE + kg * STEP, left = p.K - (it * WK + kg) * kBK;
    auto piece = [&](int a, int c) {
      const u32x4 v = *reinterpret_cast<const u32x4*>(lds + a);
      return frag(!last || 8 * c < left ? v : u32x4{0u, 0u, 0u, 0u});
    };
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      bf16x8 a[MT], b[PT][2];
#pragma unroll
      for (int j = 0; j < PT; ++j)
#pragma unroll
        for (int t = 0; t < 2; ++t) b[j][t] = piece(at + (baddr ^ (h << 6)) + j * 4096 + t * 512, 4 * h + g);
#pragma unroll
      for (int i = 0; i < MT; ++i) a[i] = piece(at + (aaddr ^ (h << 6)) + i * 2048, 4 * h + g);
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < PT; ++j)
#pragma unroll
          for (int t = 0; t < 2; ++t)
            acc[i][j][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j][t], a[i], acc[i][j][t], 0, 0, 0);
    }
  };
#pragma unroll
  for (int i = 0; i < NS - 1; ++i)
    if (i < nit) load(i);
  for (int it = 0; it < nit; ++it) {
    // this iteration's loads landed; NS - 2 younger ones may fly
    if (it + NS - 1 <= nit) wait_vm_here<(NS - 2) * (NA + NB)>();
    else wait_vm_here<0>();
    wait_lds_here();
    __builtin_amdgcn_s_barrier();  // everyone's, and stage it - 1 is out of LDS
    asm volatile("" ::: "memory");
    if (it + NS - 1 < nit) load(it + NS - 1);
    if (it + 1 < nit) step(it, false);
    else step(it, true);
  }

  if constexpr (WK > 1) {
    f32x4* part = reinterpret_cast<f32x4*>(lds);
    __syncthreads();
    if (kg > 0) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < PT; ++j)
#pragma unroll
          for (int t = 0; t < 2; ++t) part[((((kg - 1) * GW + gw) * MT + i) * PT + j) * 128 + t * 64 + lane] = acc[i][j][t];
    }
    __syncthreads();
    if (kg > 0) return;
#pragma unroll
    for (int v = 0; v < WK - 1; ++v)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < PT; ++j)
#pragma unroll
          for (int t = 0; t < 2; ++t) acc[i][j][t] += part[(((v * GW + gw) * MT + i) * PT + j) * 128 + t * 64 + lane];
  }
  with_act(p.act, [&](auto act) {
#pragma unroll
    for (int j = 0; j < PT; ++j) {
      const int n = n0 + wn0 + 32 * j + 8 * g;
      float b[8];
      load_bias(p, n, b);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int m = m0 + wm0 + 16 * i + fr;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = acc[i][j][e >> 2][e & 3];
        if (m < p.M) finish<act, 8>(p, m, n, v, b);
      }
    }
  });
}

// ---------------------------------------------------------------------------
// 256 x 256 tiles, K in steps of 64: eight waves of 128 x 64, two on each
// SIMD, which take turns: while one runs the 16 MFMAs of a phase, the other
// reads the LDS operands of its own next phase, so the matrix pipe does not
// wait for LDS. Waves 4..7 run one barrier behind waves 0..3 for that.
//
// A step of K is four phases; the x rows (A) and w rows (B) of the tile are
// halves A0, A1, B0, B1 of 128 rows, of which a wave owns 64 and 32:
//   phase       1        2        3        4
//   reads       A0       B1       A1       B0 of the next step
//   product     A0 B0    A0 B1    A1 B0    A1 B1
//   loads       A1 s+1   B0 s+2   A0 s+2   B1 s+2     (of step s, into LDS)
// LDS holds two steps (128 KB). A half is overwritten two phases after its
// last read (the late waves' operands are in registers by then) and is
// waited for, with ten younger loads of the wave still flying, one phase and
// a barrier before its first read: a load has five phases to land.
//
// A workgroup stays on its CU and takes tile after tile: the first halves of
// the next tile are loaded before the finished one goes through its epilogue,
// whose 16 or more stores per wave then drain under the next tile's first
// five phases (their waits count those 16 too; where a tile ends the matrix
// and the stores are not counted, the epilogue ends with an empty queue).
// The tiles of an XCD are taken in bands of 8 rows of tiles, columns outside:
// the 32 tiles that its CUs work on at a time share 8 x-bands and 4 w-bands
// in its L2.
//
// Piece c of an A row r sits at place c ^ (r & 7). A lane's operand row of w
// is 8 (fr / 4) + fr % 4 (+ 4 in the second tile of a pair), so that it ends
// with eight adjacent columns; piece c of a B row sits at
// c ^ (r & 3 | (r & 8) / 2), which spreads those rows over the banks.
// ---------------------------------------------------------------------------
constexpr int kHalfBytes = 128 * kBK * 2;
constexpr int kTurnCus = 256;     // one workgroup a CU: its LDS and registers fill it
constexpr int kTurnBand = 8;      // rows of tiles in a band
constexpr int kTurnMinSteps = 5;  // two steps after a tile's start and three before its end are apart

__device__ __forceinline__ void phase_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
}

__global__ __launch_bounds__(512, 2) void linear_turn_kernel(LinParams p) {
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 15, g = lane >> 4;
  const int wm = wave >> 2, wn = wave & 3;
  const int lr = lane >> 3;
  const int acol = (lane & 7) ^ lr, bcol = (lane & 7) ^ ((lr & 3) | ((wave & 1) << 2));
  const int nk = (p.K + kBK - 1) / kBK;
  // the last step's pieces past K load the row's last one instead
  const int left = p.K - (nk - 1) * kBK;

  // this XCD's run of tiles (workgroups are dealt round-robin over the XCDs)
  const int tiles_n = (p.N + 255) / 256, tiles_m = (p.M + 255) / 256;
  const int total = tiles_m * tiles_n;
  const int xcd = blockIdx.x % kXcds, rem = total % kXcds;
  const int first = xcd * (total / kXcds) + min(xcd, rem);
  const int count = total / kXcds + (xcd < rem ? 1 : 0);
  const int slots = ((int)gridDim.x + kXcds - 1 - xcd) / kXcds;
  int at = blockIdx.x / kXcds;
  if (at >= count) return;

  // of the tile whose loads are being issued
  int m0, n0;
  __amdgpu_buffer_rsrc_t xb, wb;
  auto turn_to = [&](int i) {
    const int l = first + i, per = kTurnBand * tiles_n;
    const int band = l / per, r = l - band * per, rows = min(kTurnBand, tiles_m - band * kTurnBand);
    m0 = (band * kTurnBand + r % rows) * 256;
    n0 = (r / rows) * 256;
    xb = rows_from(p.x, m0, p.M, p.ldx);
    wb = rows_from(p.w, n0, p.N, p.ldw);
  };
  // byte offsets of the pieces this lane loads: halves A0, A1, B0, B1
  uint32_t off[4][2];
#pragma unroll
  for (int h = 0; h < 4; ++h)
#pragma unroll
    for (int i = 0; i < 2; ++i)
      off[h][i] = (uint32_t)((h & 1) * 128 + (wave + 8 * i) * 8 + lr) * (uint32_t)(h < 2 ? p.ldx : p.ldw) * 2u +
                  (h < 2 ? acol : bcol) * 16u;
  auto load = [&](int h, int step, bool last) {
    uint32_t back = 0;
    if (last) {
      back = (uint32_t)max(8 * (h < 2 ? acol : bcol) - (left - 8), 0) * 2u;
      asm volatile("" : "+v"(back));  // the differences are made here, not kept
    }
    unsigned char* dst = lds + (step & 1) * (4 * kHalfBytes) + h * kHalfBytes + wave * 1024;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(h < 2 ? xb : wb, (lds_void*)(dst + i * 8192), 16,
                                               (int)(off[h][i] - back), step * (kBK * 2), 0, 0);
  };
  // a tile's first seven halves, in the order its steps go on with
  auto load_first = [&]() {
    load(2, 0, false);
    load(0, 0, false);
    load(3, 0, false);
    load(1, 0, false);
    load(2, 1, false);
    load(0, 1, false);
    load(3, 1, false);
  };

  f32x4 acc[2][4][2][2];
  const int ar = wm * 64 + fr, br = wn * 32 + 8 * (fr >> 2) + (fr & 3);
  const int aaddr = ar * 128 + ((g ^ (ar & 7)) << 4);
  const int baddr = br * 128 + ((g ^ ((br & 3) | ((br & 8) >> 1))) << 4);
  bf16x8 fa[2][4], fb[2][2][2];  // [K half][tile], [B half][K half][tile]
  auto piece = [&](int at, int c, bool last) {
    const u32x4 v = *reinterpret_cast<const u32x4*>(lds + at);
    return frag(!last || 8 * c < left ? v : u32x4{0u, 0u, 0u, 0u});
  };
  auto read_a = [&](int half, int step, bool last) {
    int st = (step & 1) * (4 * kHalfBytes) + half * kHalfBytes;
    asm volatile("" : "+s"(st));
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) fa[k][i] = piece(st + (aaddr ^ (k << 6)) + i * 2048, 4 * k + g, last);
  };
  auto read_b = [&](int half, int step, bool last) {
    int st = (step & 1) * (4 * kHalfBytes) + (2 + half) * kHalfBytes;
    asm volatile("" : "+s"(st));
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int t = 0; t < 2; ++t) fb[half][k][t] = piece(st + (baddr ^ (k << 6)) + t * 512, 4 * k + g, last);
  };
  auto product = [&](int a, int b) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int t = 0; t < 2; ++t)
          acc[a][i][b][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[b][k][t], fa[k][i], acc[a][i][b][t], 0, 0, 0);
  };
  // One step. Ten younger loads may fly at a wait; `early` waits, a tile's first
  // five, also leave out the last epilogue's 16 stores. `tail`: the loads are
  // those of the last step.
  auto wait_loads = [&](bool early) {
    if (early) wait_vm_here<26>();
    else wait_vm_here<10>();
  };
  auto full_step = [&](int s, bool early_first, bool early, bool tail) {
    read_a(0, s, false);
    load(1, s + 1, false);
    wait_loads(early_first);
    phase_barrier();
    product(0, 0);
    phase_barrier();
    read_b(1, s, false);
    load(2, s + 2, tail);
    wait_loads(early);
    phase_barrier();
    product(0, 1);
    phase_barrier();
    read_a(1, s, false);
    load(0, s + 2, tail);
    wait_loads(early);
    phase_barrier();
    product(1, 0);
    phase_barrier();
    read_b(0, s + 1, false);
    load(3, s + 2, tail);
    wait_loads(early);
    phase_barrier();
    product(1, 1);
    wait_lds_here();  // the next step's B0 is out of LDS before it may be overwritten
    phase_barrier();
  };

  turn_to(at);
  load_first();
  wait_vm_here<0>();
  for (;;) {
    wait_vm_here<26>();
    phase_barrier();
    read_b(0, 0, false);
    // lane (fr, g) will hold columns 8 g .. 8 g + 7 of row fr of each 16 x 32 pair
    const int me = m0 + wm * 64 + fr, ne = n0 + wn * 32 + 8 * g;
    const bool inside = m0 + 256 <= p.M && n0 + 256 <= p.N;
    u32x4 bias[2] = {u32x4{0u, 0u, 0u, 0u}, u32x4{0u, 0u, 0u, 0u}};
    if (inside && p.bias) {
#pragma unroll
      for (int b = 0; b < 2; ++b) bias[b] = *reinterpret_cast<const u32x4_any*>(p.bias + ne + b * 128);
    }
    if (wm == 1) phase_barrier();
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int t = 0; t < 2; ++t) acc[a][i][b][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    // (the steps' numbers are hidden from the compiler: peeled copies cost registers)
    int s = 0;
    for (; s < 2; ++s) {
      asm volatile("" : "+s"(s));
      full_step(s, true, s == 0, false);
    }
    for (; s + 3 < nk; ++s) full_step(s, false, false, false);
    asm volatile("" : "+s"(s));
    full_step(s, false, false, true);
    ++s;
    // the last step but one
    read_a(0, s, false);
    load(1, s + 1, true);
    wait_vm_here<10>();
    phase_barrier();
    product(0, 0);
    phase_barrier();
    read_b(1, s, false);
    wait_vm_here<8>();
    phase_barrier();
    product(0, 1);
    phase_barrier();
    read_a(1, s, false);
    wait_vm_here<6>();
    phase_barrier();
    product(1, 0);
    phase_barrier();
    read_b(0, s + 1, true);
    wait_vm_here<4>();
    phase_barrier();
    product(1, 1);
    phase_barrier();
    ++s;
    // the last
    read_a(0, s, true);
    wait_vm_here<2>();
    phase_barrier();
    product(0, 0);
    phase_barrier();
    read_b(1, s, true);
    wait_vm_here<0>();
    phase_barrier();
    product(0, 1);
    phase_barrier();
    read_a(1, s, true);
    wait_lds_here();  // nothing is read from LDS after this barrier: the next tile may come in
    phase_barrier();
    product(1, 0);
    product(1, 1);
    if (wm == 0) phase_barrier();

    asm volatile("" : "+v"(bias[0]), "+v"(bias[1]));  // landed long ago, on every path
    at += slots;
    const bool more = at < count;
    if (more) {
      turn_to(at);
      load_first();
      asm volatile("" ::: "memory");  // the waits count on the epilogue's stores being younger
    }
    with_act(p.act, [&](auto act) {
      if (inside) {
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const int m = me + a * 128 + 16 * i, n = ne + b * 128;
              float v[8];
#pragma unroll
              for (int e = 0; e < 8; ++e)
                v[e] = activate<act>(acc[a][i][b][e >> 2][e & 3] +
                                     __uint_as_float(e & 1 ? bias[b][e >> 1] & 0xffff0000u : bias[b][e >> 1] << 16));
              finish_pieces<8>(p, (long long)m * p.ldo + n, (long long)m * p.ldr + n, v);
            }
      } else {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float z[8];
          load_bias(p, ne + b * 128, z);
#pragma unroll
          for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float v[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] = acc[a][i][b][e >> 2][e & 3];
              if (me + a * 128 + 16 * i < p.M) finish<act, 8>(p, me + a * 128 + 16 * i, ne + b * 128, v, z);
            }
        }
      }
    });
    if (!more) break;
    if (!inside) wait_vm_here<0>();
  }
}

// ---------------------------------------------------------------------------
// Up to 16 MT rows: a workgroup takes 16 columns (rows of w), its NW waves take
// every NW-th 64-wide piece of K with the next piece's operands on their way
// during a piece's products, and their sums meet in LDS in a fixed order.
// ---------------------------------------------------------------------------
template <int MT, int NW>
__global__ __launch_bounds__(64 * NW) void linear_few_kernel(LinParams p) {
  __shared__ f32x4 part[NW][MT][64];
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
  u32x4 wv[2][2], xv[2][2][MT];  // [buffer][half of the piece]
  auto read = [&](int buf, int k0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = min(k0 + 32 * h + 8 * g, p.K - 8);  // past K: repeated, and taken as zeros
      wv[buf][h] = *reinterpret_cast<const u32x4*>(wr + k);
#pragma unroll
      for (int i = 0; i < MT; ++i) xv[buf][h][i] = *reinterpret_cast<const u32x4*>(xr[i] + k);
    }
  };
  auto product = [&](int buf, int k0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool in = k0 + 32 * h + 8 * g < p.K;
      const u32x4 z = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int i = 0; i < MT; ++i)
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(in ? wv[buf][h] : z), frag(in ? xv[buf][h][i] : z),
                                                         acc[i], 0, 0, 0);
    }
  };
  constexpr int kStep = 64 * NW;
  int k0 = wave * 64;
  if (k0 < p.K) read(0, k0);
  for (; k0 < p.K; k0 += 2 * kStep) {
    if (k0 + kStep < p.K) read(1, k0 + kStep);
    product(0, k0);
    if (k0 + kStep < p.K) {
      if (k0 + 2 * kStep < p.K) read(0, k0 + 2 * kStep);
      product(1, k0 + kStep);
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) part[wave][i][lane] = acc[i];
  __syncthreads();
  for (int i = wave; i < MT; i += NW) {
    f32x4 s = part[0][i][lane];
#pragma unroll
    for (int v = 1; v < NW; ++v) s += part[v][i][lane];
    const int m = 16 * i + fr, n = n0 + 4 * g;
    float b[4], v[4] = {s[0], s[1], s[2], s[3]};
    load_bias(p, n, b);
    if (m < p.M) with_act(p.act, [&](auto act) { finish<act, 4>(p, m, n, v, b); });
  }
}

// Rows of n elements, ld apart, into rows of n8 = n rounded up to 8, the rest
// zero, one 16-byte piece a thread: x, w or both, x first.
struct PackParams {
  const uint16_t* src[2];
  uint16_t* dst[2];
  long long ld[2], pieces[2];
  int n, n8;
};

__global__ __launch_bounds__(256) void linear_pack_kernel(PackParams p) {
  const int per = p.n8 / 8;
  for (long long u = (long long)blockIdx.x * 256 + threadIdx.x; u < p.pieces[0] + p.pieces[1];
       u += (long long)gridDim.x * 256) {
    const int which = u >= p.pieces[0];
    const long long v = which ? u - p.pieces[0] : u, r = v / per;
    const int c = (int)(v - r * per) * 8;
    const uint16_t* src = (which ? p.src[1] : p.src[0]) + r * (which ? p.ld[1] : p.ld[0]) + c;
    u32x4 t;
    if (c + 8 <= p.n) {
      t = *reinterpret_cast<const u32x4_any*>(src);
    } else {
      uint16_t e8[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) e8[e] = c + e < p.n ? src[e] : (uint16_t)0;
      __builtin_memcpy(&t, e8, 16);
    }
    *reinterpret_cast<u32x4*>((which ? p.dst[1] : p.dst[0]) + r * p.n8 + c) = t;
  }
}

size_t al256(size_t n) { return (n + 255) & ~(size_t)255; }
int up8(int n) { return (n + 7) & ~7; }
bool packs(int K, long long ld) { return K % 8 != 0 || ld % 8 != 0; }

template <int BM, int BN, int WM, int WN, int WK, int NS>
hipError_t run_ring(const LinParams& p, hipStream_t st) {
  const long long tiles = (long long)((p.M + BM - 1) / BM) * ((p.N + BN - 1) / BN);
  hipLaunchKernelGGL((linear_ring_kernel<BM, BN, WM, WN, WK, NS>), dim3((unsigned)tiles), dim3(64 * WM * WN * WK),
                     NS * WK * (BM + BN) * kBK * 2, st, p);
  return hipGetLastError();
}

template <int MT>
hipError_t run_few(const LinParams& p, hipStream_t st) {
  if (p.K > 512)
    hipLaunchKernelGGL((linear_few_kernel<MT, 16>), dim3((p.N + 15) / 16), dim3(1024), 0, st, p);
  else
    hipLaunchKernelGGL((linear_few_kernel<MT, 8>), dim3((p.N + 15) / 16), dim3(512), 0, st, p);
  return hipGetLastError();
}

hipError_t run_turn(const LinParams& p, hipStream_t st) {
  const long long tiles = (long long)((p.M + 255) / 256) * ((p.N + 255) / 256);
  hipLaunchKernelGGL(linear_turn_kernel, dim3((unsigned)(tiles < kTurnCus ? tiles : kTurnCus)), dim3(512),
                     8 * kHalfBytes, st, p);
  return hipGetLastError();
}

// The kernel follows from how many tiles there are for the 256 CUs. Measured
// (M x N x K; us, this choice / the next best): 222 x 58 x 4096 19 / 31, 700 x 1209 x
// 2384 15 / 22 (64 x 64 tiles); 1425 x 777 x 646 15 / 18 (128 x 64); 3825 x
// 610 x 3616 40 / 43, 8049 x 260 x 2952 35 / 38 (128 x 128, four stages);
// 28607 x 2031 x 224 72 / 80, 35266 x 476 x 96 17 / 19 (128 x 128, two
// stages, two workgroups a CU).
hipError_t run_rows(const LinParams& p, hipStream_t st) {
  if (p.M <= 16) return run_few<1>(p, st);
  if (p.M <= 32) return run_few<2>(p, st);
  if (p.M <= 64) return run_few<4>(p, st);
  auto tiles = [&](long long m, int bm, int bn) { return ((m + bm - 1) / bm) * ((p.N + bn - 1) / bn); };
  if (tiles(p.M, 64, 64) <= 256) return run_ring<64, 64, 2, 2, 2, 4>(p, st);
  if (tiles(p.M, 128, 64) <= 256) return run_ring<128, 64, 4, 2, 1, 3>(p, st);
  if (tiles(p.M, 128, 128) <= 256) return run_ring<128, 128, 2, 4, 1, 4>(p, st);
  // Beyond that the 256 x 256 kernel takes 1.35 us a step and 10 us a tile, all
  // CUs in step, and the 128 x 128 one 0.95 us and 7 us for each 512 tiles, one
  // round of smaller tiles 1.2 us and 5 (bfloat16 outputs, no residual; the model
  // knows neither): 15161 x 3143 x 1512 168 against 198, 4096 x 4096 x 1024 32
  // against 39, each in one launch. Rows beyond the 256 x 256 tiles' last whole
  // round go to a launch of their own where that is the least (calls with it /
  // without): 19706 x 1024 x 1024 70 / 86 us with a float32 residual, 44 / 49 in
  // bfloat16 without; 15161 x 3143 x 1512 142 / 168; 8917 x 2079 x 3552 130 /
  // 153. Over 45 drawn sizes it gained 4% on average, from 7% slower to 38%
  // faster: what the model leaves out.
  const int nk = (p.K + kBK - 1) / kBK;
  auto ring = [&](long long m) {
    const long long n = tiles(m, 128, 128);
    return n <= 256 ? 1.2 * nk + 5.0 : (double)((n + 511) / 512) * (0.95 * nk + 7.0);
  };
  if (nk >= kTurnMinSteps) {
    const double round = 1.35 * nk + 10.0;
    const long long n = tiles(p.M, 256, 256), whole = n / kTurnCus;
    const double turn = (double)((n + kTurnCus - 1) / kTurnCus) * round, all = ring(p.M);
    const long long head = whole * kTurnCus / tiles(1, 256, 256) * 256;  // rows of the whole rounds
    if (head > 0 && head < p.M && (double)whole * round + ring(p.M - head) < 0.95 * (turn < all ? turn : all)) {
      LinParams first = p, rest = p;
      first.M = (int)head;
      const hipError_t e = run_turn(first, st);
      if (e != hipSuccess) return e;
      const long long size = p.out_f32 ? 4 : 2;
      rest.M = (int)(p.M - head);
      rest.x = p.x + head * p.ldx;
      if (p.res) rest.res = static_cast<const uint8_t*>(p.res) + head * p.ldr * size;
      rest.out = static_cast<uint8_t*>(p.out) + head * p.ldo * size;
      return run_rows(rest, st);
    }
    if (turn <= all) return run_turn(p, st);
  }
  return run_ring<128, 128, 4, 2, 1, 2>(p, st);
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
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  PackParams pk{};
  pk.n = a.K;
  pk.n8 = p.K;
  auto pack = [&](int which, const uint16_t*& src, int& ld, int rows) {
    pk.src[which] = src;
    pk.ld[which] = ld;
    pk.dst[which] = reinterpret_cast<uint16_t*>(ws);
    pk.pieces[which] = (long long)rows * (p.K / 8);
    ws += al256((size_t)rows * p.K * 2);
    src = pk.dst[which];
    ld = p.K;
  };
  if (packs(a.K, a.ldx)) pack(0, p.x, p.ldx, a.M);
  if (packs(a.K, a.ldw)) pack(1, p.w, p.ldw, a.N);
  if (const long long n = pk.pieces[0] + pk.pieces[1]; n > 0) {
    const long long wgs = (n + 255) / 256;
    hipLaunchKernelGGL(linear_pack_kernel, dim3((unsigned)(wgs < 4096 ? wgs : 4096)), dim3(256), 0, st, pk);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return run_rows(p, st);
}

}  // namespace gkd
