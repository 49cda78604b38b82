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
  int vec;             // finish() may move whole pieces
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
// smooth, so a polynomial of degree 7 (minimax on 0..6.5, fitted with the
// error weighted as it enters the result) leaves 1.8e-7 of error in z Phi(z)
// and, as a factor, keeps 5e-5 relative in the tail down to z = -6; further
// out P falls on without bound and the tail goes to 0. 11 VALU operations and
// one quarter-rate one.
__device__ __forceinline__ float gelu(float z) {
  const float a = fminf(fabsf(z), 64.f);  // Phi(-64) is 0 in float32
  float y = fmaf(-1.61419405e-06f, a, 5.75573977e-05f);
  y = fmaf(y, a, -0.000903298729f);
  y = fmaf(y, a, 0.00842618756f);
  y = fmaf(y, a, -0.053858351f);
  y = fmaf(y, a, -0.458490729f);
  y = fmaf(y, a, -1.15127611f);
  y = fmaf(y, a, -0.999987483f);
  return fmaf(-a, __builtin_amdgcn_exp2f(y), z < 0.f ? 0.f : z);
}

template <int ACT>
__device__ __forceinline__ float activate(float z) {
  if constexpr (ACT == GKD_ACT_RELU) return z < 0.f ? 0.f : z;  // a NaN stays one
  if constexpr (ACT == GKD_ACT_GELU) return gelu(z);
  // z / (1 + exp(-c z)): for z far below 0 exp gives infinity and the quotient 0
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

// The residual and the store of W columns in whole pieces, at elements o
// (out) and r (residual).
template <int W>
__device__ __forceinline__ void finish_pieces(const LinParams& p, long long o, long long r, float (&v)[W]) {
  if (p.out_f32) {
#pragma unroll
    for (int q = 0; q < W / 4; ++q) {
      f32x4 t = {v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
      if (p.res) t += *reinterpret_cast<const f32x4*>(static_cast<const float*>(p.res) + r + 4 * q);
      *reinterpret_cast<f32x4*>(static_cast<float*>(p.out) + o + 4 * q) = t;
    }
  } else {
    typedef uint32_t words __attribute__((ext_vector_type(W / 2)));
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
// of row m < M; columns past N are left out. Whole pieces where the rows
// allow it (p.vec: W adjacent columns are aligned in out and residual), else
// one by one.
template <int ACT, int W>
__device__ __forceinline__ void finish(const LinParams& p, int m, int n, float (&v)[W], const float (&b)[W]) {
  if (n >= p.N) return;
  const long long o = (long long)m * p.ldo + n, r = (long long)m * p.ldr + n;
#pragma unroll
  for (int e = 0; e < W; ++e) v[e] = activate<ACT>(v[e] + b[e]);
  if (n + W <= p.N && p.vec) {
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
  with_act(p.act, [&](auto act) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int n = n0 + wn0 + 16 * j + 4 * g;
      float b[4];
      load_bias(p, n, b);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int m = m0 + wm0 + 16 * i + fr;
        float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
        if (m < p.M) finish<act, 4>(p, m, n, v, b);
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
  // the matrices from the tile's first row on; rows past the last one are past
  // the end of the buffer (they come out as zeros, and are not stored)
  __amdgpu_buffer_rsrc_t xb, wb;
  auto rows_from = [&](const uint16_t* base, int row, int rows, int ld) {
    const long long bytes = (long long)(rows - row) * ld * 2;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(base + (long long)row * ld), 0,
                                             (int)(uint32_t)min(bytes, 0xffffffffLL), 0x00020000);
  };
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
    const bool inside = m0 + 256 <= p.M && n0 + 256 <= p.N && p.vec;
    u32x4 bias[2] = {u32x4{0u, 0u, 0u, 0u}, u32x4{0u, 0u, 0u, 0u}};
    if (inside && p.bias) {
#pragma unroll
      for (int b = 0; b < 2; ++b) bias[b] = *reinterpret_cast<const u32x4*>(p.bias + ne + b * 128);
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
    const int m = 16 * i + fr, n = n0 + 4 * g;
    float b[4], v[4] = {s[0], s[1], s[2], s[3]};
    load_bias(p, n, b);
    if (m < p.M) with_act(p.act, [&](auto act) { finish<act, 4>(p, m, n, v, b); });
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
  // 16-byte pieces: eight bf16 columns (the 4-column kernels need half), four float32 ones
  const int unit = a.out_f32 ? 4 : 8;
  p.vec = ((reinterpret_cast<uintptr_t>(a.out) | reinterpret_cast<uintptr_t>(a.residual) |
            reinterpret_cast<uintptr_t>(a.bias)) & 15u) == 0 &&
          a.ldo % unit == 0 && (a.residual == nullptr || a.ldr % unit == 0);
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
  if ((long long)p.M * p.N >= 256LL * 256 * 256 && p.K > (kTurnMinSteps - 1) * kBK) {
    const long long tiles = (long long)((p.M + 255) / 256) * ((p.N + 255) / 256);
    hipLaunchKernelGGL(linear_turn_kernel, dim3((unsigned)(tiles < kTurnCus ? tiles : kTurnCus)), dim3(512),
                       8 * kHalfBytes, st, p);
    return hipGetLastError();
  }
  return run_tiles<128, 128, 2, 2>(p, st);
}

}  // namespace gkd
