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
#include <cstdlib>

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

// `rows` rows of `bytes` bytes as a buffer: what lies past them comes out as zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_of(const void* base, long long rows, long long ld, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)(uint32_t)((rows - 1) * ld + bytes), 0x00020000);
}
constexpr uint32_t kNowhere = 0xf0000000u;  // past every such buffer: 2^31 bytes at most

typedef __attribute__((address_space(3))) void lds_void;

template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0f70 | (N & 15) | ((N >> 4) << 14));  // vmcnt(N), the other counters left alone
  asm volatile("" ::: "memory");
}

// A stage of a wave's ring: 256 of K of 16 NT rows of w and MX rows of x (two at least, as
// a load brings two), 16-byte piece c of a row at piece c ^ (row / 2) % 8 of w and
// c ^ row % 16 of x, so that 16 lanes that read the same piece of 16 rows share no bank.
// Scale bytes come four at a time where rows of them are whole words, else (BYTES) one by
// one, each into a word.
template <int MX, int NT, bool BYTES>
struct FewStage {
  static constexpr int kRowsX = MX < 2 ? 2 : MX, kLoadsS = BYTES ? 2 * NT : (NT + 1) / 2;
  static constexpr int kScales = 2048 * NT, kX = kScales + 256 * kLoadsS, kBytes = kX + 512 * kRowsX;
  static constexpr int kLoads = 2 * NT + kLoadsS + kRowsX / 2;
};

// MX rows of x at most and 16 NT rows of w a workgroup. Each of its NW waves takes a range
// of K through a ring of STAGES stages of its own in LDS, and the sums meet in LDS in a fixed
// order. Loads go straight to LDS, whole lines of memory at a time: what bounds reading here
// is the number of loads and lines a CU asks for. Rows of w are often a multiple of 4 KB
// long, over which the memory channels repeat: so the waves' ranges lie apart, and workgroups
// begin at different places in them. Pieces past a range, and rows past the matrices, come
// out as zeros.
template <int MX, int NT, int NW, int STAGES, bool BYTES>
__global__ __launch_bounds__(64 * NW) void fp4_few_kernel(Fp4Params p) {
  typedef FewStage<MX, NT, BYTES> St;
  constexpr int MT = (MX + 15) / 16;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 15, g = lane >> 4;
  const int tiles_n = (p.N + 16 * NT - 1) / (16 * NT), tm = blockIdx.x / tiles_n;
  const int n0 = (blockIdx.x - tm * tiles_n) * 16 * NT, m0 = tm * MX;
  const long long rows = min(16 * NT, p.N - n0);
  const auto cb = rows_of(p.codes + (long long)n0 * (p.K / 2), rows, p.K / 2, p.K / 2);
  const auto sb = rows_of(p.scales + (long long)n0 * (p.K / 32), rows, p.K / 32, p.K / 32);
  const auto xb = rows_of(p.x + (long long)m0 * p.ldx, min(MX, p.M - m0), 2LL * p.ldx, 2 * p.K);

  // What a lane loads: row and k of its 16 bytes of codes (8 rows a load), its scales (32
  // rows a load, or 8), its 16 bytes of x (2 rows).
  const int cr = lane >> 3, sr = BYTES ? lane >> 3 : lane >> 1, xr = lane >> 5;
  const int pieces = (p.K + 255) / 256, from = pieces * wave / NW, n = pieces * (wave + 1) / NW - from;
  int at = n > 0 ? blockIdx.x % n : 0, left = n;  // the next piece to load, and how many
  unsigned char* ring = lds + wave * STAGES * St::kBytes;
  auto load = [&](int stage) {
    unsigned char* dst = ring + stage * St::kBytes;
    const int k0 = left > 0 ? (from + at) * 256 : p.K;  // past K: zeros
#pragma unroll
    for (int i = 0; i < 2 * NT; ++i) {
      const int r = 8 * i + cr, k = k0 + 32 * ((lane & 7) ^ ((r >> 1) & 7));
      const uint32_t a = k < p.K ? (uint32_t)r * (p.K / 2) + k / 2 : kNowhere;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(cb, (lds_void*)(dst + i * 1024), 16, (int)a, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < St::kLoadsS; ++i) {
      const int r = (BYTES ? 8 : 32) * i + sr, k = k0 + (BYTES ? 32 * (lane & 7) : 128 * (lane & 1));
      const uint32_t a = k < p.K ? (uint32_t)r * (p.K / 32) + k / 32 : kNowhere;
      if constexpr (BYTES)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(sb, (lds_void*)(dst + St::kScales + i * 256), 1, (int)a, 0, 0, 0);
      else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(sb, (lds_void*)(dst + St::kScales + i * 256), 4, (int)a, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < St::kRowsX / 2; ++i) {
      const int r = 2 * i + xr, k = k0 + 8 * ((lane & 31) ^ (r & 15));
      const uint32_t a = k < p.K && r < MX ? (uint32_t)r * (uint32_t)p.ldx * 2u + 2 * k : kNowhere;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(xb, (lds_void*)(dst + St::kX + i * 1024), 16, (int)a, 0, 0, 0);
    }
    if (++at == n) at = 0;
    --left;
  };

  f32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int xrow = MX < 16 ? fr % MX : fr;  // (columns past MX hold anything)
  auto product = [&](int stage) {
    const unsigned char* src = ring + stage * St::kBytes;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      u32x4 c[NT];
      float unit[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        c[j] = *reinterpret_cast<const u32x4*>(src + (16 * j + fr) * 128 + (((4 * h + g) ^ (fr >> 1)) << 4));
        unit[j] = fp4_unit(src[St::kScales + ((16 * j + fr) * 8 + 4 * h + g) * (BYTES ? 4 : 1)]);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        bf16x8 x[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i)
          x[i] = frag(*reinterpret_cast<const u32x4*>(src + St::kX + (16 * i + xrow) * 512 +
                                                      (((16 * h + 4 * g + t) ^ xrow) << 4)));
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const bf16x8 w = frag(fp4_values(c[j][t], unit[j]));
#pragma unroll
          for (int i = 0; i < MT; ++i) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x[i], acc[i][j], 0, 0, 0);
        }
      }
    }
  };
  if (n > 0) {
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) load(i);
    for (int i = 0, stage = 0; i < n; ++i) {
      load(stage == 0 ? STAGES - 1 : stage - 1);  // the stage before: it has been read
      wait_vm<(STAGES - 1) * St::kLoads>();
      product(stage);
      stage = stage + 1 < STAGES ? stage + 1 : 0;
    }
    wait_vm<0>();
  }
  __syncthreads();  // the ring's places are the sums'
  f32x4* part = reinterpret_cast<f32x4*>(lds);  // [NW][MT][NT][64]
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) part[((wave * MT + i) * NT + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  for (int u = wave; u < MT * NT; u += NW) {
    const int i = u / NT, j = u % NT;
    f32x4 sum = part[u * 64 + lane];
#pragma unroll
    for (int v = 1; v < NW; ++v) sum += part[(v * MT * NT + u) * 64 + lane];
    const int m = m0 + 16 * i + fr, col = n0 + 16 * j + 4 * g;
    float b[4], v[4] = {sum[0], sum[1], sum[2], sum[3]};
    load_bias(p, col, b);
    if (m < p.M && 16 * i + fr < MX) with_act(p.act, [&](auto act) { finish<act, 4>(p, m, col, v, b); });
  }
}

template <int MX, int NT, int NW, int STAGES, bool BYTES>
hipError_t launch_few(const Fp4Params& p, hipStream_t st) {
  constexpr int kRing = NW * STAGES * FewStage<MX, NT, BYTES>::kBytes, kJoin = NW * ((MX + 15) / 16) * NT * 1024;
  constexpr int kLds = kRing > kJoin ? kRing : kJoin;
  static_assert(kLds <= 160 * 1024, "the ring fits");
  const long long tiles = (long long)((p.N + 16 * NT - 1) / (16 * NT)) * ((p.M + MX - 1) / MX);
  hipLaunchKernelGGL((fp4_few_kernel<MX, NT, NW, STAGES, BYTES>), dim3((unsigned)tiles), dim3(64 * NW), kLds, st, p);
  return hipGetLastError();
}

template <int MX, int NT, int NW, int STAGES>
hipError_t run_few(const Fp4Params& p, hipStream_t st) {
  return p.K % 128 == 0 ? launch_few<MX, NT, NW, STAGES, false>(p, st) : launch_few<MX, NT, NW, STAGES, true>(p, st);
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
  const char* e = getenv("GKD_F");
  const int f = e ? atoi(e) : 0;
  if (f == 1) return run_few<1, 1, 4, 2>(p, st);
  if (f == 2) return run_few<1, 1, 4, 3>(p, st);
  if (f == 3) return run_few<1, 1, 8, 2>(p, st);
  if (f == 4) return run_few<1, 1, 8, 3>(p, st);
  if (f == 5) return run_few<1, 1, 16, 2>(p, st);
  if (f == 6) return run_few<1, 2, 4, 2>(p, st);
  if (f == 7) return run_few<1, 2, 8, 2>(p, st);
  if (f == 8) return run_few<1, 2, 4, 3>(p, st);
  if (f == 9) return run_few<16, 1, 4, 2>(p, st);
  if (f == 10) return run_few<16, 1, 4, 3>(p, st);
  if (f == 12) return run_few<16, 2, 4, 2>(p, st);
  if (f == 13) return run_few<16, 2, 4, 3>(p, st);
  if (f == 14) return run_few<32, 1, 4, 2>(p, st);
  if (f == 15) return run_few<32, 2, 2, 2>(p, st);
  if (f == 16) return run_few<4, 1, 8, 2>(p, st);
  if (f == 17) return run_few<4, 1, 4, 3>(p, st);
  if (p.M <= 1) return run_few<1, 1, 8, 2>(p, st);
  if (p.M <= 4) return run_few<4, 1, 8, 2>(p, st);
  if (p.M <= 16) return run_few<16, 1, 4, 2>(p, st);
  return run_few<32, 1, 4, 2>(p, st);
}

}  // namespace gkd
