// fp4_linear.hip - matrix product with four-bit weights (gkd_linear_fp4):
// out = act(x w^T + bias) + residual.
//
// A lane holds part of one group of 32 codes of a row of w and its scale byte, which the
// conversion instructions turn into the first operand of v_mfma_f32_16x16x32_bf16, eight
// values at a time and exactly. Which k a lane's place in the instruction stands for is
// free as long as x is read alike: place (g, i) of product t is k = 32 g + 8 t + i, so a
// lane's 16 bytes of codes are its operands of four products. Both operands go through
// rings in LDS, for loads of whole lines and many of them under way; nothing is rounded on
// the way, and sums of ranges of K meet in a fixed order.
//
// What bounds it: few rows, the codes' way from memory. 1 x 4096 x 16384 takes 10.3 us,
// 3.4 TB/s where a large copy on the same card moves 5.0; 13 x 16384 x 4095 13.4 us
// (2.7 TB/s); 1 x 1024 x 1024 2.8 us, little more than a launch. Up to some hundreds of
// rows, the loads that a CU has under way, x from L2 beside the codes: 37 x 1024 x 4096
// 6.0 us, 128 x 8192 x 8192 30 to 32 us, 0.54 PF. Beyond, x's way through L2 for tiles of 128
// rows and the conversions for each of them: 256, 1024 and 4096 x 8192 x 8192 48, 161 and
// 607 us (0.71, 0.86 and 0.91 PF), where gkd_linear takes 67, 150 and 374 with weights in
// bfloat16; 256 and 4096 x 1024 x 4096 20 and 83 against 8.5 and 32. (The registers alone,
// without LDS, took 13.8, 21.2, 2.8, 8.4 and 128 us for the first five.)
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

// `rows` rows of `bytes` bytes as a buffer: what lies past them comes out as zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_of(const void* base, long long rows, long long ld, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)(uint32_t)((rows - 1) * ld + bytes), 0x00020000);
}
constexpr uint32_t kNowhere = 0xf0000000u;  // past every such buffer: 2^31 bytes at most

// Rows of w and x are often a multiple of 4 KB long, over which the channels of L2 and of
// memory repeat: workgroups that went through K in step would all ask the same channel. So
// each begins elsewhere in its n pieces; those of an XCD (every eighth) at neighbouring ones.
__device__ __forceinline__ int first_piece(int n) {
  return n > 0 ? (int)((blockIdx.x / kXcds + blockIdx.x % kXcds * ((n + kXcds - 1) / kXcds)) % n) : 0;
}

// Bytes at `from` of a buffer straight to LDS, 16, 4 or 1 a lane: to dst + 16 lane or dst + 4
// lane. (Functions of their own: in a template the host's pass does not take the builtin.)
__device__ __forceinline__ void load16(__amdgpu_buffer_rsrc_t b, unsigned char* dst, uint32_t from) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (lds_void*)dst, 16, (int)from, 0, 0, 0);
}
__device__ __forceinline__ void load4(__amdgpu_buffer_rsrc_t b, unsigned char* dst, uint32_t from) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (lds_void*)dst, 4, (int)from, 0, 0, 0);
}
__device__ __forceinline__ void load1(__amdgpu_buffer_rsrc_t b, unsigned char* dst, uint32_t from) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (lds_void*)dst, 1, (int)from, 0, 0, 0);
}

// The place of piece c of row r of x, in rows of 256 bytes, is c ^ turned(r). Sixteen lanes
// that LDS serves together are, of a wave's 16-byte reads, lanes 0-3, 12-15 and 20-27 (and
// the like): rows of two neighbouring g, whose pieces differ in bit 2. So bit 3 is made to
// tell them apart (c ^ r: two lanes to a bank, 43% of the LDS cycles of 128 x 8192 x 8192).
__device__ __forceinline__ int turned(int r) { return (r & 15) ^ ((r & 4) << 1); }

// All waves, with what they read of LDS in their registers.
__device__ __forceinline__ void meet() {
  wait_lds();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// A stage of a wave's ring: 256 of K of 16 NT rows of w and MX rows of x (two at least, as
// a load brings two), 16-byte piece c of a row at piece c ^ (row / 2) % 8 of w and
// c ^ turned(row) of x, so that 16 lanes that read the same piece of 16 rows share no bank.
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
  int at = first_piece(n), left = n;  // the next piece to load, and how many
  unsigned char* ring = lds + wave * STAGES * St::kBytes;
  auto load = [&](int stage) {
    unsigned char* dst = ring + stage * St::kBytes;
    const int k0 = left > 0 ? (from + at) * 256 : p.K;  // past K: zeros
#pragma unroll
    for (int i = 0; i < 2 * NT; ++i) {
      const int r = 8 * i + cr, k = k0 + 32 * ((lane & 7) ^ ((r >> 1) & 7));
      const uint32_t a = k < p.K ? (uint32_t)r * (p.K / 2) + k / 2 : kNowhere;
      load16(cb, dst + i * 1024, a);
    }
#pragma unroll
    for (int i = 0; i < St::kLoadsS; ++i) {
      const int r = (BYTES ? 8 : 32) * i + sr, k = k0 + (BYTES ? 32 * (lane & 7) : 128 * (lane & 1));
      const uint32_t a = k < p.K ? (uint32_t)r * (p.K / 32) + k / 32 : kNowhere;
      if constexpr (BYTES)
        load1(sb, dst + St::kScales + i * 256, a);
      else
        load4(sb, dst + St::kScales + i * 256, a);
    }
#pragma unroll
    for (int i = 0; i < St::kRowsX / 2; ++i) {
      const int r = 2 * i + xr, k = k0 + 8 * ((lane & 31) ^ turned(r));
      const uint32_t a = k < p.K && r < MX ? (uint32_t)r * (uint32_t)p.ldx * 2u + 2 * k : kNowhere;
      load16(xb, dst + St::kX + i * 1024, a);
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
                                                      (((16 * h + 4 * g + t) ^ turned(xrow)) << 4)));
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
      wait_lds();
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

// ---------------------------------------------------------------------------
// More rows: tiles of BM = 16 MT WM rows of x and BN = 16 NT WN rows of w, two groups of
// WM x WN waves that take half of each product's k and join at the end. Both operands go
// through rings in LDS: x in DX stages of KC of K, the codes in DC stages of 256, which are
// whole lines of memory. One group loads x, the other the codes: a wave's loads return in
// order, so were they loaded by one wave, waiting for x, which comes from L2, would be
// waiting for the codes behind it, which come from memory. Where there are few tiles,
// `splits` workgroups share a tile's K and their sums meet in a kernel of their own.
// ---------------------------------------------------------------------------
template <int MT, int NT, int WM, int WN, int KC, bool BYTES>
struct TileStage {
  static constexpr int BM = 16 * MT * WM, BN = 16 * NT * WN, W = WM * WN;
  static constexpr int kRowsS = BYTES ? 8 : 32;  // rows of scales a load
  static constexpr int kNC = BN / 8, kNS = (BN + kRowsS - 1) / kRowsS, kNX = BM * KC / 512;
  static constexpr int kScales = BN * 128, kBytesC = kScales + 256 * kNS, kBytesX = BM * KC * 2;
  static constexpr int kLoadsC = (kNC + W - 1) / W + (kNS + W - 1) / W, kLoadsX = (kNX + W - 1) / W;  // a wave
};

struct TileParams {
  Fp4Params p;
  int splits;
  float* part;   // [splits][M][ldp] sums, or null
  int ldp;
};

template <int MT, int NT, int WM, int WN, int KC, int DX, int DC, bool BYTES>
__global__ __launch_bounds__(128 * WM * WN) void fp4_tile_kernel(TileParams tp) {
  typedef TileStage<MT, NT, WM, WN, KC, BYTES> St;
  const Fp4Params& p = tp.p;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];  // x's ring, then the codes'
  unsigned char* const codes = lds + DX * St::kBytesX;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 15, g = lane >> 4;
  const int split = blockIdx.x % tp.splits, tile = blockIdx.x / tp.splits;
  const int tiles_n = (p.N + St::BN - 1) / St::BN, tm = tile / tiles_n;
  const int n0 = (tile - tm * tiles_n) * St::BN, m0 = tm * St::BM;
  const int kg = wave / St::W, gw = wave % St::W, wm = gw / WN, wn = gw % WN;
  const auto cb = rows_of(p.codes + (long long)n0 * (p.K / 2), min(0 + St::BN, p.N - n0), p.K / 2, p.K / 2);
  const auto sb = rows_of(p.scales + (long long)n0 * (p.K / 32), min(0 + St::BN, p.N - n0), p.K / 32, p.K / 32);
  const auto xb = rows_of(p.x + (long long)m0 * p.ldx, min(0 + St::BM, p.M - m0), 2LL * p.ldx, 2 * p.K);
  const int steps = (p.K + 255) / 256;
  const int from = (int)((long long)steps * split / tp.splits), n = (int)((long long)steps * (split + 1) / tp.splits) - from;

  constexpr int SUB = 256 / KC, XR = 512 / KC, XP = KC / 8;  // rows of x a load brings, pieces of a row
  int at = first_piece(n), left = n, sub = 0, stage = 0;  // what to load next: step, how many, part of it; its stage
  auto load_x = [&] {
    unsigned char* dst = lds + stage * St::kBytesX;
    const int k0 = left > 0 ? (from + at) * 256 + sub * KC : p.K;  // past K: zeros
#pragma unroll
    for (int u = 0; u < St::kLoadsX; ++u) {
      const int i = (gw + u * St::W) % St::kNX, r = i * XR + lane / XP, k = k0 + 8 * ((lane % XP) ^ turned(r));
      const uint32_t a = k < p.K ? (uint32_t)r * (uint32_t)p.ldx * 2u + 2 * k : kNowhere;
      load16(xb, dst + i * 1024, a);
    }
    stage = stage + 1 < DX ? stage + 1 : 0;
    if (++sub < SUB) return;
    sub = 0;
    if (++at == n) at = 0;
    --left;
  };
  auto load_codes = [&] {
    unsigned char* dst = codes + stage * St::kBytesC;
    const int k0 = left > 0 ? (from + at) * 256 : p.K;
#pragma unroll
    for (int u = 0; u < (St::kNC + St::W - 1) / St::W; ++u) {
      const int i = (gw + u * St::W) % St::kNC, r = i * 8 + lane / 8, k = k0 + 32 * ((lane & 7) ^ ((r >> 1) & 7));
      const uint32_t a = k < p.K ? (uint32_t)r * (p.K / 2) + k / 2 : kNowhere;
      load16(cb, dst + i * 1024, a);
    }
#pragma unroll
    for (int u = 0; u < (St::kNS + St::W - 1) / St::W; ++u) {
      const int i = (gw + u * St::W) % St::kNS;
      constexpr int PER = BYTES ? 8 : 2;  // loads of a row
      const int r = i * St::kRowsS + lane / PER, k = k0 + lane % PER * (BYTES ? 32 : 128);
      const uint32_t a = k < p.K ? (uint32_t)r * (p.K / 32) + k / 32 : kNowhere;
      if constexpr (BYTES)
        load1(sb, dst + St::kScales + i * 256, a);
      else
        load4(sb, dst + St::kScales + i * 256, a);
    }
    stage = stage + 1 < DC ? stage + 1 : 0;
    if (++at == n) at = 0;
    --left;
  };

  f32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int wrow = wn * 16 * NT + fr, xrow = wm * 16 * MT + fr;
  // 128 of K, the h-th of their stages; this wave's half of each group, by turns the first and
  // the second for neighbouring g, whose lanes would meet in a bank otherwise
  const int half = kg ^ (g & 1);
  auto product = [&](const unsigned char* sx, int hx, const unsigned char* sc, int hc) {
    u32x2 c[NT];
    float unit[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      c[j] = *reinterpret_cast<const u32x2*>(sc + (wrow + 16 * j) * 128 + (((4 * hc + g) ^ (fr >> 1)) << 4) + 8 * half);
      unit[j] = fp4_unit(sc[St::kScales + ((wrow + 16 * j) * 8 + 4 * hc + g) * (BYTES ? 4 : 1)]);
    }
    bf16x8 x[2][MT];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < MT; ++i)
        x[u][i] = frag(*reinterpret_cast<const u32x4*>(sx + (xrow + 16 * i) * (2 * KC) +
                                                       (((16 * hx + 4 * g + 2 * half + u) ^ turned(fr)) << 4)));
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const bf16x8 w = frag(fp4_values(c[j][u], unit[j]));
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x[u][i], acc[i][j], 0, 0, 0);
      }
  };
  if (kg == 0) {
#pragma unroll
    for (int i = 0; i < DX - 1; ++i) load_x();
  } else {
#pragma unroll
    for (int i = 0; i < DC - 1; ++i) load_codes();
  }
  for (int it = 0, sx = 0, sc = 0; it < n; ++it) {
#pragma unroll
    for (int part = 0; part < SUB; ++part) {
      if (kg == 0) wait_vm<(DX - 2) * St::kLoadsX>();
      else if (part == 0) wait_vm<(DC - 2) * St::kLoadsC>();
      meet();  // everyone's loads of the part are here, and everyone has read the part before
      if (kg == 0) load_x();
      else if (part == 0) load_codes();
#pragma unroll
      for (int h = 0; h < KC / 128; ++h)
        product(lds + sx * St::kBytesX, h, codes + sc * St::kBytesC, part * (KC / 128) + h);
      sx = sx + 1 < DX ? sx + 1 : 0;
    }
    sc = sc + 1 < DC ? sc + 1 : 0;
  }
  wait_vm<0>();
  f32x4* other = reinterpret_cast<f32x4*>(lds) + gw * MT * NT * 64 + lane;
  meet();
  if (kg > 0) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) other[(i * NT + j) * 64] = acc[i][j];
  }
  __syncthreads();
  if (kg > 0) return;

#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int col = n0 + wn * 16 * NT + 16 * j + 4 * g;
    float b[4];
    if (!tp.part) load_bias(p, col, b);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int m = m0 + xrow + 16 * i;
      const f32x4 sum = acc[i][j] + other[(i * NT + j) * 64];
      if (m >= p.M || col >= p.N) continue;
      if (tp.part) {
        *reinterpret_cast<f32x4*>(tp.part + ((long long)split * p.M + m) * tp.ldp + col) = sum;
      } else {
        float v[4] = {sum[0], sum[1], sum[2], sum[3]};
        with_act(p.act, [&](auto act) { finish<act, 4>(p, m, col, v, b); });
      }
    }
  }
}

// The sums of a tile's splits, in their order, and the epilogue; four columns a thread.
__global__ __launch_bounds__(256) void fp4_join_kernel(TileParams tp) {
  const Fp4Params& p = tp.p;
  const int per = tp.ldp / 4;
  const long long u = (long long)blockIdx.x * 256 + threadIdx.x;
  const int m = (int)(u / per), col = (int)(u - (long long)m * per) * 4;
  if (m >= p.M) return;
  const float* at = tp.part + (long long)m * tp.ldp + col;
  const long long step = (long long)p.M * tp.ldp;
  f32x4 sum = *reinterpret_cast<const f32x4*>(at);
#pragma unroll 4
  for (int i = 1; i < tp.splits; ++i) sum += *reinterpret_cast<const f32x4*>(at + i * step);
  float b[4], v[4] = {sum[0], sum[1], sum[2], sum[3]};
  load_bias(p, col, b);
  with_act(p.act, [&](auto act) { finish<act, 4>(p, m, col, v, b); });
}

// Which kernel takes more than 16 rows, and in how many splits: by what both take, in us, as
// measured (M x K x N, few / tiles: 20 x 2048 x 16384 14.0 / 8.8, 64 x 4096 x 4096 10.8 / 15.7,
// 64 x 8192 x 8192 35.7 / 21.8, 128 x 1024 x 4096 9.9 / 13.6, 128 x 2048 x 16384 47.8 / 22.5,
// 128 x 8192 x 8192 67 / 31): the few rows' kernel 1.03 for each 1024 of K of 256 tiles of
// 16 x 32, tiles 0.7, 1.4 or 2.0 for each 256 of K of as many as there are CUs, their join
// 2.5 and the time of its bytes at 4 TB/s. With a short K both take their starts and ends
// instead, 2 for each 256 of the few rows' tiles and 4 to 12 for a round of tiles; 0.5 for
// the former tells them apart (17 x 256 x 4096 3.7 / 4.4, 32 x 256 x 16384 9.9 / 4.6, 64 x 256
// x 16384 18.4 / 7.3, 128 x 256 x 4096 9.8 / 11.8, 256 x 256 x 4096 18.2 / 11.9, 1024 x 32 x 1024
// 19.3 / 12.1, 1024 x 256 x 16384 264 / 44).
struct TilePlan {
  int bm, bn, splits;  // bm 0: the few rows' kernel
};

TilePlan tile_plan(int M, int N, int K) {
  TilePlan best{0, 0, 1};
  if (M <= 16) return best;
  const int bm = M <= 32 ? 32 : M <= 64 ? 64 : 128, bn = bm == 32 ? 64 : 128;
  const double step = bm == 32 ? 0.7 : bm == 64 ? 1.4 : 2.0;
  auto over = [](long long a, long long b) { return (a + b - 1) / b; };
  const long long few = over(M, 16) * over(N, 32), tiles = over(M, bm) * over(N, bn), steps = over(K, 256);
  double least = 2.5 + (double)over(few, 256) * (K < 500 ? 0.5 : K / 1024.0 * 1.03);
  for (int s = 1; s == 1 || (s <= 8 && 2 * s <= steps && tiles * s <= 256); ++s) {
    const double t = 3.0 + (double)over(tiles * s, 256) * (double)over(steps, s) * step +
                     (s > 1 ? 2.5 + s * 8e-6 * M * N / 4.0 : 0.0);
    if (t < least) {
      least = t;
      best = TilePlan{bm, bn, s};
    }
  }
  return best;
}

template <int MT, int NT, int WM, int WN, int KC, int DX, int DC, bool BYTES>
hipError_t launch_tile(const TileParams& tp, hipStream_t st) {
  typedef TileStage<MT, NT, WM, WN, KC, BYTES> St;
  constexpr int kLds = DX * St::kBytesX + DC * St::kBytesC;
  static_assert(kLds <= 160 * 1024 && DX >= 2 && DC >= 2 && (DX - 2) * St::kLoadsX < 64 && (DC - 2) * St::kLoadsC < 64, "the rings fit");
  static_assert(WM * WN * MT * NT * 1024 <= kLds, "the sums fit");
  const long long tiles = (long long)((tp.p.M + St::BM - 1) / St::BM) * ((tp.p.N + St::BN - 1) / St::BN);
  hipLaunchKernelGGL((fp4_tile_kernel<MT, NT, WM, WN, KC, DX, DC, BYTES>), dim3((unsigned)(tiles * tp.splits)),
                     dim3(128 * WM * WN), kLds, st, tp);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !tp.part) return e;
  const long long n = (long long)tp.p.M * (tp.ldp / 4);
  hipLaunchKernelGGL(fp4_join_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, tp);
  return hipGetLastError();
}

template <int MT, int NT, int WM, int WN, int KC, int DX, int DC>
hipError_t run_tile(const TileParams& tp, hipStream_t st) {
  return tp.p.K % 128 == 0 ? launch_tile<MT, NT, WM, WN, KC, DX, DC, false>(tp, st)
                           : launch_tile<MT, NT, WM, WN, KC, DX, 3, true>(tp, st);
}

}  // namespace

size_t linear_fp4_workspace_bytes(int M, int N, int K) {
  const TilePlan t = tile_plan(M, N, K);
  return t.splits == 1 ? 0 : (size_t)t.splits * M * ((N + 3) / 4 * 4) * 4;
}

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
  const TilePlan t = tile_plan(p.M, p.N, p.K);
  if (t.bm > 0) {
    TileParams tp{p, t.splits, t.splits > 1 ? static_cast<float*>(a.ws) : nullptr, (p.N + 3) / 4 * 4};
    if (t.bm == 32) return run_tile<2, 1, 1, 4, 256, 3, 3>(tp, st);
    if (t.bm == 64) return run_tile<4, 2, 1, 4, 128, 3, 3>(tp, st);
    return run_tile<4, 4, 2, 2, 128, 3, 3>(tp, st);
  }
  // Eight waves share a long K, four a short one (M x K x N; us, eight / four): 1 x 1024 x
  // 1024 2.9 / 2.6, 1 x 2048 x 16384 6.5 / 5.9, 1 x 8192 x 8192 9.4 / 10.0,
  // 1 x 16384 x 4096 8.9 / 11.5; 3 x 16384 x 4096 9.7 / 10.7.
  if (p.M == 1) return p.K < 4096 ? run_few<1, 1, 4, 2>(p, st) : run_few<1, 1, 8, 2>(p, st);
  if (p.M <= 4) return p.K < 4096 ? run_few<4, 1, 4, 3>(p, st) : run_few<4, 1, 8, 2>(p, st);
  // 16 rows of w a workgroup while that is no more than one a CU, 32 beyond, which load x half
  // as often (us, 16 / 32): 16 x 16384 x 4096 15.7 / 20.8, 20 x 1024 x 4096 5.0 / 3.5, 16 x 8192 x
  // 8192 16.5 / 12.6.
  const long long tiles = (long long)((p.M + 15) / 16) * ((p.N + 15) / 16);
  return tiles <= 256 ? run_few<16, 1, 4, 2>(p, st) : run_few<16, 2, 4, 2>(p, st);
}

}  // namespace gkd
