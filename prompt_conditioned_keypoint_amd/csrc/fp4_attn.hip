// fp4_attn.hip - attention over a cache of four-bit keys and values in pages
// (gkd_cache_attention).
//
// A row is one query of one query head; the rows of a sequence's key head are
// numbered i = t G + g (G = Hq / Hk query heads share the key head). A workgroup
// takes 16 R of them and a range of keys, its waves every NW-th step of 32 keys.
// A wave reads a step's codes straight into registers, where the conversion
// instructions make bfloat16 of them (0.5 instructions a value, exact), and takes
//   S^T = K Q^T    keys as rows, queries as columns,
//   O^T = V^T P^T  head elements as rows, queries as columns,
// so that the probabilities leave the first product in the very places that the
// second one wants them: a lane's eight scores of a step are its eight k of the
// operand P^T, if V's keys are taken in that order (place (g, i) is key
// 16 (i / 4) + 4 g + i % 4). Nothing passes through LDS before the waves join.
//
// The softmax runs online, in base 2: a row keeps its reference point m, the sum l
// of 2^(s - m) and the output O scaled alike, and ranges of keys are joined by
//   m = max_i m_i,  l = sum_i l_i 2^(m_i - m),  O = sum_i O_i 2^(m_i - m).
// The reference point moves only where a score passes it by 8, row by row, which
// spares the exchange between lanes and the rescaling at nearly every step.
// Probabilities are rounded to bfloat16 (2^-8 of each) for the product with V, whose
// instruction takes both sides in that type; l sums the rounded ones, in the same
// product with a column of ones.
#include "fp4_device.hpp"
#include "fp4_launch.hpp"

namespace gkd {
namespace {

struct CaParams {
  Heads q, out;
  Pages c;
  const int32_t *length, *q_len;
  int B, Tq, G;
  float scale;      // times log2(e)
  int causal;
  int tiles, parts, groups;  // tiles of rows, parts of the keys; B Hk parts
  float* po;        // [parts][B Hk Tq G][D]
  float* ml;        // [parts][B Hk Tq G][2]
};

constexpr float kFar = -3e38f;  // a reference point before any key: below every score
constexpr float kSlack = 8.f;

__device__ __forceinline__ bf16x8 frag(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  const bf16x2 h = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
  return __builtin_bit_cast(uint32_t, h);
}

template <int D>
struct StepCodes;
// A step's codes of a lane: of keys fr and 16 + fr the D/4 elements from g D/4, with
// their group's scale byte; of the values the D/16 elements from fr D/16 of eight
// keys, with the scale bytes of four neighbouring keys a piece.
template <>
struct StepCodes<128> {
  u32x4 k[2];
  uint32_t ks[2], v[8];
  u32x4 vs[2];
};
template <>
struct StepCodes<64> {
  u32x2 k[2];
  uint32_t ks[2], v[8];
  u32x2 vs[2];
};

template <int D, int R, int NW>
__global__ __launch_bounds__(64 * NW) void cache_attn_kernel(CaParams p) {
  constexpr int KT = D / 32, DT = D / 16;  // products of a score, tiles of the output
  constexpr int LD = D + 4;
  extern __shared__ __attribute__((aligned(16))) float lds[];  // [NW][16][LD], [NW][16][2]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 15, g = lane >> 4;
  const ItemCoord at = xcd_item(blockIdx.x, p.tiles);
  if (at.crop >= p.groups) return;
  const int part = at.crop % p.parts, bh = at.crop / p.parts;
  const int b = bh / p.c.Hk, hk = bh - b * p.c.Hk;
  const int cap = p.c.L * p.c.page;
  const int len = p.length ? min(max(p.length[b], 0), cap) : cap;
  const int tq = p.q_len ? min(max(p.q_len[b], 0), p.Tq) : p.Tq;
  const int live = tq * p.G, row0 = at.item * 16 * R;
  if (row0 >= live) return;
  const int rl = min(row0 + 16 * R, live) - 1;
  // keys that the last row sees, and those that every row sees
  const int last = p.causal ? max(len - tq + rl / p.G + 1, 0) : len;
  const int all = p.causal ? max(len - tq + row0 / p.G + 1, 0) : len;
  const int steps = (last + 31) / 32, per = (steps + p.parts - 1) / p.parts;
  const int s0 = part * per, s1 = min(steps, s0 + per);

  bf16x8 qf[R][KT];
  int lim[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = min(row0 + 16 * r + fr, rl), t = i / p.G, h = hk * p.G + i - t * p.G;
    const uint16_t* q = static_cast<const uint16_t*>(p.q.p) + b * p.q.b + t * p.q.t + h * p.q.h + g * (D / 4);
#pragma unroll
    for (int k = 0; k < KT; ++k) qf[r][k] = frag(*reinterpret_cast<const u32x4*>(q + 8 * k));
    lim[r] = p.causal ? len - tq + t + 1 : len;
  }
  f32x4 o[R][DT], l[R];
  float m[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    m[r] = kFar;
    l[r] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < DT; ++j) o[r][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  // The step's place: page column and row in it.
  int col = 0, row = (s0 + wave) * 32;
  if (row >= p.c.page) {
    col = row / p.c.page;
    row -= col * p.c.page;
  }
  const int32_t* table = p.c.table + (long long)b * p.c.L;
  const long long head_rows = (long long)p.c.Hk * p.c.page;
  const long long first_row = (long long)hk * p.c.page;
  int page = s0 + wave < s1 ? table[col] : -1;

  // Reads step s (at page, row) and moves on to step s + NW. False: it has no page.
  StepCodes<D> buf[2];
  auto read = [&](StepCodes<D>& c, int s) -> bool {
    const bool there = page >= 0 && page < p.c.pages;
    if (there) {
      const long long kr = (long long)page * 2 * head_rows + first_row + row, vr = kr + head_rows;
      const uint8_t* kc = p.c.codes + kr * (D / 2) + fr * (D / 2) + g * (D / 8);
      const uint8_t* ks = p.c.scales + kr * (D / 32) + fr * (D / 32) + (D == 128 ? g : g / 2);
      const uint8_t* vc = p.c.codes + vr * (D / 2) + g * (2 * D) + fr * (D / 32);
      const uint8_t* vs = p.c.scales + vr * (D / 32) + g * (D / 8);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        c.k[i] = *reinterpret_cast<const decltype(c.k[0] + c.k[0])*>(kc + i * 8 * D);
        c.ks[i] = ks[i * (D / 2)];
        c.vs[i] = *reinterpret_cast<const decltype(c.vs[0] + c.vs[0])*>(vs + i * (D / 2));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint8_t* a = vc + i * 8 * D + e * (D / 2);
          c.v[4 * i + e] = D == 128 ? *reinterpret_cast<const uint32_t*>(a) : *reinterpret_cast<const uint16_t*>(a);
        }
      }
    }
    row += 32 * NW;
    while (row >= p.c.page) {
      row -= p.c.page;
      ++col;
    }
    page = s + NW < s1 ? table[col] : -1;
    return there;
  };

  auto take = [&](StepCodes<D>& c, int s) {
    f32x4 st[R][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int r = 0; r < R; ++r) st[r][i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < KT; ++k) {
        const bf16x8 kf = frag(fp4_values(c.k[i][k], fp4_unit(c.ks[i])));
#pragma unroll
        for (int r = 0; r < R; ++r)
          st[r][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[r][k], st[r][i], 0, 0, 0);
      }
    }
    const int key = 32 * s + 4 * g;  // of place 0; place 4 i + e is 16 i + e further on
    if (32 * s + 32 > len) {
      // rows past the last token hold anything: no NaN of theirs may meet a 0
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (key + 16 * (i / 4) + i % 4 >= len) {
          c.v[i] = 0;
          if constexpr (D == 128) c.vs[i / 4][i % 4] = 0;
          else c.vs[i / 4][i % 4 / 2] &= i % 2 ? 0x0000ffffu : 0xffff0000u;
        }
    }
    u32x4 pf[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = st[r][i / 4][i % 4] * p.scale;
      if (32 * s + 32 > all) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (key + 16 * (i / 4) + i % 4 >= lim[r]) x[i] = -INFINITY;
      }
      float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
      if (__any(top > m[r] + kSlack)) {
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float to = top > m[r] + kSlack ? top : m[r];
        const float f = __builtin_amdgcn_exp2f(m[r] - to);
        m[r] = to;
        l[r] *= f;
#pragma unroll
        for (int j = 0; j < DT; ++j) o[r][j] *= f;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        pf[r][i] = bf16_pair(__builtin_amdgcn_exp2f(x[2 * i] - m[r]), __builtin_amdgcn_exp2f(x[2 * i + 1] - m[r]));
      const u32x4 ones = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
      l[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(ones), frag(pf[r]), l[r], 0, 0, 0);
    }
    // elements fr D/16 + (2 h, 2 h + 1) of the eight keys, turned into two operands
    float unit[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (D == 128) unit[i] = fp4_unit((c.vs[i / 4][i % 4] >> (8 * (fr / 4))) & 255u);
      else unit[i] = fp4_unit((c.vs[i / 4][i % 4 / 2] >> (16 * (i % 2) + 8 * (fr / 8))) & 255u);
    }
#pragma unroll
    for (int h = 0; h < DT / 2; ++h) {
      uint32_t a[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        a[i] = h == 0 ? fp4_pair<0>(c.v[i], unit[i]) : h == 1 ? fp4_pair<1>(c.v[i], unit[i])
             : h == 2 ? fp4_pair<2>(c.v[i], unit[i]) : fp4_pair<3>(c.v[i], unit[i]);
      u32x4 lo, hi;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        lo[i] = __builtin_amdgcn_perm(a[2 * i + 1], a[2 * i], 0x05040100u);
        hi[i] = __builtin_amdgcn_perm(a[2 * i + 1], a[2 * i], 0x07060302u);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        o[r][2 * h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(lo), frag(pf[r]), o[r][2 * h], 0, 0, 0);
        o[r][2 * h + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(hi), frag(pf[r]), o[r][2 * h + 1], 0, 0, 0);
      }
    }
  };

  bool there[2] = {false, false};
  int s = s0 + wave;
  if (s < s1) there[0] = read(buf[0], s);
  for (; s < s1; s += 2 * NW) {
    if (s + NW < s1) there[1] = read(buf[1], s + NW);
    if (there[0]) take(buf[0], s);
    if (s + NW < s1) {
      if (s + 2 * NW < s1) there[0] = read(buf[0], s + 2 * NW);
      if (there[1]) take(buf[1], s + NW);
    }
  }

  // The waves join, 16 rows at a time.
  constexpr int TPR = 64 * NW / 16, PER = D / TPR;  // threads of a row, elements of a thread
  float* stat = lds + NW * 16 * LD;
  const int jr = threadIdx.x / TPR, jd = threadIdx.x % TPR * PER;
  const long long rows = (long long)p.B * p.c.Hk * p.Tq * p.G;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (r > 0) __syncthreads();
    // element j + e D/16 of the lane's D/4 from g D/4 is o[j][e]
    float* mine = lds + (wave * 16 + fr) * LD + g * (D / 4);
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int j = 0; j < DT; j += 4)
        *reinterpret_cast<f32x4*>(mine + e * DT + j) =
            f32x4{o[r][j][e], o[r][j + 1][e], o[r][j + 2][e], o[r][j + 3][e]};
    if (g == 0) {
      stat[(wave * 16 + fr) * 2] = m[r];
      stat[(wave * 16 + fr) * 2 + 1] = l[r][0];
    }
    __syncthreads();
    const int i = row0 + 16 * r + jr;
    if (i > rl) continue;
    float top = kFar, sum = 0.f, y[PER];
#pragma unroll
    for (int w = 0; w < NW; ++w) top = fmaxf(top, stat[(w * 16 + jr) * 2]);
#pragma unroll
    for (int d = 0; d < PER; ++d) y[d] = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float f = __builtin_amdgcn_exp2f(stat[(w * 16 + jr) * 2] - top);
      sum = fmaf(f, stat[(w * 16 + jr) * 2 + 1], sum);
#pragma unroll
      for (int d = 0; d < PER; ++d) y[d] = fmaf(f, lds[(w * 16 + jr) * LD + jd + d], y[d]);
    }
    if (p.parts == 1) {
      const int t = i / p.G, h = hk * p.G + i - t * p.G;
      uint16_t* out = static_cast<uint16_t*>(p.out.p) + b * p.out.b + t * p.out.t + h * p.out.h + jd;
      const float f = sum == 0.f ? 0.f : 1.f / sum;  // no key: O is 0
#pragma unroll
      for (int d = 0; d < PER; d += 2) reinterpret_cast<uint32_t*>(out)[d / 2] = bf16_pair(y[d] * f, y[d + 1] * f);
    } else {
      const long long at_row = (long long)part * rows + (long long)bh * p.Tq * p.G + i;
#pragma unroll
      for (int d = 0; d < PER; ++d) p.po[at_row * D + jd + d] = y[d];
      if (jd == 0) {
        p.ml[at_row * 2] = top;
        p.ml[at_row * 2 + 1] = sum;
      }
    }
  }
}

// Joins the parts of a row, a wave a row.
template <int D>
__global__ __launch_bounds__(256) void cache_join_kernel(CaParams p) {
  constexpr int PER = D / 64;
  const int lane = threadIdx.x & 63;
  const int per = p.Tq * p.G;
  const long long rows = (long long)p.B * p.c.Hk * per;
  const long long at = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (at >= rows) return;
  const int bh = (int)(at / per), i = (int)(at - (long long)bh * per);
  const int b = bh / p.c.Hk, hk = bh - b * p.c.Hk, t = i / p.G, h = hk * p.G + i - t * p.G;
  if (p.q_len && t >= p.q_len[b]) return;
  float m = kFar, l = 0.f;
  if (lane < p.parts) {
    m = p.ml[(lane * rows + at) * 2];
    l = p.ml[(lane * rows + at) * 2 + 1];
  }
  float top = m;
#pragma unroll
  for (int x = 32; x >= 1; x >>= 1) top = fmaxf(top, __shfl_xor(top, x));
  const float f = __builtin_amdgcn_exp2f(m - top);
  const float sum = wave_sum(f * l);
  float y[PER];
#pragma unroll
  for (int d = 0; d < PER; ++d) y[d] = 0.f;
  for (int x = 0; x < p.parts; ++x) {
    const float fx = __shfl(f, x);
#pragma unroll
    for (int d = 0; d < PER; ++d) y[d] = fmaf(fx, p.po[(x * rows + at) * D + lane * PER + d], y[d]);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  uint16_t* out = static_cast<uint16_t*>(p.out.p) + b * p.out.b + t * p.out.t + h * p.out.h + lane * PER;
  if constexpr (PER == 2) *reinterpret_cast<uint32_t*>(out) = bf16_pair(y[0] * inv, y[1] * inv);
  else *out = f32_to_bf16_bits(y[0] * inv);
}

struct Plan {
  int R, tiles, parts;
};

constexpr int kWaves = 4;
constexpr int kMaxParts = 64;  // a lane of the join each

Plan plan_for(int B, int Tq, int Hq, int Hk, int D, int page, int L) {
  Plan x;
  const int rows = Tq * (Hq / Hk);
  x.R = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
  x.tiles = (rows + 16 * x.R - 1) / (16 * x.R);
  const long long items = (long long)B * Hk * x.tiles, steps = ((long long)L * page + 31) / 32;
  long long parts = (512 + items - 1) / items;
  const long long most = steps / (2 * kWaves);
  if (parts > most) parts = most;
  if (parts > kMaxParts) parts = kMaxParts;
  x.parts = parts < 1 ? 1 : (int)parts;
  return x;
}

size_t al256(size_t n) { return (n + 255) & ~(size_t)255; }

template <int D, int R>
hipError_t run(const CaParams& p, hipStream_t st) {
  const long long groups8 = ((long long)p.groups + kXcds - 1) / kXcds * kXcds;
  hipLaunchKernelGGL((cache_attn_kernel<D, R, kWaves>), dim3((unsigned)(groups8 * p.tiles)), dim3(64 * kWaves),
                     kWaves * 16 * (D + 4 + 2) * 4, st, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.parts == 1) return e;
  const long long rows = (long long)p.B * p.c.Hk * p.Tq * p.G;
  hipLaunchKernelGGL(cache_join_kernel<D>, dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, st, p);
  return hipGetLastError();
}

template <int D>
hipError_t run_rows(const CaParams& p, int R, hipStream_t st) {
  return R == 1 ? run<D, 1>(p, st) : R == 2 ? run<D, 2>(p, st) : run<D, 4>(p, st);
}

}  // namespace

size_t cache_attn_workspace_bytes(int B, int Tq, int Hq, int Hk, int D, int page, int L) {
  const Plan x = plan_for(B, Tq, Hq, Hk, D, page, L);
  if (x.parts == 1) return 0;
  const size_t rows = (size_t)B * Tq * Hq;
  return al256(x.parts * rows * D * 4) + al256(x.parts * rows * 8);
}

hipError_t launch_cache_attn(const CacheAttnArgs& a, hipStream_t st) {
  // (the plan goes by the table's size also where the cache has no pages)
  const Plan x = plan_for(a.B, a.Tq, a.Hq, a.c.Hk, a.c.D, a.c.page, a.c.L);
  CaParams p{};
  p.q = a.q;
  p.out = a.out;
  p.c = a.c;
  p.length = a.length;
  p.q_len = a.q_len;
  p.B = a.B;
  p.Tq = a.Tq;
  p.G = a.Hq / a.c.Hk;
  p.scale = a.scale * 1.4426950408889634f;
  p.causal = a.causal;
  p.tiles = x.tiles;
  p.parts = x.parts;
  p.groups = a.B * a.c.Hk * x.parts;
  const size_t rows = (size_t)a.B * a.Tq * a.Hq;
  p.po = static_cast<float*>(a.ws);
  if (x.parts > 1) p.ml = p.po + al256(x.parts * rows * a.c.D * 4) / 4;
  return a.c.D == 128 ? run_rows<128>(p, x.R, st) : run_rows<64>(p, x.R, st);
}

}  // namespace gkd
