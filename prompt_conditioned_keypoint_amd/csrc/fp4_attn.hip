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

// Read through the scalar cache: the compiler does not prove that no store changes it.
typedef const __attribute__((address_space(4))) int32_t const_int;

__device__ __forceinline__ bf16x8 frag(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  const bf16x2 h = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
  return __builtin_bit_cast(uint32_t, h);
}

// score * scale, rounded, less m: 0 for the score that m is the rounded product of,
// however far out.
__device__ __forceinline__ float far_exponent(float score, float scale, float m) {
#pragma clang fp contract(off)
  const float t = score * scale;
  return t - m;
}

// A step's codes of a lane: of keys fr and 16 + fr the D/4 elements from g D/4, with
// their group's scale byte; of the values the D/16 elements from fr D/16 of eight
// keys, with the scale bytes of four neighbouring keys a piece.
template <int D>
struct Codes {
  typedef uint32_t piece __attribute__((ext_vector_type(D / 32)));
  piece k[2], vs[2];
  uint32_t ks[2], v[8];
};

// What a workgroup works on: R tiles of rows from row0, the last one rl, and the steps
// [s0, s1) of a sequence's keys.
struct Work {
  int b, hk, bh, part, row0, rl;
  int len, tq;  // tokens, queries
  int all;      // keys that every row sees
  int s0, s1;
};

// Few rows: a step's codes are on their way during the whole step before it, in registers
// of their own. More tiles leave no room for those: keys are read again as soon as they
// are multiplied, and values likewise, and most rows keep their queries in LDS.
template <int D, int R, int NW>
__device__ __forceinline__ void attend(const CaParams& p, const Work& w, float* lds) {
  constexpr int KT = D / 32, DT = D / 16;  // products of a score, tiles of the output
  constexpr int LD = D + 4;
  constexpr bool kAhead = R * D <= 128, kQueriesInLds = R * D > 256;
  typedef typename Codes<D>::piece piece;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 15, g = lane >> 4;
  const float scale = p.scale;

  bf16x8 qf[kQueriesInLds ? 1 : R][KT];
  u32x4* ql = reinterpret_cast<u32x4*>(lds);  // [R][KT][lane]
  int lim[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = min(w.row0 + 16 * r + fr, w.rl), t = i / p.G, h = w.hk * p.G + i - t * p.G;
    const uint16_t* q = static_cast<const uint16_t*>(p.q.p) + w.b * p.q.b + t * p.q.t + h * p.q.h + g * (D / 4);
    if constexpr (kQueriesInLds) {
      for (int k = wave; k < KT; k += NW) ql[(r * KT + k) * 64 + lane] = *reinterpret_cast<const u32x4*>(q + 8 * k);
    } else {
#pragma unroll
      for (int k = 0; k < KT; ++k) qf[r][k] = frag(*reinterpret_cast<const u32x4*>(q + 8 * k));
    }
    lim[r] = p.causal ? w.len - w.tq + t + 1 : w.len;
  }
  if constexpr (kQueriesInLds) __syncthreads();
  f32x4 o[R][DT], l[R];
  float m[R];  // reference points
#pragma unroll
  for (int r = 0; r < R; ++r) {
    m[r] = kFar;
    l[r] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < DT; ++j) o[r][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  bool far = false;  // some reference point is 2^24 or more out

  int s = w.s0 + wave;
  int col = 0, row = s * 32;  // the next step's page column and row in the page
  if (row >= p.c.page) {
    col = row / p.c.page;
    row -= col * p.c.page;
  }
  const_int* table = (const_int*)(uintptr_t)(p.c.table + (long long)w.b * p.c.L);
  const long long head_rows = (long long)p.c.Hk * p.c.page;
  const uint8_t* kcodes = p.c.codes + w.hk * (long long)p.c.page * (D / 2) + fr * (D / 2) + g * (D / 8);
  const uint8_t* kscales = p.c.scales + w.hk * (long long)p.c.page * (D / 32) + fr * (D / 32) + (D == 128 ? g : g / 2);
  const uint8_t* vcodes = p.c.codes + (w.hk * (long long)p.c.page + head_rows) * (D / 2) + g * (2 * D) + fr * (D / 32);
  const uint8_t* vscales = p.c.scales + (w.hk * (long long)p.c.page + head_rows) * (D / 32) + g * (D / 8);
  int page = s < w.s1 ? table[col] : -1;

  // A step's first row among a head's rows of the cache, and whether it has a page
  // (else page 0 is read, and nothing of it counts). move_on: to step `then` if there
  // is one, else the same step is read again: loads without a branch around them stay
  // in flight.
  struct Place {
    long long at;
    bool there;
  };
  auto place = [&]() -> Place {
    const bool there = page >= 0 && page < p.c.pages;
    return Place{(long long)(there ? page : 0) * 2 * head_rows + row, there};
  };
  auto move_on = [&](int then) {
    if (then < w.s1) {
      row += 32 * NW;
      while (row >= p.c.page) {
        row -= p.c.page;
        ++col;
      }
      page = table[col];
    }
  };
  auto read_keys = [&](Codes<D>& c, long long at) {
    const uint8_t* kc = kcodes + at * (D / 2);
    const uint8_t* ks = kscales + at * (D / 32);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      c.k[i] = *reinterpret_cast<const piece*>(kc + i * 8 * D);
      c.ks[i] = ks[i * (D / 2)];
    }
  };
  auto read_values = [&](Codes<D>& c, long long at) {
    const uint8_t* vc = vcodes + at * (D / 2);
    const uint8_t* vs = vscales + at * (D / 32);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      c.vs[i] = *reinterpret_cast<const piece*>(vs + i * (D / 2));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint8_t* a = vc + i * 8 * D + e * (D / 2);
        c.v[4 * i + e] = D == 128 ? *reinterpret_cast<const uint32_t*>(a) : *reinterpret_cast<const uint16_t*>(a);
      }
    }
  };

  // S^T of a step
  auto scores = [&](const Codes<D>& c, f32x4 (&st)[R][2]) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int r = 0; r < R; ++r) st[r][i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      const bf16x8 k0 = frag(fp4_values(c.k[0][k], fp4_unit(c.ks[0])));
      const bf16x8 k1 = frag(fp4_values(c.k[1][k], fp4_unit(c.ks[1])));
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const bf16x8 q = kQueriesInLds ? frag(ql[(r * KT + k) * 64 + lane]) : qf[kQueriesInLds ? 0 : r][k];
        st[r][0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k0, q, st[r][0], 0, 0, 0);
        st[r][1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k1, q, st[r][1], 0, 0, 0);
      }
    }
  };
  // Keys that a row does not see
  auto hide = [&](f32x4 (&st)[R][2], int s, bool there) {
    const int key = (there ? 32 * s : 0x7fffff00) + 4 * g;  // of place 0; place 4 i + e is 16 i + e further on
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (key + 16 * (i / 4) + i % 4 >= lim[r]) st[r][i / 4][i % 4] = -INFINITY;
  };
  // Rows past the last token hold anything: no NaN of theirs may meet a 0
  auto clear = [&](Codes<D>& c, int s, bool there) {
    const int key = (there ? 32 * s : 0x7fffff00) + 4 * g;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (key + 16 * (i / 4) + i % 4 >= w.len) {
        c.v[i] = 0;
        if constexpr (D == 128) c.vs[i / 4][i % 4] = 0;
        else c.vs[i / 4][i % 4 / 2] &= i % 2 ? 0x0000ffffu : 0xffff0000u;
      }
  };
  // The exponents of a step against the reference points as they are, and the largest
  // of them (compared as integers: that orders positive ones, which is what counts).
  auto exponents = [&](const f32x4 (&st)[R][2], f32x4 (&x)[R][2]) -> int {
    int top = 0;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[r][i / 4][i % 4] = fmaf(st[r][i / 4][i % 4], scale, -m[r]);
        top = max(top, __float_as_int(x[r][i / 4][i % 4]));
      }
    return top;
  };
  // Where one passes the slack, its row's reference point moves to the row's largest
  // score of the step.
  auto move = [&](const f32x4 (&st)[R][2], f32x4 (&x)[R][2]) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float top = st[r][0][0];
#pragma unroll
      for (int i = 1; i < 8; ++i) top = fmaxf(top, st[r][i / 4][i % 4]);
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32)) * scale;
      const float to = top > m[r] + kSlack ? top : m[r];
      const float f = __builtin_amdgcn_exp2f(m[r] - to);
      m[r] = to;
      far = far || __any(fabsf(to) >= 16777216.f && to != kFar);
      l[r] *= f;
#pragma unroll
      for (int j = 0; j < DT; ++j) o[r][j] *= f;
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        x[r][i / 4][i % 4] = far ? far_exponent(st[r][i / 4][i % 4], scale, m[r])
                                 : fmaf(st[r][i / 4][i % 4], scale, -m[r]);
  };
  // P^T of a step, the row sums with it
  auto softmax = [&](const f32x4 (&st)[R][2], u32x4 (&pf)[R]) {
    f32x4 x[R][2];
    const int top = exponents(st, x);
    if (far || __any(top > __float_as_int(kSlack))) move(st, x);
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        pf[r][i] = bf16_pair(__builtin_amdgcn_exp2f(x[r][i / 2][i % 2 * 2]),
                             __builtin_amdgcn_exp2f(x[r][i / 2][i % 2 * 2 + 1]));
      const u32x4 ones = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
      l[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(ones), frag(pf[r]), l[r], 0, 0, 0);
    }
  };
  // O^T += V^T P^T: elements fr D/16 + (2 h, 2 h + 1) of the eight keys, turned into two
  // operands. The lane's scale byte of a key is turned to the exponent's place: the
  // conversions look at nothing else.
  auto output = [&](const Codes<D>& c, const u32x4 (&pf)[R]) {
    float unit[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t word = D == 128 ? c.vs[i / 4][i % 4] : c.vs[i / 4][i % 4 / 2];
      const int from = D == 128 ? 8 * (fr / 4) : 16 * (i % 2) + 8 * (fr / 8);
      unit[i] = __uint_as_float(__builtin_amdgcn_alignbit(word, word, (uint32_t)(from + 9) & 31u));
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
  auto edges = [&](Codes<D>& c, f32x4 (&st)[R][2], int s, bool there) {
    const int end = there ? 32 * s + 32 : 0x7fffffff;
    if (end > w.all) {
      hide(st, s, there);
      if (end > w.len) clear(c, s, there);
    }
  };

  if (s < w.s1) {
    f32x4 st[R][2];
    u32x4 pf[R];
    if constexpr (kAhead) {
      Codes<D> c0, c1;
      Place a0 = place(), a1 = a0;
      auto step = [&](Codes<D>& c, Place& a, Codes<D>& cn, Place& an) {
        an = place();
        read_keys(cn, an.at);
        read_values(cn, an.at);
        move_on(s + 2 * NW);
        scores(c, st);
        edges(c, st, s, a.there);
        softmax(st, pf);
        output(c, pf);
        s += NW;
      };
      read_keys(c0, a0.at);
      read_values(c0, a0.at);
      move_on(s + NW);
      for (;;) {
        step(c0, a0, c1, a1);
        if (s >= w.s1) break;
        step(c1, a1, c0, a0);
        if (s >= w.s1) break;
      }
    } else {
      Codes<D> c;
      Place a = place();
      read_keys(c, a.at);
      read_values(c, a.at);
      move_on(s + NW);
      for (; s < w.s1; s += NW) {
        const Place n = place();
        scores(c, st);
        read_keys(c, n.at);
        move_on(s + 2 * NW);
        edges(c, st, s, a.there);
        softmax(st, pf);
        output(c, pf);
        read_values(c, n.at);
        a = n;
      }
    }
  }
  if constexpr (kQueriesInLds) __syncthreads();

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
    const int i = w.row0 + 16 * r + jr;
    if (i > w.rl) continue;
    float top = kFar, sum = 0.f, y[PER];
#pragma unroll
    for (int v = 0; v < NW; ++v) top = fmaxf(top, stat[(v * 16 + jr) * 2]);
#pragma unroll
    for (int d = 0; d < PER; ++d) y[d] = 0.f;
#pragma unroll
    for (int v = 0; v < NW; ++v) {
      const float f = __builtin_amdgcn_exp2f(stat[(v * 16 + jr) * 2] - top);
      sum = fmaf(f, stat[(v * 16 + jr) * 2 + 1], sum);
#pragma unroll
      for (int d = 0; d < PER; ++d) y[d] = fmaf(f, lds[(v * 16 + jr) * LD + jd + d], y[d]);
    }
    if (p.parts == 1) {
      const int t = i / p.G, h = w.hk * p.G + i - t * p.G;
      uint16_t* out = static_cast<uint16_t*>(p.out.p) + w.b * p.out.b + t * p.out.t + h * p.out.h + jd;
      const float f = sum == 0.f ? 0.f : 1.f / sum;  // no key: O is 0
#pragma unroll
      for (int d = 0; d < PER; d += 2) reinterpret_cast<uint32_t*>(out)[d / 2] = bf16_pair(y[d] * f, y[d + 1] * f);
    } else {
      const long long at_row = (long long)w.part * rows + (long long)w.bh * p.Tq * p.G + i;
#pragma unroll
      for (int d = 0; d < PER; ++d) p.po[at_row * D + jd + d] = y[d];
      if (jd == 0) {
        p.ml[at_row * 2] = top;
        p.ml[at_row * 2 + 1] = sum;
      }
    }
  }
}

// A workgroup of R tiles of rows; where the last ones hold no row in use, the work of
// fewer tiles.
template <int D, int R, int NW>
__global__ __launch_bounds__(64 * NW, 2) void cache_attn_kernel(CaParams p) {
  extern __shared__ __attribute__((aligned(16))) float lds[];  // [NW][16][D + 4], [NW][16][2]
  const ItemCoord at = xcd_item(blockIdx.x, p.tiles);
  if (at.crop >= p.groups) return;
  Work w;
  w.part = at.crop % p.parts;
  w.bh = at.crop / p.parts;
  w.b = w.bh / p.c.Hk;
  w.hk = w.bh - w.b * p.c.Hk;
  const int cap = p.c.L * p.c.page;
  w.len = p.length ? min(max(p.length[w.b], 0), cap) : cap;
  w.tq = p.q_len ? min(max(p.q_len[w.b], 0), p.Tq) : p.Tq;
  const int live = w.tq * p.G;
  w.row0 = at.item * 16 * R;
  if (w.row0 >= live) return;
  w.rl = min(w.row0 + 16 * R, live) - 1;
  const int last = p.causal ? max(w.len - w.tq + w.rl / p.G + 1, 0) : w.len;  // keys that the last row sees
  w.all = p.causal ? max(w.len - w.tq + w.row0 / p.G + 1, 0) : w.len;
  const int steps = (last + 31) / 32, per = (steps + p.parts - 1) / p.parts;
  w.s0 = w.part * per;
  w.s1 = min(steps, w.s0 + per);
  const int tiles = (w.rl - w.row0) / 16 + 1;
  if constexpr (R >= 4) {
    if (tiles == 3) return attend<D, 3, NW>(p, w, lds);
  }
  if constexpr (R >= 3) {
    if (tiles == 2) return attend<D, 2, NW>(p, w, lds);
  }
  if constexpr (R >= 2) {
    if (tiles == 1) return attend<D, 1, NW>(p, w, lds);
  }
  attend<D, R, NW>(p, w, lds);
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
  x.R = rows <= 16 ? 1 : rows <= 32 ? 2 : D == 128 || rows <= 48 ? 3 : 4;
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
  if constexpr (D == 64) {
    if (R == 4) return run<D, 4>(p, st);
  }
  return R == 1 ? run<D, 1>(p, st) : R == 2 ? run<D, 2>(p, st) : run<D, 3>(p, st);
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
  // (a step without a page reads the first one; where there is none, no token has a page)
  if (p.c.pages == 0) p.c.L = 0;
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
