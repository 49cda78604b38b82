// fp4_attn.hip - attention over a cache of four-bit keys and values in pages
// (gkd_cache_attention).
//
// A row is one query of one query head; the rows of a sequence's key head are
// numbered i = t G + g (G = Hq / Hk query heads share the key head). A workgroup
// takes 16 R of them and a range of keys, its waves every NW-th step of 32 keys.
// Each wave loads its steps straight to a ring of its own in LDS, one ahead of the
// one at work, so that no wave waits for another before they join. The conversion
// instructions make bfloat16 of the codes (0.5 instructions a value, exact), and
//   S^T = K Q^T    has keys as rows, queries as columns,
//   O^T = V^T P^T  head elements as rows, queries as columns,
// so that the probabilities leave the first product in the very places that the
// second one wants them: a lane's eight scores of a step are its eight k of the
// operand P^T, if V's keys are taken in that order (place (g, i) is key
// 16 (i / 4) + 4 g + i % 4). They never leave the registers.
//
// The softmax runs online, in base 2: a row keeps its reference point m, the sum l
// of 2^(s - m) and the output O scaled alike, and ranges of keys are joined by
//   m = max_i m_i,  l = sum_i l_i 2^(m_i - m),  O = sum_i O_i 2^(m_i - m).
// The reference point moves only where a score passes it by 8, row by row, which
// spares the exchange between lanes and the rescaling at nearly every step.
// Probabilities are rounded to bfloat16 (2^-8 of each) for the product with V, whose
// instruction takes both sides in that type; l sums the rounded ones, in the same
// product with a column of ones. Outputs of thousands of random keys are 0.0023 of their
// size off the exact ones so, 0.0017 of which is their own rounding. A second product
// with what the rounding left would take them to 0.0017, for 158 -> 204 us (4 sequences of
// 128 rows of 32 heads on 8 of 128), 33 -> 41 (37 x 80 rows) and 2 to 5% with few rows.
//
// What bounds it: few rows, memory. 48 sequences of 32 heads on 8 heads of 128 and up to
// 8192 tokens, one new token each: 316 MB in 69 to 76 us, 4.2 to 4.5 TB/s, where a large
// copy on the same card moves 5.0. One sequence of 262144 tokens: 279 MB in 61 to 67 us (the
// less the fewer other inputs pass through the last cache between its calls).
// Many rows, the issue of instructions: a step of 32 rows of 128 elements takes 16 products
// for S, 16 for O and 2 for l, beside 1024 exponents and what turns codes and scores into
// operands, and 16 sequences of 128 rows of 32 heads on 8 take 298 us behind 8192 tokens,
// 0.92 PF (a large product of the library 1.3 to 1.4).
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
  int tiles;        // tiles of 16 R rows that a sequence's key head can have
  int shares;       // workgroups that share the work; 0: each takes a tile with all its keys
  int group;        // sequences of an entry of the running sum of the work
  int32_t* ends;    // [B Hk tiles][2] first and last share of a cut tile; first -1: not cut
  float* po;        // [shares][2][16 R][D] parts of rows
  float* ml;        // [shares][2][16 R][2]
};

constexpr float kFar = -3e38f;  // a reference point before any key: below every score
constexpr float kSlack = 8.f;
constexpr int kStages = 2;      // of a wave's ring

typedef __attribute__((address_space(1))) void glb_void;

// Read through the scalar cache: the compiler does not prove that no store changes it.
typedef const __attribute__((address_space(4))) int32_t const_int;
__device__ __forceinline__ const_int* scalar(const int32_t* p) { return (const_int*)(uintptr_t)p; }

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ long long uniform(long long v) {
  const uint32_t lo = (uint32_t)uniform((int)(uint32_t)v), hi = (uint32_t)uniform((int)(v >> 32));
  return (long long)((unsigned long long)hi << 32 | lo);
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  const bf16x2 h = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
  return __builtin_bit_cast(uint32_t, h);
}

// A reference point 2^24 or more out, where float32 has no halves: its row's exponents are
// rounded products less the rounded product that it is.
__device__ __forceinline__ bool is_far(float m) { return fabsf(m) >= 16777216.f && m != kFar; }

// score * scale, rounded, less m: 0 for the score that m is the rounded product of,
// however far out.
__device__ __forceinline__ float far_exponent(float score, float scale, float m) {
#pragma clang fp contract(off)
  const float t = score * scale;
  return t - m;
}

// A step's place in a wave's ring in LDS: the codes of 32 keys, those of their values,
// and the scale bytes of both. LDS has 64 banks of 4 bytes, a row of codes is D/2 bytes,
// and rows are placed so that no reading below meets itself in a bank:
//   keys     16-byte piece c of row r at piece c ^ turned(r / 4) (D 64: c ^ (r / 8) % 2), for
//            lanes that read the same piece of 16 rows;
//   values   row 4 g + e of 16 at row 4 g + (e ^ g) (D 64: e ^ (g & 2)), for lanes that
//            read all of the rows 4 g + e, g = 0 .. 3.
// Loads go straight to LDS, so it is the lanes' global addresses that are permuted.
template <int D>
struct Stage {
  static constexpr int kCodes = 32 * D / 2, kValues = kCodes, kScales = 2 * kCodes;
  static constexpr int kBytes = 2 * kCodes + 256, kLoads = D == 128 ? 5 : 3;
};

// 0 1 2 3 -> 0 2 3 1. LDS serves lanes 0-3, 12-15 and 20-27 (and the like) of 16-byte reads
// together: rows r / 4 of 0 and 3 with one g, of 1 and 2 with the next, so that
// g ^ (r / 4) would send two lanes to a bank.
__device__ __forceinline__ int turned(int j) { return (j & 1 ^ j >> 1 & 1) << 1 | (j >> 1 & 1); }

// A sequence's work: `tiles` tiles of `sub` times 16 rows of each key head, `steps`
// steps of keys each. A step is taken to cost 3 + sub, its conversions beside the
// products and exponents of its rows, and a tile kStart more, the wait for its queries and
// first keys and its waves' join (without that dozens of tiles of one step each would be
// one share: 48 sequences of one row of 32 heads on 8 of 128, 1 to 8192 tokens, 75 us, with it
// 52; 16 of 128 rows of 32 heads on as many, in shares 436 and 241).
constexpr int kStart = 64;
struct Sequence {
  int len, tq, live, tiles, sub, steps;
  __device__ int weight() const { return 3 + sub; }
  __device__ long long tile_work() const { return steps > 0 ? kStart + (long long)steps * weight() : 0; }
};

template <int R>
__device__ __forceinline__ Sequence sequence(const CaParams& p, int b) {
  Sequence q;
  const int cap = p.c.L * p.c.page;
  q.len = p.length ? min(max(scalar(p.length)[b], 0), cap) : cap;
  q.tq = p.q_len ? min(max(scalar(p.q_len)[b], 0), p.Tq) : p.Tq;
  q.live = q.tq * p.G;
  const int subs = (q.live + 15) / 16;
  q.tiles = (subs + R - 1) / R;
  q.sub = q.tiles > 0 ? (subs + q.tiles - 1) / q.tiles : 1;  // spread evenly
  q.steps = (q.len + 31) / 32;
  return q;
}

// a / b for 0 <= a < 2^53, b > 0, without the long way of 64-bit division.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  long long q = (long long)((double)a / (double)b);
  const long long r = a - q * b;
  if (r < 0) --q;
  if (r >= b) ++q;
  return q;
}

// The work (below 2^51: 2^21 tiles of 2^26 steps) is cut into `n` equal shares; share i
// begins at total i / n.
struct Shares {
  long long each;
  int rest, n;
  __device__ long long begin(int i) const { return each * i + (uint32_t)(rest * i) / (uint32_t)n; }
};

__device__ __forceinline__ Shares shares_of(long long total, int n) {
  Shares x;
  x.each = quotient(total, n);
  x.rest = (int)(total - x.each * n);
  x.n = n;
  return x;
}

// The steps of a tile that begins at `tile` which lie before `at`: a step belongs to the
// share that holds its first unit of work, and kStart lies between the first two steps' first
// units.
__device__ __forceinline__ int steps_before(const Sequence& q, long long tile, long long at) {
  if (at <= tile) return 0;
  if (at - tile >= q.tile_work()) return q.steps;
  const int x = (int)(at - tile) - kStart, w = q.weight();
  return x <= w ? 1 : (int)((uint32_t)(x + w - 1) / (uint32_t)w);
}

// Row i's query: i / G
__device__ __forceinline__ int query_of(const CaParams& p, int i) {
  return (p.G & (p.G - 1)) == 0 ? i >> (31 - __builtin_clz(p.G)) : (int)((uint32_t)i / (uint32_t)p.G);
}

// A share holds at least kStart + 8 units, so more than lie between any two steps' first
// units (a step costs 6 at most): the join counts on that.
__device__ __forceinline__ int share_count(const CaParams& p, long long total) {
  return (int)min((long long)p.shares, max(quotient(total, kStart + 8), 1LL));
}

// What a workgroup works on: rows row0 .. rl of a key head, and the steps [s0, s1) of
// the sequence's keys; `part`: -1 where these are all its keys, else where the partial
// results go.
struct Work {
  int b, hk, row0, rl;
  int len, tq;  // tokens, queries
  int all;      // keys that every row sees
  int s0, s1, part;
};
constexpr int kWorkInts = sizeof(Work) / 4;

template <int R>
__device__ __forceinline__ Work work_of(const CaParams& p, const Sequence& q, int b, int hk, int tile, int s0, int s1,
                                        int part) {
  Work w;
  w.b = b;
  w.hk = hk;
  w.row0 = tile * 16 * q.sub;
  w.rl = min(w.row0 + 16 * q.sub, q.live) - 1;
  w.len = q.len;
  w.tq = q.tq;
  w.all = p.causal ? max(q.len - q.tq + query_of(p, w.row0) + 1, 0) : q.len;
  const int last = p.causal ? max(q.len - q.tq + query_of(p, w.rl) + 1, 0) : q.len;  // keys that the last row sees
  w.s0 = s0;
  w.s1 = min(s1, (last + 31) / 32);
  w.part = part;
  return w;
}

// R tiles of 16 rows against the steps of `w`, the waves taking turns at them.
template <int D, int R, int NW, int RMAX>
__device__ __forceinline__ void attend(const CaParams& p, const Work& w, unsigned char* lds) {
  constexpr int KT = D / 32, DT = D / 16;  // products of a score, tiles of the output
  constexpr int LD = D + 4;
  typedef Stage<D> St;
  typedef uint32_t piece __attribute__((ext_vector_type(D / 32)));
  int thread = threadIdx.x;
  asm volatile("" : "+v"(thread));  // what follows from it is not kept in registers from tile to tile
  const int lane = thread & 63, wave = uniform(thread >> 6);
  const int fr = lane & 15, g = lane >> 4;
  const float scale = p.scale;

  bf16x8 qf[R][KT];
  int lim[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = min(w.row0 + 16 * r + fr, w.rl), t = query_of(p, i), h = w.hk * p.G + i - t * p.G;
    const uint16_t* q = static_cast<const uint16_t*>(p.q.p) + w.b * p.q.b + t * p.q.t + h * p.q.h + g * (D / 4);
#pragma unroll
    for (int k = 0; k < KT; ++k) qf[r][k] = frag(*reinterpret_cast<const u32x4*>(q + 8 * k));
    lim[r] = p.causal ? w.len - w.tq + t + 1 : w.len;
  }
  f32x4 o[R][DT], l[R];
  float m[R];  // reference points
#pragma unroll
  for (int r = 0; r < R; ++r) {
    m[r] = kFar;
    l[r] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < DT; ++j) o[r][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  bool far = false;  // one of the wave's reference points is far out

  int s = w.s0 + wave;
  int col = 0, row = s * 32;  // the next step's page column and row in the page
  if (row >= p.c.page) {
    col = row / p.c.page;
    row -= col * p.c.page;
  }
  const_int* table = scalar(p.c.table + (long long)w.b * p.c.L);
  const long long head_rows = (long long)p.c.Hk * p.c.page, first_row = w.hk * (long long)p.c.page;
  int page = s < w.s1 ? table[col] : -1;

  // What a lane loads of a step, 16 bytes of codes and 4 of scales at a time.
  constexpr int PR = D / 32;  // 16-byte pieces of a row
  const int lr = lane / PR, lc = lane % PR;
  const int kc = lc ^ (D == 128 ? turned(lr >> 2) : (lr >> 3) & 1);
  const int vr = (lr & ~3) | ((lr & 3) ^ (D == 128 ? (lr >> 2) & 3 : (lr >> 2) & 2));
  const uint8_t* kcodes = p.c.codes + first_row * (D / 2) + lr * (D / 2) + kc * 16;
  const uint8_t* vcodes = p.c.codes + (first_row + head_rows) * (D / 2) + vr * (D / 2) + lc * 16;
  const int ls = lane % (2 * D / 4), half = ls >= D / 4;  // D / 4 lanes for the keys' scales, as many for the values'
  const uint8_t* scales = p.c.scales + (first_row + (half ? head_rows : 0)) * (D / 32) + (ls - half * (D / 4)) * 4;

  // Loads the next step to a stage and moves on, to step `then` if there is one; else the
  // same step is loaded again, so that as many loads are under way as are waited for.
  // False: the step has no page (page 0 is loaded, and nothing of it counts).
  unsigned char* ring = lds + wave * kStages * St::kBytes;
  auto load = [&](int stage, int then) -> bool {
    const bool there = page >= 0 && page < p.c.pages;
    const long long at = (long long)(there ? page : 0) * 2 * head_rows + row;
    unsigned char* dst = ring + stage * St::kBytes;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      __builtin_amdgcn_global_load_lds((glb_void*)(kcodes + at * (D / 2) + i * 1024), (lds_void*)(dst + i * 1024), 16, 0, 0);
      __builtin_amdgcn_global_load_lds((glb_void*)(vcodes + at * (D / 2) + i * 1024),
                                       (lds_void*)(dst + St::kValues + i * 1024), 16, 0, 0);
    }
    __builtin_amdgcn_global_load_lds((glb_void*)(scales + at * (D / 32)), (lds_void*)(dst + St::kScales), 4, 0, 0);
    if (then < w.s1) {
      row += 32 * NW;
      while (row >= p.c.page) {
        row -= p.c.page;
        ++col;
      }
      page = table[col];
    }
    return there;
  };

  // Where a lane reads: of keys fr and 16 + fr the D/4 elements from g D/4, with their
  // group's scale byte; of the values the D/16 elements from fr D/16 of eight keys, with
  // the scale bytes of four neighbouring keys at a time.
  const int kat = D == 128 ? fr * 64 + ((g ^ turned(fr >> 2)) << 4) : fr * 32 + (((g >> 1) ^ (fr >> 3)) << 4) + (g & 1) * 8;
  const int ksat = St::kScales + fr * (D / 32) + (D == 128 ? g : g / 2);
  const int vsat = St::kScales + D + g * (D / 8);
  int vat[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    vat[e] = St::kValues + (4 * g + (e ^ (D == 128 ? g : g & 2))) * (D / 2) + fr * (D / 32);

  // S^T of a step
  auto scores = [&](const unsigned char* at, f32x4 (&st)[R][2]) {
    piece k[2];
    float unit[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      k[i] = *reinterpret_cast<const piece*>(at + kat + i * 8 * D);
      unit[i] = fp4_unit(at[ksat + i * (D / 2)]);
#pragma unroll
      for (int r = 0; r < R; ++r) st[r][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
#pragma unroll
    for (int x = 0; x < KT; ++x)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bf16x8 kf = frag(fp4_values(k[i][x], unit[i]));
#pragma unroll
        for (int r = 0; r < R; ++r)
          st[r][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[r][x], st[r][i], 0, 0, 0);
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
  // score of the step. Each row goes by its own exponents and reference point alone, so that
  // its result does not depend on the rows beside it.
  auto move = [&](const f32x4 (&st)[R][2], f32x4 (&x)[R][2]) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float top = st[r][0][0];
#pragma unroll
      for (int i = 1; i < 8; ++i) top = fmaxf(top, st[r][i / 4][i % 4]);
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      const float to = fmaf(top, scale, -m[r]) > kSlack ? top * scale : m[r];
      const float f = __builtin_amdgcn_exp2f(m[r] - to);
      m[r] = to;
      far = far || __any(is_far(to));
      l[r] *= f;
#pragma unroll
      for (int j = 0; j < DT; ++j) o[r][j] *= f;
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        x[r][i / 4][i % 4] = is_far(m[r]) ? far_exponent(st[r][i / 4][i % 4], scale, m[r])
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
  auto output = [&](const unsigned char* at, const u32x4 (&pf)[R], int s, bool there) {
    uint32_t v[8];
    float unit[8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const piece word = *reinterpret_cast<const piece*>(at + vsat + i * (D / 2));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const unsigned char* c = at + vat[e] + i * 8 * D;
        v[4 * i + e] = D == 128 ? *reinterpret_cast<const uint32_t*>(c) : *reinterpret_cast<const uint16_t*>(c);
        const uint32_t x = D == 128 ? word[e] : word[e / 2];
        const int from = D == 128 ? 8 * (fr / 4) : 16 * (e % 2) + 8 * (fr / 8);
        unit[4 * i + e] = __uint_as_float(__builtin_amdgcn_alignbit(x, x, (uint32_t)(from + 9) & 31u));
      }
    }
    if ((there ? 32 * s + 32 : 0x7fffffff) > w.len) {
      // rows past the last token hold anything: no NaN of theirs may meet a 0
      const int key = (there ? 32 * s : 0x7fffff00) + 4 * g;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (key + 16 * (i / 4) + i % 4 >= w.len) {
          v[i] = 0;
          unit[i] = 1.f;
        }
    }
#pragma unroll
    for (int h = 0; h < DT / 2; ++h) {
      uint32_t a[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        a[i] = h == 0 ? fp4_pair<0>(v[i], unit[i]) : h == 1 ? fp4_pair<1>(v[i], unit[i])
             : h == 2 ? fp4_pair<2>(v[i], unit[i]) : fp4_pair<3>(v[i], unit[i]);
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

  if (s < w.s1) {
    bool there[kStages];
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) there[i] = load(i, s + (i + 1) * NW);
    there[kStages - 1] = false;
    for (int stage = 0; s < w.s1; s += NW) {
      const int next = stage == 0 ? kStages - 1 : stage - 1;  // the stage of the step before: it has been read
      wait_lds();
      there[kStages - 1] = load(next, s + kStages * NW);
      wait_vm<(kStages - 1) * St::kLoads>();
      const unsigned char* at = ring + stage * St::kBytes;
      f32x4 st[R][2];
      u32x4 pf[R];
      scores(at, st);
      if ((there[0] ? 32 * s + 32 : 0x7fffffff) > w.all) hide(st, s, there[0]);
      softmax(st, pf);
      output(at, pf, s, there[0]);
#pragma unroll
      for (int i = 0; i + 1 < kStages; ++i) there[i] = there[i + 1];
      stage = stage + 1 < kStages ? stage + 1 : 0;
    }
    wait_vm<0>();
  }
  __syncthreads();  // the ring's places are the join's

  // The waves join, 16 rows at a time.
  constexpr int TPR = 64 * NW / 16, PER = D / TPR;  // threads of a row, elements of a thread
  static_assert(PER >= 2 && PER * TPR == D);
  float* join = reinterpret_cast<float*>(lds);  // [NW][16][LD], then [NW][16][2]
  float* stat = join + NW * 16 * LD;
  const int jr = thread / TPR, jd = thread % TPR * PER;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (r > 0) __syncthreads();
    // element j + e D/16 of the lane's D/4 from g D/4 is o[j][e]
    float* mine = join + (wave * 16 + fr) * LD + g * (D / 4);
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
      for (int d = 0; d < PER; ++d) y[d] = fmaf(f, join[(v * 16 + jr) * LD + jd + d], y[d]);
    }
    if (w.part < 0) {
      const int t = query_of(p, i), h = w.hk * p.G + i - t * p.G;
      uint16_t* out = static_cast<uint16_t*>(p.out.p) + w.b * p.out.b + t * p.out.t + h * p.out.h + jd;
      const float f = sum == 0.f ? 0.f : 1.f / sum;  // no key: O is 0
#pragma unroll
      for (int d = 0; d < PER; d += 2) reinterpret_cast<uint32_t*>(out)[d / 2] = bf16_pair(y[d] * f, y[d + 1] * f);
    } else {
      const long long at = (long long)w.part * (16 * RMAX) + 16 * r + jr;
#pragma unroll
      for (int d = 0; d < PER; ++d) p.po[at * D + jd + d] = y[d];
      if (jd == 0) {
        p.ml[at * 2] = top;
        p.ml[at * 2 + 1] = sum;
      }
    }
  }
}

// A tile of up to R times 16 rows.
template <int D, int R, int NW>
__device__ __forceinline__ void attend_tile(const CaParams& p, const Work& w, unsigned char* lds) {
  const int tiles = (w.rl - w.row0) / 16 + 1;
  if constexpr (R >= 3) {
    if (tiles == 2) return attend<D, 2, NW, R>(p, w, lds);
  }
  if constexpr (R >= 2) {
    if (tiles == 1) return attend<D, 1, NW, R>(p, w, lds);
  }
  attend<D, R, NW, R>(p, w, lds);
}

// Waves a SIMD that the registers are shared out to, and so workgroups of four waves that a
// compute unit holds.
constexpr int waves_of(int D, int R) { return (D == 128 ? 5 : 6) - R; }

// Entries of the running sum of the work, of a sequence each or a group of them. (1025 sequences
// of 8 heads on 1 of 128, one of 262144 tokens among short ones: 68 us, a workgroup a tile 1480;
// at 1 to 16384 tokens 235 and 271, all of 16384 432 and 426, all short 26 and 10.)
constexpr int kMaxEntries = 1024;

// A workgroup a tile, with all its keys.
template <int D, int R, int NW>
__global__ __launch_bounds__(64 * NW, waves_of(D, R)) void cache_attn_kernel(CaParams p) {
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  const ItemCoord at = xcd_item(blockIdx.x, p.tiles);
  if (at.crop >= p.B * p.c.Hk) return;
  const int b = at.crop / p.c.Hk;
  const Sequence q = sequence<R>(p, b);
  if (at.item >= q.tiles) return;
  attend_tile<D, R, NW>(p, work_of<R>(p, q, b, at.crop - b * p.c.Hk, at.item, 0, q.steps, -1), lds);
}

// Where a workgroup is in its share: the next tile (of sequence b, whose work begins at
// `base`; -1: from the share's begin) and what is listed. b -1: all of it is.
constexpr int kPieces = 32;
struct Listing {
  long long begin, end, base;
  int share, b, tile, n;
};

// The workgroup's share, and the first sequence of the entry of `cum` that it begins in.
__device__ __forceinline__ void find_share(const CaParams& p, const long long* cum, int entries, Listing* list) {
  const long long total = uniform(cum[entries]);
  const int count = uniform(share_count(p, total));
  const bool any = (int)blockIdx.x < count && total > 0;
  // neighbouring shares, which read the same keys, on one XCD
  const int x = blockIdx.x % kXcds, share = x * (count / kXcds) + min(x, count % kXcds) + blockIdx.x / kXcds;
  const Shares shares = shares_of(total, count);
  const long long begin = any ? uniform(shares.begin(share)) : 0, end = any ? uniform(shares.begin(share + 1)) : 0;
  int lo = 0, hi = entries;  // cum[lo] <= begin < cum[hi]
  while (any && hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (uniform(cum[mid]) <= begin) lo = mid;
    else hi = mid;
  }
  const long long base = uniform(cum[lo]);
  if (threadIdx.x == 0) *list = Listing{begin, end, base, share, any ? lo * p.group : -1, -1, 0};
}

template <int R>
__device__ __forceinline__ void list_pieces(const CaParams& p, int32_t (*piece)[kWorkInts], Listing* list) {
  const bool first = threadIdx.x == 0;
  int n = 0, b = uniform(list->b), tile = uniform(list->tile);
  const int share = uniform(list->share);
  const long long begin = uniform(list->begin), end = uniform(list->end);
  long long base = uniform(list->base);
  for (; b >= 0 && b < p.B && base < end; ++b, tile = -1) {
    const Sequence q = sequence<R>(p, b);
    const long long per = uniform(q.tile_work());
    if (per == 0 || q.tiles == 0) continue;
    // (past the sequence's tiles where it lies before the share)
    if (tile < 0) tile = begin > base ? (int)min(uniform(quotient(begin - base, per)), (1LL << 30)) : 0;
    for (; tile < q.tiles * p.c.Hk && n < kPieces; ++tile) {
      const long long at = base + tile * per;
      if (at >= end) break;
      const int s0 = uniform(steps_before(q, at, begin)), s1 = uniform(steps_before(q, at, end));
      if (s0 >= s1) continue;
      const int hk = uniform(tile / q.tiles), i = tile - hk * q.tiles;
      const bool whole = s0 == 0 && s1 == q.steps;
      const Work w = work_of<R>(p, q, b, hk, i, s0, s1, whole ? -1 : 2 * share + (s0 == 0 ? 1 : 0));
      if (first) {
        __builtin_memcpy(piece[n], &w, sizeof w);
        int32_t* ends = p.ends + (((long long)b * p.c.Hk + hk) * p.tiles + i) * 2;
        if (s0 == 0) ends[0] = whole ? -1 : share;
        if (s1 == q.steps) ends[1] = share;
      }
      ++n;
    }
    if (n == kPieces) break;
    base += per * q.tiles * p.c.Hk;
  }
  if (first) {
    list->n = n;
    list->b = n == kPieces ? b : -1;
    list->tile = tile;
    list->base = base;
  }
}

// An equal share of all steps a workgroup: the sequences' tiles stand one after another,
// and a share may begin and end within a tile. What it holds of such tiles goes to two
// places of its own: the tile that it begins within to the first, the one that it leaves
// unfinished to the second.
template <int D, int R, int NW>
__global__ __launch_bounds__(64 * NW, waves_of(D, R)) void cache_share_kernel(CaParams p) {
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  __shared__ int32_t piece[kPieces][kWorkInts];
  __shared__ Listing list;
  long long* cum = reinterpret_cast<long long*>(lds);  // [entries + 1] work before each group of sequences
  const int entries = (p.B + p.group - 1) / p.group;
  for (int i = threadIdx.x; i < entries; i += 64 * NW) {
    long long sum = 0;
    for (int b = i * p.group; b < min((i + 1) * p.group, p.B); ++b) {
      const Sequence q = sequence<R>(p, b);
      sum += q.tile_work() * q.tiles * p.c.Hk;
    }
    cum[i + 1] = sum;
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    long long sum = 0;
    for (int i0 = 0; i0 < entries; i0 += 64) {
      const int i = i0 + threadIdx.x;
      long long v = i < entries ? cum[i + 1] : 0;
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const long long u = __shfl_up(v, d);
        if ((int)threadIdx.x >= d) v += u;
      }
      if (i < entries) cum[i + 1] = sum + v;
      sum += __shfl(v, 63);
    }
    if (threadIdx.x == 0) cum[0] = 0;
    find_share(p, cum, entries, &list);
  }
  __syncthreads();
  // The share's pieces are listed some at a time, and nothing of the sharing stays in
  // registers while they are worked on.
  for (;;) {
    if (threadIdx.x < 64) list_pieces<R>(p, piece, &list);
    __syncthreads();
    const int n = uniform(list.n);
    const bool last = uniform(list.b) < 0;
    for (int k = 0; k < n; ++k) {
      int32_t v[kWorkInts];
#pragma unroll
      for (int i = 0; i < kWorkInts; ++i) v[i] = uniform(piece[k][i]);
      Work w;
      __builtin_memcpy(&w, v, sizeof w);
      __syncthreads();  // the last piece's join, or the listing, has been read
      attend_tile<D, R, NW>(p, w, lds);
    }
    __syncthreads();
    if (last) break;
  }
}

// Rows whose tiles were cut, and zeros for rows without a key. The parts of a tile lie in
// the second place of its first share and the first place of every one after it (a share
// holds more than a step, so none between them is empty). D/4 lanes take a row, four
// elements each; with FEW all of a workgroup's lanes take one row, its parts dealt to
// them in turn.
template <int D, int R, bool FEW>
__global__ __launch_bounds__(256) void cache_join_kernel(CaParams p) {
  constexpr int GL = D / 4, GROUPS = 256 / GL;
  __shared__ f32x4 part[FEW ? GROUPS : 1][GL];
  __shared__ float stat[FEW ? GROUPS : 1][2];
  const int lane = threadIdx.x % GL, group = threadIdx.x / GL;
  const int blocks = FEW ? p.Tq * p.G : (p.Tq * p.G + GROUPS - 1) / GROUPS;  // of a key head
  const int bh = blockIdx.x / blocks, b = bh / p.c.Hk, hk = bh - b * p.c.Hk;
  const Sequence q = sequence<R>(p, b);
  const int i = (blockIdx.x - bh * blocks) * (FEW ? 1 : GROUPS) + (FEW ? 0 : group);
  if (i >= q.live) return;
  const int t = query_of(p, i), h = hk * p.G + i - t * p.G;
  int tile = i / 16;  // by q.sub
  if (q.sub == 2) tile /= 2;
  if (q.sub == 3) tile /= 3;
  const int r = i - tile * 16 * q.sub;
  float m = kFar, l = 0.f;
  f32x4 y = {0.f, 0.f, 0.f, 0.f};
  if (q.steps > 0) {
    const int32_t* ends = p.ends + ((long long)bh * p.tiles + tile) * 2;
    const int first = ends[0], n = ends[1] - first + 1;
    if (first < 0) return;  // written as it is
    auto slot = [&](int k) { return (long long)(2 * (first + k) + (k == 0 ? 1 : 0)) * (16 * R) + r; };
    constexpr int STEP = FEW ? GROUPS : 1, BATCH = 8;
    for (int k0 = FEW ? group : 0; k0 < n; k0 += BATCH * STEP) {
      float pm[BATCH], pl[BATCH];
      f32x4 v[BATCH];
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        const int x = k0 + k * STEP;
        const long long from = slot(x < n ? x : k0);
        pm[k] = x < n ? p.ml[from * 2] : kFar;
        pl[k] = x < n ? p.ml[from * 2 + 1] : 0.f;
        v[k] = reinterpret_cast<const f32x4*>(p.po + from * D)[lane];
      }
      float to = m;
#pragma unroll
      for (int k = 0; k < BATCH; ++k) to = fmaxf(to, pm[k]);
      const float f = __builtin_amdgcn_exp2f(m - to);
      m = to;
      l *= f;
      y *= f;
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        const float g = k0 + k * STEP < n ? __builtin_amdgcn_exp2f(pm[k] - to) : 0.f;
        l = fmaf(pl[k], g, l);
        y += v[k] * g;
      }
    }
  }
  if constexpr (FEW) {
    part[group][lane] = y;
    if (lane == 0) {
      stat[group][0] = m;
      stat[group][1] = l;
    }
    __syncthreads();
    if (group > 0) return;
    float to = m;
    for (int k = 1; k < GROUPS; ++k) to = fmaxf(to, stat[k][0]);
    const float f = __builtin_amdgcn_exp2f(m - to);
    l *= f;
    y *= f;
    for (int k = 1; k < GROUPS; ++k) {
      const float g = __builtin_amdgcn_exp2f(stat[k][0] - to);
      l = fmaf(stat[k][1], g, l);
      y += part[k][lane] * g;
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint16_t* out = static_cast<uint16_t*>(p.out.p) + b * p.out.b + t * p.out.t + h * p.out.h + lane * 4;
  *reinterpret_cast<u32x2*>(out) = u32x2{bf16_pair(y[0] * inv, y[1] * inv), bf16_pair(y[2] * inv, y[3] * inv)};
}

struct Plan {
  int R, tiles;
  int waves;   // of a workgroup
  int shares;  // 0: a workgroup a tile
};

constexpr int kWaves = 4, kManyWaves = 8;
constexpr int kLong = 128;

// R, tiles of 16 rows that go through the keys together, and a workgroup's waves. With no
// more than a tile of 16 rows for each compute unit, every tile has a workgroup of eight
// waves (80 rows of 2 x 8 heads of 64, 2304 tokens: 11.1 us, in twos 17.3; one row of 16
// heads and 2304 tokens: 10.8 us, with four waves 13.8; 384 tiles of 2048 tokens would take
// 24.9 with eight, 22.2 with four). Else four waves (37 x 80 rows of 16 heads of 64, 2304
// tokens: two 64 us, four 61, eight 70), and up to three tiles go together (37 x 40 rows of 16
// heads of 64, 2304 tokens: 39 us, in twos 47), and more than three in twos: as fast as in
// threes where all have as many (37 x 80 rows: 65 us and 62; 16 x 128 rows of 32 heads of
// 128, 4096 tokens: 165 and 166) and ahead where not (37 sets of up to 80 rows: 35 and 44).
//
// A workgroup a tile, or equal shares: listing and joining the shares takes 10 us beside the
// reading, and spares the others' wait for the longest tile, 0.8 us a step and wave. One
// sequence of 32 heads on 8 of 128: 2048 tokens 12.2 us in tiles and 15.2 in shares, 4096
// 20.1 and 14.0, 32768 128 and 20; 16 of them: 4096 tokens 22 and 25, 8192 37 and 36; 48 at
// 8192 81 and 93, at lengths from 1 to 8192 54 and 46, one at 8000 among short ones 47 and
// 22.
//
// Among four times as many tiles as stay resident, a workgroup a tile again, if the longest
// possible tile does not outlast the others by much: at most kLong steps for each round of
// tiles (a round takes 4 to 5 us however short its tiles are, a step of the longest 0.18), or
// a sequence that has so many tiles by itself; and if the XCDs, each of which takes whole key
// heads, get nearly the same. Us, in tiles / in shares: 512 sequences of 32 heads on 8 of 128,
// all of 16384 tokens 1464 / 1505, 1 to 16384 805 / 804, one of 16384 among short ones 101 / 48,
// of 32768 193 / 50, of 262144 1493 / 89; 256 x 64 rows of 16 heads of 64, all of 32768 tokens
// 3439 / 4364; 4096 rows of 32 heads of 128 behind 16384 tokens on 8 key heads 1093 / 1252, on
// 4 2142 / 1268, of 24 heads on 12 1101 / 921.
Plan plan_for(int B, int Tq, int Hq, int Hk, int D, int page, int L) {
  const int rows = Tq * (Hq / Hk), subs = (rows + 15) / 16;
  const long long heads = (long long)B * Hk, steps = ((long long)L * page + 31) / 32;
  const bool few = heads * subs <= 256;
  Plan x;
  x.R = few ? 1 : subs <= 3 ? subs : 2;
  x.tiles = (subs + x.R - 1) / x.R;
  x.waves = few ? kManyWaves : kWaves;
  x.shares = 0;
  const long long items = heads * x.tiles;
  if (steps <= 96 + (items < 640 ? items : 640) / 4) return x;
  // (shares are even whatever the tiles are, so theirs are as large as can be)
  const int R = subs < 3 ? subs : 3, tiles = (subs + R - 1) / R, resident = 256 * waves_of(D, R);
  const bool bounded = steps * resident <= kLong * heads * tiles || (long long)Hk * tiles >= 4 * resident;
  const bool even = 8 * ((heads + kXcds - 1) / kXcds * kXcds) <= 9 * heads;
  if (heads * tiles >= 4 * resident && bounded && even) return x;
  const long long most = heads * tiles * steps / (2 * kWaves);
  x.R = R;
  x.tiles = tiles;
  x.waves = kWaves;
  x.shares = most < resident ? (int)most : resident;
  return x;
}

size_t al256(size_t n) { return (n + 255) & ~(size_t)255; }
size_t ends_bytes(const Plan& x, int B, int Hk) { return al256((size_t)B * Hk * x.tiles * 8); }
size_t po_bytes(const Plan& x, int D) { return al256((size_t)x.shares * 2 * 16 * x.R * D * 4); }

template <int D, int NW>
constexpr int lds_bytes() {
  constexpr int kRing = NW * kStages * Stage<D>::kBytes, kJoin = NW * 16 * (D + 4 + 2) * 4;
  static_assert((kMaxEntries + 1) * 8 <= kRing, "the running sum fits");
  return kRing > kJoin ? kRing : kJoin;
}

template <int D, int R, int NW>
hipError_t run_tiles(const CaParams& p, hipStream_t st) {
  const long long groups8 = ((long long)p.B * p.c.Hk + kXcds - 1) / kXcds * kXcds;
  hipLaunchKernelGGL((cache_attn_kernel<D, R, NW>), dim3((unsigned)(groups8 * p.tiles)), dim3(64 * NW),
                     (lds_bytes<D, NW>()), st, p);
  return hipGetLastError();
}

template <int D, int R>
hipError_t run(const CaParams& p, int waves, hipStream_t st) {
  if (p.shares == 0) {
    if constexpr (R == 1) {
      if (waves == kManyWaves) return run_tiles<D, 1, kManyWaves>(p, st);
    }
    return run_tiles<D, R, kWaves>(p, st);
  }
  constexpr int kLds = lds_bytes<D, kWaves>();
  hipLaunchKernelGGL((cache_share_kernel<D, R, kWaves>), dim3((unsigned)p.shares), dim3(64 * kWaves), kLds, st, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const long long heads = (long long)p.B * p.c.Hk, rows = (long long)p.Tq * p.G;
  constexpr int kRows = 1024 / D;  // of a workgroup
  if (heads * rows <= 512)
    hipLaunchKernelGGL((cache_join_kernel<D, R, true>), dim3((unsigned)(heads * rows)), dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL((cache_join_kernel<D, R, false>), dim3((unsigned)(heads * ((rows + kRows - 1) / kRows))), dim3(256),
                       0, st, p);
  return hipGetLastError();
}

template <int D>
hipError_t run_rows(const CaParams& p, const Plan& x, hipStream_t st) {
  return x.R == 1 ? run<D, 1>(p, x.waves, st) : x.R == 2 ? run<D, 2>(p, x.waves, st) : run<D, 3>(p, x.waves, st);
}

}  // namespace

size_t cache_attn_workspace_bytes(int B, int Tq, int Hq, int Hk, int D, int page, int L) {
  const Plan x = plan_for(B, Tq, Hq, Hk, D, page, L);
  if (x.shares == 0) return 0;
  return ends_bytes(x, B, Hk) + po_bytes(x, D) + al256((size_t)x.shares * 2 * 16 * x.R * 8);
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
  p.shares = x.shares;
  p.group = (a.B + kMaxEntries - 1) / kMaxEntries;
  if (x.shares > 0) {
    uint8_t* ws = static_cast<uint8_t*>(a.ws);
    p.ends = reinterpret_cast<int32_t*>(ws);
    ws += ends_bytes(x, a.B, a.c.Hk);
    p.po = reinterpret_cast<float*>(ws);
    p.ml = reinterpret_cast<float*>(ws + po_bytes(x, a.c.D));
  }
  return a.c.D == 128 ? run_rows<128>(p, x, st) : run_rows<64>(p, x, st);
}

}  // namespace gkd
