// prefix_attn.hip - attention of a batch that shares one long prefix of keys
// (gkd_prefix_attention).
//
// A row is one query of one query head; the rows of a key head are numbered
// R = (b Tq + t) G + g (G = Hq / Hk query heads share the key head). The
// softmax runs online: a row keeps its running maximum m, the sum l of
// exp(s - m) and the output O scaled alike, and ranges of keys that were
// taken apart are joined by
//   m = max_i m_i,  l = sum_i l_i exp(m_i - m),  O = sum_i O_i exp(m_i - m).
// Probabilities are rounded to bfloat16 (2^-8 of each) for the product with V,
// whose instruction takes both sides in that type; l sums the rounded ones, so a
// row's weights add to one and what is left is an error of the size of the
// output's own rounding (2.3e-3 of an output in the mean, 1.7e-3 of it the
// latter). Two products, of the high and the low half, would take half as many
// matrix instructions again.
//
// So the prefix can be taken once for the rows of all sequences together
// (their keys pass through LDS once per tile of rows, not once per
// sequence), own keys sequence by sequence, and long ranges in parts.
//
// Two tiles:
//   wide   128 rows, four waves of 32 rows, key chunks of 64 shared by them;
//   thin   16 rows, four or eight waves that take every fourth or eighth
//          32-key chunk and join at the end: for few rows, where reading the
//          keys is all there is.
//
// Measured (bfloat16, a call, inputs that change from call to call):
//   8 x 1024 queries, 32 heads of 128 (8 of keys), causal, behind 8192 keys:
//     1.08-1.10 ms, 1.07 PFLOP/s. A wave's chunk is 68 matrix instructions and
//     the exponents between them; two waves a SIMD take turns with both.
//   48 x 1 query, the same heads, 1024 own keys at most, behind 32768: 82 us,
//     287 MB at 3.5 TB/s. Up to 128 rows it is the reading (32 sequences: 52 us,
//     4.5 TB/s); these 192 are two tiles, which read the prefix through L2 and
//     take its products twice.
//   37 x 80 queries at most, 16 heads of 64, behind 2304: 40 us, 35 of them the
//     products' kernel; a lone query behind 576 keys 8 us on the GPU.
#include "gkd_device.hpp"
#include "tokens_launch.hpp"

#include <type_traits>

namespace gkd {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) void lds_void;

// A list of work items, [part of the keys][tile of rows][key head].
struct List {
  int wide;    // its tiles are wide ones, else thin ones
  int seq;     // they stay within a sequence, else the rows of all sequences are packed
  int keys;    // 0: the prefix, 1: own keys, 2: both, prefix first
  int tiles;   // tiles of rows per key head
  int parts;
  int slot;    // the first part's slot among a row's partial results
  int n;       // items
};

struct PaParams {
  Heads q, kp, vp, ko, vo, out;
  int P, S;
  const int32_t *own_len, *q_len;
  const uint8_t* mask;
  int B, Tq, Hk, G;
  int RS, RT;          // rows of a sequence, of all sequences (per key head)
  float c;             // scale * log2(e)
  int causal;
  List first, second;  // the plan: the workgroups of both lists, one after the other
  int slots;           // partial results a row has; 1: written as they are
  float* po;                   // [slots][Hk][RT][D]
  float* ml;                   // [slots][Hk][RT][2]
};

__device__ __forceinline__ bf16x8 frag(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

// A tile's rows and keys, the same for both kinds of tile.
struct TileWork {
  int hk;            // key head
  int b;             // sequence of the own keys, -1: prefix keys only
  int row0, n;       // packed tiles: first packed row; others: first row R, rows
  bool packed;       // rows are those in use of all sequences, one after another
  int p0, p1;        // prefix keys
  int s0, s1;        // own keys
  int slot;
};

// Query rows of a lane: their places, and how far they see.
struct RowPlace {
  int R;             // row of the key head
  bool live;
  int lim;           // own keys below this are visible
  long long q, out;  // element offsets
};

__device__ __forceinline__ int own_length(const PaParams& p, int b) {
  return p.own_len ? min(max(p.own_len[b], 0), p.S) : p.S;
}
__device__ __forceinline__ int query_length(const PaParams& p, int b) {
  return p.q_len ? min(max(p.q_len[b], 0), p.Tq) : p.Tq;
}

// Row i of the tile. `cum`: for packed tiles, the packed rows before each
// sequence (B + 1 of them, in LDS).
__device__ __forceinline__ RowPlace place_row(const PaParams& p, const TileWork& w, const int* cum, int i) {
  RowPlace r;
  r.live = i < w.n;
  unsigned b, rr;
  if (w.packed && p.q_len) {
    const int at = w.row0 + (r.live ? i : w.n - 1);
    int lo = 0, hi = p.B;  // cum[lo] <= at < cum[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cum[mid] <= at) lo = mid;
      else hi = mid;
    }
    b = lo;
    rr = at - cum[lo];
  } else {
    const unsigned at = w.row0 + (r.live ? i : w.n - 1);
    b = at / (unsigned)p.RS;
    rr = at - b * p.RS;
  }
  const unsigned t = rr / (unsigned)p.G;
  const int h = w.hk * p.G + (int)(rr - t * p.G);
  r.R = (int)(b * p.RS + rr);
  r.lim = 0x7fffffff;
  if (p.causal && w.b >= 0) r.lim = own_length(p, w.b) - query_length(p, w.b) + (int)t + 1;
  r.q = b * p.q.b + t * p.q.t + h * p.q.h;
  r.out = b * p.out.b + t * p.out.t + h * p.out.h;
  return r;
}

// The own keys that the tile's last row sees, and those that every row sees.
__device__ __forceinline__ void own_ends(const PaParams& p, const TileWork& w, int& last, int& all) {
  last = all = w.s1;
  if (w.b < 0) return;
  const int len = own_length(p, w.b);
  last = all = min(w.s1, len);
  if (p.causal) {
    const int first = w.row0 - w.b * p.RS, before = len - query_length(p, w.b) + 1;
    last = min(last, before + (int)((unsigned)(first + w.n - 1) / (unsigned)p.G));
    all = min(all, before + (int)((unsigned)first / (unsigned)p.G));
  }
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  const bf16x2 h = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
  return __builtin_bit_cast(uint32_t, h);
}

// A row's result: O^T[dim 16 j + 4 g + e] in o[j][e], l and m (base 2) the same
// in all its lanes.
template <int D>
__device__ __forceinline__ void write_row(const PaParams& p, const TileWork& w, const RowPlace& r, int g,
                                          float m, float l, const f32x4 (&o)[D / 16], bool any_keys) {
  if (!r.live) return;
  if (p.slots == 1) {
    const float inv = l > 0.f ? 1.f / l : 0.f;
    uint16_t* dst = static_cast<uint16_t*>(p.out.p) + r.out + 4 * g;
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
      *reinterpret_cast<u32x2*>(dst + 16 * j) =
          u32x2{bf16_pair(o[j][0] * inv, o[j][1] * inv), bf16_pair(o[j][2] * inv, o[j][3] * inv)};
    return;
  }
  const long long at = ((long long)w.slot * p.Hk + w.hk) * p.RT + r.R;
  if (g == 0) *reinterpret_cast<f32x2*>(p.ml + 2 * at) = f32x2{m, l};
  if (!any_keys) return;  // the statistics say that there is nothing
#pragma unroll
  for (int j = 0; j < D / 16; ++j) *reinterpret_cast<f32x4*>(p.po + at * D + 16 * j + 4 * g) = o[j];
}

// V's rows lie in LDS with piece c of key row r at place c ^ v_turn(r). A
// transposing read takes 16 bytes' halves of pieces 2 j and 2 j + 1 of eight
// keys at a time: with rows of 256 bytes (D = 128) these meet in different
// banks only if keys differ by an even number of pieces (turned by r like K's
// rows, a third of the LDS cycles were conflicts); rows of 128 bytes alternate
// between the halves of the banks by themselves.
template <int D>
__device__ __forceinline__ int v_turn(int r) {
  return (D == 128 ? 2 * r : r) & (D / 8 - 1);
}

// max over the four 16-lane groups of a wave
__device__ __forceinline__ float group_max(float x) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

// ---------------------------------------------------------------------------
// 16 rows, WK waves that take every WK-th 32-key chunk and join at the end. A
// wave's K rows go straight into registers as the product's operand and its V
// rows into its own 32 rows of LDS (the product takes them transposed), with
// nothing in flight beside them: what hides a chunk's latency are the other
// waves of the CU, 16 KB of keys each (D = 128).
// ---------------------------------------------------------------------------
template <int D, int WK>
struct ThinTile {
  static constexpr int KC = 32, kRows = 16;
  static constexpr bool kPacked = false;  // thin tiles stay within a sequence
  static constexpr int kPieces = D / 8, kDK = D / 32, kND = D / 16;
  static constexpr int kMat = KC * D * 2;
  static constexpr int kJoin = (WK - 1) * (kND * 1024 + 512);  // the waves' results at the end
  static constexpr int kLds = WK * kMat > kJoin ? WK * kMat : kJoin;
  static constexpr int kLoads = kMat / 1024, kBlkRows = 64 / kPieces;

  static __device__ __forceinline__ void run(const PaParams& p, const TileWork& w, unsigned char* lds, const int*) {
    const int lane = threadIdx.x & 63;
    const int wk = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int fr = lane & 15, g = lane >> 4;
    const RowPlace row = place_row(p, w, nullptr, fr);
    bf16x8 qf[kDK];
#pragma unroll
    for (int k = 0; k < kDK; ++k)
      qf[k] = frag(row.live ? *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p.q.p) + row.q + 32 * k + 8 * g)
                            : u32x4{0u, 0u, 0u, 0u});
    int own_end, all_see;
    own_ends(p, w, own_end, all_see);
    const int nprefix = w.p1 > w.p0 ? (w.p1 - w.p0 + KC - 1) / KC : 0;
    const int nown = own_end > w.s0 ? (own_end - w.s0 + KC - 1) / KC : 0;
    const int nc = nprefix + nown;

    f32x4 o[kND];
    float m = -INFINITY, l = 0.f;
#pragma unroll
    for (int j = 0; j < kND; ++j) o[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    unsigned char* sV = lds + wk * kMat;
    const int lr = lane / kPieces, vkey = 4 * g + (fr >> 2);
    for (int c = wk; c < nc; c += WK) {
      const bool pre = c < nprefix;
      const int base = pre ? w.p0 + c * KC : w.s0 + (c - nprefix) * KC;
      const int end = pre ? w.p1 : own_end;
      const int keys = min(end - base, KC);
      const Heads& hk = pre ? p.kp : p.ko;
      const Heads& hv = pre ? p.vp : p.vo;
      const long long ob = pre ? 0 : (long long)w.b;
      uint16_t* ks = static_cast<uint16_t*>(hk.p) + ob * hk.b + w.hk * hk.h + (long long)base * hk.t;
      uint16_t* vs = static_cast<uint16_t*>(hv.p) + ob * hv.b + w.hk * hv.h + (long long)base * hv.t;
      const uint32_t kt = (uint32_t)hk.t * 2u, vt = (uint32_t)hv.t * 2u;
      // rows past the last key are past the buffer's end and come out as zeros
      const auto kb = __builtin_amdgcn_make_buffer_rsrc(ks, 0, (int)((uint32_t)(keys - 1) * kt + D * 2), 0x00020000);
      const auto vb = __builtin_amdgcn_make_buffer_rsrc(vs, 0, (int)((uint32_t)(keys - 1) * vt + D * 2), 0x00020000);
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): the last chunk's V is out of LDS
      asm volatile("" ::: "memory");
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = i * kBlkRows + lr;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(vb, (lds_void*)(sV + i * 1024), 16,
                                                 (int)(r * vt + 16 * ((lane % kPieces) ^ v_turn<D>(r))), 0, 0, 0);
      }
      bf16x8 kf[2][kDK];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int k = 0; k < kDK; ++k)
          kf[t][k] = frag(__builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
              kb, (int)((16 * t + fr) * kt + 64 * k + 16 * g), 0, 0)));
      uint32_t bits = ~0u;  // keys in use
      if (!pre && p.mask) {
        const bool on = lane < keys && p.mask[(long long)w.b * p.S + base + lane] != 0;
        bits = (uint32_t)__ballot(on);
      }
      f32x4 sc[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        sc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < kDK; ++k) sc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf[t][k], qf[k], sc[t], 0, 0, 0);
      }
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0): V is in LDS
      asm volatile("" ::: "memory");
      if (~bits != 0u) {
        // masked values may hold anything: they enter the product as zeros
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
          if (!((bits >> (i * kBlkRows + lr)) & 1))
            *reinterpret_cast<u32x4*>(sV + i * 1024 + lane * 16) = u32x4{0u, 0u, 0u, 0u};
      }
      if (base + KC > (pre ? end : all_see) || ~bits != 0u) {
        const int seen = min(max((pre ? end : min(end, row.lim)) - base, 0), KC);
        const uint32_t mine = (seen < KC ? bits & ((1u << seen) - 1u) : bits) >> (4 * g);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t keep = (uint32_t)__builtin_amdgcn_sbfe((int)mine, 16 * t + e, 1);
            sc[t][e] = __uint_as_float((__float_as_uint(sc[t][e]) & keep) | (0xff800000u & ~keep));
          }
      }
      float x = -INFINITY;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) x = fmaxf(x, sc[t][e]);
      // m is a product as it comes: differences of scores are taken first and
      // scaled then, so the largest one's exponent is 0 at any size (the rounding
      // of score times c is 2^7 and more from 2^31 on)
      const float mn = fmaxf(m, group_max(x));
      const float ref = mn == -INFINITY ? 0.f : mn;
      const float alpha = __builtin_amdgcn_exp2f((m - ref) * p.c);
      m = mn;
      l *= alpha;
#pragma unroll
      for (int j = 0; j < kND; ++j) o[j] *= alpha;
      uint32_t pk[2][2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        float e4[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) e4[e] = __builtin_amdgcn_exp2f((sc[t][e] - ref) * p.c);
        pk[t][0] = bf16_pair(e4[0], e4[1]);
        pk[t][1] = bf16_pair(e4[2], e4[3]);
        // the sum takes the probabilities as the product does, so weights add to one
#pragma unroll
        for (int e = 0; e < 2; ++e) l += __uint_as_float(pk[t][e] << 16) + __uint_as_float(pk[t][e] & 0xffff0000u);
      }
      // O^T += V^T P^T: k-slots 8 g .. 8 g + 7 carry keys 4 g + (0..3) and
      // 16 + 4 g + (0..3) on both sides
      const bf16x8 pf = frag(u32x4{pk[0][0], pk[0][1], pk[1][0], pk[1][1]});
#pragma unroll
      for (int j = 0; j < kND; ++j) {
        const unsigned char* v = sV + vkey * D * 2 + (((2 * j + ((fr & 3) >> 1)) ^ v_turn<D>(vkey)) << 4) + (fr & 1) * 8;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)v);
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(v + 16 * D * 2));
        const u32x2 l2 = __builtin_bit_cast(u32x2, lo), h2 = __builtin_bit_cast(u32x2, hi);
        o[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(u32x4{l2[0], l2[1], h2[0], h2[1]}), pf, o[j], 0, 0, 0);
      }
    }
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);

    // the waves join in LDS, in order
    f32x4* so = reinterpret_cast<f32x4*>(lds);
    f32x2* sm = reinterpret_cast<f32x2*>(lds + (WK - 1) * kND * 1024);
    __syncthreads();  // V is read
    if (wk > 0) {
#pragma unroll
      for (int j = 0; j < kND; ++j) so[((wk - 1) * kND + j) * 64 + lane] = o[j];
      sm[(wk - 1) * 64 + lane] = f32x2{m, l};
    }
    __syncthreads();
    if (wk > 0) return;
    float top = m;
#pragma unroll
    for (int v = 0; v < WK - 1; ++v) top = fmaxf(top, sm[v * 64 + lane][0]);
    const float ref = top == -INFINITY ? 0.f : top;
    const float a = __builtin_amdgcn_exp2f((m - ref) * p.c);
    m = top;
    l *= a;
#pragma unroll
    for (int j = 0; j < kND; ++j) o[j] *= a;
    for (int v = 0; v < WK - 1; ++v) {
      const f32x2 x = sm[v * 64 + lane];
      const float wgt = __builtin_amdgcn_exp2f((x[0] - ref) * p.c);
      l = fmaf(x[1], wgt, l);
#pragma unroll
      for (int j = 0; j < kND; ++j) o[j] += so[(v * kND + j) * 64 + lane] * wgt;
    }
    write_row<D>(p, w, row, g, m * p.c, l, o, nc > 0);
  }
};

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

// The keys that a tile reads, chunk by chunk: first the prefix's, then own ones.
struct KeyWalk {
  const uint16_t *k, *v;  // the next chunk's first key
  int kt, vt;             // token strides (below 2^25)
  int left;               // keys from there on
};

// The reference point m of a row's exponents stays where it is while the
// row's scores pass it by no more than 8: float32 sums and bfloat16 products
// bear probabilities of up to 2^8 as well as those below 1. So the scores'
// maximum is found, and l and O are scaled, on the first chunk and a few times
// after it; elsewhere a chunk costs seven integer maxima over the rounded
// probabilities (positive bfloat16 values order like their bits): one of 2^8
// or more sends the wave to look, and then the rows that passed 8 move and no
// others, so a row's results do not depend on its neighbours'.
constexpr float kSlack = 8.f;
constexpr uint32_t kSlackBits = 0x4380u;  // 2^8 in bfloat16
constexpr float kNowhere = -3e38f;        // m before a row's first key: any score passes it

// How far a score s passes m, base 2. One fused operation, while the rounding of
// m (a score times c) is at most 1/2; a row that is further out takes the
// rounded product, of which m is one, so that its largest score is at 0 and not
// at that rounding (half of 2^9 at scores of 2^32, which leaves the row with
// nothing or with infinities).
constexpr float kFar = 16777216.f;
__device__ __forceinline__ bool far_out(float m) { return fabsf(m) >= kFar && m != kNowhere; }
__device__ __forceinline__ float passed(float s, float c, float m, bool far) {
#pragma clang fp contract(off)
  const float t = s * c;
  return far ? t - m : fmaf(s, c, -m);
}

template <int D, int WR, int QT>
struct WideTile {
  static constexpr int KC = 64;
  static constexpr int kRows = 16 * QT * WR;
  static constexpr bool kPacked = true;
  static constexpr int kPieces = D / 8;                 // 16-byte pieces of a key row
  static constexpr int kMat = KC * D * 2;               // bytes of a chunk's K (or V)
  static constexpr int kStage = 2 * kMat;
  static constexpr int kLds = 2 * kStage;
  static constexpr int kNT = KC / 16, kDK = D / 32, kND = D / 16;
  static constexpr int kLoads = kMat / (WR * 1024);     // 1-KB loads a wave and matrix
  static constexpr int kBlkRows = 64 / kPieces;         // key rows of one load

  static __device__ __forceinline__ void run(const PaParams& p, const TileWork& w, unsigned char* lds, const int* cum) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wr = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int fr = lane & 15, g = lane >> 4;
    const int hk = w.hk, b_own = w.b, p0 = w.p0, p1 = w.p1, s0 = w.s0;

    bf16x8 qf[QT][kDK];
    RowPlace row[QT];
#pragma unroll
    for (int u = 0; u < QT; ++u) {
      row[u] = place_row(p, w, cum, (wr * QT + u) * 16 + fr);
      const uint16_t* src = static_cast<const uint16_t*>(p.q.p) + row[u].q;
#pragma unroll
      for (int k = 0; k < kDK; ++k)
        qf[u][k] = frag(row[u].live ? *reinterpret_cast<const u32x4*>(src + 32 * k + 8 * g) : u32x4{0u, 0u, 0u, 0u});
    }
    if (cum) __syncthreads();  // looked up by all before keys come into its place
    const bool idle = wr * QT * 16 >= w.n;  // a wave without rows: it loads, and leaves the pipes to others
    int own_end, all_see;
    own_ends(p, w, own_end, all_see);
    const int nprefix = p1 > p0 ? (p1 - p0 + KC - 1) / KC : 0;
    const int nown = own_end > s0 ? (own_end - s0 + KC - 1) / KC : 0;
    const int nc = nprefix + nown;
    KeyWalk own{}, walk{};
    if (nown > 0) {
      own.k = static_cast<const uint16_t*>(p.ko.p) + (long long)b_own * p.ko.b + hk * p.ko.h + (long long)s0 * p.ko.t;
      own.v = static_cast<const uint16_t*>(p.vo.p) + (long long)b_own * p.vo.b + hk * p.vo.h + (long long)s0 * p.vo.t;
      own.kt = (int)p.ko.t;
      own.vt = (int)p.vo.t;
      own.left = own_end - s0;
    }
    if (nprefix > 0) {
      walk.k = static_cast<const uint16_t*>(p.kp.p) + hk * p.kp.h + (long long)p0 * p.kp.t;
      walk.v = static_cast<const uint16_t*>(p.vp.p) + hk * p.vp.h + (long long)p0 * p.vp.t;
      walk.kt = (int)p.kp.t;
      walk.vt = (int)p.vp.t;
      walk.left = p1 - p0;
    } else {
      walk = own;
    }

    f32x4 o[QT][kND], l[QT];
    float m[QT];
    bool wary = false;  // a row of the wave is far out
#pragma unroll
    for (int u = 0; u < QT; ++u) {
      m[u] = kNowhere;
      l[u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < kND; ++j) o[u][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    // this lane's piece of the wave's first load: key row lr, piece (place ^
    // row), so that the 16 rows of an operand read lie in different banks
    const int lr = wr * kBlkRows + lane / kPieces;
    const int lp = 16 * ((lane % kPieces) ^ (lr & (kPieces - 1))), vp = 16 * ((lane % kPieces) ^ v_turn<D>(lr));
    auto load = [&](int c, int buf) {
      if (c == nprefix) walk = own;
      const int keys = min(walk.left, KC);
      // rows past the last key are past the buffer's end and come out as zeros
      const auto kb = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(walk.k), 0,
                                                        (int)((uint32_t)(keys - 1) * (uint32_t)walk.kt * 2u + D * 2), 0x00020000);
      const auto vb = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(walk.v), 0,
                                                        (int)((uint32_t)(keys - 1) * (uint32_t)walk.vt * 2u + D * 2), 0x00020000);
      unsigned char* st = lds + buf * kStage + wr * 1024;
      uint32_t off = (uint32_t)lr * (uint32_t)walk.kt * 2u + lp;
#pragma unroll
      for (int i = 0; i < kLoads; ++i, off += (uint32_t)walk.kt * (WR * kBlkRows * 2))
        __builtin_amdgcn_raw_ptr_buffer_load_lds(kb, (lds_void*)(st + i * WR * 1024), 16, (int)off, 0, 0, 0);
      off = (uint32_t)lr * (uint32_t)walk.vt * 2u + vp;
#pragma unroll
      for (int i = 0; i < kLoads; ++i, off += (uint32_t)walk.vt * (WR * kBlkRows * 2))
        __builtin_amdgcn_raw_ptr_buffer_load_lds(vb, (lds_void*)(st + kMat + i * WR * 1024), 16, (int)off, 0, 0, 0);
      walk.k += (long long)walk.kt * KC;
      walk.v += (long long)walk.vt * KC;
      walk.left -= KC;
    };

    // operand addresses in a stage: K row fr of a 16-row group, piece 4 k + g;
    // V rows 4 g + fr / 4 (and 16 further), 8 bytes of dims 16 j + 4 (fr % 4)
    int kat[kDK], vat[kND];
#pragma unroll
    for (int k = 0; k < kDK; ++k) kat[k] = (fr * kPieces + ((4 * k + g) ^ (fr & (kPieces - 1)))) * 16;
    const int vkey = 4 * g + (fr >> 2);
#pragma unroll
    for (int j = 0; j < kND; ++j)
      vat[j] = kMat + vkey * D * 2 + (((2 * j + ((fr & 3) >> 1)) ^ v_turn<D>(vkey)) << 4) + (fr & 1) * 8;
    bf16x8 ones;
#pragma unroll
    for (int e = 0; e < 8; ++e) ones[e] = static_cast<__bf16>(1.f);

    auto step = [&](int c, auto buf) {
      const unsigned char* st = lds + buf * kStage;
      __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0): this wave's loads of chunk c landed
      __syncthreads();                     // everyone's, and chunk c - 1 is read
      if (c + 1 < nc) load(c + 1, 1 - buf);
      const bool pre = c < nprefix;
      const int base = pre ? p0 + c * KC : s0 + (c - nprefix) * KC;
      const int end = pre ? p1 : own_end;
      unsigned long long bits = ~0ull;
      if (!pre && p.mask) {
        // masked values may hold anything: they enter the product as zeros
        const bool on = base + lane < end && p.mask[(long long)b_own * p.S + base + lane] != 0;
        bits = __ballot(on);
        unsigned char* z = lds + buf * kStage + kMat;
        for (int i = tid; i < KC * kPieces; i += 64 * WR)
          if (!((bits >> (i / kPieces)) & 1)) *reinterpret_cast<u32x4*>(z + i * 16) = u32x4{0u, 0u, 0u, 0u};
        __syncthreads();
      }
      if (idle) return;
      // S^T = K Q^T, the next 16 keys' operands read ahead of their products
      f32x4 sc[QT][kNT];
      bf16x8 kf[2][kDK];
      auto read_k = [&](int t) {
#pragma unroll
        for (int k = 0; k < kDK; ++k)
          kf[t & 1][k] = frag(*reinterpret_cast<const u32x4*>(st + kat[k] + t * 16 * D * 2));
      };
      read_k(0);
#pragma unroll
      for (int t = 0; t < kNT; ++t) {
        if (t + 1 < kNT) read_k(t + 1);
#pragma unroll
        for (int u = 0; u < QT; ++u) sc[u][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < kDK; ++k)
#pragma unroll
          for (int u = 0; u < QT; ++u)
            sc[u][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf[t & 1][k], qf[u][k], sc[u][t], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
      // keys that no row or not every row sees
      if (base + KC > (pre ? end : all_see) || (!pre && p.mask)) {
#pragma unroll
        for (int u = 0; u < QT; ++u) {
          // bits of this lane's keys 16 t + 4 g + e, from the first one on
          const int seen = min(max((pre ? end : min(end, row[u].lim)) - base, 0), KC);
          const unsigned long long mine = (seen < KC ? bits & ((1ull << seen) - 1ull) : bits) >> (4 * g);
#pragma unroll
          for (int t = 0; t < kNT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t keep = (uint32_t)__builtin_amdgcn_sbfe((int)(t < 2 ? mine : mine >> 32), (16 * t + e) & 31, 1);
              sc[u][t][e] = __uint_as_float((__float_as_uint(sc[u][t][e]) & keep) | (0xff800000u & ~keep));
            }
        }
      }
      uint32_t pk[QT][kNT][2];
      auto exponents = [&](auto any_size) -> bool {
        u16x2 top = {0, 0};
#pragma unroll
        for (int u = 0; u < QT; ++u) {
          const float ref = m[u];
          const bool far = any_size && far_out(ref);
#pragma unroll
          for (int t = 0; t < kNT; ++t) {
            float e4[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) e4[e] = __builtin_amdgcn_exp2f(passed(sc[u][t][e], p.c, ref, far));
            pk[u][t][0] = bf16_pair(e4[0], e4[1]);
            pk[u][t][1] = bf16_pair(e4[2], e4[3]);
            top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, pk[u][t][0]));
            top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, pk[u][t][1]));
          }
        }
        return max(top[0], top[1]) >= kSlackBits;
      };
      bool move = c == 0 || wary;
      if (!move) move = __any(exponents(std::false_type{}));
      if (move) {
        bool far = false;
#pragma unroll
        for (int u = 0; u < QT; ++u) {
          float x = -INFINITY;
#pragma unroll
          for (int t = 0; t < kNT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) x = fmaxf(x, sc[u][t][e]);
          x = group_max(x);
          // base-2 scores (c > 0), passed as the exponents above see it
          const float mn = passed(x, p.c, m[u], far_out(m[u])) > kSlack ? x * p.c : m[u];
          const float alpha = __builtin_amdgcn_exp2f(m[u] - mn);
          m[u] = mn;
          far = far || far_out(mn);
          l[u] *= alpha;
#pragma unroll
          for (int j = 0; j < kND; ++j) o[u][j] *= alpha;
        }
        wary = __any(far);
        exponents(std::true_type{});
      }
      // O^T += V^T P^T: k-slots 8 g .. 8 g + 7 carry keys 32 c + 4 g + (0..3)
      // and 32 c + 16 + 4 g + (0..3) on both sides; a row of ones in the place
      // of V^T gives l, the sum of the probabilities as the product takes them
      constexpr int kGroup = 4, kPer = kND / kGroup, kGroups = KC / 32 * kPer;  // of four 16-dim columns
      bf16x8 vf[2][kGroup];
      auto read_v = [&](int n) {
#pragma unroll
        for (int j = 0; j < kGroup; ++j) {
          const unsigned char* v = st + vat[(n % kPer) * kGroup + j] + (n / kPer) * 32 * D * 2;
          const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)v);
          const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(v + 16 * D * 2));
          const u32x2 l2 = __builtin_bit_cast(u32x2, lo), h2 = __builtin_bit_cast(u32x2, hi);
          vf[n & 1][j] = frag(u32x4{l2[0], l2[1], h2[0], h2[1]});
        }
      };
      read_v(0);
#pragma unroll
      for (int n = 0; n < kGroups; ++n) {
        if (n + 1 < kGroups) read_v(n + 1);
        const int cc = n / kPer;
        bf16x8 pf[QT];
#pragma unroll
        for (int u = 0; u < QT; ++u) {
          pf[u] = frag(u32x4{pk[u][2 * cc][0], pk[u][2 * cc][1], pk[u][2 * cc + 1][0], pk[u][2 * cc + 1][1]});
          if (n % kPer == 0) l[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, pf[u], l[u], 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < kGroup; ++j)
#pragma unroll
          for (int u = 0; u < QT; ++u) {
            f32x4& acc = o[u][(n % kPer) * kGroup + j];
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf[n & 1][j], pf[u], acc, 0, 0, 0);
          }
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    if (nc > 0) load(0, 0);
    for (int c = 0; c < nc; c += 2) {
      step(c, std::integral_constant<int, 0>{});
      if (c + 1 < nc) step(c + 1, std::integral_constant<int, 1>{});
    }

#pragma unroll
    for (int u = 0; u < QT; ++u) write_row<D>(p, w, row[u], g, m[u], l[u][0], o[u], nc > 0);
  }
};

// One part of a list of keys n, cut at multiples of `unit` (n rounded up to
// that may pass 2^31: prefix and own keys have up to 2^30 each).
__device__ __forceinline__ void part_range(int n, int parts, int part, int unit, int& lo, int& hi) {
  const long long nu = ((long long)n + unit - 1) / unit;
  lo = (int)min(nu * part / parts * unit, (long long)n);
  hi = (int)min(nu * (part + 1) / parts * unit, (long long)n);
}

template <int D>
using Wide = WideTile<D, 4, 2>;

constexpr int kMostPacked = 1024;  // sequences whose packed rows a workgroup looks up

// Item `item` of a list: key heads innermost, so that neighbours in the list
// (dealt round-robin over the XCDs) read different heads, and the tiles of one
// head and part, which read the same keys, meet in one L2.
template <class T>
__device__ __forceinline__ void run_item(const PaParams& p, const List& list, unsigned char* lds, int item) {
  const int tiles = list.tiles, parts = list.parts;
  TileWork w;
  w.hk = item % p.Hk;
  const int rest = item / p.Hk;
  const int tile = rest % tiles, part = rest / tiles;
  w.b = -1;
  w.packed = T::kPacked && !list.seq;
  const int* cum = nullptr;
  if (!w.packed) {
    const int per = tiles / p.B;
    int b = tile / per, first = (tile - b * per) * T::kRows;
    if (p.causal) {
      // every sequence's last rows, which see the most keys, come first, and the
      // short ones fill the gaps at the end (8 x 1024 rows, 16 heads of 128, no
      // prefix: 65 -> 53 us; 32 heads, 8 of keys, behind 8192 1125 -> 1083; but
      // 33 x 464 rows of 120 heads of 64, 15 of keys, no prefix 239 -> 251, as own
      // keys leave L2 between their tiles)
      const int turned = tiles - 1 - tile;
      b = turned % p.B;
      first = turned / p.B * T::kRows;
    }
    w.row0 = b * p.RS + first;
    w.n = min(query_length(p, b) * p.G - first, T::kRows);
    if (list.keys != 0) w.b = b;
  } else {
    int rows = p.RT;
    if (p.q_len) {
      // packed rows before each sequence: a running sum, 256 sequences at a time
      int* c = reinterpret_cast<int*>(lds);
      int* part_sum = c + kMostPacked + 1;
      const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
      int carry = 0;
      for (int b0 = 0; b0 < p.B; b0 += 256) {
        const int b = b0 + tid;
        int n = tid < 256 && b < p.B ? query_length(p, b) * p.G : 0, x = n;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
          const int y = __shfl_up(x, d);
          if (lane >= d) x += y;
        }
        if (lane == 63 && wave < 4) part_sum[wave] = x;
        __syncthreads();
        int before = carry;
        for (int v = 0; v < 4; ++v) {
          if (v < wave) before += part_sum[v];
          carry += part_sum[v];
        }
        if (tid < 256 && b < p.B) c[b] = before + x - n;
        __syncthreads();
      }
      if (tid == 0) c[p.B] = carry;
      __syncthreads();
      rows = carry;
      cum = c;
    }
    w.row0 = tile * T::kRows;
    w.n = min(rows - w.row0, T::kRows);
  }
  if (w.n <= 0) return;
  w.p0 = w.p1 = w.s0 = w.s1 = 0;
  w.slot = list.slot + part;
  if (list.keys == 0) {
    part_range(p.P, parts, part, 64, w.p0, w.p1);
  } else if (list.keys == 1) {
    part_range(p.S, parts, part, 64, w.s0, w.s1);
  } else {
    // prefix (rounded up to whole chunks) and own keys as one list
    const int pp = (p.P + 63) & ~63;
    int lo, hi;
    part_range(pp + p.S, parts, part, 64, lo, hi);
    w.p0 = min(lo, p.P);
    w.p1 = min(hi, p.P);
    w.s0 = max(lo - pp, 0);
    w.s1 = max(hi - pp, 0);
  }
  T::run(p, w, lds, cum);
}

// Both lists in one launch: thin items, which wait for memory, run beside wide
// ones, which compute, and short ones fill in behind long ones.
template <int D>
__global__ __launch_bounds__(256, 2) void prefix_mixed_kernel(PaParams p) {
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  const int bid = blockIdx.x;
  if (bid < p.first.n) run_item<Wide<D>>(p, p.first, lds, bid);
  else run_item<ThinTile<D, 4>>(p, p.second, lds, bid - p.first.n);
}

template <int D>
__global__ __launch_bounds__(256, 2) void prefix_wide_kernel(PaParams p) {
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  const int bid = blockIdx.x;
  const bool second = bid >= p.first.n;
  run_item<Wide<D>>(p, second ? p.second : p.first, lds, second ? bid - p.first.n : bid);
}

template <int D>
__global__ __launch_bounds__(512, 4) void prefix_thin_kernel(PaParams p) {
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  run_item<ThinTile<D, 8>>(p, p.first, lds, blockIdx.x);
}

// Joins a row's partial results, D / 4 lanes a row: kGroups groups of slots
// side by side (four loads of each in flight together), then the groups in
// order. Up to eight slots take one group.
template <int D, int kGroups>
__global__ __launch_bounds__(256) void prefix_join_kernel(PaParams p) {
  constexpr int LPR = D / 4, kRowsWg = 256 / (LPR * kGroups);
  __shared__ f32x4 so[kGroups][kRowsWg][LPR];
  __shared__ float sl[kGroups][kRowsWg];
  const int lane = threadIdx.x % LPR, grp = threadIdx.x / LPR % kGroups, rw = threadIdx.x / (LPR * kGroups);
  const long long rows = (long long)p.Hk * p.RT;
  const long long row = min((long long)blockIdx.x * kRowsWg + rw, rows - 1);  // hk * RT + R
  const int hk = (int)(row / p.RT), R = (int)(row - (long long)hk * p.RT);
  const int b = (int)((unsigned)R / (unsigned)p.RS), rr = R - b * p.RS, t = (int)((unsigned)rr / (unsigned)p.G);
  const bool used = (long long)blockIdx.x * kRowsWg + rw < rows && t < query_length(p, b);
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  float l = 0.f;
  // the lanes look at the slots' maxima side by side
  float m = -INFINITY;
  for (int s = lane; s < p.slots; s += LPR) m = fmaxf(m, p.ml[2 * (s * rows + row)]);
#pragma unroll
  for (int d = 1; d < LPR; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
  const float ref = m == -INFINITY ? 0.f : m;
  if (used) {
    constexpr int U = 4;  // slots whose loads are in flight together
    for (int s0 = grp; s0 < p.slots; s0 += U * kGroups) {
      f32x2 x[U];
      f32x4 y[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const long long at = min(s0 + u * kGroups, p.slots - 1) * rows + row;
        x[u] = *reinterpret_cast<const f32x2*>(p.ml + 2 * at);
        y[u] = *reinterpret_cast<const f32x4*>(p.po + at * D + 4 * lane);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (s0 + u * kGroups >= p.slots || !(x[u][1] > 0.f)) continue;  // nothing there, O not written
        const float wgt = __builtin_amdgcn_exp2f(x[u][0] - ref);
        l = fmaf(x[u][1], wgt, l);
        o += y[u] * wgt;
      }
    }
  }
  so[grp][rw][lane] = o;
  if (lane == 0) sl[grp][rw] = l;
  __syncthreads();
  if (grp > 0 || !used) return;
#pragma unroll
  for (int v = 1; v < kGroups; ++v) {
    o += so[v][rw][lane];
    l += sl[v][rw];
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  const int h = hk * p.G + (rr - t * p.G);
  uint16_t* dst = static_cast<uint16_t*>(p.out.p) + (long long)b * p.out.b + (long long)t * p.out.t +
                  (long long)h * p.out.h + 4 * lane;
  *reinterpret_cast<u32x2*>(dst) = u32x2{bf16_pair(o[0] * inv, o[1] * inv), bf16_pair(o[2] * inv, o[3] * inv)};
}

// How the rows and keys are dealt to workgroups: from the sizes alone, so
// the workspace's size follows from them too.
struct Plan {
  List first, second;
  int slots;
};

int cdiv(long long a, long long b) { return (int)((a + b - 1) / b); }

// Parts of n keys so that about `want` workgroups run, none under `least` keys.
int parts_for(long long n, long long items, long long want, long long least) {
  long long parts = items > 0 ? (want + items - 1) / items : 1;
  const long long most = (n + least - 1) / least;
  if (parts > most) parts = most;
  return (int)(parts < 1 ? 1 : parts);
}

// Parts for wide tiles within sequences, 512 of which run at a time: as many
// as fit into one round, if that is filled to four fifths, else about a round
// and a half, and never a little over one: 2 x 300 rows of 16 heads of 128
// behind 9000 keys, 96 tiles, take 71 us in 5 parts and 88 in 6.
int wide_parts(long long n, long long items) {
  const long long fit = 512 / (items > 0 ? items : 1);
  return parts_for(n, items, fit * items * 5 >= 512 * 4 ? fit * items : 768, 256);
}

Plan make_plan(int B, int Tq, int Hq, int Hk, int P, int S) {
  Plan pl{};
  const int G = Hq / Hk;
  const long long RS = (long long)Tq * G, RT = (long long)B * RS;
  auto list = [&](int wide, int seq, int keys, int tiles, int parts, int slot) {
    return List{wide, seq, keys, tiles, parts, slot, (int)((long long)tiles * Hk * parts)};
  };
  // Packing the rows of all sequences reads the prefix once for 128 of them
  // and costs a second list of items, partial results and a join; tiles within
  // a sequence leave 128 - RS of their rows empty instead. Measured (us, packed
  // / in sequence): 64 x 1 row of 16 heads of 64 behind 4096 keys 17 / 80,
  // behind 256 14 / 12; two sequences behind 16384 20 / 20; 37 x 80 rows behind
  // 2304 53 / 69, and with half of them in use (q_len) 40 / 65; 64 x 96 rows of 8
  // heads of 128 behind 8192 229 / 242, behind 2304 88 / 77; 8 x 80 rows behind
  // 2304 27 / 27. The rule sees neither the rows in use nor the heads: 37 x 80
  // rows, half in use, behind 1024 stay in sequence, 31 / 41. It asks for own
  // keys, and for 1024 sequences at most, whose lengths fit LDS: prefix keys
  // alone, or longer batches, take tiles in sequence.
  // (The last limit keeps the join's threads below 2^32.)
  const bool packed = S > 0 && B <= kMostPacked && RT * Hk < (1 << 25) &&
                      (RS <= 16 ? B >= 4 && P >= 1024
                                : B >= 16 && RS < 128 && P >= 2048 && (128 - RS) * P >= 90000);
  if (!packed) {
    // every tile stays in its sequence and takes prefix and own keys
    const int wide = RS > 16, tiles = B * cdiv(RS, wide ? 128 : 16);
    const int parts = wide ? wide_parts((long long)P + S, (long long)tiles * Hk)
                           : parts_for((long long)P + S, (long long)tiles * Hk, 256, (long long)P + S <= 1024 ? 1024 : 512);
    pl.first = list(wide, 1, 2, tiles, parts, 0);
    pl.slots = parts;
    return pl;
  }
  // the prefix for the rows of all sequences together, own keys apart
  // (beside thin items one wide one a CU: with 512 the 48 sequences with 1024
  // own keys behind 32768 take 83 instead of 75 us; but where own keys are
  // few, 384: 16 sequences with 256 behind 65536 61 instead of 69 us; among
  // wide ones half as many again as the CUs hold, which fill each other's gaps:
  // 37 x 80 rows of 8 heads of 128 behind 8192 125 us, with 512 149, with 1024 137)
  const int wide = RS > 16, tiles = cdiv(RT, 128);
  const int parts = parts_for(P, (long long)tiles * Hk, wide ? 768 : P / 64 >= S ? 384 : 256, 256);
  pl.first = list(1, 0, 0, tiles, parts, 0);
  const int own_tiles = B * cdiv(RS, wide ? 128 : 16);
  pl.second = list(wide, 1, 1, own_tiles, parts_for(S, (long long)own_tiles * Hk, 256, 256), parts);
  pl.slots = parts + pl.second.parts;
  return pl;
}

size_t al256(size_t n) { return (n + 255) & ~(size_t)255; }

template <int D>
hipError_t run(const PaParams& p, const Plan& pl, hipStream_t st) {
  const dim3 grid((unsigned)(pl.first.n + pl.second.n));
  constexpr int wide = Wide<D>::kLds, thin4 = ThinTile<D, 4>::kLds, thin8 = ThinTile<D, 8>::kLds;
  if (!pl.first.wide)
    hipLaunchKernelGGL((prefix_thin_kernel<D>), grid, dim3(512), thin8, st, p);
  else if (pl.second.n == 0 || pl.second.wide)
    hipLaunchKernelGGL((prefix_wide_kernel<D>), grid, dim3(256), wide, st, p);
  else
    hipLaunchKernelGGL((prefix_mixed_kernel<D>), grid, dim3(256), wide > thin4 ? wide : thin4, st, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || pl.slots == 1) return e;
  const long long rows = (long long)p.Hk * p.RT;
  constexpr int many = 256 / D, few = 1024 / D;  // rows a workgroup
  if (pl.slots > 8)
    hipLaunchKernelGGL((prefix_join_kernel<D, 4>), dim3((unsigned)cdiv(rows, many)), dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL((prefix_join_kernel<D, 1>), dim3((unsigned)cdiv(rows, few)), dim3(256), 0, st, p);
  return hipGetLastError();
}

}  // namespace

size_t prefix_attn_workspace_bytes(int B, int Tq, int Hq, int Hk, int D, int P, int S) {
  const Plan pl = make_plan(B, Tq, Hq, Hk, P, S);
  if (pl.slots == 1) return 0;
  const size_t rows = (size_t)pl.slots * B * Tq * Hq;
  return al256(rows * D * 4) + al256(rows * 8);
}

hipError_t launch_prefix_attn(const PrefixAttnArgs& a, hipStream_t st) {
  const Plan pl = make_plan(a.B, a.Tq, a.Hq, a.Hk, a.P, a.S);
  PaParams p{};
  p.q = a.q;
  p.kp = a.kp;
  p.vp = a.vp;
  p.ko = a.ko;
  p.vo = a.vo;
  p.out = a.out;
  p.P = a.P;
  p.S = a.S;
  p.own_len = a.own_len;
  p.q_len = a.q_len;
  p.mask = a.mask;
  p.B = a.B;
  p.Tq = a.Tq;
  p.Hk = a.Hk;
  p.G = a.Hq / a.Hk;
  p.RS = a.Tq * p.G;
  p.RT = a.B * p.RS;
  p.c = a.scale * 1.4426950408889634f;
  p.causal = a.causal;
  p.first = pl.first;
  p.second = pl.second;
  p.slots = pl.slots;
  if (pl.slots > 1) {
    const size_t rows = (size_t)pl.slots * a.B * a.Tq * a.Hq;
    p.po = static_cast<float*>(a.ws);
    p.ml = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + al256(rows * a.D * 4));
  }
  return a.D == 64 ? run<64>(p, pl, st) : run<128>(p, pl, st);
}

}  // namespace gkd
