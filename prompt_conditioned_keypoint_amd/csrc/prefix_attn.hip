// prefix_attn.hip - attention of a batch that shares one long prefix of keys
// (gkd_prefix_attention).
//
// A row is one query of one query head; the rows of a key head are numbered
// R = (b Tq + t) G + g (G = Hq / Hk query heads share the key head). The
// softmax runs online: a row keeps its running maximum m, the sum l of
// exp(s - m) and the output O scaled alike, and ranges of keys that were
// taken apart are joined by
//   m = max_i m_i,  l = sum_i l_i exp(m_i - m),  O = sum_i O_i exp(m_i - m).
// So the prefix can be taken once for the rows of all sequences together
// (their keys pass through LDS once per tile of rows, not once per
// sequence), own keys sequence by sequence, and long ranges in parts.
//
// Two tiles, of 256 threads each:
//   wide   128 rows, four waves of 32 rows, key chunks of 64 shared by them;
//   thin   16 rows, four waves that take every fourth 32-key chunk and join
//          at the end: for few rows, where reading the keys is all there is.
#include "gkd_device.hpp"
#include "tokens_launch.hpp"

#include <type_traits>

namespace gkd {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) void lds_void;

struct PaParams {
  Heads q, kp, vp, ko, vo, out;
  int P, S;
  const int32_t *own_len, *q_len;
  const uint8_t* mask;
  int B, Tq, Hk, G;
  int RS, RT;          // rows of a sequence, of all sequences (per key head)
  float c;             // scale * log2(e)
  int causal;
  // the plan: wide items first, then thin ones; an item list is [part][tile][key head]
  int wide_seq, thin_seq;      // its tiles stay within a sequence
  int wide_tiles, thin_tiles;  // tiles of rows per key head
  int wide_parts, thin_parts;
  int wide_own, thin_own;      // 0: prefix keys, 1: own keys, 2: both, prefix first
  int n_wide;                  // workgroups of the wide list
  int slots;                   // partial results a row has; 1: written as they are
  int thin_slot;               // first slot of the thin list
  float* po;                   // [slots][Hk][RT][D]
  float* ml;                   // [slots][Hk][RT][2]
};

__device__ __forceinline__ bf16x8 frag(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

template <int D, int WR, int WK, int QT, int KC>
struct ThinTile {
  static constexpr int kRows = 16 * QT * WR;
  static constexpr int kPieces = D / 8;                       // 16-byte pieces of a key row
  static constexpr int kNP = KC * kPieces / (64 * WR);        // pieces a thread stages, K and V each
  static constexpr int kMat = KC * D * 2;                     // bytes of a chunk's K (or V)
  static constexpr int kStage = WK * 2 * kMat;
  static constexpr int kLds = 2 * kStage;
  static constexpr int kNT = KC / 16, kDK = D / 32, kND = D / 16;

  static __device__ __forceinline__ void run(const PaParams& p, unsigned char* lds, int hk, int b_own,
                                             int row0, int row_end, int p0, int p1, int s0, int s1,
                                             int slot) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wr = wave % WR, wk = wave / WR;
    const int fr = lane & 15, g = lane >> 4;
    const int tidc = wr * 64 + lane;  // thread within its key column

    // this lane's rows (query fr of each of its 16-row groups)
    bf16x8 qf[QT][kDK];
    int R[QT];
    bool live[QT];
    int lim[QT];      // own keys below this are visible
    long long oaddr[QT];
    int own_end = s1;
#pragma unroll
    for (int u = 0; u < QT; ++u) {
      live[u] = (wr * QT + u) * 16 + fr < row_end - row0;
      R[u] = live[u] ? row0 + (wr * QT + u) * 16 + fr : row_end - 1;
      const int b = (int)((unsigned)R[u] / (unsigned)p.RS), rr = R[u] - b * p.RS;
      const int t = (int)((unsigned)rr / (unsigned)p.G), h = hk * p.G + (rr - t * p.G);
      const int ql = p.q_len ? min(max(p.q_len[b], 0), p.Tq) : p.Tq;
      live[u] = live[u] && t < ql;
      lim[u] = 0x7fffffff;
      if (p.causal && b_own >= 0) {
        const int len = p.own_len ? min(max(p.own_len[b], 0), p.S) : p.S;
        lim[u] = len - ql + t + 1;
      }
      const uint16_t* src = static_cast<const uint16_t*>(p.q.p) + b * p.q.b + t * p.q.t + h * p.q.h;
#pragma unroll
      for (int k = 0; k < kDK; ++k)
        qf[u][k] = frag(*reinterpret_cast<const u32x4*>(src + 32 * k + 8 * g));
      oaddr[u] = b * p.out.b + t * p.out.t + h * p.out.h;
    }
    if (b_own >= 0) {
      own_end = min(s1, p.own_len ? min(max(p.own_len[b_own], 0), p.S) : p.S);
      if (p.causal) {  // no row of the tile sees past its last one's limit
        const int first = row0 - b_own * p.RS, last = min(first + kRows, row_end - b_own * p.RS) - 1;
        const int t = (int)((unsigned)last / (unsigned)p.G);
        const int ql = p.q_len ? min(max(p.q_len[b_own], 0), p.Tq) : p.Tq;
        const int len = p.own_len ? min(max(p.own_len[b_own], 0), p.S) : p.S;
        own_end = min(own_end, len - ql + t + 1);
      }
    }
    const int nprefix = p1 > p0 ? (p1 - p0 + KC - 1) / KC : 0;
    const int nown = own_end > s0 ? (own_end - s0 + KC - 1) / KC : 0;
    const int nc = nprefix + nown;
    const int nit = (nc + WK - 1) / WK;

    f32x4 o[QT][kND];
    float m[QT], l[QT];
#pragma unroll
    for (int u = 0; u < QT; ++u) {
      m[u] = -INFINITY;
      l[u] = 0.f;
#pragma unroll
      for (int j = 0; j < kND; ++j) o[u][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    u32x4 kreg[kNP], vreg[kNP];
    // chunk c of this column: where its keys are
    auto load = [&](int it) {
      const int c = it * WK + wk;
      const u32x4 z = {0u, 0u, 0u, 0u};
      const bool pre = c < nprefix;
      const int base = pre ? p0 + c * KC : s0 + (c - nprefix) * KC;
      const int end = c >= nc ? base : pre ? p1 : own_end;
      const Heads& hk_ = pre ? p.kp : p.ko;
      const Heads& hv_ = pre ? p.vp : p.vo;
      const long long ob = pre ? 0 : (long long)b_own;
      const uint16_t* ks = static_cast<const uint16_t*>(hk_.p) + ob * hk_.b + hk * hk_.h;
      const uint16_t* vs = static_cast<const uint16_t*>(hv_.p) + ob * hv_.b + hk * hv_.h;
#pragma unroll
      for (int i = 0; i < kNP; ++i) {
        const int s = tidc + 64 * WR * i, r = s / kPieces, pc = s % kPieces;
        const long long key = base + r;
        bool in = key < end;
        kreg[i] = vreg[i] = z;
        if (in) {
          kreg[i] = *reinterpret_cast<const u32x4*>(ks + key * hk_.t + 8 * pc);
          // masked values may hold anything: they enter the product as zeros
          if (!pre && p.mask) in = p.mask[ob * p.S + key] != 0;
          if (in) vreg[i] = *reinterpret_cast<const u32x4*>(vs + key * hv_.t + 8 * pc);
        }
      }
    };
    auto store = [&](int buf) {
      unsigned char* st = lds + buf * kStage + wk * 2 * kMat;
#pragma unroll
      for (int i = 0; i < kNP; ++i) {
        const int s = tidc + 64 * WR * i, r = s / kPieces, pc = s % kPieces;
        const int at = (r * kPieces + (pc ^ (r & (kPieces - 1)))) * 16;
        *reinterpret_cast<u32x4*>(st + at) = kreg[i];
        *reinterpret_cast<u32x4*>(st + kMat + at) = vreg[i];
      }
    };

    if (nit > 0) {
      load(0);
      store(0);
    }
    __syncthreads();
    for (int it = 0; it < nit; ++it) {
      if (it + 1 < nit) load(it + 1);
      const int c = it * WK + wk;
      if (c < nc) {
        const unsigned char* sK = lds + (it & 1) * kStage + wk * 2 * kMat;
        const unsigned char* sV = sK + kMat;
        const bool pre = c < nprefix;
        const int base = pre ? p0 + c * KC : s0 + (c - nprefix) * KC;
        const int end = pre ? p1 : own_end;
        f32x4 sc[QT][kNT];
#pragma unroll
        for (int t = 0; t < kNT; ++t) {
#pragma unroll
          for (int u = 0; u < QT; ++u) sc[u][t] = f32x4{0.f, 0.f, 0.f, 0.f};
          const int kr = 16 * t + fr;
#pragma unroll
          for (int k = 0; k < kDK; ++k) {
            const bf16x8 kf = frag(*reinterpret_cast<const u32x4*>(
                sK + (kr * kPieces + ((4 * k + g) ^ (kr & (kPieces - 1)))) * 16));
#pragma unroll
            for (int u = 0; u < QT; ++u)
              sc[u][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[u][k], sc[u][t], 0, 0, 0);
          }
        }
        // keys that no row or not every row sees
        if (base + KC > end || (!pre && (p.causal || p.mask))) {
          unsigned long long bits = ~0ull;
          if (!pre && p.mask) {
            const bool on = base + lane < end && lane < KC && p.mask[(long long)b_own * p.S + base + lane] != 0;
            bits = __ballot(on);
          }
#pragma unroll
          for (int u = 0; u < QT; ++u) {
            const int stop = pre ? end : min(end, lim[u]);
#pragma unroll
            for (int t = 0; t < kNT; ++t)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int kk = 16 * t + 4 * g + e;
                if (base + kk >= stop || !((bits >> kk) & 1)) sc[u][t][e] = -INFINITY;
              }
          }
        }
        uint32_t pk[QT][kNT][2];
#pragma unroll
        for (int u = 0; u < QT; ++u) {
          float cm = -INFINITY;
#pragma unroll
          for (int t = 0; t < kNT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) cm = fmaxf(cm, sc[u][t][e]);
          cm = fmaxf(cm, __shfl_xor(cm, 16));
          cm = fmaxf(cm, __shfl_xor(cm, 32));
          cm *= p.c;  // base-2 scores (c > 0)
          const float mn = fmaxf(m[u], cm);
          const float ref = mn == -INFINITY ? 0.f : mn;
          const float alpha = __builtin_amdgcn_exp2f(m[u] - ref);
          m[u] = mn;
          float ps = 0.f;
#pragma unroll
          for (int t = 0; t < kNT; ++t) {
            float e4[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              e4[e] = __builtin_amdgcn_exp2f(fmaf(sc[u][t][e], p.c, -ref));
              ps += e4[e];
            }
            const bf16x2 lo = {static_cast<__bf16>(e4[0]), static_cast<__bf16>(e4[1])};
            const bf16x2 hi = {static_cast<__bf16>(e4[2]), static_cast<__bf16>(e4[3])};
            pk[u][t][0] = __builtin_bit_cast(uint32_t, lo);
            pk[u][t][1] = __builtin_bit_cast(uint32_t, hi);
          }
          l[u] = l[u] * alpha + ps;
#pragma unroll
          for (int j = 0; j < kND; ++j) o[u][j] *= alpha;
        }
        // O^T += V^T P^T: k-slots 8 g .. 8 g + 7 carry keys 32 c + 4 g + (0..3)
        // and 32 c + 16 + 4 g + (0..3) on both sides
        const int vkey = 4 * g + (fr >> 2);
#pragma unroll
        for (int cc = 0; cc < KC / 32; ++cc) {
          const int kr = 32 * cc + vkey;
          const unsigned char* vrow = sV + kr * D * 2 + (fr & 1) * 8;
#pragma unroll
          for (int j = 0; j < kND; ++j) {
            const int pc = 2 * j + ((fr & 3) >> 1);
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_s16x4*)(vrow + ((pc ^ (kr & (kPieces - 1))) << 4)));
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_s16x4*)(vrow + 16 * D * 2 + ((pc ^ ((kr + 16) & (kPieces - 1))) << 4)));
            const u32x2 l2 = __builtin_bit_cast(u32x2, lo), h2 = __builtin_bit_cast(u32x2, hi);
            const bf16x8 vf = frag(u32x4{l2[0], l2[1], h2[0], h2[1]});
#pragma unroll
            for (int u = 0; u < QT; ++u)
              o[u][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  vf, frag(u32x4{pk[u][2 * cc][0], pk[u][2 * cc][1], pk[u][2 * cc + 1][0], pk[u][2 * cc + 1][1]}),
                  o[u][j], 0, 0, 0);
          }
        }
      }
      if (it + 1 < nit) store((it + 1) & 1);
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < QT; ++u) {
      l[u] += __shfl_xor(l[u], 16);
      l[u] += __shfl_xor(l[u], 32);
    }

    if constexpr (WK > 1) {
      // the columns join in LDS, in order
      constexpr int kPer = QT * kND * 64;  // f32x4 a wave
      static_assert((WK - 1) * WR * (kPer * 16 + QT * 64 * 8) <= kLds, "the joined results fit");
      f32x4* so = reinterpret_cast<f32x4*>(lds);
      f32x2* sm = reinterpret_cast<f32x2*>(lds + (WK - 1) * WR * kPer * 16);
      if (wk > 0) {
        const int w = (wk - 1) * WR + wr;
#pragma unroll
        for (int u = 0; u < QT; ++u) {
#pragma unroll
          for (int j = 0; j < kND; ++j) so[w * kPer + (u * kND + j) * 64 + lane] = o[u][j];
          sm[(w * QT + u) * 64 + lane] = f32x2{m[u], l[u]};
        }
      }
      __syncthreads();
      if (wk > 0) return;
#pragma unroll
      for (int v = 0; v < WK - 1; ++v) {
        const int w = v * WR + wr;
#pragma unroll
        for (int u = 0; u < QT; ++u) {
          const f32x2 x = sm[(w * QT + u) * 64 + lane];
          const float mn = fmaxf(m[u], x[0]);
          const float ref = mn == -INFINITY ? 0.f : mn;
          const float a = __builtin_amdgcn_exp2f(m[u] - ref), bsc = __builtin_amdgcn_exp2f(x[0] - ref);
          m[u] = mn;
          l[u] = l[u] * a + x[1] * bsc;
#pragma unroll
          for (int j = 0; j < kND; ++j) o[u][j] = o[u][j] * a + so[w * kPer + (u * kND + j) * 64 + lane] * bsc;
        }
      }
    }

    // o[u][j][e] = O^T[dim 16 j + 4 g + e][row]
#pragma unroll
    for (int u = 0; u < QT; ++u) {
      if (!live[u]) continue;
      if (p.slots == 1) {
        const float inv = l[u] > 0.f ? 1.f / l[u] : 0.f;
        uint16_t* dst = static_cast<uint16_t*>(p.out.p) + oaddr[u] + 4 * g;
#pragma unroll
        for (int j = 0; j < kND; ++j) {
          const bf16x2 lo = {static_cast<__bf16>(o[u][j][0] * inv), static_cast<__bf16>(o[u][j][1] * inv)};
          const bf16x2 hi = {static_cast<__bf16>(o[u][j][2] * inv), static_cast<__bf16>(o[u][j][3] * inv)};
          *reinterpret_cast<u32x2*>(dst + 16 * j) =
              u32x2{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
        }
      } else {
        const long long at = ((long long)slot * p.Hk + hk) * p.RT + R[u];
        if (g == 0) *reinterpret_cast<f32x2*>(p.ml + 2 * at) = f32x2{m[u], l[u]};
        if (nc == 0) continue;  // the statistics say that there is nothing
#pragma unroll
        for (int j = 0; j < kND; ++j) *reinterpret_cast<f32x4*>(p.po + at * D + 16 * j + 4 * g) = o[u][j];
      }
    }
  }
};

// max over the four 16-lane groups of a wave
__device__ __forceinline__ float group_max(float x) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

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

template <int D, int WR, int QT>
struct WideTile {
  static constexpr int KC = 64;
  static constexpr int kRows = 16 * QT * WR;
  static constexpr int kPieces = D / 8;                 // 16-byte pieces of a key row
  static constexpr int kMat = KC * D * 2;               // bytes of a chunk's K (or V)
  static constexpr int kStage = 2 * kMat;
  static constexpr int kLds = 2 * kStage;
  static constexpr int kNT = KC / 16, kDK = D / 32, kND = D / 16;
  static constexpr int kLoads = kMat / (WR * 1024);     // 1-KB loads a wave and matrix
  static constexpr int kBlkRows = 64 / kPieces;         // key rows of one load

  static __device__ __forceinline__ void run(const PaParams& p, unsigned char* lds, int hk, int b_own,
                                             int row0, int row_end, int p0, int p1, int s0, int s1,
                                             int slot) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wr = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int fr = lane & 15, g = lane >> 4;

    bf16x8 qf[QT][kDK];
    int lim[QT];      // own keys below this are visible
    bool live[QT];
    long long oaddr[QT];
#pragma unroll
    for (int u = 0; u < QT; ++u) {
      const int n = (wr * QT + u) * 16 + fr;
      live[u] = n < row_end - row0;
      const unsigned r = live[u] ? row0 + n : row_end - 1;
      const unsigned b = r / (unsigned)p.RS, rr = r - b * p.RS, t = rr / (unsigned)p.G;
      const int h = hk * p.G + (int)(rr - t * p.G);
      const int ql = p.q_len ? min(max(p.q_len[b], 0), p.Tq) : p.Tq;
      live[u] = live[u] && (int)t < ql;
      lim[u] = 0x7fffffff;
      if (p.causal && b_own >= 0) {
        const int len = p.own_len ? min(max(p.own_len[b], 0), p.S) : p.S;
        lim[u] = len - ql + (int)t + 1;
      }
      const uint16_t* src = static_cast<const uint16_t*>(p.q.p) + b * p.q.b + t * p.q.t + h * p.q.h;
#pragma unroll
      for (int k = 0; k < kDK; ++k)
        qf[u][k] = frag(live[u] ? *reinterpret_cast<const u32x4*>(src + 32 * k + 8 * g) : u32x4{0u, 0u, 0u, 0u});
      oaddr[u] = b * p.out.b + t * p.out.t + h * p.out.h;
    }
    int own_end = s1, all_see = s1;  // own keys of the tile; those that every row sees
    if (b_own >= 0) {
      const int len = p.own_len ? min(max(p.own_len[b_own], 0), p.S) : p.S;
      own_end = all_see = min(s1, len);
      if (p.causal) {
        const int ql = p.q_len ? min(max(p.q_len[b_own], 0), p.Tq) : p.Tq;
        const int first = row0 - b_own * p.RS, last = min(first + kRows, row_end - b_own * p.RS) - 1;
        own_end = min(own_end, len - ql + (int)((unsigned)last / (unsigned)p.G) + 1);
        all_see = min(all_see, len - ql + (int)((unsigned)first / (unsigned)p.G) + 1);
      }
    }
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
    const int lp = 16 * ((lane % kPieces) ^ (lr & (kPieces - 1)));
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
      off = (uint32_t)lr * (uint32_t)walk.vt * 2u + lp;
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
      vat[j] = kMat + vkey * D * 2 + (((2 * j + ((fr & 3) >> 1)) ^ (vkey & (kPieces - 1))) << 4) + (fr & 1) * 8;
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
          const int seen = min(max((pre ? end : min(end, lim[u])) - base, 0), KC);
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
      auto exponents = [&]() -> bool {
        u16x2 top = {0, 0};
#pragma unroll
        for (int u = 0; u < QT; ++u) {
          const float ref = m[u];
#pragma unroll
          for (int t = 0; t < kNT; ++t) {
            float e4[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) e4[e] = __builtin_amdgcn_exp2f(fmaf(sc[u][t][e], p.c, -ref));
            const bf16x2 lo = {static_cast<__bf16>(e4[0]), static_cast<__bf16>(e4[1])};
            const bf16x2 hi = {static_cast<__bf16>(e4[2]), static_cast<__bf16>(e4[3])};
            pk[u][t][0] = __builtin_bit_cast(uint32_t, lo);
            pk[u][t][1] = __builtin_bit_cast(uint32_t, hi);
            top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, lo));
            top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, hi));
          }
        }
        return max(top[0], top[1]) >= kSlackBits;
      };
      bool move = c == 0;
      if (!move) move = __any(exponents());
      if (move) {
#pragma unroll
        for (int u = 0; u < QT; ++u) {
          float x = -INFINITY;
#pragma unroll
          for (int t = 0; t < kNT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) x = fmaxf(x, sc[u][t][e]);
          x = group_max(x);
          // base-2 scores (c > 0), passed as the exponents above see it
          const float mn = fmaf(x, p.c, -m[u]) > kSlack ? x * p.c : m[u];
          const float alpha = __builtin_amdgcn_exp2f(m[u] - mn);
          m[u] = mn;
          l[u] *= alpha;
#pragma unroll
          for (int j = 0; j < kND; ++j) o[u][j] *= alpha;
        }
        exponents();
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

    // o[u][j][e] = O^T[dim 16 j + 4 g + e][row]
#pragma unroll
    for (int u = 0; u < QT; ++u) {
      if (!live[u]) continue;
      if (p.slots == 1) {
        const float inv = l[u][0] > 0.f ? 1.f / l[u][0] : 0.f;
        uint16_t* dst = static_cast<uint16_t*>(p.out.p) + oaddr[u] + 4 * g;
#pragma unroll
        for (int j = 0; j < kND; ++j) {
          const bf16x2 lo = {static_cast<__bf16>(o[u][j][0] * inv), static_cast<__bf16>(o[u][j][1] * inv)};
          const bf16x2 hi = {static_cast<__bf16>(o[u][j][2] * inv), static_cast<__bf16>(o[u][j][3] * inv)};
          *reinterpret_cast<u32x2*>(dst + 16 * j) =
              u32x2{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
        }
      } else {
        const long long at = ((long long)slot * p.Hk + hk) * p.RT + row0 + (wr * QT + u) * 16 + fr;
        if (g == 0) *reinterpret_cast<f32x2*>(p.ml + 2 * at) = f32x2{m[u], l[u][0]};
        if (nc == 0) continue;  // the statistics say that there is nothing
#pragma unroll
        for (int j = 0; j < kND; ++j) *reinterpret_cast<f32x4*>(p.po + at * D + 16 * j + 4 * g) = o[u][j];
      }
    }
  }
};

// One part of a list of keys n, cut at multiples of `unit`.
__device__ __forceinline__ void part_range(int n, int parts, int part, int unit, int& lo, int& hi) {
  const int nu = (n + unit - 1) / unit;
  lo = min((int)((long long)nu * part / parts) * unit, n);
  hi = min((int)((long long)nu * (part + 1) / parts) * unit, n);
}

template <int D>
using Wide = WideTile<D, 4, 2>;
template <int D>
using Thin = ThinTile<D, 1, 4, 1, 32>;

template <class T>
__device__ __forceinline__ void run_item(const PaParams& p, unsigned char* lds, int item, int seq, int tiles,
                                         int parts, int own, int slot0) {
  // key heads innermost: neighbours in the list read neighbouring heads of the same keys
  const int hk = item % p.Hk;
  const int rest = item / p.Hk;
  const int tile = rest % tiles, part = rest / tiles;
  int row0, row_end;
  int b = -1;
  if (seq) {
    const int per = tiles / p.B;
    b = tile / per;
    row0 = b * p.RS + (tile - b * per) * T::kRows;
    row_end = b * p.RS + (p.q_len ? min(max(p.q_len[b], 0), p.Tq) * p.G : p.RS);
    if (row0 >= row_end) return;
  } else {
    row0 = tile * T::kRows;
    row_end = p.RT;
  }
  int p0 = 0, p1 = 0, s0 = 0, s1 = 0;
  if (own == 0) {
    part_range(p.P, parts, part, 64, p0, p1);
  } else if (own == 1) {
    part_range(p.S, parts, part, 64, s0, s1);
  } else {
    // prefix (rounded up to whole chunks) and own keys as one list
    const int pp = (p.P + 63) & ~63;
    int lo, hi;
    part_range(pp + p.S, parts, part, 64, lo, hi);
    p0 = min(lo, p.P);
    p1 = min(hi, p.P);
    s0 = max(lo - pp, 0);
    s1 = max(hi - pp, 0);
  }
  T::run(p, lds, hk, own == 0 ? -1 : b, row0, row_end, p0, p1, s0, s1, slot0 + part);
}

// KIND: 1 wide items, 2 thin items, 3 both lists in one launch (the thin ones,
// which wait for memory, beside the wide ones, which compute).
template <int D, int KIND>
__global__ __launch_bounds__(256, 2) void prefix_attn_kernel(PaParams p) {
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  const int bid = blockIdx.x;
  if (KIND == 1 || (KIND == 3 && bid < p.n_wide))
    run_item<Wide<D>>(p, lds, bid, p.wide_seq, p.wide_tiles, p.wide_parts, p.wide_own, 0);
  else
    run_item<Thin<D>>(p, lds, bid - p.n_wide, p.thin_seq, p.thin_tiles, p.thin_parts, p.thin_own, p.thin_slot);
}

// Joins a row's partial results; D / 4 lanes a row.
template <int D>
__global__ __launch_bounds__(256) void prefix_join_kernel(PaParams p) {
  constexpr int LPR = D / 4;
  const long long row = (long long)blockIdx.x * (256 / LPR) + threadIdx.x / LPR;  // hk * RT + R
  const int d = (threadIdx.x % LPR) * 4;
  const long long rows = (long long)p.Hk * p.RT;
  if (row >= rows) return;
  const int hk = (int)(row / p.RT);
  const int R = (int)(row - (long long)hk * p.RT);
  const int b = R / p.RS, rr = R - b * p.RS, t = rr / p.G;
  if (p.q_len && t >= p.q_len[b]) return;
  float m = -INFINITY;
  for (int s = 0; s < p.slots; ++s) m = fmaxf(m, p.ml[2 * (s * rows + row)]);
  const float ref = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < p.slots; ++s) {
    const f32x2 x = *reinterpret_cast<const f32x2*>(p.ml + 2 * (s * rows + row));
    if (!(x[1] > 0.f)) continue;  // nothing there, O not written
    const float w = __builtin_amdgcn_exp2f(x[0] - ref);
    l += x[1] * w;
    o += *reinterpret_cast<const f32x4*>(p.po + (s * rows + row) * D + d) * w;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  const int h = hk * p.G + (rr - t * p.G);
  uint16_t* dst = static_cast<uint16_t*>(p.out.p) + (long long)b * p.out.b + (long long)t * p.out.t +
                  (long long)h * p.out.h + d;
  const bf16x2 lo = {static_cast<__bf16>(o[0] * inv), static_cast<__bf16>(o[1] * inv)};
  const bf16x2 hi = {static_cast<__bf16>(o[2] * inv), static_cast<__bf16>(o[3] * inv)};
  *reinterpret_cast<u32x2*>(dst) = u32x2{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
}

// How the rows and keys are dealt to workgroups: from the sizes alone, so
// the workspace's size follows from them too.
struct Plan {
  int wide_seq, wide_tiles, wide_parts, wide_own;
  int thin_seq, thin_tiles, thin_parts, thin_own;
  int slots, thin_slot;
  long long n_wide, n_thin;
};

int cdiv(long long a, long long b) { return (int)((a + b - 1) / b); }

// Parts of n keys so that about `want` workgroups run, none under `least` keys.
int parts_for(long long n, long long items, long long want, long long least) {
  long long parts = items > 0 ? (want + items - 1) / items : 1;
  const long long most = (n + least - 1) / least;
  if (parts > most) parts = most;
  return (int)(parts < 1 ? 1 : parts);
}

Plan make_plan(int B, int Tq, int Hq, int Hk, int P, int S) {
  Plan pl{};
  const int G = Hq / Hk;
  const long long RS = (long long)Tq * G, RT = (long long)B * RS;
  const bool both = RS >= 64 || B == 1 || S == 0 || P == 0;
  if (both) {
    // every tile stays in its sequence and takes prefix and own keys
    const bool thin = RS <= 16;
    const int rows = thin ? 16 : 128;
    const int tiles = B * cdiv(RS, rows);
    const int parts = parts_for((long long)P + S, (long long)tiles * Hk, 512, 256);
    if (thin) {
      pl.thin_seq = 1, pl.thin_tiles = tiles, pl.thin_parts = parts, pl.thin_own = 2;
      pl.n_thin = (long long)tiles * Hk * parts;
    } else {
      pl.wide_seq = 1, pl.wide_tiles = tiles, pl.wide_parts = parts, pl.wide_own = 2;
      pl.n_wide = (long long)tiles * Hk * parts;
    }
    pl.slots = parts;
    return pl;
  }
  // the prefix for the rows of all sequences together, own keys apart
  pl.wide_tiles = cdiv(RT, 128);
  pl.wide_parts = parts_for(P, (long long)pl.wide_tiles * Hk, 256, 256);
  pl.n_wide = (long long)pl.wide_tiles * Hk * pl.wide_parts;
  pl.thin_seq = 1, pl.thin_own = 1;
  pl.thin_tiles = B * cdiv(RS, 16);
  pl.thin_parts = parts_for(S, (long long)pl.thin_tiles * Hk, 256, 256);
  pl.n_thin = (long long)pl.thin_tiles * Hk * pl.thin_parts;
  pl.thin_slot = pl.wide_parts;
  pl.slots = pl.wide_parts + pl.thin_parts;
  return pl;
}

size_t al256(size_t n) { return (n + 255) & ~(size_t)255; }

template <int D>
hipError_t run(const PaParams& p, const Plan& pl, hipStream_t st) {
  const dim3 grid((unsigned)(pl.n_wide + pl.n_thin));
  constexpr int both = Wide<D>::kLds > Thin<D>::kLds ? Wide<D>::kLds : Thin<D>::kLds;
  if (pl.n_thin == 0)
    hipLaunchKernelGGL((prefix_attn_kernel<D, 1>), grid, dim3(256), Wide<D>::kLds, st, p);
  else if (pl.n_wide == 0)
    hipLaunchKernelGGL((prefix_attn_kernel<D, 2>), grid, dim3(256), Thin<D>::kLds, st, p);
  else
    hipLaunchKernelGGL((prefix_attn_kernel<D, 3>), grid, dim3(256), both, st, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || pl.slots == 1) return e;
  const long long rows = (long long)p.Hk * p.RT;
  hipLaunchKernelGGL((prefix_join_kernel<D>), dim3((unsigned)cdiv(rows, 1024 / D)), dim3(256), 0, st, p);
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
  p.wide_seq = pl.wide_seq;
  p.thin_seq = pl.thin_seq;
  p.wide_tiles = pl.wide_tiles;
  p.thin_tiles = pl.thin_tiles;
  p.wide_parts = pl.wide_parts;
  p.thin_parts = pl.thin_parts;
  p.wide_own = pl.wide_own;
  p.thin_own = pl.thin_own;
  p.n_wide = (int)pl.n_wide;
  p.slots = pl.slots;
  p.thin_slot = pl.thin_slot;
  if (pl.slots > 1) {
    const size_t rows = (size_t)pl.slots * a.B * a.Tq * a.Hq;
    p.po = static_cast<float*>(a.ws);
    p.ml = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + al256(rows * a.D * 4));
  }
  return a.D == 64 ? run<64>(p, pl, st) : run<128>(p, pl, st);
}

}  // namespace gkd
