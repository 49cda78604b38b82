// rope.hip - norm of every query and key head and rotary positions with
// several axes, in one pass (gkd_qk_norm_rope).
//
// A token's angles phi_i = sum_a pos[a] freqs[a,i] are the same for all its
// heads, so a workgroup takes a run of tokens, puts the cosines and sines of
// each into LDS once, and then streams the heads past them: one read and one
// write of q and k, which is all the traffic there is (the work is ~10
// float operations an element, far below what the memory leaves room for).
//
// phi in float64: pos and freqs are float32, so their product is exact, and
// a float32 angle of 10^5 would be off by 2^-8 of a radian. For bfloat16 heads
// it is reduced to one turn there (phi / 2 pi minus the nearest whole number)
// and the rest, in [-1/2, 1/2], goes to float32 (2^-26 of a turn) and to the
// hardware's functions; for float32 heads it stays in float64 up to the cosine
// and sine, which are rounded once.
//
// Measured (a call; the card copies at 5.08 TB/s): 2 x 18432 tokens, 40 heads of
// 128, three axes, norm, bfloat16: 755 MB in 141 us, 5.3 TB/s; 64 x 581 tokens,
// 32 heads of 64: 305 MB in 59 us, 5.1 TB/s; 8 tokens 4.8 us on the GPU. Split
// pairs of odd halves (kLoose) are at half that rate, their partners looked up
// in LDS one by one: 9 x 2193 tokens, 16 heads of 96, 121 MB in 44 us.
#include "gkd_device.hpp"
#include "tokens_launch.hpp"

namespace gkd {
namespace {

struct RopeParams {
  Heads q, k, qo, ko;
  int Hq, H;                // query heads; query and key heads together
  long long n_tok;          // B * T
  int T, D, half;           // half: rot / 2
  const float* pos;
  long long pos_batch;
  int n_axes;
  const float* freqs;
  const void *wq, *wk;      // or null
  float eps, inv_d;
  int tt;                   // tokens a workgroup
  long long first;          // first token (head, rope_any_kernel) of this launch
};

// T: the heads' type.
template <typename T>
__device__ __forceinline__ void rope_angle(const RopeParams& p, const float* pos, int i, float& c,
                                           float& s) {
  double phi = 0.0;
  for (int a = 0; a < p.n_axes; ++a)
    phi = fma((double)pos[a], (double)p.freqs[(long long)a * p.half + i], phi);
  if constexpr (sizeof(T) == 2) {
    const double turns = phi * 0.15915494309189533576888;  // 1 / (2 pi)
    const float r = (float)(turns - rint(turns));
    // the hardware's functions take turns; with the angle's rounding they are
    // right to 1.8e-7 (measured), three float32 steps of a value near 1 and
    // nothing beside the output's rounding to bfloat16 (2^-8)
    s = __builtin_amdgcn_sinf(r);
    c = __builtin_amdgcn_cosf(r);
  } else {
    // the nearest whole number k of quarter turns, and Taylor series of the rest,
    // |h| <= pi / 4, whose first terms left out are h^13 / 13! and h^12 / 12! (1.2e-10)
    const double quarters = phi * 0.63661977236758134308;  // 2 / pi
    const double q = rint(quarters), h = (quarters - q) * 1.57079632679489661923, u = h * h;
    const int k = (int)fma(-4.0, rint(0.25 * q), q) & 3;
    double x = fma(u, -1.0 / 39916800, 1.0 / 362880);
    x = fma(u, x, -1.0 / 5040);
    x = fma(u, x, 1.0 / 120);
    x = fma(u, x, -1.0 / 6);
    const float sh = (float)fma(h * u, x, h);
    double y = fma(u, -1.0 / 3628800, 1.0 / 40320);
    y = fma(u, y, -1.0 / 720);
    y = fma(u, y, 1.0 / 24);
    y = fma(u, y, -0.5);
    const float ch = (float)fma(u, y, 1.0);
    const float sk = k & 1 ? ch : sh, ck = k & 1 ? sh : ch;
    s = k & 2 ? -sk : sk;
    c = (k + 1) & 2 ? -ck : ck;
  }
}

// 16 bytes of T as floats and back (one rounding to nearest even).
template <typename T>
struct Piece;
template <>
struct Piece<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(u32x4 v, float* f) {
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = __uint_as_float(v[e]);
  }
  static __device__ __forceinline__ u32x4 pack(const float* f) {
    return u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                 __float_as_uint(f[3])};
  }
};
template <>
struct Piece<uint16_t> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(u32x4 v, float* f) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[2 * e] = __uint_as_float(v[e] << 16);
      f[2 * e + 1] = __uint_as_float(v[e] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ u32x4 pack(const float* f) {
    u32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bf16x2 h = {static_cast<__bf16>(f[2 * e]), static_cast<__bf16>(f[2 * e + 1])};
      v[e] = __builtin_bit_cast(uint32_t, h);
    }
    return v;
  }
};

// Whole 16-byte pieces. A head is np = ceil(D / (2 N)) pairs of pieces, one
// pair a lane, the head's lanes padded to LP (a power of two) so the norm's
// sum is LP-wide lane exchanges. Pair j holds, for pairs of elements side by
// side, pieces 2 j and 2 j + 1; for split pairs (i, i + rot/2), pieces j and
// rot/2/N + j while they rotate, then the rest of the head two by two. In
// both orders the lane's pairs are N j .. N j + N - 1, so cosines and sines
// are read as whole float4s (past rot/2 the table is not used). Split pairs
// whose half is no whole number of pieces (kLoose) keep pieces 2 j and 2 j + 1
// and find each element's partner in LDS, where the head's lanes put their
// values. Every lane reads its two pieces before it writes them and no lane
// touches another's, so an output may be its input.
enum { kSplit = 0, kSide = 1, kLoose = 2 };
__host__ __device__ constexpr int loose_floats(int npair) { return 2 * npair + 2 * npair / 8; }

template <typename T, int LP, int PAIRS>
__global__ __launch_bounds__(256) void rope_kernel(RopeParams p) {
  constexpr int N = Piece<T>::N;
  constexpr bool IL = PAIRS == kSide;
  extern __shared__ __attribute__((aligned(16))) float cs[];  // [tt][2][npair], kLoose: and the heads' values
  const int tid = threadIdx.x;
  const int np = (p.D + 2 * N - 1) / (2 * N), npair = np * N;
  const long long tok0 = p.first + (long long)blockIdx.x * p.tt;
  const int nt = (int)min((long long)p.tt, p.n_tok - tok0);
  const long long seq0 = tok0 / p.T;
  const uint32_t at0 = (uint32_t)(tok0 - seq0 * p.T);
  // sequence of the workgroup's token t, and its place there
  auto place = [&](int t, long long& b, uint32_t& tb) {
    const uint32_t at = at0 + (uint32_t)t, over = at / (uint32_t)p.T;
    b = seq0 + over;
    tb = at - over * (uint32_t)p.T;
  };

  const int j = tid & (LP - 1);
  // the pair's two pieces (element offsets; b1: the second one exists)
  const int hp = p.half / N;
  int e0, e1;
  if (PAIRS != kSplit) {
    e0 = 2 * j * N;
    e1 = e0 + N;
  } else if (j < hp) {
    e0 = j * N;
    e1 = e0 + p.half;
  } else {
    e0 = 2 * p.half + 2 * (j - hp) * N;
    e1 = e0 + N;
  }
  const bool b0 = j < np && e0 < p.D, b1 = j < np && e1 < p.D;
  const bool turn = PAIRS != kSplit || j < hp;
  // kLoose: this head's values, a gap after every 8 so that lanes 16 apart meet
  // different banks
  float* mine = cs + 2 * p.tt * npair + (tid / LP) * loose_floats(npair);
  auto gap = [](int e) { return e + (e >> 3); };
  const u32x4 z4 = {0u, 0u, 0u, 0u};
  u32x4 wq0 = z4, wq1 = z4, wk0 = z4, wk1 = z4;  // gains, as stored
  auto gain = [&](const void* w, int e, bool in) {
    if ((reinterpret_cast<uintptr_t>(w) & 15u) == 0)
      return in ? *reinterpret_cast<const u32x4*>(static_cast<const T*>(w) + e) : z4;
    T t[N];
#pragma unroll
    for (int i = 0; i < N; ++i) t[i] = in ? static_cast<const T*>(w)[e + i] : T(0);
    u32x4 v;
    __builtin_memcpy(&v, t, 16);
    return v;
  };
  if (p.wq) wq0 = gain(p.wq, e0, b0), wq1 = gain(p.wq, e1, b1);
  if (p.wk) wk0 = gain(p.wk, e0, b0), wk1 = gain(p.wk, e1, b1);

  // A head is on its way while the one before is worked on, the first one
  // while the table is made. Not so with kLoose, where it gains nothing on
  // average (76 of 96 rotated, 9 x 2193 tokens, 16 heads, norm: 44.7 us with it,
  // 43.9 without; 90 rotated, 62 x 455 tokens, 25 heads, no norm: 85.4, 87.7).
  constexpr int kStep = 256 / LP;  // heads a round
  const int units = nt * p.H;
  u32x4 next0 = z4, next1 = z4;
  T* next_dst = nullptr;
  auto fetch = [&](int u) {
    const int t = (int)((uint32_t)u / (uint32_t)p.H), hh = u - t * p.H;
    const bool isk = hh >= p.Hq;
    const int h = isk ? hh - p.Hq : hh;
    long long b;
    uint32_t tb;
    place(t, b, tb);
    const Heads& in = isk ? p.k : p.q;
    const Heads& out = isk ? p.ko : p.qo;
    const T* src = static_cast<const T*>(in.p) + b * in.b + tb * in.t + h * in.h;
    next_dst = static_cast<T*>(out.p) + b * out.b + tb * out.t + h * out.h;
    next0 = b0 ? *reinterpret_cast<const u32x4*>(src + e0) : z4;
    next1 = b1 ? *reinterpret_cast<const u32x4*>(src + e1) : z4;
  };
  if (PAIRS != kLoose && tid / LP < units) fetch(tid / LP);

  for (int i = tid; i < nt * npair; i += 256) {
    const int t = (int)((uint32_t)i / (uint32_t)npair), pr = i - t * npair;
    long long b;
    uint32_t tb;
    place(t, b, tb);
    float c = 1.f, s = 0.f;
    if (pr < p.half) rope_angle<T>(p, p.pos + b * p.pos_batch + (long long)tb * p.n_axes, pr, c, s);
    cs[(2 * t) * npair + pr] = c;
    cs[(2 * t + 1) * npair + pr] = s;
  }
  __syncthreads();

  for (int u = tid / LP; u < units; u += kStep) {
    const int t = (int)((uint32_t)u / (uint32_t)p.H);
    const bool isk = u - t * p.H >= p.Hq;
    if (PAIRS == kLoose) fetch(u);
    T* dst = next_dst;
    float x0[N], x1[N];
    Piece<T>::unpack(next0, x0);
    Piece<T>::unpack(next1, x1);
    if (PAIRS != kLoose && u + kStep < units) fetch(u + kStep);
    if ((isk ? p.wk : p.wq) != nullptr) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) ss = fmaf(x0[i], x0[i], fmaf(x1[i], x1[i], ss));
#pragma unroll
      for (int d = 1; d < LP; d <<= 1) ss += __shfl_xor(ss, d);
      const float rs = 1.f / sqrtf(fmaf(ss, p.inv_d, p.eps));
      float g0[N], g1[N];
      Piece<T>::unpack(isk ? wk0 : wq0, g0);
      Piece<T>::unpack(isk ? wk1 : wq1, g1);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        x0[i] = x0[i] * rs * g0[i];
        x1[i] = x1[i] * rs * g1[i];
      }
    }
    float y0[N], y1[N];
    if constexpr (PAIRS == kLoose) {
      if (b0) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          mine[gap(e0 + i)] = x0[i];
          mine[gap(e1 + i)] = x1[i];
        }
      }
      asm volatile("" ::: "memory");  // the head's lanes are in one wave, whose LDS accesses keep their order
      __builtin_amdgcn_wave_barrier();
      const float* c = cs + (2 * t) * npair;
      const float* s = c + npair;
      auto turned = [&](int e, float x) {
        const bool second = e >= p.half;
        if (e >= 2 * p.half || e >= p.D) return x;
        const int i = second ? e - p.half : e;
        const float y = mine[gap(second ? i : e + p.half)];
        return second ? x * c[i] + y * s[i] : x * c[i] - y * s[i];
      };
#pragma unroll
      for (int i = 0; i < N; ++i) {
        y0[i] = turned(e0 + i, x0[i]);
        y1[i] = turned(e1 + i, x1[i]);
      }
      asm volatile("" ::: "memory");
      __builtin_amdgcn_wave_barrier();
    } else if (turn && b0) {
      const float* c = cs + (2 * t) * npair + N * j;
      const float* s = c + npair;
      if (IL) {
        // elements past rot are copied, not turned by (1, 0): an infinite or NaN
        // neighbour times 0 would make them NaN
        const int left = p.half - N * j;  // pairs that turn, from the lane's first on
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
          const bool t0 = i < left, t1 = N / 2 + i < left;
          y0[2 * i] = t0 ? x0[2 * i] * c[i] - x0[2 * i + 1] * s[i] : x0[2 * i];
          y0[2 * i + 1] = t0 ? x0[2 * i + 1] * c[i] + x0[2 * i] * s[i] : x0[2 * i + 1];
          y1[2 * i] = t1 ? x1[2 * i] * c[N / 2 + i] - x1[2 * i + 1] * s[N / 2 + i] : x1[2 * i];
          y1[2 * i + 1] = t1 ? x1[2 * i + 1] * c[N / 2 + i] + x1[2 * i] * s[N / 2 + i] : x1[2 * i + 1];
        }
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          y0[i] = x0[i] * c[i] - x1[i] * s[i];
          y1[i] = x1[i] * c[i] + x0[i] * s[i];
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        y0[i] = x0[i];
        y1[i] = x1[i];
      }
    }
    if (b0) *reinterpret_cast<u32x4*>(dst + e0) = Piece<T>::pack(y0);
    if (b1) *reinterpret_cast<u32x4*>(dst + e1) = Piece<T>::pack(y1);
  }
}

__device__ __forceinline__ float rope_load(const float* p) { return *p; }
__device__ __forceinline__ float rope_load(const uint16_t* p) { return bf16_bits_to_f32(*p); }
__device__ __forceinline__ void rope_store(float* p, float v) { *p = v; }
__device__ __forceinline__ void rope_store(uint16_t* p, float v) { *p = f32_to_bf16_bits(v); }

// Any alignment and head width: one wave a head, elements
// one by one (D <= 512: at most 4 rotated pairs and 8 other elements a
// lane). A lane reads all its elements before it writes them.
template <typename T>
__global__ __launch_bounds__(256) void rope_any_kernel(RopeParams p, bool interleaved) {
  const int lane = threadIdx.x & 63;
  const long long u = p.first + (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (u >= p.n_tok * p.H) return;
  const long long tok = u / p.H, b = tok / p.T, tb = tok - b * p.T;
  const int hh = (int)(u - tok * p.H);
  const bool isk = hh >= p.Hq;
  const int h = isk ? hh - p.Hq : hh;
  const Heads& in = isk ? p.k : p.q;
  const Heads& out = isk ? p.ko : p.qo;
  const T* src = static_cast<const T*>(in.p) + b * in.b + tb * in.t + h * in.h;
  T* dst = static_cast<T*>(out.p) + b * out.b + tb * out.t + h * out.h;
  const T* w = static_cast<const T*>(isk ? p.wk : p.wq);
  const float* pos = p.pos + b * p.pos_batch + tb * p.n_axes;
  float a0[4], a1[4], rest[8];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int pr = lane + 64 * i;
    a0[i] = a1[i] = 0.f;
    if (pr < p.half) {
      a0[i] = rope_load(src + (interleaved ? 2 * pr : pr));
      a1[i] = rope_load(src + (interleaved ? 2 * pr + 1 : pr + p.half));
    }
    ss = fmaf(a0[i], a0[i], fmaf(a1[i], a1[i], ss));
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = 2 * p.half + lane + 64 * i;
    rest[i] = e < p.D ? rope_load(src + e) : 0.f;
    ss = fmaf(rest[i], rest[i], ss);
  }
  float rs = 1.f;
  if (w != nullptr) rs = 1.f / sqrtf(fmaf(wave_sum(ss), p.inv_d, p.eps));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int pr = lane + 64 * i;
    if (pr >= p.half) continue;
    const int e0 = interleaved ? 2 * pr : pr, e1 = interleaved ? 2 * pr + 1 : pr + p.half;
    float c, s;
    rope_angle<T>(p, pos, pr, c, s);
    const float u0 = w ? a0[i] * rs * rope_load(w + e0) : a0[i];
    const float u1 = w ? a1[i] * rs * rope_load(w + e1) : a1[i];
    rope_store(dst + e0, u0 * c - u1 * s);
    rope_store(dst + e1, u1 * c + u0 * s);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = 2 * p.half + lane + 64 * i;
    if (e < p.D) rope_store(dst + e, w ? rest[i] * rs * rope_load(w + e) : rest[i]);
  }
}

// A launch has at most 2^32 work items; longer batches take several.
constexpr long long kMostWgs = 1 << 23;

template <typename T, int LP>
hipError_t run_pieces(RopeParams p, int pairs, hipStream_t st) {
  constexpr int N = Piece<T>::N;
  const int npair = (p.D + 2 * N - 1) / (2 * N) * N;
  // about 1024 pairs of pieces a workgroup (four rounds of its lanes), fewer
  // where that leaves less than four workgroups a CU (in a captured graph: 3 x
  // 1001 tokens of 8 heads of 96 in float32 8.3 us, with 1024 10.6; 4 x 300 of 5
  // heads of 128 4.4, 8.6), while its table stays within 16 KB of LDS
  const long long round = 256 / ((long long)p.H * LP);
  long long tt = 1024 / ((long long)p.H * LP);
  if (tt > p.n_tok / 1024) tt = p.n_tok / 1024 > round ? p.n_tok / 1024 : round;
  tt = tt < 1 ? 1 : tt;
  const long long most = 16384 / (8 * npair);
  if (tt > most) tt = most;
  p.tt = (int)tt;
  const size_t lds = (size_t)tt * npair * 8 + (pairs == kLoose ? (size_t)(256 / LP) * loose_floats(npair) * 4 : 0);
  for (; p.first < p.n_tok; p.first += kMostWgs * tt) {
    const long long wgs = (p.n_tok - p.first + tt - 1) / tt;
    const dim3 grid((unsigned)(wgs < kMostWgs ? wgs : kMostWgs));
    if (pairs == kSide)
      hipLaunchKernelGGL((rope_kernel<T, LP, kSide>), grid, dim3(256), lds, st, p);
    else if (pairs == kSplit)
      hipLaunchKernelGGL((rope_kernel<T, LP, kSplit>), grid, dim3(256), lds, st, p);
    else
      hipLaunchKernelGGL((rope_kernel<T, LP, kLoose>), grid, dim3(256), lds, st, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename T>
hipError_t run_typed(const RopeArgs& a, RopeParams p, hipStream_t st) {
  constexpr int N = Piece<T>::N;
  auto whole = [](const Heads& h) {
    return (reinterpret_cast<uintptr_t>(h.p) & 15u) == 0 && h.b % N == 0 && h.t % N == 0 && h.h % N == 0;
  };
  bool pieces = a.D % N == 0 && whole(a.q) && whole(a.qo);
  const int pairs = a.interleaved ? kSide : p.half % N == 0 ? kSplit : kLoose;
  if (a.Hk > 0) pieces = pieces && whole(a.k) && whole(a.ko);
  if (pieces) {
    const int np = (a.D + 2 * N - 1) / (2 * N);
    if (np <= 4) return run_pieces<T, 4>(p, pairs, st);
    if (np <= 8) return run_pieces<T, 8>(p, pairs, st);
    if (np <= 16) return run_pieces<T, 16>(p, pairs, st);
    if (np <= 32) return run_pieces<T, 32>(p, pairs, st);
    return run_pieces<T, 64>(p, pairs, st);
  }
  for (; p.first < p.n_tok * p.H; p.first += kMostWgs * 4) {
    const long long wgs = (p.n_tok * p.H - p.first + 3) / 4;
    hipLaunchKernelGGL((rope_any_kernel<T>), dim3((unsigned)(wgs < kMostWgs ? wgs : kMostWgs)),
                       dim3(256), 0, st, p, a.interleaved);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, hipStream_t st) {
  RopeParams p{};
  p.q = a.q;
  p.k = a.k;
  p.qo = a.qo;
  p.ko = a.ko;
  p.Hq = a.Hq;
  p.H = a.Hq + a.Hk;
  p.n_tok = (long long)a.B * a.T;
  p.T = a.T;
  p.D = a.D;
  p.half = a.rot / 2;
  p.pos = a.pos;
  p.pos_batch = a.pos_batch;
  p.n_axes = a.n_axes;
  p.freqs = a.freqs;
  p.wq = a.wq;
  p.wk = a.wk;
  p.eps = a.eps;
  p.inv_d = 1.f / (float)a.D;
  return a.bf16 ? run_typed<uint16_t>(a, p, st) : run_typed<float>(a, p, st);
}

}  // namespace gkd
