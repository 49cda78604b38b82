// fp4_cache.hip - values into four-bit codes and back: rows of weights
// (gkd_quantize_fp4), tokens into a cache's pages (gkd_cache_append) and out of
// them (gkd_cache_read).
//
// A thread takes 8 neighbouring values, one 16-byte piece of bfloat16; four
// neighbouring lanes hold a group and agree on its largest magnitude.
//
// A token's keys lie together outside a cache, a head's tokens together in its pages. So
// a workgroup takes up to 32 tokens, the lanes of a wave neighbouring tokens of a head:
// both sides move in whole lines, and a thread's place, the same for all its heads, is
// looked up once, while its values are on their way. (Heads neighbouring in a wave instead:
// the same time; a place looked up for every piece: 1.6 times as long.)
//
// Memory bounds both. 64 x 581 tokens of 16 heads of 64, 193 MB each way: 48 to 57 us to
// append (3.4 to 4.0 TB/s) and 43 us to read (4.5; 31 where what was just appended is still in
// the last cache); a large copy on the same card moves 5.0. In float32 72 us to append (4.8).
// One token of 48 sequences, 8 heads of 128: 3.3 and 3.1 us, a launch's time. 16384 x 4096
// weights: 33 us in bfloat16, 58 in float32, 5.2 TB/s.
#include "fp4_device.hpp"
#include "fp4_launch.hpp"

namespace gkd {
namespace {

// Values i .. i + 8 of an array in bfloat16 or float32.
template <bool BF16>
__device__ __forceinline__ void load8(const void* base, long long i, float (&v)[8]) {
  if constexpr (BF16) {
    const u32x4 w = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(base) + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = __uint_as_float(w[e] << 16);
      v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
  } else {
    const f32x4* q = reinterpret_cast<const f32x4*>(static_cast<const float*>(base) + i);
    const f32x4 a = q[0], b = q[1];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = a[e];
      v[4 + e] = b[e];
    }
  }
}

// The group's largest magnitude, as bits (which order like integers, NaN last), of
// its four lanes: quad permutes [1,0,3,2] and [2,3,0,1].
__device__ __forceinline__ uint32_t group_max(const float (&v)[8]) {
  uint32_t a = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) a = max(a, __float_as_uint(v[e]) & 0x7fffffffu);
  a = max(a, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a, 0xB1, 0xf, 0xf, false));
  return max(a, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a, 0x4E, 0xf, 0xf, false));
}

struct QuantParams {
  const void* x;
  long long ldx, pieces;
  int per;  // pieces a row
  uint8_t *codes, *scales;
};

template <bool BF16>
__global__ __launch_bounds__(256) void fp4_quantize_kernel(QuantParams p) {
  for (long long u = (long long)blockIdx.x * 256 + threadIdx.x; u < p.pieces; u += (long long)gridDim.x * 256) {
    const long long r = u / p.per;
    const int c = (int)(u - r * p.per);
    float v[8];
    load8<BF16>(p.x, r * p.ldx + 8 * c, v);
    const uint32_t s = fp4_scale(group_max(v));
    reinterpret_cast<uint32_t*>(p.codes)[u] = fp4_codes(v, s);
    if ((u & 3) == 0) p.scales[u >> 2] = (uint8_t)s;
  }
}

// A thread's heads, keys' and values': loads under way against registers (64 x 581 tokens
// appended and read, us: 1 head 64 and 64, 2 heads 54 and 51, 4 heads 48 and 43, 8 appended 51).
constexpr int kHeads = 4;

struct MoveParams {
  Heads k, v;
  Pages c;
  int T, dlog, tlog;   // D / 8 pieces of a row and 2^tlog tokens of a workgroup: 256 threads at most
  int chunks, blocks;  // of a sequence's tokens, of a chunk's heads
  const int32_t *start, *count;
  long long groups;
};

// A thread's piece of a token: place `piece` of its row, and the heads it takes.
struct Piece {
  int t, d, head, step;  // the first head, of 2 Hk, and how far the next one is
  long long at[2];       // element offset of the row in k, in v
  long long code;        // piece of head 0's codes in the cache, -1 without a place
  bool live;
};

__device__ __forceinline__ Piece piece(const MoveParams& p, long long group) {
  Piece w;
  const int hb = (int)(group % p.blocks), chunk = (int)(group / p.blocks % p.chunks);
  const int b = (int)(group / p.blocks / p.chunks);
  const int x = threadIdx.x;
  w.d = x & ((1 << p.dlog) - 1);
  w.t = (chunk << p.tlog) + ((x >> p.dlog) & ((1 << p.tlog) - 1));
  w.step = 256 >> (p.dlog + p.tlog);
  w.head = hb * kHeads * w.step + (x >> (p.dlog + p.tlog));
  w.at[0] = b * p.k.b + w.t * p.k.t + 8 * w.d;
  w.at[1] = b * p.v.b + w.t * p.v.t + 8 * w.d;
  w.live = w.t < p.T && (!p.count || w.t < p.count[b]);
  w.code = -1;
  const long long pos = (long long)(p.start ? p.start[b] : 0) + w.t;
  if (w.live && pos >= 0 && pos < (long long)p.c.L * p.c.page) {
    const int col = (int)((uint32_t)pos / (uint32_t)p.c.page), row = (int)pos - col * p.c.page;
    const int page = p.c.table[(long long)b * p.c.L + col];
    if (page >= 0 && page < p.c.pages) w.code = (((long long)page * 2 * p.c.Hk * p.c.page + row) << p.dlog) + w.d;
  }
  return w;
}

// Its heads, one after another: f(j, value, element offset, piece of the cache's codes).
template <class F>
__device__ __forceinline__ void heads_of(const MoveParams& p, const Piece& w, F&& f) {
#pragma unroll
  for (int j = 0; j < kHeads; ++j) {
    const int h = w.head + j * w.step;
    if (h >= 2 * p.c.Hk) break;
    const bool value = h >= p.c.Hk;
    const long long at = value ? w.at[1] + (h - p.c.Hk) * p.v.h : w.at[0] + h * p.k.h;
    f(j, value, at, w.code + (((long long)h * p.c.page) << p.dlog));
  }
}

template <bool BF16>
__global__ __launch_bounds__(256) void fp4_append_kernel(MoveParams p) {
  for (long long group = blockIdx.x; group < p.groups; group += gridDim.x) {
    const Piece w = piece(p, group);
    float v[kHeads][8];
    if (w.live) heads_of(p, w, [&](int j, bool value, long long at, long long) {
      load8<BF16>(value ? p.v.p : p.k.p, at, v[j]);
    });
    if (w.code >= 0) heads_of(p, w, [&](int j, bool, long long, long long code) {  // the four lanes of a group alike
      const uint32_t s = fp4_scale(group_max(v[j]));
      reinterpret_cast<uint32_t*>(p.c.codes)[code] = fp4_codes(v[j], s);
      if ((code & 3) == 0) p.c.scales[code >> 2] = (uint8_t)s;
    });
  }
}

__global__ __launch_bounds__(256) void fp4_read_kernel(MoveParams p) {
  for (long long group = blockIdx.x; group < p.groups; group += gridDim.x) {
    const Piece w = piece(p, group);
    if (!w.live) continue;
    uint32_t c[kHeads] = {}, s[kHeads] = {};
    if (w.code >= 0) heads_of(p, w, [&](int j, bool, long long, long long code) {
      c[j] = reinterpret_cast<const uint32_t*>(p.c.codes)[code];
      s[j] = p.c.scales[code >> 2];
    });
    heads_of(p, w, [&](int j, bool value, long long at, long long) {
      *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(value ? p.v.p : p.k.p) + at) = fp4_values(c[j], fp4_unit(s[j]));
    });
  }
}

unsigned groups_for(long long pieces) {
  const long long n = (pieces + 255) / 256;
  return (unsigned)(n < 8192 ? n : 8192);
}

MoveParams move_params(const CacheMoveArgs& a) {
  MoveParams p{};
  p.k = a.k;
  p.v = a.v;
  p.c = a.c;
  p.T = a.T;
  p.dlog = a.c.D == 64 ? 3 : 4;
  while (p.dlog + p.tlog < 8 && (1 << p.tlog) < a.T) ++p.tlog;
  p.chunks = (int)(((long long)a.T + (1 << p.tlog) - 1) >> p.tlog);
  const int heads = kHeads * (256 >> (p.dlog + p.tlog));
  p.blocks = (2 * a.c.Hk + heads - 1) / heads;
  p.start = a.start;
  p.count = a.count;
  p.groups = (long long)a.B * p.chunks * p.blocks;
  return p;
}

unsigned grid_for(long long groups) { return (unsigned)(groups < (1 << 20) ? groups : 1 << 20); }

}  // namespace

hipError_t launch_quantize_fp4(const QuantizeArgs& a, hipStream_t st) {
  QuantParams p{a.x, a.ldx, (long long)a.N * (a.K / 8), a.K / 8, a.codes, a.scales};
  if (a.bf16)
    hipLaunchKernelGGL(fp4_quantize_kernel<true>, dim3(groups_for(p.pieces)), dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL(fp4_quantize_kernel<false>, dim3(groups_for(p.pieces)), dim3(256), 0, st, p);
  return hipGetLastError();
}

hipError_t launch_cache_append(const CacheMoveArgs& a, hipStream_t st) {
  const MoveParams p = move_params(a);
  if (a.bf16)
    hipLaunchKernelGGL(fp4_append_kernel<true>, dim3(grid_for(p.groups)), dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL(fp4_append_kernel<false>, dim3(grid_for(p.groups)), dim3(256), 0, st, p);
  return hipGetLastError();
}

hipError_t launch_cache_read(const CacheMoveArgs& a, hipStream_t st) {
  const MoveParams p = move_params(a);
  hipLaunchKernelGGL(fp4_read_kernel, dim3(grid_for(p.groups)), dim3(256), 0, st, p);
  return hipGetLastError();
}

}  // namespace gkd
