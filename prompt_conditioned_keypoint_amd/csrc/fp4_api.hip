// fp4_api.hip - the C ABI of the four-bit token operators (gkdfp4.h): argument
// validation and dispatch to the kernel launchers. Every check runs before the
// first HIP call, in the order flags, dtype, shapes, the empty case, NULL
// pointers, alignment, workspace.
#include "gkdfp4.h"
#include "fp4_launch.hpp"
#include "status.hpp"
#include "tokens_checks.hpp"

namespace {

using gkd::aligned;
using gkd::check_heads;
using gkd::check_out;
using gkd::check_workspace;
using gkd::fail;
using gkd::heads;
using gkd::hip_status;
using gkd::ok;

gkd_status check_flags(const char* fn, uint32_t flags, uint32_t known) {
  if ((flags & ~known) != 0) return fail(GKD_ERR_UNSUPPORTED, "%s: unknown flags 0x%x", fn, (unsigned)flags);
  return GKD_OK;
}

gkd_status check_dtype(const char* fn, gkd_dtype dtype) {
  if (dtype != GKD_DTYPE_F32 && dtype != GKD_DTYPE_BF16)
    return fail(GKD_ERR_DTYPE, "%s: unknown dtype %d", fn, (int)dtype);
  return GKD_OK;
}

gkd_status check_codes(const char* fn, const uint8_t* codes, const uint8_t* scales) {
  if (!codes || !scales) return fail(GKD_ERR_NULL, "%s: NULL codes or scales", fn);
  if (!aligned(codes, 16) || !aligned(scales, 16))
    return fail(GKD_ERR_ALIGN, "%s: codes and scales need 16-byte alignment", fn);
  return GKD_OK;
}

bool linear_sizes_ok(int M, int N, int K) {
  return M >= 0 && N >= 0 && K >= 1 && M < (1 << 26) && N < (1 << 25) && K < (1 << 22) && (int64_t)M * N < (1LL << 31);
}

// A cache's sizes: what a page holds of a head is addressed with 32 bits.
bool pages_ok(int pages, int page, int Hk, int L) {
  return pages >= 0 && page >= 1 && Hk >= 1 && Hk <= 65536 && L >= 0 && page <= 65536 &&
         (int64_t)L * page < (1 << 30);
}

gkd_status check_cache(const char* fn, const gkd_cache* c, int L) {
  if (c == nullptr) return fail(GKD_ERR_NULL, "%s: NULL cache", fn);
  if (!pages_ok(c->pages, c->page, c->Hk, L) || c->D < 1)
    return fail(GKD_ERR_SHAPE, "%s: bad cache of %d pages of %d, Hk=%d D=%d, L=%d", fn, c->pages, c->page, c->Hk, c->D,
                L);
  if ((c->D != 64 && c->D != 128) || c->page % 32 != 0)
    return fail(GKD_ERR_UNSUPPORTED, "%s: needs D 64 or 128 and pages of a multiple of 32", fn);
  return GKD_OK;
}

// Its arrays. A cache without pages, or a table without columns, needs none.
gkd_status check_arrays(const char* fn, const gkd_cache* c, const int32_t* table, int L) {
  if (c->pages > 0) {
    const gkd_status st = check_codes(fn, c->codes, c->scales);
    if (st != GKD_OK) return st;
  }
  if (L > 0 && !table) return fail(GKD_ERR_NULL, "%s: NULL table", fn);
  if (!aligned(table, 4)) return fail(GKD_ERR_ALIGN, "%s: the table needs 4-byte alignment", fn);
  return GKD_OK;
}

gkd_status check_lengths(const char* fn, const int32_t* a, const int32_t* b) {
  if (!aligned(a, 4) || !aligned(b, 4))
    return fail(GKD_ERR_ALIGN, "%s: lengths and places need 4-byte alignment", fn);
  return GKD_OK;
}

gkd::Pages pages_of(const gkd_cache* c, const int32_t* table, int L) {
  return gkd::Pages{c->codes, c->scales, c->pages, c->page, c->Hk, c->D, table, L};
}

// Tokens to move: a workgroup's last token is counted in 32 bits, in use or not.
bool move_sizes_ok(int B, int T) { return B >= 0 && T >= 0 && T < (1 << 30) && (int64_t)B * T <= 0x7fffffffLL; }

bool attn_sizes_ok(int B, int Tq, int Hq, int Hk) {
  if (B < 0 || Tq < 0 || Hq < 1 || Hk < 1) return false;
  if (B == 0 || Tq == 0) return true;
  if ((int64_t)B * Tq > 0x7fffffffLL / Hq) return false;
  const int64_t tiles = ((int64_t)Tq * (Hq / Hk) + 15) / 16;
  return (int64_t)B * Hk < (1 << 21) && (int64_t)B * Hk * (tiles > 0 ? tiles : 1) < (1 << 21);
}

}  // namespace

extern "C" {

int gkd_fp4_version(void) { return GKD_FP4_VERSION; }

gkd_status gkd_quantize_fp4(const void* x, int64_t ldx, int N, int K, gkd_dtype dtype, uint32_t flags,
                            uint8_t* codes, uint8_t* scales, hipStream_t stream) {
  const char* fn = "gkd_quantize_fp4";
  gkd_status st;
  if ((st = check_flags(fn, flags, 0)) != GKD_OK) return st;
  if ((st = check_dtype(fn, dtype)) != GKD_OK) return st;
  if (N < 0 || K < 1 || ldx < K)
    return fail(GKD_ERR_SHAPE, "%s: bad shape N=%d K=%d ldx=%lld", fn, N, K, (long long)ldx);
  if (K % 32 != 0) return fail(GKD_ERR_UNSUPPORTED, "%s: needs K %% 32 == 0", fn);
  if (N == 0) return ok();
  if (!x) return fail(GKD_ERR_NULL, "%s: NULL x", fn);
  if ((st = check_codes(fn, codes, scales)) != GKD_OK) return st;
  if (!aligned(x, 16) || ldx % (dtype == GKD_DTYPE_F32 ? 4 : 8) != 0)
    return fail(GKD_ERR_ALIGN, "%s: x needs 16-byte aligned data and rows", fn);
  return hip_status(gkd::launch_quantize_fp4({x, (long long)ldx, N, K, dtype == GKD_DTYPE_BF16, codes, scales}, stream),
                    fn);
}

size_t gkd_linear_fp4_workspace_size(int M, int N, int K) {
  if (!linear_sizes_ok(M, N, K) || K % 32 != 0 || M == 0 || N == 0) return 0;
  return gkd::linear_fp4_workspace_bytes(M, N, K);
}

gkd_status gkd_linear_fp4(const void* x, int64_t ldx, const uint8_t* codes, const uint8_t* scales,
                          const void* bias, const void* residual, int64_t ldr, int M, int N, int K,
                          gkd_activation act, gkd_dtype out_dtype, uint32_t flags, void* out, int64_t ldo,
                          void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const char* fn = "gkd_linear_fp4";
  gkd_status st;
  if ((st = check_flags(fn, flags, 0)) != GKD_OK) return st;
  if ((st = check_dtype(fn, out_dtype)) != GKD_OK) return st;
  if ((int)act < GKD_ACT_NONE || (int)act > GKD_ACT_SILU)
    return fail(GKD_ERR_VALUE, "%s: unknown activation %d", fn, (int)act);
  if (!linear_sizes_ok(M, N, K) || ldx < K || ldx >= (1 << 22))
    return fail(GKD_ERR_SHAPE, "%s: bad shape M=%d N=%d K=%d ldx=%lld", fn, M, N, K, (long long)ldx);
  if (K % 32 != 0) return fail(GKD_ERR_UNSUPPORTED, "%s: needs K %% 32 == 0", fn);
  if (ldo < N || (residual != nullptr && ldr < N))
    return fail(GKD_ERR_SHAPE, "%s: ldo=%lld or ldr=%lld below N=%d", fn, (long long)ldo, (long long)ldr, N);
  if (M == 0 || N == 0) return ok();
  if (!x || !out) return fail(GKD_ERR_NULL, "%s: NULL pointer argument", fn);
  if ((st = check_codes(fn, codes, scales)) != GKD_OK) return st;
  const unsigned size = out_dtype == GKD_DTYPE_F32 ? 4 : 2;
  if (!aligned(x, 16) || ldx % 8 != 0)
    return fail(GKD_ERR_ALIGN, "%s: x needs 16-byte aligned data and rows", fn);
  if (!aligned(bias, 2) || !aligned(residual, size) || !aligned(out, size))
    return fail(GKD_ERR_ALIGN, "%s: bias, residual and out need their element's alignment", fn);
  if ((st = check_workspace(fn, workspace, workspace_bytes, gkd::linear_fp4_workspace_bytes(M, N, K))) != GKD_OK)
    return st;
  gkd::LinearFp4Args a;
  a.x = static_cast<const uint16_t*>(x);
  a.codes = codes;
  a.scales = scales;
  a.bias = static_cast<const uint16_t*>(bias);
  a.residual = residual;
  a.out = out;
  a.ldx = ldx;
  a.ldr = ldr;
  a.ldo = ldo;
  a.M = M;
  a.N = N;
  a.K = K;
  a.act = (int)act;
  a.out_f32 = out_dtype == GKD_DTYPE_F32;
  a.ws = workspace;
  return hip_status(gkd::launch_linear_fp4(a, stream), fn);
}

gkd_status gkd_cache_append(const gkd_heads* k, const gkd_heads* v, int B, int T, const int32_t* start,
                            const int32_t* count, const gkd_cache* cache, const int32_t* table, int L,
                            gkd_dtype dtype, uint32_t flags, hipStream_t stream) {
  const char* fn = "gkd_cache_append";
  gkd_status st;
  if ((st = check_flags(fn, flags, 0)) != GKD_OK) return st;
  if ((st = check_dtype(fn, dtype)) != GKD_OK) return st;
  if (!move_sizes_ok(B, T))
    return fail(GKD_ERR_SHAPE, "%s: bad shape B=%d T=%d", fn, B, T);
  if ((st = check_cache(fn, cache, L)) != GKD_OK) return st;
  if (B == 0 || T == 0) return ok();
  const unsigned size = dtype == GKD_DTYPE_F32 ? 4 : 2;
  if ((st = check_heads(fn, "k", k, size, 16)) != GKD_OK) return st;
  if ((st = check_heads(fn, "v", v, size, 16)) != GKD_OK) return st;
  if ((st = check_arrays(fn, cache, table, L)) != GKD_OK) return st;
  if ((st = check_lengths(fn, start, count)) != GKD_OK) return st;
  if (cache->pages == 0 || L == 0) return ok();  // no place for any token
  return hip_status(gkd::launch_cache_append({heads(k), heads(v), pages_of(cache, table, L), B, T, start, count,
                                              dtype == GKD_DTYPE_BF16}, stream), fn);
}

gkd_status gkd_cache_read(const gkd_cache* cache, const int32_t* table, int L, int B, int T,
                          const int32_t* start, const int32_t* count, uint32_t flags, const gkd_heads* k,
                          const gkd_heads* v, hipStream_t stream) {
  const char* fn = "gkd_cache_read";
  gkd_status st;
  if ((st = check_flags(fn, flags, 0)) != GKD_OK) return st;
  if (!move_sizes_ok(B, T))
    return fail(GKD_ERR_SHAPE, "%s: bad shape B=%d T=%d", fn, B, T);
  if ((st = check_cache(fn, cache, L)) != GKD_OK) return st;
  if (B == 0 || T == 0) return ok();
  if ((st = check_out(fn, "k", k, 2, 16, B, T, cache->Hk)) != GKD_OK) return st;
  if ((st = check_out(fn, "v", v, 2, 16, B, T, cache->Hk)) != GKD_OK) return st;
  if ((st = check_arrays(fn, cache, table, L)) != GKD_OK) return st;
  if ((st = check_lengths(fn, start, count)) != GKD_OK) return st;
  return hip_status(gkd::launch_cache_read({heads(k), heads(v), pages_of(cache, table, L), B, T, start, count, true},
                                           stream), fn);
}

size_t gkd_cache_attention_workspace_size(int B, int Tq, int Hq, int Hk, int D, int page, int L) {
  if (!attn_sizes_ok(B, Tq, Hq, Hk) || !pages_ok(0, page, Hk, L) || page % 32 != 0 || Hq % Hk != 0 ||
      (D != 64 && D != 128) || B == 0 || Tq == 0)
    return 0;
  return gkd::cache_attn_workspace_bytes(B, Tq, Hq, Hk, D, page, L);
}

gkd_status gkd_cache_attention(const gkd_heads* q, const gkd_cache* cache, const int32_t* table, int L,
                               const int32_t* length, const int32_t* q_len, int B, int Tq, int Hq, float scale,
                               uint32_t flags, const gkd_heads* out, void* workspace, size_t workspace_bytes,
                               hipStream_t stream) {
  const char* fn = "gkd_cache_attention";
  gkd_status st;
  if ((st = check_flags(fn, flags, GKD_ATTN_CAUSAL)) != GKD_OK) return st;
  if ((st = check_cache(fn, cache, L)) != GKD_OK) return st;
  if (!attn_sizes_ok(B, Tq, Hq, cache->Hk))
    return fail(GKD_ERR_SHAPE, "%s: bad shape B=%d Tq=%d Hq=%d Hk=%d", fn, B, Tq, Hq, cache->Hk);
  if (Hq % cache->Hk != 0) return fail(GKD_ERR_UNSUPPORTED, "%s: needs Hq %% Hk == 0", fn);
  // (the kernels take base-2 scores: scale log2(e) must be finite too)
  if (!(scale > 0.f) || !(scale <= 2e38f))
    return fail(GKD_ERR_VALUE, "%s: scale must be above 0 and at most 2e38", fn);
  if (B == 0 || Tq == 0) return ok();
  if ((st = check_heads(fn, "q", q, 2, 16)) != GKD_OK) return st;
  if ((st = check_out(fn, "out", out, 2, 16, B, Tq, Hq)) != GKD_OK) return st;
  if ((st = check_arrays(fn, cache, table, L)) != GKD_OK) return st;
  if ((st = check_lengths(fn, length, q_len)) != GKD_OK) return st;
  if ((st = check_workspace(fn, workspace, workspace_bytes,
                            gkd::cache_attn_workspace_bytes(B, Tq, Hq, cache->Hk, cache->D, cache->page, L))) != GKD_OK)
    return st;
  gkd::CacheAttnArgs a;
  a.q = heads(q);
  a.out = heads(out);
  a.c = pages_of(cache, table, L);
  a.length = length;
  a.q_len = q_len;
  a.B = B;
  a.Tq = Tq;
  a.Hq = Hq;
  a.scale = scale;
  a.causal = (flags & GKD_ATTN_CAUSAL) != 0;
  a.ws = workspace;
  return hip_status(gkd::launch_cache_attn(a, stream), fn);
}

}  // extern "C"
