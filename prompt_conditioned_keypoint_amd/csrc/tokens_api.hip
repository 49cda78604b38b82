// tokens_api.hip - the C ABI of the token operators (gkdtokens.h): argument
// validation and dispatch to the kernel launchers. Every check runs before
// the first HIP call, in the order flags, dtype, shapes, the empty case,
// NULL pointers, alignment, workspace.
#include "gkdtokens.h"
#include "status.hpp"
#include "tokens_checks.hpp"
#include "tokens_launch.hpp"

#include <cmath>

namespace {

using gkd::aligned;
using gkd::check_heads;
using gkd::check_out;
using gkd::check_workspace;
using gkd::fail;
using gkd::heads;
using gkd::hip_status;
using gkd::ok;

// Keys and values of the attention: a chunk of 64 of them is addressed with
// 32 bits.
gkd_status check_keys(const char* fn, const char* name, const gkd_heads* h) {
  const gkd_status st = check_heads(fn, name, h, 2, 16);
  if (st != GKD_OK) return st;
  if (h->token >= (1 << 25)) return fail(GKD_ERR_SHAPE, "%s: token stride of %s reaches 2^25", fn, name);
  return GKD_OK;
}

bool linear_sizes_ok(int M, int N, int K, int64_t ldx, int64_t ldw) {
  // (a launch has fewer than 2^32 threads)
  return M >= 0 && N >= 0 && K >= 1 && M < (1 << 26) && N < (1 << 25) && (int64_t)M * N < (1LL << 36) &&
         ldx >= K && ldw >= K && ldx < (1 << 22) && ldw < (1 << 22);
}

bool attn_sizes_ok(int B, int Tq, int Hq, int Hk, int P, int S) {
  if (B < 0 || Tq < 0 || Hk < 1 || Hq < 1 || P < 0 || S < 0 || P >= (1 << 30) || S >= (1 << 30)) return false;
  if (B == 0 || Tq == 0) return true;
  if ((long long)B * Tq > 0x7fffffffLL / Hq) return false;
  // (a launch has fewer than 2^32 threads)
  const long long tiles = ((long long)Tq * Hq / Hk + 127) / 128;
  return (long long)B * Hk < (1 << 23) && (long long)B * Hk * (tiles > 0 ? tiles : 1) < (1 << 23);
}

}  // namespace

extern "C" {

int gkd_tokens_version(void) { return GKD_TOKENS_VERSION; }

size_t gkd_linear_workspace_size(int M, int N, int K, int64_t ldx, int64_t ldw) {
  if (!linear_sizes_ok(M, N, K, ldx, ldw) || M == 0 || N == 0) return 0;
  return gkd::linear_workspace_bytes(M, N, K, ldx, ldw);
}

gkd_status gkd_linear(const void* x, int64_t ldx, const void* w, int64_t ldw, const void* bias,
                      const void* residual, int64_t ldr, int M, int N, int K, gkd_activation act,
                      gkd_dtype dtype, gkd_dtype out_dtype, uint32_t flags, void* out, int64_t ldo,
                      void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const char* fn = "gkd_linear";
  if (flags != 0) return fail(GKD_ERR_UNSUPPORTED, "%s: unknown flags 0x%x", fn, (unsigned)flags);
  if ((dtype != GKD_DTYPE_F32 && dtype != GKD_DTYPE_BF16) ||
      (out_dtype != GKD_DTYPE_F32 && out_dtype != GKD_DTYPE_BF16))
    return fail(GKD_ERR_DTYPE, "%s: unknown dtype %d / %d", fn, (int)dtype, (int)out_dtype);
  if (dtype != GKD_DTYPE_BF16) return fail(GKD_ERR_UNSUPPORTED, "%s: needs bfloat16 operands", fn);
  if ((int)act < GKD_ACT_NONE || (int)act > GKD_ACT_SILU)
    return fail(GKD_ERR_VALUE, "%s: unknown activation %d", fn, (int)act);
  if (!linear_sizes_ok(M, N, K, ldx, ldw))
    return fail(GKD_ERR_SHAPE, "%s: bad shape M=%d N=%d K=%d ldx=%lld ldw=%lld", fn, M, N, K,
                (long long)ldx, (long long)ldw);
  if (ldo < N || (residual != nullptr && ldr < N))
    return fail(GKD_ERR_SHAPE, "%s: ldo=%lld or ldr=%lld below N=%d", fn, (long long)ldo, (long long)ldr, N);
  if (M == 0 || N == 0) return ok();
  if (!x || !w || !out) return fail(GKD_ERR_NULL, "%s: NULL pointer argument", fn);
  const unsigned size = out_dtype == GKD_DTYPE_F32 ? 4 : 2;
  if (!aligned(x, 16) || !aligned(w, 16))
    return fail(GKD_ERR_ALIGN, "%s: x and w need 16-byte alignment", fn);
  if (!aligned(bias, 2) || !aligned(residual, size) || !aligned(out, size))
    return fail(GKD_ERR_ALIGN, "%s: bias, residual and out need their element's alignment", fn);
  const gkd_status st = check_workspace(fn, workspace, workspace_bytes,
                                        gkd::linear_workspace_bytes(M, N, K, ldx, ldw));
  if (st != GKD_OK) return st;
  gkd::LinearArgs a;
  a.x = static_cast<const uint16_t*>(x);
  a.w = static_cast<const uint16_t*>(w);
  a.bias = static_cast<const uint16_t*>(bias);
  a.residual = residual;
  a.out = out;
  a.ldx = ldx;
  a.ldw = ldw;
  a.ldr = ldr;
  a.ldo = ldo;
  a.M = M;
  a.N = N;
  a.K = K;
  a.act = (int)act;
  a.out_f32 = out_dtype == GKD_DTYPE_F32;
  a.ws = workspace;
  return hip_status(gkd::launch_linear(a, stream), fn);
}

gkd_status gkd_qk_norm_rope(const gkd_heads* q, int Hq, const gkd_heads* k, int Hk, int B, int T,
                            int D, const float* pos, int64_t pos_batch, int n_axes,
                            const float* freqs, int rot, const void* q_weight,
                            const void* k_weight, float eps, gkd_dtype dtype, uint32_t flags,
                            const gkd_heads* q_out, const gkd_heads* k_out, hipStream_t stream) {
  const char* fn = "gkd_qk_norm_rope";
  if ((flags & ~GKD_ROPE_INTERLEAVED) != 0)
    return fail(GKD_ERR_UNSUPPORTED, "%s: unknown flags 0x%x", fn, (unsigned)flags);
  if (dtype != GKD_DTYPE_F32 && dtype != GKD_DTYPE_BF16)
    return fail(GKD_ERR_DTYPE, "%s: unknown dtype %d", fn, (int)dtype);
  if (B < 0 || T < 0 || Hq < 1 || Hk < 0 || D < 1 || rot < 2 || rot > D || rot % 2 != 0 || n_axes < 1 ||
      pos_batch < 0)
    return fail(GKD_ERR_SHAPE, "%s: bad shape B=%d T=%d Hq=%d Hk=%d D=%d rot=%d n_axes=%d", fn, B, T, Hq,
                Hk, D, rot, n_axes);
  if (D > 512 || n_axes > 8 || Hq > 65535 || Hk > 65535)
    return fail(GKD_ERR_UNSUPPORTED, "%s: needs D <= 512, n_axes <= 8 and at most 65535 heads", fn);
  if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(GKD_ERR_VALUE, "%s: eps must be finite and >= 0", fn);
  if (B == 0 || T == 0) return ok();
  const unsigned size = dtype == GKD_DTYPE_F32 ? 4 : 2;
  if ((Hk > 0) != (k != nullptr) || (Hk > 0) != (k_out != nullptr))
    return fail(GKD_ERR_NULL, "%s: k and k_out go with Hk > 0", fn);
  gkd_status st;
  if ((st = check_heads(fn, "q", q, size, size)) != GKD_OK) return st;
  if ((st = check_out(fn, "q_out", q_out, size, size, B, T, Hq)) != GKD_OK) return st;
  if (Hk > 0) {
    if ((st = check_heads(fn, "k", k, size, size)) != GKD_OK) return st;
    if ((st = check_out(fn, "k_out", k_out, size, size, B, T, Hk)) != GKD_OK) return st;
  }
  if (!pos || !freqs) return fail(GKD_ERR_NULL, "%s: NULL pos or freqs", fn);
  if (!aligned(pos, 4) || !aligned(freqs, 4) || !aligned(q_weight, size) || !aligned(k_weight, size))
    return fail(GKD_ERR_ALIGN, "%s: arrays need their element's alignment", fn);
  gkd::RopeArgs a;
  a.q = heads(q);
  a.k = heads(k);
  a.qo = heads(q_out);
  a.ko = heads(k_out);
  a.Hq = Hq;
  a.Hk = Hk;
  a.B = B;
  a.T = T;
  a.D = D;
  a.pos = pos;
  a.pos_batch = pos_batch;
  a.n_axes = n_axes;
  a.freqs = freqs;
  a.rot = rot;
  a.wq = q_weight;
  a.wk = k_weight;
  a.eps = eps;
  a.bf16 = dtype == GKD_DTYPE_BF16;
  a.interleaved = (flags & GKD_ROPE_INTERLEAVED) != 0;
  return hip_status(gkd::launch_rope(a, stream), fn);
}

size_t gkd_prefix_attention_workspace_size(int B, int Tq, int Hq, int Hk, int D, int P, int S) {
  if (!attn_sizes_ok(B, Tq, Hq, Hk, P, S) || Hq % Hk != 0 || (D != 64 && D != 128) || B == 0 || Tq == 0)
    return 0;
  return gkd::prefix_attn_workspace_bytes(B, Tq, Hq, Hk, D, P, S);
}

gkd_status gkd_prefix_attention(const gkd_heads* q, const gkd_heads* k_prefix,
                                const gkd_heads* v_prefix, int P, const gkd_heads* k_own,
                                const gkd_heads* v_own, int S, const int32_t* own_len,
                                const int32_t* q_len, const uint8_t* own_mask, int B, int Tq,
                                int Hq, int Hk, int D, float scale, gkd_dtype dtype, uint32_t flags,
                                const gkd_heads* out, void* workspace, size_t workspace_bytes,
                                hipStream_t stream) {
  const char* fn = "gkd_prefix_attention";
  if ((flags & ~GKD_ATTN_CAUSAL) != 0)
    return fail(GKD_ERR_UNSUPPORTED, "%s: unknown flags 0x%x", fn, (unsigned)flags);
  if (dtype != GKD_DTYPE_F32 && dtype != GKD_DTYPE_BF16)
    return fail(GKD_ERR_DTYPE, "%s: unknown dtype %d", fn, (int)dtype);
  if (dtype != GKD_DTYPE_BF16) return fail(GKD_ERR_UNSUPPORTED, "%s: needs bfloat16 operands", fn);
  if (!attn_sizes_ok(B, Tq, Hq, Hk, P, S) || D < 1)
    return fail(GKD_ERR_SHAPE, "%s: bad shape B=%d Tq=%d Hq=%d Hk=%d D=%d P=%d S=%d", fn, B, Tq, Hq, Hk, D, P, S);
  if ((D != 64 && D != 128) || Hq % Hk != 0)
    return fail(GKD_ERR_UNSUPPORTED, "%s: needs D 64 or 128 and Hq %% Hk == 0", fn);
  // (the kernels take base-2 scores: scale log2(e) must be finite too)
  if (!(scale > 0.f) || !(scale <= 2e38f))
    return fail(GKD_ERR_VALUE, "%s: scale must be above 0 and at most 2e38", fn);
  if (B == 0 || Tq == 0) return ok();
  gkd_status st;
  if ((st = check_heads(fn, "q", q, 2, 16)) != GKD_OK) return st;
  if ((st = check_out(fn, "out", out, 2, 16, B, Tq, Hq)) != GKD_OK) return st;
  if (P > 0) {
    if ((st = check_keys(fn, "k_prefix", k_prefix)) != GKD_OK) return st;
    if ((st = check_keys(fn, "v_prefix", v_prefix)) != GKD_OK) return st;
  }
  if (S > 0) {
    if ((st = check_keys(fn, "k_own", k_own)) != GKD_OK) return st;
    if ((st = check_keys(fn, "v_own", v_own)) != GKD_OK) return st;
  }
  if (!aligned(own_len, 4) || !aligned(q_len, 4))
    return fail(GKD_ERR_ALIGN, "%s: lengths need 4-byte alignment", fn);
  if ((st = check_workspace(fn, workspace, workspace_bytes,
                            gkd::prefix_attn_workspace_bytes(B, Tq, Hq, Hk, D, P, S))) != GKD_OK)
    return st;
  gkd::PrefixAttnArgs a;
  a.q = heads(q);
  a.kp = heads(P > 0 ? k_prefix : nullptr);
  a.vp = heads(P > 0 ? v_prefix : nullptr);
  a.ko = heads(S > 0 ? k_own : nullptr);
  a.vo = heads(S > 0 ? v_own : nullptr);
  a.out = heads(out);
  a.P = P;
  a.S = S;
  a.own_len = own_len;
  a.q_len = q_len;
  a.mask = S > 0 ? own_mask : nullptr;
  a.B = B;
  a.Tq = Tq;
  a.Hq = Hq;
  a.Hk = Hk;
  a.D = D;
  a.scale = scale;
  a.causal = (flags & GKD_ATTN_CAUSAL) != 0;
  a.ws = workspace;
  return hip_status(gkd::launch_prefix_attn(a, stream), fn);
}

}  // extern "C"
