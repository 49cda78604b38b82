/*
 * gkdtokens.h - C ABI of libgkdhead's token operators: the pieces of a
 * transformer block over image tokens and prompt rows, as calls of their
 * own (gkdhead.h's gkd_kg_transformer runs a whole transformer).
 *
 *   gkd_linear            matrix product with bias, activation and residual
 *                         in its epilogue
 *   gkd_qk_norm_rope      norm of each query and key head and rotary
 *                         positions with several axes, in one pass
 *   gkd_prefix_attention  attention of a batch that shares one long prefix
 *                         of keys (an image's tokens, a common prompt), each
 *                         sequence with own keys behind it
 *
 * They run forward only, like the rest of the library: it trains nothing.
 *
 * Conventions are those of gkdhead.h (device pointers owned by the caller,
 * asynchronous calls ordered on `stream`, checks before any launch, status
 * codes and gkd_last_error(), no allocation, no state kept between calls),
 * with these differences, made for long caches and packed projections:
 *   - operands have strides, in elements; offsets are 64-bit, so an array
 *     may hold more than 2^31 elements (each size by itself is an int).
 *   - alignment is stated at each call.
 *   - a call that takes a workspace needs it to itself until it has run:
 *     calls that share one must not overlap, also when they are replayed
 *     from captured graphs. Its contents on entry do not matter.
 *   - `stream` belongs to the current device, and so do the arrays.
 *
 * These entry points joined the library without a change to gkdhead.h's:
 * GKD_ABI_VERSION counts the latter, GKD_TOKENS_VERSION these.
 */
#ifndef GKDTOKENS_H
#define GKDTOKENS_H

#include "gkdhead.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GKD_TOKENS_VERSION 1

/* GKD_TOKENS_VERSION of the loaded library. */
GKD_API int gkd_tokens_version(void);

typedef enum {
    GKD_ACT_NONE = 0,
    GKD_ACT_RELU = 1,       /* max(z, 0) */
    GKD_ACT_GELU = 2,       /* z (1 + erf(z / sqrt 2)) / 2 */
    GKD_ACT_QUICK_GELU = 3, /* z / (1 + exp(-1.702 z)) */
    GKD_ACT_SILU = 4        /* z / (1 + exp(-z)) */
} gkd_activation;

/* Heads in memory: element (b, t, h, d) of a [B, T, H, D] operand is
 * data[b*batch + t*token + h*head + d]. Strides are in elements, none
 * negative; a head's D values are adjacent. An output's elements all have
 * places of their own: a stride of 0 over a size above one is refused there
 * (GKD_ERR_SHAPE), and allowed for inputs. */
typedef struct {
    void *data;
    int64_t batch, token, head;
} gkd_heads;

/*
 * Matrix product with bias, activation and residual:
 *   out[m,n] = act(sum_k x[m,k] w[n,k] + bias[n]) + residual[m,n]
 * (w as a torch Linear weight). bfloat16 operands, float32 accumulation and
 * epilogue, one rounding to out_dtype at the end. The activations are right
 * to 2^-20 |z| (GELU by a polynomial, in its tail down to z = -6 to 2^-12 of
 * itself; quick GELU and SiLU by the hardware's exponential and reciprocal).
 *
 *   x        [M,K] bf16, row stride ldx >= K, 16-byte aligned
 *   w        [N,K] bf16, row stride ldw >= K, 16-byte aligned
 *   bias     [N]   bf16 or NULL
 *   residual [M,N] out_dtype or NULL, row stride ldr >= N
 *   out      [M,N] out_dtype (bf16 or f32), row stride ldo >= N; may be
 *            `residual` itself (same pointer and stride), else it overlaps
 *            no input
 *   workspace  gkd_linear_workspace_size() bytes, 256-byte aligned (NULL
 *            where that is 0). Operands whose rows do not all start on
 *            16-byte boundaries (ldx or ldw % 8 != 0, or K % 8 != 0) are
 *            first copied there; any other layout runs in place.
 * Any M, N >= 0 and K >= 1 (M < 2^26, N < 2^25, M N < 2^36, ldx, ldw < 2^22,
 * else GKD_ERR_SHAPE);
 * dtype must be GKD_DTYPE_BF16. flags must be 0. M == 0 or N == 0: nothing
 * is launched.
 */
GKD_API size_t gkd_linear_workspace_size(int M, int N, int K, int64_t ldx, int64_t ldw);
GKD_API gkd_status gkd_linear(const void *x, int64_t ldx, const void *w, int64_t ldw,
                              const void *bias, const void *residual, int64_t ldr, int M, int N,
                              int K, gkd_activation act, gkd_dtype dtype, gkd_dtype out_dtype,
                              uint32_t flags, void *out, int64_t ldo, void *workspace,
                              size_t workspace_bytes, hipStream_t stream);

/* gkd_qk_norm_rope flag: pair i is elements (2i, 2i + 1) instead of
 * (i, i + rot/2). */
#define GKD_ROPE_INTERLEAVED 0x1u

/*
 * Head norm and rotary positions of queries and keys, in one pass.
 * For each token t of sequence b and each head x (D values):
 *   u = x / sqrt(mean(x^2) + eps) * weight      (weight NULL: u = x)
 *   phi_i = sum_a pos[b,t,a] freqs[a,i]          0 <= i < rot/2
 *   y_p = u_p cos phi_i - u_q sin phi_i
 *   y_q = u_q cos phi_i + u_p sin phi_i          (p, q) = (i, i + rot/2)
 * and y = u for the elements past rot. A frequency that belongs to one axis
 * alone has 0 in the other axes' rows, so sections of frequencies per axis
 * (time, height, width), frequencies dealt to the axes in turn and mixed
 * ones are all this one table. phi is summed and reduced to one turn in
 * float64 (positions of 10^6 keep their angle), cosines and sines are right
 * to 2^-25 for f32 and to 2^-22 for bf16 heads (the hardware's functions);
 * norms, rotation and weights are float32 (a head's squares must stay
 * finite there), rounded once to dtype. Without a norm a value that is not
 * finite stays within its pair, and past rot within its element.
 *
 *   q, q_out [B,T,Hq,D] dtype; k, k_out [B,T,Hk,D] dtype, or both NULL with
 *            Hk = 0. An output may be its input itself (same data and
 *            strides), else it overlaps no input.
 *   pos      [B,T,n_axes] float32, sequence b at pos + b*pos_batch (0: one
 *            table for all sequences); whole numbers or coordinates. Tokens
 *            without a position (class, storage tokens) take zeros.
 *   freqs    [n_axes, rot/2] float32
 *   q_weight, k_weight [D] dtype or NULL
 * Limits: D <= 512, rot even, 2 <= rot <= D, 1 <= n_axes <= 8, eps >= 0
 * and finite. dtype: f32 or bf16. Arrays are aligned to their elements.
 * Where data pointers and strides are multiples of 16 bytes and D fills
 * whole 16-byte pieces, 16-byte accesses are used.
 */
GKD_API gkd_status gkd_qk_norm_rope(const gkd_heads *q, int Hq, const gkd_heads *k, int Hk, int B,
                                    int T, int D, const float *pos, int64_t pos_batch, int n_axes,
                                    const float *freqs, int rot, const void *q_weight,
                                    const void *k_weight, float eps, gkd_dtype dtype,
                                    uint32_t flags, const gkd_heads *q_out,
                                    const gkd_heads *k_out, hipStream_t stream);

/* gkd_prefix_attention flag: query i of sequence b (q_len[b] queries, the
 * last of its own_len[b] own tokens) sees own keys
 * j <= own_len[b] - q_len[b] + i only. */
#define GKD_ATTN_CAUSAL 0x1u

/*
 * Attention of a batch with a shared prefix of keys:
 *   out[b,i,h] = softmax_j(scale q[b,i,h] . K_j) V_j
 * over the P prefix keys, the same for every sequence and held once for the
 * whole batch, and the sequence's own keys j < own_len[b] with own_mask[b,j]
 * set (and, with GKD_ATTN_CAUSAL, visible to query i). Head h reads key
 * head h / (Hq / Hk). A query that sees no key gives zeros.
 *
 *   q, out   [B,Tq,Hq,D] bf16. Queries i >= q_len[b] are not computed and
 *            their rows of out not written.
 *   k_prefix, v_prefix [P,Hk,D] bf16 (their batch stride is not used);
 *            NULL allowed if P == 0
 *   k_own, v_own [B,S,Hk,D] bf16; NULL allowed if S == 0
 *   own_len  [B] int32 or NULL (S); values are clamped to 0..S
 *   q_len    [B] int32 or NULL (Tq); values are clamped to 0..Tq
 *   own_mask [B,S] uint8 or NULL (all set)
 *   workspace  gkd_prefix_attention_workspace_size() bytes, 256-byte
 *            aligned (NULL where that is 0)
 * Own keys and values past own_len or masked may hold anything, NaN
 * included, and so may queries past q_len; every other input must be
 * finite, and the products q . K_j, as they are and scaled, at most 1e38
 * in magnitude. Scores, softmax statistics and outputs are float32;
 * probabilities are rounded to bfloat16 for the product with V and summed
 * as they are there. Limits: D 64 or 128, Hq a multiple of Hk, B Tq Hq
 * below 2^31, B Hk ceil(Tq Hq / Hk / 128) below 2^23, P and S below 2^30,
 * 0 < scale <= 2e38; dtype must be GKD_DTYPE_BF16. q, k, v and out:
 * 16-byte aligned data, strides multiples of 8 (else GKD_ERR_ALIGN); token
 * strides of keys and values below 2^25 (else GKD_ERR_SHAPE). `out`
 * overlaps no input.
 */
GKD_API size_t gkd_prefix_attention_workspace_size(int B, int Tq, int Hq, int Hk, int D, int P,
                                                   int S);
GKD_API gkd_status gkd_prefix_attention(const gkd_heads *q, const gkd_heads *k_prefix,
                                        const gkd_heads *v_prefix, int P, const gkd_heads *k_own,
                                        const gkd_heads *v_own, int S, const int32_t *own_len,
                                        const int32_t *q_len, const uint8_t *own_mask, int B,
                                        int Tq, int Hq, int Hk, int D, float scale,
                                        gkd_dtype dtype, uint32_t flags, const gkd_heads *out,
                                        void *workspace, size_t workspace_bytes,
                                        hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GKDTOKENS_H */
