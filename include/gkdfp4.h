/*
 * gkdfp4.h - C ABI of libgkdhead's four-bit token operators: products with
 * weights, and attention over a cache of keys and values, that are held in
 * 4.25 bits a value (gkdtokens.h's gkd_linear and gkd_prefix_attention hold
 * both in bfloat16).
 *
 *   gkd_quantize_fp4     rows of values -> codes and scales (weights, once)
 *   gkd_linear_fp4       matrix product with such weights, bias, activation
 *                        and residual
 *   gkd_cache_append     new tokens' keys and values into a cache's pages
 *   gkd_cache_read       a cache's tokens back, in bfloat16
 *   gkd_cache_attention  attention over a cache
 *
 * THE FORMAT. 32 neighbouring values are a group with one scale byte s; each
 * value has a code of 4 bits: the sign (bit 3) and the size 0, 0.5, 1, 1.5,
 * 2, 3, 4 or 6 (bits 2..0). A value is code * 2^(s - 127); s = 255 makes the
 * whole group NaN. A byte holds two codes, the earlier value's in its low
 * half. n values (n a multiple of 32) take n/2 bytes of codes and n/32 of
 * scales. (These are the element and scale types of the Open Compute
 * Project's MXFP4, which this GPU converts by itself.) Values come from the
 * scale byte by exact arithmetic where bfloat16 has them; code * 2^(s - 127)
 * past its range is infinite, and below 2^-126 may count as 0 in products.
 *
 * QUANTISING takes the largest magnitude a of a group and the least whole e
 * with a < 7 * 2^e, kept within -125..125: s = e + 127. The codes are the
 * nearest ones to value / 2^e, ties to the even code, sizes past 6 as 6. So
 * no value of a group is off by more than half its code's step, except past
 * 7 * 2^125. A group with a value that is not finite gets s = 255 and codes
 * of 0.
 *
 * Conventions are those of gkdtokens.h: strides in elements, offsets in 64
 * bits, checks before any launch, a workspace to itself until its call has
 * run, `stream` and all arrays of the current device. Codes and scales are
 * dense and 16-byte aligned. Forward only.
 *
 * GKD_FP4_VERSION counts these entry points.
 */
#ifndef GKDFP4_H
#define GKDFP4_H

#include "gkdtokens.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GKD_FP4_VERSION 1

/* GKD_FP4_VERSION of the loaded library. */
GKD_API int gkd_fp4_version(void);

/*
 * Rows of values into codes and scales.
 *   x      [N,K] dtype (f32 or bf16), row stride ldx >= K; 16-byte aligned
 *          data and rows
 *   codes  [N,K/2] uint8, scales [N,K/32] uint8
 * K a multiple of 32 (else GKD_ERR_UNSUPPORTED) and >= 32, N >= 0. flags
 * must be 0. N == 0: nothing is launched. Outputs overlap no input.
 */
GKD_API gkd_status gkd_quantize_fp4(const void *x, int64_t ldx, int N, int K, gkd_dtype dtype,
                                    uint32_t flags, uint8_t *codes, uint8_t *scales,
                                    hipStream_t stream);

/*
 * Matrix product with four-bit weights:
 *   out[m,n] = act(sum_k x[m,k] w[n,k] + bias[n]) + residual[m,n]
 * with float32 accumulation and epilogue and one rounding to out_dtype at
 * the end, as gkd_linear (activations, bias and residual are its own).
 *   x        [M,K] bf16, row stride ldx >= K, 16-byte aligned data and rows
 *            (ldx % 8 == 0)
 *   codes    [N,K/2], scales [N,K/32]
 *   bias     [N]   bf16 or NULL
 *   residual [M,N] out_dtype or NULL, row stride ldr >= N
 *   out      [M,N] out_dtype (bf16 or f32), row stride ldo >= N; may be
 *            `residual` itself (same pointer and stride), else it overlaps
 *            no input
 * K a multiple of 32 (else GKD_ERR_UNSUPPORTED), 32 <= K < 2^22, M < 2^26,
 * N < 2^25, M N < 2^31, ldx < 2^22 (else GKD_ERR_SHAPE). flags must be 0.
 * M == 0 or N == 0: nothing is launched.
 *   workspace  gkd_linear_fp4_workspace_size() bytes, 256-byte aligned (NULL
 *            where that is 0)
 */
GKD_API size_t gkd_linear_fp4_workspace_size(int M, int N, int K);
GKD_API gkd_status gkd_linear_fp4(const void *x, int64_t ldx, const uint8_t *codes,
                                  const uint8_t *scales, const void *bias, const void *residual,
                                  int64_t ldr, int M, int N, int K, gkd_activation act,
                                  gkd_dtype out_dtype, uint32_t flags, void *out, int64_t ldo,
                                  void *workspace, size_t workspace_bytes, hipStream_t stream);

/* A cache of keys and values in pages of `page` tokens: page p's keys are
 * [p,0], its values [p,1] of
 *   codes  [pages, 2, Hk, page, D/2] uint8
 *   scales [pages, 2, Hk, page, D/32] uint8
 * A table [B,L] int32 names the pages of each sequence: its token i is in row
 * i % page of page table[b, i / page]. An entry outside 0..pages - 1 stands
 * for no page: what would go there is dropped, and its tokens are not
 * attended to. Sequences may share pages.
 * D 64 or 128; page a multiple of 32, at most 65536; 1 <= Hk <= 65536;
 * pages >= 0; L >= 0, L page < 2^30. */
typedef struct {
    uint8_t *codes, *scales;
    int pages, page, Hk, D;
} gkd_cache;

/*
 * New tokens' keys and values, quantised into a cache's pages: token t of
 * sequence b, t < count[b], goes to place start[b] + t. Places below 0, past
 * the table's pages or without a page are dropped.
 *   k, v   [B,T,Hk,D] dtype (f32 or bf16), 16-byte aligned data and strides
 *   start  [B] int32 or NULL (0)
 *   count  [B] int32 or NULL (T); values are clamped to 0..T
 * Two tokens of a call must not have the same place (which of them, or what
 * mixture, stays is undefined). Nothing but the tokens' places is written.
 * B T below 2^31, T below 2^30. flags must be 0.
 */
GKD_API gkd_status gkd_cache_append(const gkd_heads *k, const gkd_heads *v, int B, int T,
                                    const int32_t *start, const int32_t *count,
                                    const gkd_cache *cache, const int32_t *table, int L,
                                    gkd_dtype dtype, uint32_t flags, hipStream_t stream);

/*
 * Tokens of a cache, as values in bfloat16 (exact, but where 2^(s - 127)
 * leaves its range): token t < count[b] of sequence b is the one at place
 * start[b] + t; zeros where there is no such place or page. Tokens past
 * count[b] are not written. Arguments as gkd_cache_append's; k and v
 * [B,T,Hk,D] bf16 are the outputs, 16-byte aligned data and strides.
 */
GKD_API gkd_status gkd_cache_read(const gkd_cache *cache, const int32_t *table, int L, int B,
                                  int T, const int32_t *start, const int32_t *count,
                                  uint32_t flags, const gkd_heads *k, const gkd_heads *v,
                                  hipStream_t stream);

/*
 * Attention over a cache:
 *   out[b,i,h] = softmax_j(scale q[b,i,h] . K_j) V_j
 * over the tokens j < length[b] of sequence b; with GKD_ATTN_CAUSAL, where
 * the q_len[b] queries are the last tokens, over j <= length[b] - q_len[b] + i.
 * Head h reads key head h / (Hq / Hk). A query that sees no key gives zeros.
 *   q, out   [B,Tq,Hq,D] bf16, 16-byte aligned data and strides. Queries
 *            i >= q_len[b] are not computed and their rows of out not written.
 *   length   [B] int32 or NULL (L page); values are clamped to 0..L page
 *   q_len    [B] int32 or NULL (Tq); values are clamped to 0..Tq
 *   workspace  gkd_cache_attention_workspace_size() bytes, 256-byte aligned
 *            (NULL where that is 0)
 * Pages' rows past length[b] may hold anything, NaN included, and so may
 * queries past q_len; the other values must be finite, the products q . K_j,
 * as they are and scaled, at most 1e38 and the values V_j at most 1e24 in
 * magnitude (sums hold up to 2^30 of them, times 2^16 at most). Scores, softmax
 * statistics and outputs are float32; probabilities are rounded to bfloat16
 * for the product with V and summed as they are there. Hq a multiple of Hk,
 * B Tq Hq below 2^31, B Hk ceil(Tq Hq / Hk / 16) below 2^21, 0 < scale <=
 * 2e38. `out` overlaps no input.
 */
GKD_API size_t gkd_cache_attention_workspace_size(int B, int Tq, int Hq, int Hk, int D, int page,
                                                  int L);
GKD_API gkd_status gkd_cache_attention(const gkd_heads *q, const gkd_cache *cache,
                                       const int32_t *table, int L, const int32_t *length,
                                       const int32_t *q_len, int B, int Tq, int Hq, float scale,
                                       uint32_t flags, const gkd_heads *out, void *workspace,
                                       size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GKDFP4_H */
