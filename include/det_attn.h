/*
 * Attention operators on GB300 (sm_103a): rotary positions, appending to a
 * paged key-value cache, attention of one new token over that cache, and
 * attention of packed sequences with its gradients. Part of libdet_gemm.so;
 * status codes, BF16 values and streams are det_gemm.h's.
 *
 * Like the library's products these are deterministic and batch-invariant:
 * a token's output is a function of its own sequence alone, whatever else
 * is in the batch and however a prompt is cut in chunks; every sum has a
 * fixed order and nothing is added with atomics. That holds for each operator
 * by itself: det_attn and det_attn_decode sum the same keys in orders of their
 * own, and the same token has other bits from one than from the other.
 *
 * Conventions: an array of heads is [tokens, heads, D] BF16 with unit stride
 * in D and a stride (in elements) for each other axis, so that views of one
 * projection's output are taken as they are; D is a multiple of 8, at most
 * 128. Base pointers are 16-byte aligned and strides multiples of 16 bytes;
 * rows of an array do not overlap. KV heads divide H: query head h reads KV
 * head h / (H / KV). Work is enqueued on `stream` and the call returns without
 * waiting; argument errors come back before anything is enqueued; an empty
 * output enqueues nothing; nothing is allocated, and a workspace is device
 * memory of the size that the function of its name gives, 256-byte aligned,
 * used until the enqueued work is done, until when inputs (lengths, tables
 * and bounds among them) stay as they are. Outputs must not overlap inputs or
 * each other, by their first and last bytes (DET_GEMM_ERR_INVALID_ARG).
 * What only the device can see (a position outside the tables, a slot or
 * page outside the cache, a length that the page table does not hold,
 * bounds that go down or leave the array) is made harmless there, set in a
 * status word and reported by det_ops_check(); a row that two sequences of
 * such bounds hold gets the results of either. Sizes are below 2^31 - 4096.
 *
 * Visible keys: query i of a sequence of n keys and m queries is at position
 * i + n - m (its last query at its last key) and sees the keys j at or
 * before it with position - j < window or j < sinks. window 0: no window.
 * A query that sees no key, or none whose score is above -infinity, gives
 * zeros (and lse -inf). Scores are scale q.k;
 * scale is positive and at most 2^127. What masked keys and values hold, infinities
 * and NaN included, does not reach the output. In det_attn a visible value that
 * is not finite is added as it is, however small its weight, and in det_attn_bwd
 * so is such a row of dout; det_attn_decode multiplies it with its weight in FP32
 * (NaN where that is zero).
 *
 * Precision: sums, maxima, exponentials and lse are FP32. The weights P are
 * rounded to BF16 for their product with the values, and results once. The
 * sum that det_attn divides by is that of P before this rounding,
 * det_attn_decode's that of the rounded ones.
 */
#ifndef DET_ATTN_H
#define DET_ATTN_H

#include "det_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define DET_ATTN_MAX_HEADS 1024
#define DET_ATTN_MAX_HEAD_DIM 128
#define DET_ATTN_MAX_SHARED 64

/*
 * Rotary positions: y = x with the first `rot` columns (even) of every head
 * turned. Column pairs (i, i + rot / 2), or (2i, 2i + 1) with interleaved,
 * (a, b) become (a c - b s, b c + a s), c and s being cos and sin [P, rot / 2]
 * (FP32, rows ldt apart) at the token's position; FP32, rounded once.
 * inverse != 0 turns back, which is also the gradient. A position outside
 * [0, P) gives a zero row and is reported. y may be x itself.
 */
det_gemm_status det_rope(const det_gemm_bf16 *x, const float *cosine, const float *sine, const int32_t *positions,
                         det_gemm_bf16 *y, int64_t T, int64_t H, int64_t D, int64_t rot, int64_t P, int interleaved,
                         int inverse, int64_t xt, int64_t xh, int64_t ldt, int64_t yt, int64_t yh,
                         det_gemm_stream stream);

/*
 * Appending: k turned as by det_rope and v as it is go to row slots[t] of the
 * caches, row s being token s % page_size of page s / page_size; q (or NULL)
 * turned goes to q_out. Slot -1 stores nothing. A slot outside the cache, or a
 * token whose position is outside the tables, stores nothing and is reported.
 * Slots other than -1 are distinct: of a slot that occurs twice the row holds
 * parts of either token. Caches have strides for page, token and head, and
 * may lie between one another (a buffer whose pages, tokens or heads hold
 * keys and then values).
 */
det_gemm_status det_kv_append(const det_gemm_bf16 *q, const det_gemm_bf16 *k, const det_gemm_bf16 *v, const float *cosine,
                              const float *sine, const int32_t *positions, const int32_t *slots, det_gemm_bf16 *q_out,
                              det_gemm_bf16 *k_cache, det_gemm_bf16 *v_cache, int64_t T, int64_t H, int64_t KV, int64_t D,
                              int64_t rot, int64_t P, int64_t pages, int64_t page_size, int interleaved, int64_t qt,
                              int64_t qh, int64_t kt, int64_t kh, int64_t vt, int64_t vh, int64_t ldt, int64_t ot,
                              int64_t oh, int64_t kcp, int64_t kcs, int64_t kch, int64_t vcp, int64_t vcs, int64_t vch,
                              det_gemm_stream stream);

/*
 * One new token a sequence: out[b] = attention of q[b] [H, D] over the first
 * lengths[b] tokens of sequence b, whose token j is token j % page_size of
 * page table[b * ldt + j / page_size]; the query is the last of them. Keys
 * are taken in chunks of 256 at fixed places, joined in a fixed order. Pages
 * past a sequence's length are not read, nor are those that the window hides.
 * A length outside [0, max_pages * page_size] counts as the nearest of the
 * two, a page outside the cache as hidden keys; both are reported. page_size
 * is a multiple of 8, H / KV at most DET_ATTN_MAX_SHARED.
 */
int64_t det_attn_decode_workspace(int64_t B, int64_t H, int64_t KV, int64_t D, int64_t max_tokens);
det_gemm_status det_attn_decode(const det_gemm_bf16 *q, const det_gemm_bf16 *k_cache, const det_gemm_bf16 *v_cache,
                                const int32_t *table, const int32_t *lengths, det_gemm_bf16 *out, int64_t B, int64_t H,
                                int64_t KV, int64_t D, int64_t pages, int64_t page_size, int64_t max_pages, float scale,
                                int64_t window, int64_t sinks, int64_t qt, int64_t qh, int64_t kcp, int64_t kcs,
                                int64_t kch, int64_t vcp, int64_t vcs, int64_t vch, int64_t ldt, int64_t ot, int64_t oh,
                                void *workspace, int64_t workspace_bytes, det_gemm_stream stream);

/*
 * Packed sequences: sequence n has the queries [q_bounds[n], q_bounds[n+1])
 * and the keys [k_bounds[n], k_bounds[n+1]), int32 [N+1] on the device.
 * k_bounds NULL: the same as the queries'. q_bounds NULL as well: one sequence
 * (N = 1) of all T queries and S keys. out [T, H, D]; lse [H, T] FP32,
 * contiguous: log of the sum of exp(scores). Queries outside every sequence
 * give zeros and -inf.
 */
det_gemm_status det_attn(const det_gemm_bf16 *q, const det_gemm_bf16 *k, const det_gemm_bf16 *v, const int32_t *q_bounds,
                         const int32_t *k_bounds, det_gemm_bf16 *out, float *lse, int64_t N, int64_t T, int64_t S,
                         int64_t H, int64_t KV, int64_t D, float scale, int64_t window, int64_t sinks, int64_t qt,
                         int64_t qh, int64_t kt, int64_t kh, int64_t vt, int64_t vh, int64_t ot, int64_t oh,
                         det_gemm_stream stream);

/*
 * Gradients of det_attn: dq [T, H, D], dk and dv [S, KV, D] from dout, the
 * inputs, out and lse. With P = exp(scores - lse): dv = P^T dout, dS = P
 * (dout v^T - rowsum(dout out)), dq = scale dS k, dk = scale dS^T q, summed over
 * the query heads that share a KV head. out and lse may be those of more keys
 * than these (results over several ranges of keys, joined). A query that sees
 * a single key, and whose lse is that key's score, has dS = 0 and not the
 * rounding of its two terms. P and dS are rounded to BF16 for their second
 * products. Rows outside every sequence become zero.
 */
int64_t det_attn_bwd_workspace(int64_t N, int64_t T, int64_t S, int64_t H, int64_t KV, int64_t D, int64_t window,
                               int64_t sinks);
det_gemm_status det_attn_bwd(const det_gemm_bf16 *dout, const det_gemm_bf16 *q, const det_gemm_bf16 *k,
                             const det_gemm_bf16 *v, const det_gemm_bf16 *out, const float *lse, const int32_t *q_bounds,
                             const int32_t *k_bounds, det_gemm_bf16 *dq, det_gemm_bf16 *dk, det_gemm_bf16 *dv, int64_t N,
                             int64_t T, int64_t S, int64_t H, int64_t KV, int64_t D, float scale, int64_t window,
                             int64_t sinks, int64_t dot, int64_t doh, int64_t qt, int64_t qh, int64_t kt, int64_t kh,
                             int64_t vt, int64_t vh, int64_t ot, int64_t oh, int64_t dqt, int64_t dqh, int64_t dkt,
                             int64_t dkh, int64_t dvt, int64_t dvh, void *workspace, int64_t workspace_bytes,
                             det_gemm_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* DET_ATTN_H */
