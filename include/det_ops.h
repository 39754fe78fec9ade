/*
 * Operators around det_gemm's products for mixture-of-experts language
 * models on GB300 (sm_103a): routing to experts, dispatch and combine, 8-bit
 * (e4m3) matrix products with a scale for each block of 128, and the
 * embedding with its gradient. Part of libdet_gemm.so; status codes, BF16
 * values and streams are det_gemm.h's.
 *
 * Like det_gemm's products these are deterministic and batch-invariant: a
 * token's output is a function of that token's inputs (and the weights)
 * alone, every sum has a fixed order, and nothing is added with atomics.
 *
 * Conventions: matrices are row-major with a leading dimension in elements;
 * pointers are device pointers owned by the caller; base pointers of BF16
 * and e4m3 matrices are 16-byte aligned and their row pitches multiples of
 * 16 bytes; work is enqueued on `stream` and the call returns without
 * waiting; argument errors come back before anything is enqueued; an empty
 * output enqueues nothing; nothing is allocated. Outputs must not overlap
 * inputs (DET_GEMM_ERR_INVALID_ARG). What only the device can see (a token
 * outside the vocabulary, group bounds that decrease or leave the matrix, a
 * bounded wait that expired) is made harmless there, set in a status word
 * and reported by det_ops_check(). Not reported, because dropped pairs are
 * ordinary: an expert id outside [0, E), and a pair or row index outside its
 * range, count as -1. Sizes are below 2^31 - 4096, a vocabulary below 2^27 - 1
 * for its gradient.
 */
#ifndef DET_OPS_H
#define DET_OPS_H

#include "det_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define DET_MOE_MAX_EXPERTS 512
#define DET_MOE_MAX_TOP_K 32
#define DET_MOE_MAX_GROUPS 32
#define DET_FP8_BLOCK 128

/*
 * Routing. logits [T,E] are FP32 (logits_fp32 != 0) or BF16. Scores are
 * softmax (score 0) or sigmoid (score 1) of a token's logits; the choice is
 * score + bias (bias [E] FP32 or NULL). With n_groups > 1 the experts form
 * that many equal consecutive groups, a group's value is the sum of its best
 * group_best (1 or 2) choices, and only experts of the best top_groups
 * groups stay. ids[t] are the top_k largest choices in descending order,
 * ties (of experts and of groups) to the lower index; weights[t] their
 * scores (without the bias), divided by their sum when renormalize != 0 (a
 * sigmoid's sum plus 1e-20), times scale. An expert whose logit is -inf or
 * NaN, or whose bias is, is masked; a choice that is left over is id -1 with
 * weight 0. A logit of +inf is chosen like the largest finite FP32 value (no
 * smaller one goes before it), and the softmax weights of its row are NaN. A bias of +inf puts its
 * expert, and its group, first.
 * Which experts win is decided with 43 bits or more wherever FP32 cannot tell.
 * weights [T,top_k] FP32 and ids [T,top_k] are contiguous.
 */
det_gemm_status det_moe_route(const void *logits, int logits_fp32, const float *bias, float *weights, int32_t *ids,
                              int64_t T, int64_t E, int64_t ldl, int top_k, int score, int n_groups, int top_groups,
                              int group_best, int renormalize, float scale, det_gemm_stream stream);

/* dlogits [T,E] (the logits' type) from dweights [T,top_k] FP32, the logits
 * and the ids of det_moe_route; the choice itself is held fixed. */
det_gemm_status det_moe_route_bwd(const float *dweights, const void *logits, int logits_fp32, const int32_t *ids,
                                  void *dlogits, int64_t T, int64_t E, int64_t ldl, int64_t ldd, int top_k, int score,
                                  int renormalize, float scale, det_gemm_stream stream);

/*
 * Dispatch: the (token, choice) pairs f = t * top_k + j of ids [T,top_k] in
 * the order of their experts, pairs of one expert in ascending f. offsets
 * [E+1]: expert e's rows are [offsets[e], offsets[e+1]); rows [T*top_k]: the
 * pair of each row, -1 past offsets[E]; slots [T,top_k]: the row of each
 * pair, -1 for an id outside [0, E). All int32, contiguous.
 */
det_gemm_status det_moe_dispatch(const int32_t *ids, int32_t *offsets, int32_t *rows, int32_t *slots, int64_t T,
                                 int64_t E, int top_k, det_gemm_stream stream);

/* xs[r] = x[rows[r] / top_k], zero where rows[r] < 0. x [T,H], xs [R,H] BF16. */
det_gemm_status det_moe_gather(const det_gemm_bf16 *x, const int32_t *rows, det_gemm_bf16 *xs, int64_t T, int64_t R,
                               int64_t H, int top_k, int64_t ldx, int64_t ldxs, det_gemm_stream stream);

/* y[t] = sum over j of weights[t,j] * ys[slots[t,j]] (FP32, ascending j, one
 * rounding); weights NULL: 1 (the gather's gradient). ys [R,H], y [T,H]. */
det_gemm_status det_moe_combine(const det_gemm_bf16 *ys, const int32_t *slots, const float *weights, det_gemm_bf16 *y,
                                int64_t T, int64_t R, int64_t H, int top_k, int64_t ldys, int64_t ldy,
                                det_gemm_stream stream);

/* Gradients of det_moe_combine: dys[r] = weight * dy[token] (zero where no
 * token owns the row), dweights[t,j] = dy[t] . ys[slots[t,j]] (0 for slot
 * -1). rows and slots are det_moe_dispatch's, R = T * top_k. */
det_gemm_status det_moe_combine_bwd(const det_gemm_bf16 *dy, const det_gemm_bf16 *ys, const int32_t *rows,
                                    const int32_t *slots, const float *weights, det_gemm_bf16 *dys, float *dweights,
                                    int64_t T, int64_t H, int top_k, int64_t lddy, int64_t ldys, int64_t lddys,
                                    det_gemm_stream stream);

/*
 * e4m3 quantisers. For each block of 128: amax = max(max|x|, 2^-100),
 * s = amax / 448 (FP32), q = x * 448 / amax rounded once to e4m3 (nearest,
 * ties to even). A block that holds an infinity or a NaN gets s = NaN.
 * Scales are stored block-major: the scale of row r, block b is
 * s[b * lds + r].
 *
 * rows: blocks along a row. x [T,K] -> q [M,K], s [ceil(K/128), M]. With
 * `rows` (int32 [M], from det_moe_dispatch) output row r is x[rows[r] /
 * top_k], a zero row where rows[r] < 0; otherwise M == T.
 */
det_gemm_status det_fp8_quantize_rows(const det_gemm_bf16 *x, const int32_t *rows, uint8_t *q, float *s, int64_t T,
                                      int64_t M, int64_t K, int top_k, int64_t ldx, int64_t ldq, int64_t lds,
                                      det_gemm_stream stream);

/*
 * cols: blocks along a column, transposed, for products that contract over
 * the tokens. x [M,K] -> qt [K, nb*128], s [nb, K], nb blocks of 128 rows,
 * the last one padded with zeros: nb = ceil(M/128). With offsets (int32
 * [G+1]) each group's rows form their own blocks, one group after the other;
 * the blocks that exist number at most ceil(M/128) + G, which is what
 * max_blocks, the room in qt and s, has to be at least (max_blocks =
 * ceil(M/128) without offsets). Blocks that no group has are left alone, or
 * become zero where the bounds are reported.
 */
det_gemm_status det_fp8_quantize_cols(const det_gemm_bf16 *x, const int32_t *offsets, uint8_t *qt, float *s, int64_t M,
                                      int64_t K, int64_t G, int64_t max_blocks, int64_t ldx, int64_t ldqt, int64_t lds,
                                      det_gemm_stream stream);

/*
 * tiles: one scale for each 128 x 128 tile of G matrices w [N,K] (gw
 * elements apart). Writes q [N,K] with s [ceil(N/128), ceil(K/128)], and/or
 * the transpose qt [K,N] with st [ceil(K/128), ceil(N/128)]; either pair may
 * be NULL. Scales here are row-major and contiguous per matrix (gs apart).
 */
det_gemm_status det_fp8_quantize_tiles(const det_gemm_bf16 *w, uint8_t *q, float *s, uint8_t *qt, float *st, int64_t G,
                                       int64_t N, int64_t K, int64_t ldw, int64_t gw, int64_t ldq, int64_t gq,
                                       int64_t ldqt, int64_t gqt, det_gemm_stream stream);

/*
 * C[M,N] = sum over blocks b of 128 of sa[m,b] * sb[n/128,b] * (A_b . W_b):
 * A [M,K] e4m3 with the scale of row m, block b at sa[m * sa_row + b *
 * sa_blk]; W [N,K] e4m3 with the scale of tile (n/128, b) at sb[(n/128) *
 * sb_row + b]. The sum over a block is the tensor core's, in FP32; blocks
 * are added in ascending order in FP32 and C is rounded once (BF16, or FP32
 * with out_fp32). The input gradient is the same product with W transposed
 * (det_fp8_quantize_tiles writes both).
 */
det_gemm_status det_fp8_gemm(const uint8_t *A, const float *sa, const uint8_t *W, const float *sb, void *C,
                             int out_fp32, int64_t M, int64_t N, int64_t K, int64_t lda, int64_t sa_row,
                             int64_t sa_blk, int64_t ldw, int64_t sb_row, int64_t ldc, det_gemm_stream stream);

/*
 * The same per expert: rows [offsets[g], offsets[g+1]) of A with W_g (gw
 * elements apart, scales gsb apart). offsets (int32 [G+1]) is read on the
 * device. Rows of C outside every group become zero; all of them, where the
 * bounds go down somewhere.
 */
det_gemm_status det_fp8_gemm_grouped(const uint8_t *A, const float *sa, const uint8_t *W, const float *sb,
                                     const int32_t *offsets, void *C, int out_fp32, int64_t G, int64_t M, int64_t N,
                                     int64_t K, int64_t lda, int64_t sa_row, int64_t sa_blk, int64_t ldw, int64_t gw,
                                     int64_t sb_row, int64_t gsb, int64_t ldc, det_gemm_stream stream);

/*
 * Weight gradient: dW[N,K] = sum over the tokens of dY[m,n] X[m,k], from
 * det_fp8_quantize_cols of dY (Yt [N, *], scales sy [*, N]) and of X (Xt
 * [K, *], sx [*, K]), made with the same offsets. M is the number of tokens;
 * with offsets, dW is G matrices gdw elements apart, an expert without rows
 * gets zeros.
 */
det_gemm_status det_fp8_gemm_wgrad(const uint8_t *Yt, const float *sy, const uint8_t *Xt, const float *sx,
                                   const int32_t *offsets, void *dW, int out_fp32, int64_t G, int64_t M, int64_t N,
                                   int64_t K, int64_t max_blocks, int64_t ldyt, int64_t ldsy, int64_t ldxt,
                                   int64_t ldsx, int64_t lddw, int64_t gdw, det_gemm_stream stream);

/* out[t] = bf16(scale * table[tokens[t]]). table [V,H], out [T,H] BF16;
 * tokens int64 (tokens64 != 0) or int32. A token outside [0, V) gives a zero
 * row and DET_GEMM_ERR_INVALID_ARG from det_ops_check(). */
det_gemm_status det_embedding(const void *tokens, int tokens64, const det_gemm_bf16 *table, det_gemm_bf16 *out,
                              int64_t T, int64_t V, int64_t H, float scale, int64_t ldt, int64_t ldo,
                              det_gemm_stream stream);

/*
 * dtable[v] = scale * sum of dy[t] over tokens[t] == v, FP32: a token's
 * occurrences in ascending t in chunks of 32, chunks in ascending order; one
 * rounding to dtable's type (FP32 with out_fp32, else BF16). With accumulate
 * the sum is added to dtable and other rows are left alone; without, rows
 * that never occur become zero. padding_idx (or -1) gets no gradient. A
 * token outside [0, V) adds nothing and is reported as in det_embedding.
 * workspace: device memory of det_embedding_grad_workspace(T, V, H) bytes,
 * 256-byte aligned, used until the enqueued work is done.
 */
int64_t det_embedding_grad_workspace(int64_t T, int64_t V, int64_t H);
det_gemm_status det_embedding_grad(const det_gemm_bf16 *dy, const void *tokens, int tokens64, void *dtable,
                                   int out_fp32, int64_t T, int64_t V, int64_t H, float scale, int64_t padding_idx,
                                   int accumulate, int64_t lddy, int64_t ldd, void *workspace, int64_t workspace_bytes,
                                   det_gemm_stream stream);

/* Synchronises the stream, then reads and clears these operators' status
 * word of the current device (det_gemm_check does the same for det_gemm's). */
det_gemm_status det_ops_check(det_gemm_stream stream);

/* Test hook: while `enable` is nonzero, the 8-bit products' copy warp waits
 * on a barrier that nothing signals, for about 50 ms (see
 * det_gemm_debug_force_timeout). */
det_gemm_status det_ops_debug_force_timeout(int enable);

#ifdef __cplusplus
}
#endif

#endif /* DET_OPS_H */
