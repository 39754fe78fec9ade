// Internal declarations of the mixture-of-experts operators (include/det_ops.h):
// what the C entry points hand to the kernel launchers.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace deto {

constexpr int kBlock = 128;          // contraction elements (and weight rows) one scale covers
constexpr int kMaxExperts = 512;
constexpr int kMaxTopK = 32;
constexpr float kE4M3Max = 448.0f;
constexpr float kAmaxMin = 7.888609052210118e-31f;   // 2^-100: keeps every scale a normal number
constexpr int kStatusInvalid = 1;    // DET_GEMM_ERR_INVALID_ARG, found by a kernel

// ---- routing
struct RouteParams {
    const void *logits;
    const float *bias;               // or null
    float *weights;                  // [T, k]
    int32_t *ids;                    // [T, k]
    const float *dw;                 // backward: [T, k]
    void *dlogits;                   // backward: [T, E]
    long long ldl, ldd;
    int tokens, experts, k, groups, top_groups, group_best, renorm, sigmoid;
    int group_mul;                   // floor(2^18 / experts of a group) + 1
    float scale;
};
cudaError_t launch_route_f32(const RouteParams &p, cudaStream_t s);
cudaError_t launch_route_bf16(const RouteParams &p, cudaStream_t s);
cudaError_t launch_route_bwd_f32(const RouteParams &p, cudaStream_t s);
cudaError_t launch_route_bwd_bf16(const RouteParams &p, cudaStream_t s);

// ---- stable sort by key (one cluster), rows to experts and back
struct SortParams {
    const void *keys;                // int32 or int64
    int keys64;
    int n, range;                    // keys in [0, range); any other goes last, as `range`
    int passes;                      // 1: the key is the digit; otherwise 9-bit digits
    // dispatch (passes == 1)
    int32_t *offsets, *rows, *slots;
    // runs: sorted keys and their original indexes, each position's run head, and which keys occur
    int32_t *kbuf[2], *ibuf[2];      // [n] each; the last pass leaves its result in buffer (passes - 1) & 1
    int32_t *head;
    uint8_t *seen;                   // [range], rounded up to 16
    void *zero;                      // rows to zero meanwhile: zero_rows of zero_cols bytes, zero_pitch bytes apart
    long long zero_rows, zero_cols, zero_pitch;
    int sms;
    int skip_key;                    // a key treated as out of range (or -1)
    int *status;
    int flag_bad;                    // report keys outside [0, range)
};
cudaError_t launch_sort(const SortParams &p, bool runs, cudaStream_t s);

struct GatherParams {
    const uint16_t *src;
    uint16_t *dst;
    const int32_t *rows;
    long long lds, ldd;
    int n, src_rows, cols, k;
};
cudaError_t launch_gather(const GatherParams &p, cudaStream_t s);

struct CombineParams {
    const uint16_t *ys, *dy;
    const int32_t *rows, *slots;
    const float *weights;            // or null: 1
    uint16_t *y, *dys;
    float *dw;
    long long ldys, ldy, lddy, lddys;
    int tokens, k, rows_n, cols;
};
cudaError_t launch_combine(const CombineParams &p, cudaStream_t s);
cudaError_t launch_combine_bwd(const CombineParams &p, cudaStream_t s);

// ---- embedding
struct EmbedParams {
    const void *tokens;
    int tokens64;
    const uint16_t *table;
    uint16_t *out;
    long long ldt, ldo;
    int n, vocab, cols;
    float scale;
    int *status;
};
cudaError_t launch_embedding(const EmbedParams &p, cudaStream_t s);

struct EmbedGradParams {
    const uint16_t *dy;
    void *dtable;
    long long lddy, ldd;
    int n, vocab, cols;
    float scale;
    int accumulate, fp32;
    const int32_t *keys, *order, *head;
    const uint8_t *seen;
    int zero_from;                   // rows from here on that never occur are zeroed
    float *partials;                 // [2 * ceil(n / 32), cols rounded up to 8]
    long long ldp;
};
cudaError_t launch_embedding_grad(const EmbedGradParams &p, cudaStream_t s);

// ---- 8-bit quantisers
struct QuantParams {
    const uint16_t *x;
    const int32_t *rows;             // rows: source row of each output row times k, or null
    const int32_t *offsets;          // columns: group bounds, or null
    uint8_t *q, *qt;
    float *s, *st;
    long long ldx, ldq, lds, ldqt, ldst;       // scale of (row m, block b): s[b * lds + m]
    long long xg, qg, sg, qtg, stg;  // tiles: strides between matrices
    int n, src_rows, cols, k, groups;
    int max_blocks;                  // columns: blocks of rows the output has room for
    int *status;
};
cudaError_t launch_quantize_rows(const QuantParams &p, cudaStream_t s);
cudaError_t launch_quantize_cols(const QuantParams &p, cudaStream_t s);
cudaError_t launch_quantize_tiles(const QuantParams &p, cudaStream_t s);

// ---- 8-bit block-scaled products: out[r, c] = sum over blocks b of
// sa(r, b) * sb(c, b) * (sum over the block of a[r, k] * b[c, k])
struct Fp8Params {
    CUtensorMap tmap_a;              // [rows, contraction]
    CUtensorMap tmap_b;              // [cols, contraction] (x experts)
    CUtensorMap tmap_sa, tmap_sb;    // weight gradient: the scales, [blocks, rows] and [blocks, cols]
    const float *sa, *sb;
    long long sa_row, sa_blk;        // scale of row r, block b: sa[r * sa_row + b * sa_blk]
    long long sb_row, sb_blk, sb_grp;
    void *out;
    long long ldo, og;               // pitch, elements between the groups' outputs (weight gradient)
    const int32_t *offsets;          // group bounds over the rows (or, weight gradient, over the contraction)
    int groups, rows, cols, kc;      // rows: all groups' rows
    int max_blocks;                  // contraction blocks that the operands and their scales hold
    int n_tiles, m_tiles;            // column tiles; row tiles when there are no offsets
    int out_fp32;
    int a_box, b_box;                // rows of the copied boxes
    int sa_box, sb_box;              // scales of the copied boxes
    int *status;
    unsigned long long timeout_ns;
    int force_timeout;
};
enum Fp8Kind { kFp8Rows = 0, kFp8Wgrad = 1 };
struct Fp8Plan {
    Fp8Kind kind;
    bool swap;                       // few rows: the weight on the MMA's row side
    int tile_m, tile_n;              // output tile: rows, columns
};
cudaError_t launch_fp8(const Fp8Params &p, const Fp8Plan &plan, int sms, cudaStream_t s);

}  // namespace deto
