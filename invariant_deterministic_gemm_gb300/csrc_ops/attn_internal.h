// Internal declarations of the attention operators (include/det_attn.h): what
// the C entry points hand to the kernel launchers.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace deto {

constexpr int kNoWindow = 0x7FFFFFFF;

// An array of heads [tokens, heads, D]: strides in elements.
struct Heads {
    uint16_t *p;
    long long t, h;
    __device__ uint16_t *row(long long token, int head) const { return p + token * t + head * h; }
};

// A cache [pages, page_size, heads, D].
struct Cache {
    uint16_t *p;
    long long page, s, h;
    __device__ uint16_t *row(int pg, int at, int head) const { return p + pg * page + at * s + head * h; }
};

struct RopeParams {
    Heads q, k, v, out;              // q -> out; k, v -> the caches
    Cache kc, vc;
    const float *cosine, *sine;      // [P, rot / 2], rows ldt apart
    const int32_t *pos, *slots;
    long long ldt;
    int T, H, KV, D, rot, P;         // KV 0: rotation alone
    int pages, page_size;
    float sign;                      // -1: back
    int *status;
};
cudaError_t launch_rope(const RopeParams &p, bool interleaved, cudaStream_t s);

struct AttnParams {
    Heads q, k, v, out, dout, dq, dk, dv;
    float *lse;                      // [H, T]
    float *delta;                    // backward: [H, T]
    float *partials;                 // backward: the first keys' gradients by pieces, [pieces][2: dv, dk][128][D]
    int sink_blocks;                 // blocks of first keys that are taken in pieces (0: none)
    const int32_t *qb, *kb;          // bounds [N + 1], or null: one sequence
    int N, T, S, H, KV, G, D;
    float scale;
    int window, sinks;
    int *status;
    unsigned long long timeout_ns;
    int force_timeout;
};
// Heads [T, H, D] as (column, head, token): inputs (o: the forward pass's output) in boxes of 64 columns of 128 tokens, outputs
// (out, or dq in its place, dk and dv) in boxes of 32 tokens.
struct AttnMaps {
    CUtensorMap q, k, v, dout, o, out, dk, dv;
};
cudaError_t launch_attn(const AttnParams &p, const AttnMaps &maps, cudaStream_t s);
// With a window the first keys, which stay visible, are seen by all queries and the others by few: their gradients are summed
// in pieces of so many queries, and the pieces joined. Only where there are at most kPieceSinks of them.
constexpr int kPiece = 512, kPieceSinks = 512;
inline int sink_blocks(long long window, long long sinks) { return window > 0 && sinks > 0 && sinks <= kPieceSinks ? static_cast<int>((sinks + 127) / 128) : 0; }
inline long long piece_slots(long long T, long long N, bool packed) { return packed ? T / kPiece + (N > 1 ? N : 1) : (T + kPiece - 1) / kPiece; }
cudaError_t launch_attn_bwd(const AttnParams &p, const AttnMaps &maps, cudaStream_t s);

// The key axis of one sequence of a decode step: chunks of 256 keys, four to a block, 16 blocks to a super block. A
// sequence's result is its super blocks joined in ascending order, each of its blocks, each of its chunks.
constexpr int kChunk = 256, kBlockChunks = 4, kSuperChunks = 64;

// Where a CTA's run begins inside a list (a sequence, KV head and part of its query heads), if no CTA before it does: the
// list's first unit and their number (0: nothing to join), chunks a unit.
struct Cut {
    long long first;
    int n, b, list, unit;
};

struct DecodeParams {
    Heads q, out;
    const int32_t *table, *lengths;
    long long ldt;
    int B, H, KV, G, D, pages, page_size, max_pages;
    int parts, heads;                // query heads of a KV head are taken in `parts` of at most `heads`
    int box;                         // tokens of one copy: a power of two that divides the page
    float scale;
    int window, sinks;
    Cut *cuts;                       // of each CTA's begin
    float *partials;                 // of each unit: [heads][D] sums, [heads] l, [heads] m
    int *status;
    unsigned long long timeout_ns;
    int force_timeout;
};
struct DecodeMaps {
    CUtensorMap q;                   // (column, head, sequence): boxes of 64 columns of 16 or 32 heads
    CUtensorMap k, v;                // (column, head, token of a page, page): boxes of 64 columns of `box` tokens
};
cudaError_t launch_attn_decode(const DecodeParams &p, const DecodeMaps &maps, int sms, cudaStream_t s);

// Units that a launch of `ctas` may leave in parts: chunks while there are few blocks, blocks while there are few super
// blocks. At most `tokens` tokens a sequence, `lists` sequences times KV heads.
constexpr int kUnitsEach = 4;        // units for every CTA that are enough
inline long long decode_slots(long long lists, long long tokens, long long ctas)
{
    const auto least = [](long long a, long long b) { return a < b ? a : b; };
    const long long chunks = least(lists * ((tokens + kChunk - 1) / kChunk), kUnitsEach * kBlockChunks * ctas);
    const long long block = kChunk * kBlockChunks, super = kChunk * kSuperChunks;
    const long long blocks = least(lists * ((tokens + block - 1) / block), kUnitsEach * (kSuperChunks / kBlockChunks) * ctas);
    const long long supers = lists * ((tokens + super - 1) / super);
    const long long most = chunks > blocks ? chunks : blocks;
    return most > supers ? most : supers;
}

// ---- sequences and what a query sees

struct Seq {
    int q0, q1, k0, k1;
    __device__ int queries() const { return q1 - q0; }
    __device__ int keys() const { return k1 - k0; }
    // Position of the query in row t.
    __device__ int position(int t) const { return t - q0 + (k1 - k0) - (q1 - q0); }
};

// Bounds of sequence n, inside the arrays whatever the numbers say.
__device__ __forceinline__ Seq seq_at(const AttnParams &p, int n)
{
    Seq s;
    s.q0 = p.qb ? min(max(p.qb[n], 0), p.T) : 0;
    s.q1 = p.qb ? min(max(p.qb[n + 1], s.q0), p.T) : p.T;
    s.k0 = p.kb ? min(max(p.kb[n], 0), p.S) : 0;
    s.k1 = p.kb ? min(max(p.kb[n + 1], s.k0), p.S) : p.S;
    return s;
}

__device__ __forceinline__ bool sees(const AttnParams &p, int position, int j)
{
    return j <= position && (position - j < p.window || j < p.sinks);
}
// A query at `position` (0 or more) sees a single key of these.
__device__ __forceinline__ bool sees_one(const AttnParams &p, int position) { return position == 0 || (p.window == 1 && p.sinks == 0); }

}  // namespace deto
