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
cudaError_t launch_rope(const RopeParams &p, bool interleaved, int sms, cudaStream_t s);

struct AttnParams {
    Heads q, k, v, out, dout, dq, dk, dv;
    float *lse;                      // [H, T]
    float *delta;                    // backward: [H, T]
    const int32_t *qb, *kb;          // bounds [N + 1], or null: one sequence
    int N, T, S, H, KV, G, D;
    float scale;
    int window, sinks;
    int *status;
    unsigned long long timeout_ns;
    int force_timeout;
};
// Heads [T, H, D] as (column, head, token), boxes of 64 columns of 128 tokens.
struct AttnMaps {
    CUtensorMap q, k, v, dout;
};
cudaError_t launch_attn(const AttnParams &p, const AttnMaps &maps, cudaStream_t s);
cudaError_t launch_attn_bwd(const AttnParams &p, const AttnMaps &maps, cudaStream_t s);

struct DecodeParams {
    Heads q, out;
    Cache kc, vc;
    const int32_t *table, *lengths;
    long long ldt;
    int B, H, KV, G, D, pages, page_size, max_pages;
    float scale;
    int window, sinks;
    int *status;
};
cudaError_t launch_attn_decode(const DecodeParams &p, int sms, cudaStream_t s);

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

// The last sequence whose first row (query, or key with of_keys) is at or before row t; its bounds need not hold t.
__device__ __forceinline__ int seq_of(const int32_t *bounds, int N, int t)
{
    int a = 0, b = N;
    while (b - a > 1) {
        const int mid = (a + b) >> 1;
        if (bounds[mid] <= t) a = mid;
        else b = mid;
    }
    return a;
}

__device__ __forceinline__ bool sees(const AttnParams &p, int position, int j)
{
    return j <= position && (position - j < p.window || j < p.sinks);
}

}  // namespace deto
