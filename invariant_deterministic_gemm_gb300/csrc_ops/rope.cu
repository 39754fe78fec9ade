// Rotary positions, and appending rotated keys and values to a paged cache.
//
//   (a, b) -> (a c - b s, b c + a s) for the column pairs of a head's first
//   `rot` columns, c and s from FP32 tables at the token's position; the other
//   columns, and values, are copied.
//
// The launch is bound by its bytes: each element is read and written once. A
// block takes one token (a part of its heads where tokens are few), a thread V
// pairs at a fixed place in the head, so the table's values are read once and
// serve all the thread's heads.
#include "attn_internal.h"
#include "launch.cuh"
#include "ops_internal.h"
#include "vec.cuh"

#include <algorithm>

namespace deto {
namespace {

constexpr int kThreads = 128;

template <int V>
struct Word;
template <>
struct Word<8> { using T = uint4; };
template <>
struct Word<4> { using T = uint2; };
template <>
struct Word<1> { using T = uint16_t; };

// V pairs: columns [x, x + V) and [y, y + V), or, interleaved, 2 V columns from x (y = x + V).
template <int V, bool INTER>
__device__ __forceinline__ void turn(uint16_t (&lo)[V], uint16_t (&hi)[V], const float (&c)[V], const float (&s)[V])
{
#pragma unroll
    for (int i = 0; i < V; ++i) {
        uint16_t &a = INTER ? (2 * i < V ? lo[(2 * i) % V] : hi[(2 * i) % V]) : lo[i];
        uint16_t &b = INTER ? (2 * i + 1 < V ? lo[(2 * i + 1) % V] : hi[(2 * i + 1) % V]) : hi[i];
        const float fa = bf_at(&a), fb = bf_at(&b);
        const uint32_t r = pack_bf16(fa * c[i] - fb * s[i], fb * c[i] + fa * s[i]);
        a = static_cast<uint16_t>(r);
        b = static_cast<uint16_t>(r >> 16);
    }
}

template <int V, bool INTER>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p)
{
    using W = typename Word<V>::T;
    if (gridDim.x * gridDim.y <= kFewBlocks) let_next_begin();
    wait_for_last();
    const int t = blockIdx.x, pairs = p.rot / 2 / V, items = pairs + (p.D - p.rot) / V;
    const int per = kThreads / items, item = threadIdx.x % items, first = threadIdx.x / items;
    const int pos = p.pos[t];
    const bool known = pos >= 0 && pos < p.P;
    int page = -1, at = 0;
    bool bad = !known;
    if (p.slots) {
        const int slot = p.slots[t];
        const long long room = static_cast<long long>(p.pages) * p.page_size;
        if (slot >= 0 && slot < room && known) {
            page = slot / p.page_size;
            at = slot - page * p.page_size;
        }
        bad |= slot < -1 || slot >= room;
    }
    if (bad && threadIdx.x == 0 && blockIdx.y == 0) atomicExch(p.status, kStatusInvalid);
    if (first >= per) return;
    float c[V], s[V];
    const bool pair_item = item < pairs;
    if (pair_item && known) {
        const float *cp = p.cosine + pos * p.ldt + item * V, *sp = p.sine + pos * p.ldt + item * V;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            c[i] = cp[i];
            s[i] = p.sign * sp[i];
        }
    }
    const int x = pair_item ? (INTER ? item * 2 * V : item * V) : p.rot + (item - pairs) * V;
    const int y = pair_item ? (INTER ? x + V : x + p.rot / 2) : x;
    const int heads = p.H + 2 * p.KV;
#pragma unroll 4
    for (int h = blockIdx.y * per + first; h < heads; h += gridDim.y * per) {
        const uint16_t *src;
        uint16_t *dst;
        if (h < p.H) {
            src = p.q.row(t, h);
            dst = p.out.row(t, h);
        } else {
            const bool key = h < p.H + p.KV;
            const int g = h - p.H - (key ? 0 : p.KV);
            src = key ? p.k.row(t, g) : p.v.row(t, g);
            if (page < 0) continue;
            dst = key ? p.kc.row(page, at, g) : p.vc.row(page, at, g);
        }
        union {
            W w;
            uint16_t e[V];
        } lo, hi;
        lo.w = *reinterpret_cast<const W *>(src + x);
        hi.w = *reinterpret_cast<const W *>(src + y);
        if (!known) {
#pragma unroll
            for (int i = 0; i < V; ++i) lo.e[i] = hi.e[i] = 0;
        } else if (pair_item && h < p.H + p.KV) {
            turn<V, INTER>(lo.e, hi.e, c, s);
        }
        *reinterpret_cast<W *>(dst + x) = lo.w;
        if (pair_item) *reinterpret_cast<W *>(dst + y) = hi.w;
    }
}

template <int V, bool INTER>
cudaError_t run(const RopeParams &p, int sms, cudaStream_t s)
{
    const int items = p.rot / 2 / V + (p.D - p.rot) / V, per = kThreads / items;
    const int turns = (p.H + 2 * p.KV + per - 1) / per;
    // Few tokens: a token's heads go to several blocks, until every SM has four.
    const int split = std::min(turns, std::max(1, 4 * sms / p.T));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.T), static_cast<unsigned>(split));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute a[1];
    a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = a;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, rope_kernel<V, INTER>, p);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

cudaError_t launch_rope(const RopeParams &p, bool interleaved, int sms, cudaStream_t s)
{
    if (p.rot % 16 == 0) return interleaved ? run<8, true>(p, sms, s) : run<8, false>(p, sms, s);
    if (p.rot % 8 == 0) return interleaved ? run<4, true>(p, sms, s) : run<4, false>(p, sms, s);
    return interleaved ? run<1, true>(p, sms, s) : run<1, false>(p, sms, s);
}

}  // namespace deto
