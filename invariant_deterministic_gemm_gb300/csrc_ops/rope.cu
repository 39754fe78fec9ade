// Rotary positions, and appending rotated keys and values to a paged cache.
//
//   (a, b) -> (a c - b s, b c + a s) for the column pairs of a head's first
//   `rot` columns, c and s from FP32 tables at the token's position; the other
//   columns, and values, are copied.
//
// The launch is bound by its bytes: each element is read and written once. A
// thread takes an item, 16 bytes of a row, or 32 where a pair's columns lie apart
// (two times 8 or 16), with the pairs' table values; the token, head and place
// come from its number by multiplications. What keeps bytes under way is threads:
// two items each took a prompt from 40 to 46 us, four to 52. Appending 8192
// tokens (32 + 8 + 8 heads of 128): 36 us, 5.7 TB/s; turning 4099 tokens of 12
// heads of 80: 4.0 us, 3.9 TB/s.
#include "attn_internal.h"
#include "launch.cuh"
#include "ops_internal.h"
#include "vec.cuh"

#include <algorithm>

namespace deto {
namespace {

constexpr int kThreads = 256;

// n / d for 0 <= n < 2^31, 1 <= d < 2^31: the upper half of n m, shifted, m the next multiple of 1 / d in 64 bits.
struct Divisor {
    uint32_t d;
    uint64_t m;                      // floor((2^64 - 1) / d) + 1 (0 for d = 1)
    __host__ explicit Divisor(uint32_t x) : d(x), m(x == 1 ? 0 : ~0ull / x + 1) {}
    __device__ uint32_t operator()(uint32_t n) const { return m ? static_cast<uint32_t>(__umul64hi(m, n)) : n; }
};

struct Plan {
    RopeParams p;
    long long items;                 // of all tokens
    Divisor token, head, page;       // items of a token, items of a head, tokens of a page
    int pairs;                       // items of a head that hold pairs
};

// The rows and columns of an item.
struct Place {
    const uint16_t *src;
    uint16_t *dst;
    int item, pos;
    bool known, turned;              // the position is in the tables; the item is turned (not a value's, nor past the pairs)
};

__device__ __forceinline__ Place place(const Plan &g, uint32_t id, long long token0)
{
    const RopeParams &p = g.p;
    const uint32_t tk = g.token(id), in = id - tk * g.token.d, h = g.head(in);
    const long long t = token0 + tk;
    Place r;
    r.item = static_cast<int>(in - h * g.head.d);
    r.pos = p.pos[t];
    r.known = r.pos >= 0 && r.pos < p.P;
    r.turned = static_cast<int>(h) < p.H + p.KV && r.item < g.pairs;
    bool bad = !r.known;
    if (static_cast<int>(h) < p.H) {
        r.src = p.q.row(t, h);
        r.dst = p.out.row(t, h);
    } else {
        const bool key = static_cast<int>(h) < p.H + p.KV;
        const int kv = static_cast<int>(h) - p.H - (key ? 0 : p.KV), slot = p.slots[t];
        const long long room = static_cast<long long>(p.pages) * p.page_size;
        r.src = key ? p.k.row(t, kv) : p.v.row(t, kv);
        r.dst = nullptr;
        if (slot >= 0 && slot < room && r.known) {
            const uint32_t page = g.page(slot);
            r.dst = (key ? p.kc : p.vc).row(page, slot - page * g.page.d, kv);
        }
        bad |= slot < -1 || slot >= room;
    }
    if (bad && r.item == 0) atomicExch(p.status, kStatusInvalid);
    return r;
}

// V neighbouring columns (of 8) and, where a pair's columns lie apart, V more.
//   MODE 0: pairs (i, i + rot / 2), V = 8 or 4: columns [V item, + V) and rot / 2 further on
//   MODE 1: pairs (2 i, 2 i + 1): columns [8 item, + 8)
// Items past the pairs are eight columns, copied.
template <int MODE, int V>
struct Data {
    union {
        uint4 w;
        uint2 n;
        uint16_t e[8];
    } lo, hi;
    __device__ __forceinline__ void load(const Place &r, int pairs, int rot)
    {
        if (MODE == 1 || r.item >= pairs) {
            lo.w = *reinterpret_cast<const uint4 *>(r.src + (MODE == 1 ? 8 * r.item : rot + 8 * (r.item - pairs)));
        } else if (V == 8) {
            lo.w = *reinterpret_cast<const uint4 *>(r.src + 8 * r.item);
            hi.w = *reinterpret_cast<const uint4 *>(r.src + 8 * r.item + rot / 2);
        } else {
            lo.n = *reinterpret_cast<const uint2 *>(r.src + 4 * r.item);
            hi.n = *reinterpret_cast<const uint2 *>(r.src + 4 * r.item + rot / 2);
        }
    }
    __device__ __forceinline__ void store(const Place &r, int pairs, int rot) const
    {
        if (MODE == 1 || r.item >= pairs) {
            *reinterpret_cast<uint4 *>(r.dst + (MODE == 1 ? 8 * r.item : rot + 8 * (r.item - pairs))) = lo.w;
        } else if (V == 8) {
            *reinterpret_cast<uint4 *>(r.dst + 8 * r.item) = lo.w;
            *reinterpret_cast<uint4 *>(r.dst + 8 * r.item + rot / 2) = hi.w;
        } else {
            *reinterpret_cast<uint2 *>(r.dst + 4 * r.item) = lo.n;
            *reinterpret_cast<uint2 *>(r.dst + 4 * r.item + rot / 2) = hi.n;
        }
    }
    __device__ __forceinline__ void clear() { lo.w = hi.w = make_uint4(0, 0, 0, 0); }
};

__device__ __forceinline__ void turn(uint16_t &a, uint16_t &b, float c, float s)
{
    const float fa = bf_at(&a), fb = bf_at(&b);
    const uint32_t r = pack_bf16(fa * c - fb * s, fb * c + fa * s);
    a = static_cast<uint16_t>(r);
    b = static_cast<uint16_t>(r >> 16);
}

template <int MODE, int V>
__global__ void __launch_bounds__(kThreads) rope_kernel(const Plan g)
{
    constexpr int N = MODE == 1 ? 4 : V;         // pairs of an item
    if (gridDim.x <= kFewBlocks) let_next_begin();
    wait_for_last();
    const RopeParams &p = g.p;
    // A block's first item's token in 64 bits; inside the block 32 are enough.
    const long long first = static_cast<long long>(blockIdx.x) * kThreads, token0 = first / g.token.d;
    if (first + threadIdx.x >= g.items) return;
    const Place r = place(g, static_cast<uint32_t>(first - token0 * g.token.d) + threadIdx.x, token0);
    if (!r.dst) return;
    Data<MODE, V> x;
    x.load(r, g.pairs, p.rot);
    if (!r.known) {
        x.clear();
    } else if (r.turned) {
        const float *cp = p.cosine + r.pos * p.ldt + r.item * N, *sp = p.sine + r.pos * p.ldt + r.item * N;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            uint16_t &a = MODE == 1 ? x.lo.e[2 * i] : x.lo.e[i], &b = MODE == 1 ? x.lo.e[2 * i + 1] : x.hi.e[i];
            turn(a, b, cp[i], p.sign * sp[i]);
        }
    }
    x.store(r, g.pairs, p.rot);
}

// Any even rot: a thread takes one pair, or one column past them.
template <int MODE>
__global__ void __launch_bounds__(kThreads) rope_single_kernel(const Plan g)
{
    if (gridDim.x <= kFewBlocks) let_next_begin();
    wait_for_last();
    const RopeParams &p = g.p;
    const long long first = static_cast<long long>(blockIdx.x) * kThreads, token0 = first / g.token.d;
    if (first + threadIdx.x >= g.items) return;
    const Place r = place(g, static_cast<uint32_t>(first - token0 * g.token.d) + threadIdx.x, token0);
    if (!r.dst) return;
    if (r.item >= g.pairs) {
        const int x = p.rot + r.item - g.pairs;
        r.dst[x] = r.known ? r.src[x] : 0;
        return;
    }
    const int x = MODE == 1 ? 2 * r.item : r.item, y = MODE == 1 ? x + 1 : x + p.rot / 2;
    uint16_t a = r.src[x], b = r.src[y];
    if (!r.known) a = b = 0;
    else if (r.turned) turn(a, b, p.cosine[r.pos * p.ldt + r.item], p.sign * p.sine[r.pos * p.ldt + r.item]);
    r.dst[x] = a;
    r.dst[y] = b;
}

cudaError_t launch(void (*fn)(Plan), const RopeParams &p, int pairs, int per_head, cudaStream_t s)
{
    const int heads = p.H + 2 * p.KV;
    const Plan g{p, static_cast<long long>(p.T) * heads * per_head, Divisor(heads * per_head), Divisor(per_head), Divisor(std::max(p.page_size, 1)), pairs};
    return launch_early(fn, (g.items + kThreads - 1) / kThreads, kThreads, 0, 1, s, g);
}

template <int MODE, int V>
cudaError_t run(const RopeParams &p, cudaStream_t s)
{
    const int pairs = MODE == 1 ? p.rot / 8 : p.rot / 2 / V;
    return launch(rope_kernel<MODE, V>, p, pairs, pairs + (p.D - p.rot) / 8, s);
}

}  // namespace

cudaError_t launch_rope(const RopeParams &p, bool interleaved, cudaStream_t s)
{
    if (p.rot % 8 == 0) return interleaved ? run<1, 8>(p, s) : p.rot % 16 == 0 ? run<0, 8>(p, s) : run<0, 4>(p, s);
    const int per_head = p.rot / 2 + p.D - p.rot;
    return launch(interleaved ? rope_single_kernel<1> : rope_single_kernel<0>, p, p.rot / 2, per_head, s);
}

}  // namespace deto
