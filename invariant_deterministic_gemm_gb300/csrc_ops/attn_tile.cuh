// What the tensor-core attention kernels share: tiles of 128 rows in shared
// memory and TMEM, which key blocks a range of queries sees, bounded waits.
//
// A tile is 128 rows (tokens of one head) of DH = 64 or 128 columns, in halves
// of 64 columns of 128 bytes a row (TMA's 128-byte swizzle). As it lies it is a
// K-major operand of a product over the columns (scores) and an MN-major
// operand of a product over the rows (values, gradients): nothing is transposed.
// Columns past D are zeros, written by TMA.
#pragma once

#include "attn_internal.h"
#include "det_gemm_kernel.cuh"
#include "launch.cuh"
#include "ops_internal.h"
#include "vec.cuh"

namespace deto {

using detg::elect_one;
using detg::idesc_bf16;
using detg::mbar_arrive;
using detg::mbar_arrive_expect_tx;
using detg::mbar_init;
using detg::mma_bf16;
using detg::mma_commit;
using detg::reg_fence;
using detg::sdesc;
using detg::smem_u32;
using detg::tc_fence_after;
using detg::tc_fence_before;
using detg::tmap_prefetch;
using detg::tmem_ld32;
using detg::tmem_st32;
using detg::tmem_wait_ld;
using detg::tmem_wait_st;

constexpr int kTile = 128;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr unsigned kWarp = 0xFFFFFFFFu;
constexpr uint32_t kNan = 0x7FFFFFFFu;

// ---- waits

struct Waits {
    volatile int *abort_flag;
    int *status;
    unsigned long long timeout_ns;
    __device__ bool one(uint32_t bar, uint32_t parity) const { return detg::wait_bounded(bar, parity, abort_flag, status, timeout_ns, true); }
    __device__ bool drain(uint32_t bar, uint32_t parity) const { return detg::wait_bounded(bar, parity, abort_flag, status, timeout_ns, false); }
    __device__ bool warp(uint32_t bar, uint32_t parity) const { return __all_sync(kWarp, one(bar, parity)); }
};

// Copies that a role has started: the barriers (a bit each, counted from one of them) of its last ones, and their phases' parities.
struct InFlight {
    uint32_t begun, parity;
    __device__ void add(int i, uint32_t p)
    {
        begun |= 1u << i;
        parity = (parity & ~(1u << i)) | p << i;
    }
};
// The end of a CTA in which a role has given up, once all roles are over: nothing may land, and no product may be under way, when its
// shared memory and TMEM go back. Whichever role gave up, and when; so not by the roles, which may have ended before.
static __device__ __noinline__ void drain_copies(const uint64_t *barriers, InFlight f, Waits wait)
{
    for (int i = 0; i < 32; ++i)
        if ((f.begun >> i) & 1u) wait.drain(smem_u32(barriers + i), (f.parity >> i) & 1u);
}
// (By the thread that issued the products; a warp's elected thread is always the same.)
__device__ __forceinline__ void drain_products(uint32_t bar, const Waits &wait)
{
    mma_commit(bar);
    wait.drain(bar, 0);
}

// Whether one of the `threads` of named barrier `id` says so; they wait for one another, and none leaves but where all do.
__device__ __forceinline__ bool any_at(int id, int threads, bool v)
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "bar.red.or.pred p, %2, %3, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(v)), "r"(id), "r"(threads)
        : "memory");
    return r != 0;
}

// ---- tensor maps and copies

// Heads [T, H, D] as (column, head, token); a box is 64 columns of `rows` tokens of one head.
__device__ __forceinline__ void load_rows(uint32_t dst, const CUtensorMap *map, uint32_t bar, int col, int head, int token)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(col), "r"(head), "r"(token)
        : "memory");
}
template <int DH>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap *map, uint32_t bar, int head, int token)
{
#pragma unroll
    for (int h = 0; h < DH / 64; ++h) load_rows(dst + h * kTile * 128, map, bar, h * 64, head, token);
}

// A warp's 32 rows of a tile (its halves 16 KB apart, as copies leave them) to rows [token, + 32) of an array.
template <int DH>
__device__ __forceinline__ void store_rows(const CUtensorMap *map, uint32_t src, int head, int token)
{
#pragma unroll
    for (int h = 0; h < DH / 64; ++h)
        asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(reinterpret_cast<uint64_t>(map)),
                     "r"(src + h * kTile * 128), "r"(h * 64), "r"(head), "r"(token)
                     : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// The thread's stores have read shared memory.
__device__ __forceinline__ void stores_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

// A warp's 32 rows of a tile, those below `rows`, to an array: at once where all are, one after the other where the sequence ends.
template <int DH>
__device__ __forceinline__ void write_rows(const CUtensorMap *map, const Heads &out, uint32_t tile, int head, int token, int warp, int lane, int rows, int D)
{
    if (warp * 32 + 32 <= rows) {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
            store_rows<DH>(map, tile + warp * 32 * 128, head, token + warp * 32);
            stores_read();
        }
        return;
    }
    __syncwarp();
    constexpr int CH = DH / 8, RW = 32 / CH;     // 16-byte chunks of a row; rows of one store instruction
#pragma unroll 1
    for (int r0 = 0; r0 < 32; r0 += RW) {
        const int r = warp * 32 + r0 + lane / CH, chunk = lane % CH;
        uint4 y;
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(y.x), "=r"(y.y), "=r"(y.z), "=r"(y.w)
                     : "r"(tile + (chunk >> 3) * (kTile * 128) + r * 128 + (((chunk & 7) ^ (r & 7)) * 16))
                     : "memory");
        if (r < rows && chunk * 8 < D) *reinterpret_cast<uint4 *>(out.row(static_cast<long long>(token) + r, head) + chunk * 8) = y;
    }
}

// ---- products

// A in TMEM (128 lanes, two BF16 of consecutive contraction elements a column).
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// d[128, 128] = A B^T over the columns of two tiles, `steps` of 16 columns. (Unrolled: an issued product costs its thread about
// 40 cycles, and 90 in a loop.)
template <int DH>
__device__ __forceinline__ void mma_scores(uint32_t d, uint32_t a, uint32_t b, int steps)
{
    const uint64_t da = sdesc(a, 16u, 1024u), db = sdesc(b, 16u, 1024u);
    constexpr uint32_t idesc = idesc_bf16(kTile, kTile, 0, 0);
#pragma unroll
    for (int k = 0; k < DH / 16; ++k) {
        if (k >= steps) break;
        const uint32_t at = (k >> 2) * (kTile * 128 / 16) + (k & 3) * 2;      // 16-byte units
        mma_bf16(d, da + at, db + at, idesc, k != 0);
    }
}

// d[128, D] (+)= A (TMEM, 128 x 128) times a tile's rows; n: D rounded up to 16.
// `gap`: columns left out between A's halves (two warpgroups wrote them, each into its own part of the scores). K: rows of b.
template <int K = kTile>
__device__ __forceinline__ void mma_rows(uint32_t d, uint32_t a_tmem, uint32_t b, int n, bool accumulate, uint32_t gap = 0)
{
    const uint64_t db = sdesc(b, kTile * 128u, 1024u);
    const uint32_t idesc = idesc_bf16(kTile, n, 0, 1);
#pragma unroll
    for (int k = 0; k < K / 16; ++k) mma_ts(d, a_tmem + k * 8 + (k >= 4 ? gap : 0), db + k * (2048 / 16), idesc, accumulate || k != 0);
}

// Which columns of some rows hold +infinity, -infinity, NaN: a bit a column.
struct NotFinite {
    uint32_t bits[3][4];
    // Adds them to the sums of columns [c, c + 8).
    __device__ __forceinline__ void add_to(uint32_t (&o)[8], int c) const
    {
        const uint32_t plus = bits[0][c >> 5] >> (c & 31), minus = bits[1][c >> 5] >> (c & 31), nan = bits[2][c >> 5] >> (c & 31);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float x = __uint_as_float(o[e]);
            if ((plus >> e) & 1u) x += INFINITY;
            if ((minus >> e) & 1u) x -= INFINITY;
            o[e] = (nan >> e) & 1u ? kNan : __float_as_uint(x);
        }
    }
};

// Sums that nothing changes any more.
__device__ __forceinline__ bool all_nan(const uint32_t (&o)[8])
{
    bool all = true;
#pragma unroll
    for (int e = 0; e < 8; ++e) all &= isnan(__uint_as_float(o[e]));
    return all;
}

// Takes what is not finite out of row r of a tile (if the tile has one), and all of it if the sequence's rows end
// before. True if something was not finite; which columns, in shared memory, is noted in `a` and `b` (either may be null). The row's
// eight chunks of 16 bytes are taken in an order of its own, for the banks.
template <int DH>
__device__ __noinline__ bool make_finite(uint32_t tile, int r, int live, NotFinite *a, NotFinite *b)
{
    if (r >= kTile) return false;
    bool found = false;
#pragma unroll
    for (int c = 0; c < DH / 8; ++c) {
        const uint32_t at = tile + (c >> 3) * (kTile * 128) + r * 128 + ((c ^ r) & 7) * 16;
        uint32_t x[4], any = 0;
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at) : "memory");
        uint32_t kinds = 0;          // 8 bits each
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = (x[i] & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u, hi = (x[i] & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u;
            any |= lo | hi;
            if (lo) kinds |= ((x[i] & 0x7Fu) ? 1u << 16 : (x[i] & 0x8000u) ? 1u << 8 : 1u) << (2 * i);
            if (hi) kinds |= ((x[i] & 0x7F0000u) ? 1u << 16 : (x[i] >> 31) ? 1u << 8 : 1u) << (2 * i + 1);
            x[i] &= r < live ? ~(lo | hi) : 0u;
        }
        if (any != 0 || r >= live)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]) : "memory");
        if (any != 0 && r < live) {
            found = true;
            for (int k = 0; k < 3; ++k) {
                const uint32_t bits = ((kinds >> (8 * k)) & 0xFFu) << (8 * (c & 3));
                if (a && bits & ~*const_cast<volatile uint32_t *>(&a->bits[k][c >> 2])) atomicOr(&a->bits[k][c >> 2], bits);
                if (b && bits & ~*const_cast<volatile uint32_t *>(&b->bits[k][c >> 2])) atomicOr(&b->bits[k][c >> 2], bits);
            }
        }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    return found;
}

// ---- arithmetic

__device__ __forceinline__ uint64_t pair(float lo, float hi)
{
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ void unpair(uint64_t v, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// ---- which keys a range of positions sees

// Queries at positions [lo, hi] of one sequence (lo may be negative: those see nothing).
struct Positions {
    int lo, hi;
};

// Blocks of 128 keys that any of them sees: [0, ns) and from w0 on, n together, ascending.
struct Blocks {
    int ns, w0, n;
    __device__ int at(int i) const { return i < ns ? i : w0 + i - ns; }
};
__device__ __forceinline__ Blocks blocks_of(const AttnParams &p, Positions q)
{
    if (q.hi < 0) return Blocks{0, 0, 0};
    Blocks b;
    b.w0 = max(0, max(q.lo, 0) - p.window + 1) / kTile;
    b.ns = min((p.sinks + kTile - 1) / kTile, b.w0);
    b.n = b.ns + q.hi / kTile - b.w0 + 1;
    return b;
}
// The first key of a position's window, counted from key a (or below all of them).
__device__ __forceinline__ int first_seen(const AttnParams &p, int position, int a)
{
    return static_cast<int>(max(-1ll, static_cast<long long>(position) - p.window + 1 - a));
}

// Bits [0, n) of 32.
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }
// Of 32 keys from k on: those up to `last` and from `first` on, or below `sink`.
__device__ __forceinline__ uint32_t seen_bits(int k, int first, int last, int sink)
{
    return below(last + 1 - k) & (~below(first - k) | below(sink - k));
}

// The blocks that a tile of queries sees, as places i in a list of blocks: the first ns (of the first keys) and [s, e]; every one of
// its queries sees all of the first nf, and of [fs, fe).
struct Places {
    int ns, s, e, nf, fs, fe;
    __device__ bool sees(int i) const { return i < ns || (i >= s && i <= e); }
    __device__ bool whole(int i) const { return i < nf || (i >= fs && i < fe); }
    // The last of them (-1: none).
    __device__ int last() const { return e >= s ? e : ns - 1; }
};
__device__ __forceinline__ Places places_of(const AttnParams &p, Positions q, const Blocks &b)
{
    if (q.hi < 0) return Places{0, 0, -1, 0, 0, 0};
    Places r;
    // (Where the list leaves nothing out, place i is block i, and the first keys' blocks may be inside the window's.)
    r.ns = min((p.sinks + kTile - 1) / kTile, q.hi / kTile + 1);
    r.s = b.ns + max(0, max(q.lo, 0) - p.window + 1) / kTile - b.w0;
    r.e = b.ns + q.hi / kTile - b.w0;
    r.nf = q.lo < 0 ? 0 : min(p.sinks / kTile, (q.lo + 1) / kTile);
    r.fs = max(b.ns, b.ns + (max(0, q.hi - p.window + 1) + kTile - 1) / kTile - b.w0);
    r.fe = q.lo < 0 ? 0 : b.ns + (q.lo + 1) / kTile - b.w0;
    return r;
}

// Whether some of the first n numbers (a multiple of 16) is not finite: their products with zero add up to zero otherwise. (Columns
// that the products do not write, past D rounded up to 16, hold what another launch left in TMEM.)
template <int N>
__device__ __forceinline__ bool not_finite(const uint32_t (&o)[N][32], int n)
{
    uint64_t z0 = 0, z1 = 0;
#pragma unroll
    for (int x = 0; x < 2 * N; ++x)
        if (16 * x < n)
#pragma unroll
            for (int j = 16 * (x & 1); j < 16 * (x & 1) + 16; j += 4) {
                z0 = fma2(pair(__uint_as_float(o[x >> 1][j]), __uint_as_float(o[x >> 1][j + 1])), 0, z0);
                z1 = fma2(pair(__uint_as_float(o[x >> 1][j + 2]), __uint_as_float(o[x >> 1][j + 3])), 0, z1);
            }
    float lo, hi;
    unpair(add2(z0, z1), lo, hi);
    return !(lo + hi == 0.0f);
}
// Columns that the second products write.
__device__ __forceinline__ int written(const AttnParams &p) { return (p.D + 15) & ~15; }

// ---- tiles of packed rows
//
// Sequence n's tiles of `rows` rows have the numbers from bounds[n] / rows + n on:
// no two sequences share one, whatever their lengths, and nothing has to be
// summed up first. Numbers that no tile has are skipped.
__host__ __device__ constexpr int tile_slots(int rows_total, int sequences, int rows) { return rows_total / rows + (sequences > 1 ? sequences : 1); }

__device__ __forceinline__ int clamped(const int32_t *bounds, int n, int limit) { return min(max(bounds[n], 0), limit); }

// The sequence of tile number x, and how many of its tiles come before: x's tile may be past its end, and is negative where x is
// below the first sequence's numbers, whose rows nobody owns.
__device__ __forceinline__ int tile_sequence(const int32_t *bounds, int N, int limit, int rows, int x, int &tile)
{
    if (!bounds) {
        tile = x;
        return 0;
    }
    int a = 0, b = N;
    while (b - a > 1) {
        const int mid = (a + b) >> 1;
        if (clamped(bounds, mid, limit) / rows + mid <= x) a = mid;
        else b = mid;
    }
    tile = x - (clamped(bounds, a, limit) / rows + a);
    return a;
}

// Bounds that go down or leave the array, by `threads` threads of the launch's first block.
__device__ __forceinline__ void report_bounds(const AttnParams &p, int thread, int threads)
{
    if (!p.qb || blockIdx.x != 0) return;
    bool bad = false;
    for (int n = thread; n < p.N; n += threads) {
        const Seq s = seq_at(p, n);
        bad |= s.q0 != p.qb[n] || s.q1 != p.qb[n + 1] || s.k0 != p.kb[n] || s.k1 != p.kb[n + 1];
    }
    if (bad) atomicExch(p.status, kStatusInvalid);
}

}  // namespace deto
