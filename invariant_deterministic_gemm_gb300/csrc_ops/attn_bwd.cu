// Gradients of packed attention.
//
//   P_ij = 2^(s_ij - lse_i log2(e)), s_ij = scale log2(e) q_i.k_j
//   delta_i = dout_i.out_i, dS_ij = P_ij (dout_i.v_j - delta_i)
//   dv_j = sum_i P_ij dout_i, dk_j = scale sum_i dS_ij q_i, dq_i = scale sum_j dS_ij k_j
//
// Two launches, each of which writes its outputs once, in a fixed order of
// sums: no atomics. The first takes 128 queries of a head and walks the keys
// that they see (three products a block: scores, dout v^T, dq), and writes delta
// for the second, which takes 128 keys of a KV head and walks the queries that
// see them, all heads that share it (four products: both transposed score
// matrices, dv, dk). The scores are made twice: seven products where five would
// do with dq added up by atomics, whose order changes bits.
//
// With a window, the first keys that stay visible are seen by all queries: they are taken in pieces of 512 queries, which a
// third launch adds up (one CTA would walk every query: 50 us of 85 for three sequences of about 700 with a window of 257).
//
// A block of dq takes 1725 to 2100 cycles (products 1536), of dk and dv 2200 to 2600
// (2048); of a packed training pass of 638 us dq is 244, dk and dv 217. dk and dv are
// bound by their blocks. Of dq they are a little more than half: 2080 CTAs of ten
// blocks each are 13.7 rounds of 152, and each begins (barriers, TMEM, copies of q,
// dout and out, delta, the first products) and ends (dq out of TMEM, its rows
// stored) with nothing of the next one under way, since a CTA holds all of TMEM:
// 7 us a round (a launch of one block a CTA takes 8.1), some 97 us. Scores of 64
// columns at a time, with both operands from shared memory, are bound by its 128
// bytes a cycle; waits for each product's end cost dk and dv 257 us.
//
// In both, a row is a TMEM lane; two warpgroups take half of a block's columns
// each. P and dS go back to TMEM in the place of the scores they came from,
// rounded to BF16 (as the tensor core wants it beside BF16 operands), and are
// the left operand of the next product from there; dS is made of the unrounded P.
//   warps 0-3, 4-7   P and dS of a block's first and last 64 columns
//   warp 8           copies (TMA)
//   warp 9           issues the products from one thread
//   warp 10          second launch: lse and delta of the queries, into shared memory
//   warp 10, 11      rows that no sequence owns
// What is masked does not reach the results: masked elements are replaced. Rows
// of the right operands that are not finite would (zero times infinity), in
// blocks that are seen in part; then the result is not finite. Such a tile is
// done a second time, with what is not finite taken out, and put back afterwards
// for those that see it. A gradient of the output (dv) is added as it is: weights
// are positive, those too that are zero in FP32. Keys (dq) and queries (dk) make
// NaN: with a score of -infinity P and dS are zero, and zero times infinity is NaN,
// as it is in blocks that are seen whole; any other such score has made NaN of dS.
#include "attn_tile.cuh"

#include <atomic>
#include <cmath>

namespace deto {
namespace {

constexpr int kThreads = 384, kLaunchRegs = 168, kMathRegs = 208, kServiceRegs = 88;
static_assert(kMathRegs * 256 + kServiceRegs * 128 <= kLaunchRegs * kThreads, "register split");
constexpr uint32_t kGap = 32;        // columns between the halves of P (or dS): 32 of 64

// ---- what both do

// P of 32 columns: 2^(s c + l) for the row's (or, PER_COLUMN, each column's) l; masked elements zero.
__device__ __forceinline__ void exp_block(uint32_t (&s)[32], uint64_t c2, uint64_t l2)
{
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        float lo, hi;
        unpair(fma2(pair(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1])), c2, l2), lo, hi);
        s[2 * j] = __float_as_uint(exp2_fast(lo));
        s[2 * j + 1] = __float_as_uint(exp2_fast(hi));
    }
}
__device__ __forceinline__ void lds4(uint32_t at, uint64_t &a, uint64_t &b) { asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(at)); }

// A query that sees a single key, whose weight P is one, has no dS whatever the score: dout v^T and delta are two sums of the same
// numbers in different orders, so its delta is that key's dout v^T, for both launches (the tensor core's sum has the same bits
// with its operands exchanged). Whether P is one its lse tells, and not its place alone: an lse over more keys than these (of
// results that were joined) is larger than the score, and P less. P is off by a few steps of 2^-24 times the argument's terms
// (score, lse: l is -lse log2(e)); 2^-18 is 64 of them, and what is left out that small a part of the two terms of dS.
__device__ __forceinline__ bool is_one(uint32_t p, float l) { return fabsf(__uint_as_float(p) - 1.0f) <= 0x1p-18f * (1.0f + fabsf(l)); }

__device__ __forceinline__ uint32_t pack_words(uint32_t lo, uint32_t hi) { return pack_bf16(__uint_as_float(lo), __uint_as_float(hi)); }

// 32 FP32 words as 16 of BF16, into TMEM.
__device__ __forceinline__ void put16(uint32_t at, const uint32_t (&v)[32])
{
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = pack_words(v[2 * j], v[2 * j + 1]);
    detg::tmem_st16(at, w);
}

// A row's sums (times f) as BF16, 32 columns from 32 x on, into a tile's place.
__device__ __forceinline__ void put_sums(uint32_t tile, int row, int x, const uint32_t (&o)[32], float f)
{
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint32_t y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = pack_bf16(__uint_as_float(o[8 * q + 2 * e]) * f, __uint_as_float(o[8 * q + 2 * e + 1]) * f);
        const int chunk = 4 * x + q;
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(tile + (chunk >> 3) * (kTile * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) * 16)),
                     "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3])
                     : "memory");
    }
}
// Rows of one axis that no sequence owns become zero in the arrays given.
__device__ void zero_outside(const int32_t *bounds, int N, int limit, int heads, int D, const Heads &a, const Heads *b, int thread, int threads)
{
    if (!bounds) return;
    const int lo = N > 0 ? clamped(bounds, 0, limit) : 0, hi = N > 0 ? max(lo, clamped(bounds, N, limit)) : 0;
    const long long rows = static_cast<long long>(lo + limit - hi) * heads;
    for (long long i = blockIdx.x; i < rows; i += gridDim.x) {
        const int r = static_cast<int>(i / heads), h = static_cast<int>(i % heads), t = r < lo ? r : hi + r - lo;
        for (int c = thread * 8; c < D; c += threads * 8) {
            *reinterpret_cast<uint4 *>(a.row(t, h) + c) = make_uint4(0, 0, 0, 0);
            if (b) *reinterpret_cast<uint4 *>(b->row(t, h) + c) = make_uint4(0, 0, 0, 0);
        }
    }
}

// ------------------------------------------------------------ queries: dq

template <int DH>
struct QCfg {
    static constexpr int TILE = kTile * DH * 2;
    static constexpr int SLOTS = DH == 128 ? 5 : 8;
    static constexpr int OFF_RING = 2 * TILE;        // query rows and dout's first
    static constexpr int OFF_DELTA = OFF_RING + SLOTS * TILE;       // [2][128] floats
    static constexpr int OFF_SHARED = OFF_DELTA + 1024;
    static constexpr int SMEM = OFF_SHARED + 512 + 1024;
    static_assert(SMEM <= 232448, "shared memory");
};

struct QWork {
    Seq s;
    int head, kv, row0, rows;
    Positions pos;
    Blocks blocks;
    Places at;
};
struct QShared {
    uint64_t q_full, o_full, o_read, full[8], empty[8], scores[2], dp, read, ds[2], done, verdict, staged, drain, never;
    uint32_t tmem;
    int abort_flag, taken, again, some;
    InFlight copies;                 // barriers from q_full on
    QWork work;
};
static_assert(sizeof(QShared) <= 512, "shared state");

__device__ __forceinline__ bool find_queries(const AttnParams &p, int unit, int slots, QWork &w)
{
    if (p.qb && p.N == 0) return false;
    w.head = unit % p.H;
    w.kv = w.head / p.G;
    int tile;
    const int n = tile_sequence(p.qb, p.N, p.T, kTile, slots - 1 - unit / p.H, tile);
    w.s = seq_at(p, n);
    const long long row0 = w.s.q0 + static_cast<long long>(kTile) * tile;
    if (tile < 0 || row0 >= w.s.q1) return false;
    w.row0 = static_cast<int>(row0);
    w.rows = min(kTile, w.s.q1 - w.row0);
    const int first = w.s.position(w.row0);
    w.pos = Positions{first, first + w.rows - 1};
    w.blocks = blocks_of(p, w.pos);
    w.at = places_of(p, w.pos, w.blocks);
    return true;
}

// Waits for the verdict: whether the tile is done again.
template <typename S>
__device__ __forceinline__ bool done_again(S &shared, const Waits &wait)
{
    return wait.one(smem_u32(&shared.verdict), 0) && *reinterpret_cast<volatile int *>(&shared.again) != 0;
}

template <int DH>
__device__ void q_copy(const AttnParams &p, const AttnMaps &maps, QShared &S, uint32_t base, const Waits &wait)
{
    using C = QCfg<DH>;
    const QWork w = S.work;
    if (w.blocks.n == 0 || (p.force_timeout && !wait.one(smem_u32(&S.never), 0))) return;
    // The output's rows, for delta, lie where the ring's last tile will.
    mbar_arrive_expect_tx(smem_u32(&S.o_full), 2 * C::TILE);
    load_tile<DH>(base + C::TILE, &maps.dout, smem_u32(&S.o_full), w.head, w.row0);
    load_tile<DH>(base + C::OFF_RING + (C::SLOTS - 1) * C::TILE, &maps.o, smem_u32(&S.o_full), w.head, w.row0);
    mbar_arrive_expect_tx(smem_u32(&S.q_full), C::TILE);
    load_tile<DH>(base, &maps.q, smem_u32(&S.q_full), w.head, w.row0);
    int slot = 0;
    uint32_t round = 0;
    bool ok = true;
    InFlight copies{3, 0};           // (q_full, o_full)
    constexpr int RING = offsetof(QShared, full) / 8 - offsetof(QShared, q_full) / 8;
    for (int again = 0; ok && again < 2; ++again) {
        if (again && !done_again(S, wait)) break;
        for (int i = 0; i < 2 * w.blocks.n; ++i) {
            ok = wait.one(smem_u32(&S.empty[slot]), round ^ 1u) && (slot < C::SLOTS - 1 || wait.one(smem_u32(&S.o_read), 0));
            if (!ok) break;
            const uint32_t bar = smem_u32(&S.full[slot]);
            mbar_arrive_expect_tx(bar, C::TILE);
            load_tile<DH>(base + C::OFF_RING + slot * C::TILE, (i & 1) ? &maps.v : &maps.k, bar, w.kv, w.s.k0 + w.blocks.at(i >> 1) * kTile);
            copies.add(RING + slot, round);
            if (++slot == C::SLOTS) {
                slot = 0;
                round ^= 1u;
            }
        }
    }
    S.copies = copies;
}

// TMEM: scores of even and odd blocks, dout v^T, dq. dS takes the scores' place, so the next dout v^T can be made as soon as
// the last has been read, and the next but one's scores once dq has taken dS.
template <int DH>
__device__ void q_issue(const AttnParams &p, QShared &S, uint32_t base, const Waits &wait)
{
    using C = QCfg<DH>;
    const QWork w = S.work;
    const uint32_t ring = base + C::OFF_RING, tm = S.tmem;
    const int steps = (p.D + 15) / 16, n = w.blocks.n;
    bool ok = n == 0 || (wait.one(smem_u32(&S.q_full), 0) && wait.one(smem_u32(&S.o_full), 0));
    // Block i of all passes: its keys are tile 2 i of the ring, its values the next.
    auto arrived = [&](int seq) {
        ok = ok && wait.one(smem_u32(&S.full[seq % C::SLOTS]), (seq / C::SLOTS) & 1);
        return ok;
    };
    auto scores = [&](int i) {
        if (!arrived(2 * i)) return;
        tc_fence_after();
        mma_scores<DH>(tm + (i & 1) * kTile, base, ring + 2 * i % C::SLOTS * C::TILE, steps);
        mma_commit(smem_u32(&S.scores[i & 1]));
    };
    auto dp = [&](int i) {
        if (!arrived(2 * i + 1)) return;
        tc_fence_after();
        mma_scores<DH>(tm + 2 * kTile, base + C::TILE, ring + (2 * i + 1) % C::SLOTS * C::TILE, steps);
        mma_commit(smem_u32(&S.dp));
        mma_commit(smem_u32(&S.empty[(2 * i + 1) % C::SLOTS]));
    };
    for (int begin = 0; ok && n > 0 && begin < 2 * n; begin += n) {
        if (begin && !done_again(S, wait)) break;
        const int end = begin + n;
        scores(begin);
        if (ok) dp(begin);
        if (ok && n > 1) scores(begin + 1);
        for (int i = begin; ok && i < end; ++i) {
            if (i + 1 < end) {
                ok = wait.one(smem_u32(&S.read), i & 1);
                if (ok) dp(i + 1);
            }
            // (dS of the next block may be there before this wait is over: two barriers, so that neither goes two phases on.)
            ok = ok && wait.one(smem_u32(&S.ds[i & 1]), (i >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            mma_rows(tm + 3 * kTile, tm + (i & 1) * kTile, ring + 2 * i % C::SLOTS * C::TILE, steps * 16, i > begin, kGap);
            mma_commit(smem_u32(&S.empty[2 * i % C::SLOTS]));
            if (i + 2 < end) scores(i + 2);
        }
        if (ok) mma_commit(smem_u32(&S.done));
    }
}

// NaN for the queries that see a key which make_finite has taken something out of.
__device__ __noinline__ void q_add_taken(const AttnParams &p, const QWork &w, uint32_t out, int position, int c0, int c1)
{
    for (int c = c0; c < c1; c += 8) {
        uint32_t o[8];
        detg::tmem_ld8(out + c, o);
        tmem_wait_ld();
        detg::reg_fence8(o);
        for (int i = 0; i < w.blocks.n && !all_nan(o); ++i) {
            const int b = w.blocks.at(i);
            if (w.at.whole(i)) continue;
            for (int j = b * kTile; j < (b + 1) * kTile && j <= position; ++j) {
                if (!sees(p, position, j)) continue;
                float f[8];
                unpack8(load8(p.k.row(w.s.k0 + j, w.kv), c, p.D), f);
                for (int e = 0; e < 8; ++e)
                    if (!isfinite(f[e])) o[e] = kNan;
            }
        }
        __syncwarp();
        detg::tmem_st8(out + c, o);
        tmem_wait_st();
    }
}

template <int DH>
__device__ void q_math(const AttnParams &p, const AttnMaps &maps, QShared &S, uint32_t base, const Waits &wait, int half, int warp, int lane)
{
    using C = QCfg<DH>;
    const QWork &w = S.work;
    const int row = warp * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t tm = S.tmem + lanes;
    const bool live = row < w.rows;
    const int position = w.pos.lo + row;             // (of a row past the tile's: never stored)
    const long long at = static_cast<long long>(w.head) * p.T + w.row0 + row;
    // delta from the copies of dout and out: a half of the row's columns each, joined in shared memory, the first half first.
    float delta = 0.0f;
    if (w.blocks.n > 0) {
        const bool ok = wait.warp(smem_u32(&S.o_full), 0);
        float part = 0.0f;
        if (ok) {
#pragma unroll
            for (int i = 0; i < DH / 16; ++i) {
                const int chunk = half * (DH / 16) + i;
                const uint32_t of = (chunk >> 3) * (kTile * 128) + row * 128 + ((chunk ^ row) & 7) * 16;
                uint4 x, y;
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(base + C::TILE + of));
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(y.x), "=r"(y.y), "=r"(y.z), "=r"(y.w)
                             : "r"(base + C::OFF_RING + (C::SLOTS - 1) * C::TILE + of));
                float f[8], g[8];
                unpack8(x, f);
                unpack8(y, g);
#pragma unroll
                for (int e = 0; e < 8; ++e) part = fmaf(f[e], g[e], part);
            }
        }
        float *deltas = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(&S) - 1024);
        deltas[half * kTile + row] = part;
        if (any_at(1, 256, !ok)) return;             // (all leave together: nobody is waited for in vain)
        // All sums have been made: the copies' places are free. (Loads come back late while products read shared memory. An arrival of
        // each warp behind its loads, but ahead of what they are for, let the ring's tile in before them now and then.)
        if (threadIdx.x == 0) mbar_arrive(smem_u32(&S.o_read));
        delta = deltas[row] + deltas[kTile + row];
    }
    const float lse = live ? p.lse[at] : 0.0f;
    // (Of a query that sees a single key: when that key's dout v^T is there.)
    if (live && half == 0 && !(position >= 0 && sees_one(p, position))) p.delta[at] = delta;
    // (A row that sees nothing has no P.)
    const float c = p.scale * kLog2e, off = lse == -INFINITY ? -INFINITY : -lse * kLog2e;
    const uint64_t c2 = pair(c, c), l2 = pair(off, off), d2 = pair(-delta, -delta);
    const Places places = w.at;
    const int n = w.blocks.n;
    const uint32_t out = tm + 3 * kTile;
    uint32_t o[DH / 64][32];
    int j = 0;                       // blocks of all passes
    for (int again = 0; n > 0; ++again) {
        for (int i = 0; i < n; ++i, ++j) {
            const bool full = places.whole(i);
            const uint32_t ts = tm + (j & 1) * kTile + half * 64;
            if (!wait.warp(smem_u32(&S.scores[j & 1]), (j >> 1) & 1)) return;
            tc_fence_after();
            uint32_t s[2][32];
            tmem_ld32(ts, s[0]);
            tmem_ld32(ts + 32, s[1]);
            tmem_wait_ld();
            reg_fence(s[0]);
            reg_fence(s[1]);
            uint32_t seen[2] = {~0u, ~0u};
            if (!full) {
                const int a = w.blocks.at(i) * kTile + half * 64, first = first_seen(p, position, a), sink = p.sinks - a;
#pragma unroll
                for (int x = 0; x < 2; ++x) seen[x] = seen_bits(32 * x, first, position - a, sink);
            }
            exp_block(s[0], c2, l2);
            exp_block(s[1], c2, l2);
            if (!wait.warp(smem_u32(&S.dp), j & 1)) return;
            tc_fence_after();
            if (again && !full) {
                // Both score matrices of the block have been made: its keys may be changed for the last product. The other
                // half's threads wait for the same, and dq for both.
                const int keys = w.s.keys() - w.blocks.at(i) * kTile;
                if (row < 64 && make_finite<DH>(base + C::OFF_RING + 2 * j % C::SLOTS * C::TILE, half * 64 + row, min(kTile, keys), nullptr, nullptr)) S.taken = 1;
                __syncwarp();
            }
            uint32_t d[2][32];
            tmem_ld32(tm + 2 * kTile + half * 64, d[0]);
            tmem_ld32(tm + 2 * kTile + half * 64 + 32, d[1]);
            tmem_wait_ld();
            reg_fence(d[0]);
            reg_fence(d[1]);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&S.read));
            if (!full && __any_sync(kWarp, sees_one(p, position))) {
                // (The one key is in the half of one of two threads, which writes delta.)
                float mine = delta;
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (sees_one(p, position) && ((seen[x] >> k) & 1u) && is_one(s[x][k], off)) {
                            mine = __uint_as_float(d[x][k]);
                            s[x][k] = 0u;
                        }
                if (live && !again && sees_one(p, position) && (seen[0] | seen[1]) != 0) p.delta[at] = mine;
            }
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    float lo, hi;
                    unpair(mul2(add2(pair(__uint_as_float(d[x][2 * k]), __uint_as_float(d[x][2 * k + 1])), d2),
                                pair(__uint_as_float(s[x][2 * k]), __uint_as_float(s[x][2 * k + 1]))), lo, hi);
                    d[x][2 * k] = __float_as_uint(lo);
                    d[x][2 * k + 1] = __float_as_uint(hi);
                }
#pragma unroll
            for (int x = 0; x < 2; ++x)
                if (__any_sync(kWarp, seen[x] != ~0u)) {
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (!(seen[x] & (1u << k))) d[x][k] = 0u;
                }
            put16(ts, d[0]);
            put16(ts + 16, d[1]);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&S.ds[j & 1]));
        }
        if (!wait.warp(smem_u32(&S.done), again)) return;
        tc_fence_after();
        if (again && *reinterpret_cast<volatile int *>(&S.taken)) q_add_taken(p, w, out, live ? position : -1, half * (DH / 2), min((half + 1) * (DH / 2), written(p)));
#pragma unroll
        for (int x = 0; x < DH / 64; ++x) tmem_ld32(out + half * (DH / 2) + 32 * x, o[x]);
        tmem_wait_ld();
#pragma unroll
        for (int x = 0; x < DH / 64; ++x) reg_fence(o[x]);
        if (again) break;
        if (__any_sync(kWarp, live && not_finite(o, written(p) - half * (DH / 2)))) S.again = 1;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&S.verdict));
        if (!wait.warp(smem_u32(&S.verdict), 0)) return;
        if (!*reinterpret_cast<volatile int *>(&S.again)) break;
    }
    // Half of the columns each, through the query tile's place; a warp's rows leave when both halves are there.
    if (n == 0) {
#pragma unroll
        for (int x = 0; x < DH / 64; ++x)
#pragma unroll
            for (int k = 0; k < 32; ++k) o[x][k] = 0u;
    }
#pragma unroll
    for (int x = 0; x < DH / 64; ++x) put_sums(base, row, half * (DH / 64) + x, o[x], p.scale);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (half) {
        if (lane == 0) mbar_arrive(smem_u32(&S.staged));
    } else if (wait.warp(smem_u32(&S.staged), 0)) {
        write_rows<DH>(&maps.out, p.dq, base, w.head, w.row0, warp, lane, w.rows, p.D);
    }
}

template <int DH>
__global__ void __launch_bounds__(kThreads, 1) attn_dq_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ AttnMaps maps, const int slots)
{
    using C = QCfg<DH>;
    extern __shared__ uint8_t attn_smem[];
    const uint32_t raw = smem_u32(attn_smem), base = (raw + 1023u) & ~1023u;
    QShared &S = *reinterpret_cast<QShared *>(attn_smem + (base - raw) + C::OFF_SHARED);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        S.abort_flag = 0;
        S.copies = InFlight{0, 0};
        S.again = S.taken = 0;
        for (int i = 0; i < C::SLOTS; ++i) {
            mbar_init(smem_u32(&S.full[i]), 1);
            mbar_init(smem_u32(&S.empty[i]), 1);
        }
        mbar_init(smem_u32(&S.q_full), 1);
        mbar_init(smem_u32(&S.o_full), 1);
        mbar_init(smem_u32(&S.o_read), 1);
        mbar_init(smem_u32(&S.scores[0]), 1);
        mbar_init(smem_u32(&S.scores[1]), 1);
        mbar_init(smem_u32(&S.dp), 1);
        mbar_init(smem_u32(&S.read), 8);
        mbar_init(smem_u32(&S.ds[0]), 8);
        mbar_init(smem_u32(&S.ds[1]), 8);
        mbar_init(smem_u32(&S.done), 1);
        mbar_init(smem_u32(&S.verdict), 8);
        mbar_init(smem_u32(&S.staged), 4);
        mbar_init(smem_u32(&S.drain), 1);
        mbar_init(smem_u32(&S.never), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 8 && lane == 0 && p.T > 0 && p.S > 0) {
        tmap_prefetch(&maps.q);
        tmap_prefetch(&maps.k);
        tmap_prefetch(&maps.v);
        tmap_prefetch(&maps.dout);
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&S.tmem)), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    begin();
    if (threadIdx.x == 32) {
        QWork w;
        S.some = find_queries(p, blockIdx.x, slots, w);
        if (S.some) S.work = w;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const Waits wait{&S.abort_flag, p.status, p.timeout_ns};
    const bool some = S.some;
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kMathRegs));
        if (some) q_math<DH>(p, maps, S, base, wait, warp >> 2, warp & 3, lane);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kServiceRegs));
        if (some && warp == 8 && elect_one()) q_copy<DH>(p, maps, S, base, wait);
        else if (some && warp == 9 && elect_one()) q_issue<DH>(p, S, base, wait);
        __syncwarp();
        if (warp >= 10) {
            report_bounds(p, threadIdx.x - 320, 64);
            zero_outside(p.qb, p.N, p.T, p.H, p.D, p.dq, nullptr, threadIdx.x - 320, 64);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (*wait.abort_flag) {
        if (warp == 8 && elect_one()) drain_copies(&S.q_full, S.copies, wait);
        if (warp == 9 && elect_one()) drain_products(smem_u32(&S.drain), wait);
        __syncwarp();
        __syncthreads();
    }
    if (warp == 9) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(S.tmem), "r"(512) : "memory");
}

// ------------------------------------------------------- keys: dk and dv

template <int DH>
struct KCfg {
    static constexpr int TILE = kTile * DH * 2;
    static constexpr int STAGES = 2;                 // of query rows and of dout
    static constexpr int OFF_Q = 2 * TILE;           // after keys and values
    static constexpr int OFF_D = OFF_Q + STAGES * TILE;
    static constexpr int OFF_VEC = OFF_D + STAGES * TILE;           // [STAGES][2][128] floats: -lse log2(e), -delta
    static constexpr int OFF_SHARED = OFF_VEC + STAGES * 1024;
    static constexpr int SMEM = OFF_SHARED + 512 + 1024;
    static_assert(SMEM <= 232448, "shared memory");
};

struct KWork {
    Seq s;
    int kv, key0, rows;              // first key's place in the sequence; keys of the tile
    int first, n;                    // first block of 128 queries; iterations: blocks times heads
    int f0, f1;                      // the blocks of which every query sees every key of the tile
    int piece;                       // of the first keys' queries, or -1: all that see the tile
};
struct KShared {
    uint64_t kv_full, q_full[2], q_empty[2], d_full[2], d_empty[2], v_full[2], v_empty[2], scores, dp, probs, ds, done, verdict, drain, never;
    uint32_t tmem;
    int abort_flag, taken, again, some;
    InFlight copies;                 // barriers from kv_full on
    NotFinite whole;                 // what was, of rows of dout that see all of the tile's keys
    KWork work;
};
static_assert(sizeof(KShared) <= 512, "shared state");

// The queries [lo, hi] of the sequence that see some of the tile's keys.
// Of a piece (units below `pieces`): those among kPiece queries.
__device__ __forceinline__ bool find_keys(const AttnParams &p, int unit, int pieces, KWork &w)
{
    if (p.kb && p.N == 0) return false;
    long long key0;
    int part = 0;
    w.piece = -1;
    if (unit < pieces) {
        w.piece = unit;
        w.kv = unit % p.KV;
        key0 = static_cast<long long>(unit / p.KV % p.sink_blocks) * kTile;
        w.s = seq_at(p, tile_sequence(p.qb, p.N, p.T, kPiece, unit / p.KV / p.sink_blocks, part));
        if (part < 0 || static_cast<long long>(part) * kPiece >= w.s.queries()) return false;
    } else {
        unit -= pieces;
        w.kv = unit % p.KV;
        int tile;
        w.s = seq_at(p, tile_sequence(p.kb, p.N, p.S, kTile, unit / p.KV, tile));
        key0 = static_cast<long long>(kTile) * tile;
        if (tile < 0 || tile < p.sink_blocks) return false;  // (the pieces')
    }
    if (key0 >= w.s.keys()) return false;
    w.key0 = static_cast<int>(key0);
    w.rows = min(kTile, w.s.keys() - w.key0);
    const int shift = w.s.keys() - w.s.queries();                    // position of query 0
    const long long lo = max(0, w.key0 - shift);
    long long hi = w.s.queries() - 1;
    if (w.key0 >= p.sinks) hi = min(hi, static_cast<long long>(w.key0) + w.rows - 1 + p.window - 1 - shift);
    long long b0 = lo / kTile, b1 = hi >= lo ? hi / kTile : b0 - 1;
    if (w.piece >= 0) {
        b0 = max(b0, static_cast<long long>(part) * (kPiece / kTile));
        b1 = min(b1, static_cast<long long>(part + 1) * (kPiece / kTile) - 1);
        if (b1 < b0) return false;
    }
    w.first = static_cast<int>(b0);
    w.n = static_cast<int>(b1 - b0 + 1) * p.G;
    const long long f0 = max(0ll, static_cast<long long>(w.key0) + kTile - 1 - shift);
    long long f1 = w.s.queries();    // whole blocks that begin before
    if (w.key0 + kTile - 1 >= p.sinks) f1 = min(f1, static_cast<long long>(w.key0) - shift + p.window);
    w.f0 = static_cast<int>((f0 + kTile - 1) / kTile);
    w.f1 = w.rows == kTile ? static_cast<int>(max(0ll, f1) / kTile) : 0;
    return true;
}

template <int DH>
__device__ void k_copy(const AttnParams &p, const AttnMaps &maps, KShared &S, uint32_t base, const Waits &wait)
{
    using C = KCfg<DH>;
    const KWork w = S.work;
    if (w.n == 0 || (p.force_timeout && !wait.one(smem_u32(&S.never), 0))) return;
    mbar_arrive_expect_tx(smem_u32(&S.kv_full), 2 * C::TILE);
    load_tile<DH>(base, &maps.k, smem_u32(&S.kv_full), w.kv, w.s.k0 + w.key0);
    load_tile<DH>(base + C::TILE, &maps.v, smem_u32(&S.kv_full), w.kv, w.s.k0 + w.key0);
    InFlight copies{1, 0};           // (kv_full)
    constexpr int Q = offsetof(KShared, q_full) / 8 - offsetof(KShared, kv_full) / 8, D = offsetof(KShared, d_full) / 8 - offsetof(KShared, kv_full) / 8;
    bool ok = true;
    for (int again = 0, j = 0; ok && again < 2; ++again) {
        if (again && !done_again(S, wait)) break;
        int row = w.s.q0 + w.first * kTile, h = 0;
        for (int i = 0; i < w.n; ++i, ++j) {
            const int st = j & 1, phase = (j >> 1) & 1, head = w.kv * p.G + h;
            ok = wait.one(smem_u32(&S.q_empty[st]), phase ^ 1);
            if (!ok) break;
            mbar_arrive_expect_tx(smem_u32(&S.q_full[st]), C::TILE);
            load_tile<DH>(base + C::OFF_Q + st * C::TILE, &maps.q, smem_u32(&S.q_full[st]), head, row);
            copies.add(Q + st, phase);
            ok = wait.one(smem_u32(&S.d_empty[st]), phase ^ 1);
            if (!ok) break;
            mbar_arrive_expect_tx(smem_u32(&S.d_full[st]), C::TILE);
            load_tile<DH>(base + C::OFF_D + st * C::TILE, &maps.dout, smem_u32(&S.d_full[st]), head, row);
            copies.add(D + st, phase);
            if (++h == p.G) {
                h = 0;
                row += kTile;
            }
        }
    }
    S.copies = copies;
}

// One warp: -lse log2(e) and -delta of each iteration's queries. A row that saw nothing gets -infinity: P is zero.
template <int DH>
__device__ void k_vectors(const AttnParams &p, KShared &S, uint8_t *smem, const Waits &wait, int lane)
{
    using C = KCfg<DH>;
    const KWork w = S.work;
    for (int again = 0, j = 0; again < 2; ++again) {
        if (again && (w.n == 0 || !__all_sync(kWarp, done_again(S, wait)))) return;
        int r0 = w.first * kTile, h = 0;
        for (int i = 0; i < w.n; ++i, ++j) {
            const int st = j & 1;
            const long long at = static_cast<long long>(w.kv * p.G + h) * p.T + w.s.q0 + r0;
            float l[4], d[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = lane + 32 * e;
                const bool live = r0 + r < w.s.queries();
                l[e] = live ? p.lse[at + r] : 0.0f;
                d[e] = live ? p.delta[at + r] : 0.0f;
            }
            if (!wait.warp(smem_u32(&S.v_empty[st]), ((j >> 1) & 1) ^ 1)) return;
            float *v = reinterpret_cast<float *>(smem + C::OFF_VEC + st * 1024);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[lane + 32 * e] = l[e] == -INFINITY ? -INFINITY : -l[e] * kLog2e;
                v[kTile + lane + 32 * e] = -d[e];
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&S.v_full[st]));
            if (++h == p.G) {
                h = 0;
                r0 += kTile;
            }
        }
    }
}

// TMEM: transposed scores (keys are the lanes), their gradients, dv, dk: all of it. While P of a block is made, the last
// block's dk and the next gradient of the scores are; while dS is, dv and the next scores.
template <int DH>
__device__ void k_issue(const AttnParams &p, KShared &S, uint32_t base, const Waits &wait)
{
    using C = KCfg<DH>;
    const KWork w = S.work;
    const uint32_t tm = S.tmem;
    const int steps = (p.D + 15) / 16;
    bool ok = w.n == 0 || wait.one(smem_u32(&S.kv_full), 0);
    auto scores = [&](int i) {
        ok = ok && wait.one(smem_u32(&S.q_full[i & 1]), (i >> 1) & 1);
        if (!ok) return;
        tc_fence_after();
        mma_scores<DH>(tm, base, base + C::OFF_Q + (i & 1) * C::TILE, steps);
        mma_commit(smem_u32(&S.scores));
    };
    auto dp = [&](int i) {
        ok = ok && wait.one(smem_u32(&S.d_full[i & 1]), (i >> 1) & 1);
        if (!ok) return;
        tc_fence_after();
        mma_scores<DH>(tm + kTile, base + C::TILE, base + C::OFF_D + (i & 1) * C::TILE, steps);
        mma_commit(smem_u32(&S.dp));
    };
    for (int begin = 0; ok && w.n > 0 && begin < 2 * w.n; begin += w.n) {
        if (begin && !done_again(S, wait)) break;
        const int end = begin + w.n;
        scores(begin);
        if (ok) dp(begin);
        for (int i = begin; ok && i < end; ++i) {
            ok = wait.one(smem_u32(&S.probs), i & 1);
            if (!ok) break;
            tc_fence_after();
            mma_rows(tm + 2 * kTile, tm, base + C::OFF_D + (i & 1) * C::TILE, steps * 16, i > begin, kGap);
            mma_commit(smem_u32(&S.d_empty[i & 1]));
            if (i + 1 < end) scores(i + 1);
            ok = ok && wait.one(smem_u32(&S.ds), i & 1);
            if (!ok) break;
            tc_fence_after();
            mma_rows(tm + 3 * kTile, tm + kTile, base + C::OFF_Q + (i & 1) * C::TILE, steps * 16, i > begin, kGap);
            mma_commit(smem_u32(&S.q_empty[i & 1]));
            if (i + 1 < end) dp(i + 1);
        }
        if (ok) mma_commit(smem_u32(&S.done));
    }
}

// What make_finite took out of the queries' rows (x: dout, or q) for the keys that they see: added to dv, NaN in dk. Row by row in
// blocks that are seen in part, `whole` for all others. key: place in the sequence, or -1.
__device__ __noinline__ void k_add_taken(const AttnParams &p, const KWork &w, const NotFinite &whole, bool is_q, uint32_t out, int key)
{
    const Heads &x = is_q ? p.q : p.dout;
    for (int c = 0; c < p.D; c += 8) {
        uint32_t o[8];
        detg::tmem_ld8(out + c, o);
        tmem_wait_ld();
        detg::reg_fence8(o);
        for (int i = 0; i < w.n && key >= 0 && !all_nan(o); ++i) {
            const int qb = w.first + i / p.G;
            if (qb >= w.f0 && qb < w.f1) continue;
            for (int r = qb * kTile; r < min((qb + 1) * kTile, w.s.queries()); ++r) {
                if (!sees(p, r + w.s.keys() - w.s.queries(), key)) continue;
                float f[8];
                unpack8(load8(x.row(w.s.q0 + r, w.kv * p.G + i % p.G), c, p.D), f);
                for (int e = 0; e < 8; ++e)
                    if (!isfinite(f[e])) o[e] = is_q ? kNan : __float_as_uint(__uint_as_float(o[e]) + f[e]);
            }
        }
        if (!is_q) whole.add_to(o, c);
        __syncwarp();
        detg::tmem_st8(out + c, o);
        tmem_wait_st();
    }
}

template <int DH>
__device__ void k_math(const AttnParams &p, const AttnMaps &maps, KShared &S, uint32_t base, const Waits &wait, int half, int warp, int lane)
{
    using C = KCfg<DH>;
    const KWork &w = S.work;
    const int row = warp * 32 + lane;
    const uint32_t tm = S.tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const bool live = row < w.rows;                  // (rows past the tile's are never stored)
    const int key = w.key0 + row;
    const float c = p.scale * kLog2e;
    const uint64_t c2 = pair(c, c);
    const int n = w.n, shift = w.s.keys() - w.s.queries(), f0 = w.f0, f1 = w.f1;
    // dv through the first warpgroup and the keys' place, dk through the second and the values'.
    const uint32_t out = tm + (half ? 3 : 2) * kTile, tile = base + half * C::TILE;
    // A piece's sums go out as they are.
    float *part = w.piece < 0 ? nullptr : p.partials + (static_cast<long long>(w.piece) * 2 + half) * kTile * p.D + static_cast<long long>(row) * p.D;
    auto put = [&](int x, const uint32_t (&o)[32]) {
        if (!part) {
            put_sums(tile, row, x, o, half ? p.scale : 1.0f);
            return;
        }
#pragma unroll
        for (int k = 0; k < 32; k += 4)
            if (32 * x + k < p.D)
                *reinterpret_cast<float4 *>(part + 32 * x + k) =
                    make_float4(__uint_as_float(o[k]), __uint_as_float(o[k + 1]), __uint_as_float(o[k + 2]), __uint_as_float(o[k + 3]));
    };
    int j = 0;                       // iterations of all passes
    for (int again = 0; n > 0; ++again) {
        int qb = w.first, h = 0;
        for (int i = 0; i < n; ++i, ++j) {
            const int st = j & 1;
            const bool full = qb >= f0 && qb < f1;
            const uint32_t vec = base + C::OFF_VEC + st * 1024 + half * 256;
            uint32_t seen[2] = {~0u, ~0u};           // of this thread's columns, the queries that see the key
            if (!full) {
                // From `first` on, up to `last`: the window's end, or the sequence's for one of the first keys.
                const int first = key - shift - qb * kTile - half * 64, end = w.s.queries() - qb * kTile - half * 64 - 1;
                const int last = key < p.sinks ? end : static_cast<int>(min(static_cast<long long>(end), static_cast<long long>(first) + p.window - 1));
#pragma unroll
                for (int x = 0; x < 2; ++x) seen[x] = below(last + 1 - 32 * x) & ~below(first - 32 * x);
            }
            if (!wait.warp(smem_u32(&S.v_full[st]), (j >> 1) & 1) || !wait.warp(smem_u32(&S.scores), j & 1)) return;
            tc_fence_after();
            uint32_t s[2][32];
            tmem_ld32(tm + half * 64, s[0]);
            tmem_ld32(tm + half * 64 + 32, s[1]);
            tmem_wait_ld();
            reg_fence(s[0]);
            reg_fence(s[1]);
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int k = 0; k < 16; k += 2) {
                    uint64_t l0, l1;
                    lds4(vec + x * 128 + k * 8, l0, l1);
                    float a0, a1, b0, b1;
                    unpair(fma2(pair(__uint_as_float(s[x][2 * k]), __uint_as_float(s[x][2 * k + 1])), c2, l0), a0, a1);
                    unpair(fma2(pair(__uint_as_float(s[x][2 * k + 2]), __uint_as_float(s[x][2 * k + 3])), c2, l1), b0, b1);
                    s[x][2 * k] = __float_as_uint(exp2_fast(a0));
                    s[x][2 * k + 1] = __float_as_uint(exp2_fast(a1));
                    s[x][2 * k + 2] = __float_as_uint(exp2_fast(b0));
                    s[x][2 * k + 3] = __float_as_uint(exp2_fast(b1));
                }
#pragma unroll
            for (int x = 0; x < 2; ++x)
                if (__any_sync(kWarp, seen[x] != ~0u)) {
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (!(seen[x] & (1u << k))) s[x][k] = 0u;
                }
            if (again && (half || !full)) {
                // When both score matrices have been made the queries' rows may be changed for the last two products: those of
                // dout everywhere, of q where the block is seen in part.
                if (!wait.warp(smem_u32(&S.dp), j & 1)) return;
                if (make_finite<DH>(base + (half ? C::OFF_D : C::OFF_Q) + st * C::TILE, row, w.s.queries() - qb * kTile, full ? &S.whole : nullptr, nullptr))
                    S.taken = 1;
                __syncwarp();
            }
            put16(tm + half * 64, s[0]);
            put16(tm + half * 64 + 16, s[1]);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&S.probs));
            if (!wait.warp(smem_u32(&S.dp), j & 1)) return;
            tc_fence_after();
            uint32_t d[2][32];
            tmem_ld32(tm + kTile + half * 64, d[0]);
            tmem_ld32(tm + kTile + half * 64 + 32, d[1]);
            tmem_wait_ld();
            reg_fence(d[0]);
            reg_fence(d[1]);
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int k = 0; k < 16; k += 2) {
                    uint64_t d0, d1;
                    lds4(vec + 512 + x * 128 + k * 8, d0, d1);
                    float a0, a1, b0, b1;
                    unpair(mul2(add2(pair(__uint_as_float(d[x][2 * k]), __uint_as_float(d[x][2 * k + 1])), d0),
                                pair(__uint_as_float(s[x][2 * k]), __uint_as_float(s[x][2 * k + 1]))), a0, a1);
                    unpair(mul2(add2(pair(__uint_as_float(d[x][2 * k + 2]), __uint_as_float(d[x][2 * k + 3])), d1),
                                pair(__uint_as_float(s[x][2 * k + 2]), __uint_as_float(s[x][2 * k + 3]))), b0, b1);
                    d[x][2 * k] = __float_as_uint(a0);
                    d[x][2 * k + 1] = __float_as_uint(a1);
                    d[x][2 * k + 2] = __float_as_uint(b0);
                    d[x][2 * k + 3] = __float_as_uint(b1);
                }
#pragma unroll
            for (int x = 0; x < 2; ++x)
                if (__any_sync(kWarp, seen[x] != ~0u)) {
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (!(seen[x] & (1u << k))) d[x][k] = 0u;
                }
            put16(tm + kTile + half * 64, d[0]);
            put16(tm + kTile + half * 64 + 16, d[1]);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_u32(&S.ds));
                mbar_arrive(smem_u32(&S.v_empty[st]));
            }
            if (++h == p.G) {
                h = 0;
                ++qb;
            }
        }
        if (!wait.warp(smem_u32(&S.done), again)) return;
        tc_fence_after();
        if (again && *reinterpret_cast<volatile int *>(&S.taken)) k_add_taken(p, w, S.whole, half != 0, out, live ? key : -1);
        bool bad = false;
#pragma unroll 1
        for (int x = 0; x < DH / 32; ++x) {
            uint32_t o[1][32];
            tmem_ld32(out + 32 * x, o[0]);
            tmem_wait_ld();
            reg_fence(o[0]);
            bad |= not_finite(o, written(p) - 32 * x);
            if (again) put(x, o[0]);
        }
        if (again) break;
        if (__any_sync(kWarp, live && bad)) S.again = 1;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&S.verdict));
        if (!wait.warp(smem_u32(&S.verdict), 0)) return;
        if (*reinterpret_cast<volatile int *>(&S.again)) continue;
#pragma unroll 1
        for (int x = 0; x < DH / 32; ++x) {
            uint32_t o[32];
            tmem_ld32(out + 32 * x, o);
            tmem_wait_ld();
            reg_fence(o);
            put(x, o);
        }
        break;
    }
    if (part) return;
    if (n == 0) {
        const uint32_t zero[32] = {};
        for (int x = 0; x < DH / 32; ++x) put_sums(tile, row, x, zero, 0.0f);
    }
    write_rows<DH>(half ? &maps.dk : &maps.dv, half ? p.dk : p.dv, tile, w.kv, w.s.k0 + w.key0, warp, lane, w.rows, p.D);
}

template <int DH>
__global__ void __launch_bounds__(kThreads, 1) attn_dkv_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ AttnMaps maps, const int pieces)
{
    using C = KCfg<DH>;
    extern __shared__ uint8_t attn_smem[];
    const uint32_t raw = smem_u32(attn_smem), base = (raw + 1023u) & ~1023u;
    uint8_t *smem = attn_smem + (base - raw);
    KShared &S = *reinterpret_cast<KShared *>(smem + C::OFF_SHARED);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        S.abort_flag = 0;
        S.copies = InFlight{0, 0};
        S.again = S.taken = 0;
        S.whole = NotFinite{};
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&S.q_full[i]), 1);
            mbar_init(smem_u32(&S.q_empty[i]), 1);
            mbar_init(smem_u32(&S.d_full[i]), 1);
            mbar_init(smem_u32(&S.d_empty[i]), 1);
            mbar_init(smem_u32(&S.v_full[i]), 1);
            mbar_init(smem_u32(&S.v_empty[i]), 8);
        }
        mbar_init(smem_u32(&S.kv_full), 1);
        mbar_init(smem_u32(&S.scores), 1);
        mbar_init(smem_u32(&S.dp), 1);
        mbar_init(smem_u32(&S.probs), 8);
        mbar_init(smem_u32(&S.ds), 8);
        mbar_init(smem_u32(&S.done), 1);
        mbar_init(smem_u32(&S.verdict), 8);
        mbar_init(smem_u32(&S.drain), 1);
        mbar_init(smem_u32(&S.never), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 8 && lane == 0 && p.T > 0 && p.S > 0) {
        tmap_prefetch(&maps.q);
        tmap_prefetch(&maps.k);
        tmap_prefetch(&maps.v);
        tmap_prefetch(&maps.dout);
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&S.tmem)), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    begin();
    if (threadIdx.x == 32) {
        KWork w;
        S.some = find_keys(p, blockIdx.x, pieces, w);
        if (S.some) S.work = w;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const Waits wait{&S.abort_flag, p.status, p.timeout_ns};
    const bool some = S.some;
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kMathRegs));
        if (some) k_math<DH>(p, maps, S, base, wait, warp >> 2, warp & 3, lane);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kServiceRegs));
        if (some && warp == 8 && elect_one()) k_copy<DH>(p, maps, S, base, wait);
        else if (some && warp == 9 && elect_one()) k_issue<DH>(p, S, base, wait);
        else if (some && warp == 10) k_vectors<DH>(p, S, smem, wait, lane);
        __syncwarp();
        if (warp == 11) {
            if (p.T == 0) report_bounds(p, lane, 32);        // (else the first launch has)
            zero_outside(p.kb, p.N, p.S, p.KV, p.D, p.dk, &p.dv, lane, 32);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (*wait.abort_flag) {
        if (warp == 8 && elect_one()) drain_copies(&S.kv_full, S.copies, wait);
        if (warp == 9 && elect_one()) drain_products(smem_u32(&S.drain), wait);
        __syncwarp();
        __syncthreads();
    }
    if (warp == 9) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(S.tmem), "r"(512) : "memory");
}

// dk and dv of the first keys from their pieces, in ascending order: a block takes kJoinRows keys of a sequence and KV head.
constexpr int kJoinRows = 8, kJoinThreads = 256;

__global__ void __launch_bounds__(kJoinThreads) attn_pieces_kernel(const AttnParams p)
{
    begin();
    constexpr int GROUPS = kTile / kJoinRows;
    int id = blockIdx.x;
    const int r0 = id % GROUPS * kJoinRows;
    id /= GROUPS;
    const int kv = id % p.KV, block = id / p.KV % p.sink_blocks, n = id / p.KV / p.sink_blocks;
    const Seq s = seq_at(p, n);
    const int key0 = block * kTile + r0, shift = s.keys() - s.queries();
    // The pieces that hold queries which see the block.
    const int lo = max(0, block * kTile - shift) / kPiece, hi = (s.queries() + kPiece - 1) / kPiece;
    const int slot0 = p.qb ? clamped(p.qb, n, p.T) / kPiece + n : 0;
    const int quads = p.D / 4;
    for (int i = threadIdx.x; i < 2 * kJoinRows * quads; i += kJoinThreads) {
        const int c = i % quads * 4, r = i / quads % kJoinRows, which = i / quads / kJoinRows;
        if (key0 + r >= s.keys()) continue;
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int x = lo; x < hi; ++x) {
            const long long piece = (static_cast<long long>(slot0 + x) * p.sink_blocks + block) * p.KV + kv;
            const float4 v = *reinterpret_cast<const float4 *>(p.partials + ((piece * 2 + which) * kTile + r0 + r) * p.D + c);
            sum = make_float4(sum.x + v.x, sum.y + v.y, sum.z + v.z, sum.w + v.w);
        }
        const float f = which ? p.scale : 1.0f;
        const Heads &out = which ? p.dk : p.dv;
        *reinterpret_cast<uint2 *>(out.row(static_cast<long long>(s.k0) + key0 + r, kv) + c) = make_uint2(pack_bf16(sum.x * f, sum.y * f), pack_bf16(sum.z * f, sum.w * f));
    }
}

template <typename F>
cudaError_t set_up(F fn, int smem)
{
    cudaFuncAttributes at;
    const cudaError_t x = cudaFuncGetAttributes(&at, fn);
    if (x != cudaSuccess) return x;
    // setmaxnreg shares out exactly the registers of the launch.
    if (at.numRegs != kLaunchRegs) return cudaErrorInvalidDeviceFunction;
    return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
}

template <int DH>
cudaError_t run(const AttnParams &p, const AttnMaps &maps, cudaStream_t s)
{
    static std::atomic<uint64_t> done{0};
    cudaError_t e = once_per_device(done, [&] {
        const cudaError_t x = set_up(attn_dq_kernel<DH>, QCfg<DH>::SMEM);
        return x == cudaSuccess ? set_up(attn_dkv_kernel<DH>, KCfg<DH>::SMEM) : x;
    });
    if (e != cudaSuccess) return e;
    if (p.T > 0) {
        const int slots = p.qb ? tile_slots(p.T, p.N, kTile) : (p.T + kTile - 1) / kTile;
        e = launch_early(attn_dq_kernel<DH>, static_cast<long long>(slots) * p.H, kThreads, QCfg<DH>::SMEM, 1, s, p, maps, slots);
        if (e != cudaSuccess) return e;
    }
    if (p.S > 0) {
        const int slots = p.kb ? tile_slots(p.S, p.N, kTile) : (p.S + kTile - 1) / kTile;
        const int pieces = static_cast<int>(piece_slots(p.T, p.N, p.qb != nullptr)) * p.sink_blocks * p.KV;
        e = launch_early(attn_dkv_kernel<DH>, pieces + static_cast<long long>(slots) * p.KV, kThreads, KCfg<DH>::SMEM, 1, s, p, maps, pieces);
        if (e != cudaSuccess || p.sink_blocks == 0 || (p.qb && p.N == 0)) return e;
        e = launch_early(attn_pieces_kernel, static_cast<long long>(p.qb ? p.N : 1) * p.sink_blocks * p.KV * (kTile / kJoinRows), kJoinThreads, 0, 1, s, p);
    }
    return e;
}

}  // namespace

cudaError_t launch_attn_bwd(const AttnParams &p, const AttnMaps &maps, cudaStream_t s)
{
    return p.D <= 64 ? run<64>(p, maps, s) : run<128>(p, maps, s);
}

}  // namespace deto
