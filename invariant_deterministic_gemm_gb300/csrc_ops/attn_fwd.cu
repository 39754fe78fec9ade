// Attention of packed sequences, forward.
//
//   m_i = max_j s_ij, p_ij = 2^(s_ij - m_i), out_i = sum_j p_ij v_j / sum_j p_ij,
//   lse_i = ln 2 (m_i + log2 sum_j p_ij),  s_ij = scale log2(e) q_i.k_j
//
// in one pass over the keys with a running maximum and sum (Milakov and
// Gimelshein, "Online normalizer calculation for softmax", 2018). Two tiles that
// take turns at the tensor core, and outputs that are rescaled only when a
// maximum has grown by much, are published schemes as well.
//
// A CTA takes 256 queries of one head as two tiles of 128 and walks the blocks
// of 128 keys that they see in ascending order. Scores and outputs stay in
// TMEM (128 columns each for two tiles: all of it); a row is one TMEM lane and
// one thread, so its maximum and sum need no exchange:
//   warps 0-3, 4-7   a tile's softmax: scores out of TMEM, P back in their place
//   warp 8           copies (TMA): both query tiles, then key and value blocks
//                    through a ring of tiles
//   warp 9           issues the products from one thread: P V of a tile, then its
//                    next scores, while the other tile's softmax runs (the
//                    scores land where that P lies: one thread's products run
//                    in the order of their issue)
// Bound by a tile's chain: scores 512 cycles, the softmax, P V 512; two chains are
// what TMEM holds. A block takes both tiles 3050 to 3300 cycles, its products 2048;
// a CTA's start and end 10 to 13 thousand.
// Prompts of 2048 queries over up to 8192 keys (32 heads of 128 on 8) 88 us, 0.50
// of the measured BF16 rate by visible pairs; 16384 tokens, window 1024, 16 heads
// 174 us. P through shared memory 98 where 94, half blocks 113, two threads a row 136.
// P is rounded to BF16, as the tensor core wants it beside BF16 values; the sum
// takes the unrounded ones.
//
// The output is rescaled only when a row's maximum has grown by more than
// 2^8 since: until then P is at most 256 and nothing is lost. The decision is
// the row's own (others in its warp are multiplied by one), so a row's bits are
// a function of its own query and keys, and blocks begin at fixed places of
// the sequence: batch, packing and chunks do not enter.
//
// What is masked does not reach the output: masked scores are replaced. A value
// that is not finite would (zero times infinity), in blocks where some row sees
// only some keys; then that row's output is not finite. Such a tile is done a
// second time, with what is not finite taken out of all values before the
// product and added to the rows that see it afterwards: as it is, since weights
// are positive, those too that are zero in FP32 (times infinity they would be NaN
// in blocks that are seen whole, which depends on where tiles begin). For such
// blocks columns are noted, the others' keys looked at again: 8192 tokens whose
// values are all infinite would take 115 ms if every row looked at every key.
#include "attn_tile.cuh"

#include <atomic>
#include <cmath>

namespace deto {
namespace {

// The softmax warps keep a row's 128 scores in registers; the third warpgroup hands over what it does not need.
constexpr int kThreads = 384, kLaunchRegs = 168, kSoftmaxRegs = 200, kServiceRegs = 104;
static_assert(kSoftmaxRegs * 256 + kServiceRegs * 128 <= kLaunchRegs * kThreads, "register split");
constexpr float kSlack = 8.0f;       // how far (log2) a row's maximum may be above what it is scaled by

template <int DH>
struct Cfg {
    static constexpr int TILE = kTile * DH * 2;      // bytes
    static constexpr int SLOTS = DH == 128 ? 5 : 8;  // ring of key and value tiles
    static constexpr int OFF_RING = 2 * TILE;
    static constexpr int OFF_SHARED = OFF_RING + SLOTS * TILE;
    static constexpr int SMEM = OFF_SHARED + 640 + 1024;
    static_assert(SMEM <= 232448, "shared memory");
};

// What a CTA works on.
struct Work {
    Seq s;
    int head, kv, row0;              // first query row
    int rows[2];                     // queries of each tile
    Positions pos[2];
    Blocks blocks;                   // of both tiles
    Places at[2];
    // What is done for the tiles `act` (a bit each): all that see something, or those that have to be done again.
    __device__ bool used(int i, unsigned act) const { return ((act & 1u) && at[0].sees(i)) || ((act & 2u) && at[1].sees(i)); }
    // All rows of such a tile see all of the block's keys.
    __device__ bool whole(int i, int t, unsigned act) const { return ((act >> t) & 1u) && at[t].sees(i) && at[t].whole(i); }
    __device__ unsigned seeing() const { return (at[0].last() >= 0 ? 1u : 0u) | (at[1].last() >= 0 ? 2u : 0u); }
};

struct Shared {
    uint64_t q_full[2], full[8], empty[8], scores[2], probs[2][2], sane[2], done[2], verdict[2], drain, never;
    uint32_t tmem;
    int abort_flag;
    InFlight copies;                 // barriers from q_full[0] on
    int again[2];                    // the tile has to be done again
    int taken;                       // some value has been taken out
    NotFinite whole[2];              // what was, of the blocks that all of a tile's rows see
    int some;                        // there is something to do
    Work work;
};
static_assert(sizeof(Shared) <= 640, "shared state");

__device__ __forceinline__ bool find_work(const AttnParams &p, int unit, int slots, Work &w)
{
    if (p.qb && p.N == 0) return false;
    w.head = unit % p.H;
    w.kv = w.head / p.G;
    int tile;
    const int n = tile_sequence(p.qb, p.N, p.T, 2 * kTile, slots - 1 - unit / p.H, tile);
    w.s = seq_at(p, n);
    const long long row0 = w.s.q0 + 2ll * kTile * tile;
    if (tile < 0 || row0 >= w.s.q1) return false;
    w.row0 = static_cast<int>(row0);
    for (int t = 0; t < 2; ++t) {
        w.rows[t] = max(0, min(kTile, w.s.q1 - w.row0 - t * kTile));
        const int first = w.s.position(w.row0 + t * kTile);
        w.pos[t] = w.rows[t] > 0 ? Positions{first, first + w.rows[t] - 1} : Positions{0, -1};
    }
    w.blocks = blocks_of(p, Positions{w.pos[0].lo, max(w.pos[0].hi, w.pos[1].hi)});
    for (int t = 0; t < 2; ++t) w.at[t] = places_of(p, w.pos[t], w.blocks);
    return true;
}

// ---- roles

// Waits for both tiles' verdicts; which of them are done again.
__device__ __forceinline__ unsigned done_again(Shared &S, const Waits &wait)
{
    for (int t = 0; t < 2; ++t)
        if (!wait.one(smem_u32(&S.verdict[t]), 0)) return 0;
    const volatile int *again = S.again;
    return (again[0] ? 1u : 0u) | (again[1] ? 2u : 0u);
}

template <int DH>
__device__ void copy_role(const AttnParams &p, const AttnMaps &maps, Shared &S, uint32_t base, const Waits &wait)
{
    using C = Cfg<DH>;
    const Work w = S.work;
    if (p.force_timeout && !wait.one(smem_u32(&S.never), 0)) return;
    const unsigned all = w.seeing();
    for (int t = 0; t < 2; ++t) {
        if (!((all >> t) & 1u)) continue;
        mbar_arrive_expect_tx(smem_u32(&S.q_full[t]), C::TILE);
        load_tile<DH>(base + t * C::TILE, &maps.q, smem_u32(&S.q_full[t]), w.head, w.row0 + t * kTile);
    }
    int slot = 0;
    uint32_t round = 0;
    bool ok = true;
    InFlight copies{all, 0};
    auto pass = [&](unsigned act) {
        for (int i = 0; ok && i < w.blocks.n; ++i) {
            if (!w.used(i, act)) continue;
            for (int kind = 0; kind < 2; ++kind) {
                ok = wait.one(smem_u32(&S.empty[slot]), round ^ 1u);
                if (!ok) return;
                const uint32_t bar = smem_u32(&S.full[slot]);
                mbar_arrive_expect_tx(bar, C::TILE);
                load_tile<DH>(base + C::OFF_RING + slot * C::TILE, kind ? &maps.v : &maps.k, bar, w.kv, w.s.k0 + w.blocks.at(i) * kTile);
                copies.add(2 + slot, round);
                if (++slot == C::SLOTS) {
                    slot = 0;
                    round ^= 1u;
                }
            }
        }
    };
    for (int again = 0; again < 2 && ok; ++again) pass(again ? done_again(S, wait) : all);
    S.copies = copies;
}

template <int DH>
__device__ void issue_role(const AttnParams &p, Shared &S, uint32_t base, const Waits &wait)
{
    using C = Cfg<DH>;
    const Work w = S.work;
    const uint32_t ring = base + C::OFF_RING, tm = S.tmem;
    const int steps = (p.D + 15) / 16, n = steps * 16;
    int slot = 0;                    // of the next tile in the ring
    uint32_t round = 0, probs = 0, sane = 0;     // phases (a bit a tile)
    bool ok = true;
    auto arrive_tile = [&](uint32_t &at) {       // waits for the next tile of the ring
        at = slot;
        ok = ok && wait.one(smem_u32(&S.full[slot]), round);
        if (++slot == C::SLOTS) {
            slot = 0;
            round ^= 1u;
        }
        return ok;
    };
    unsigned begun = 0;
    auto scores = [&](int t, uint32_t k) {
        if (!((begun >> t) & 1u)) {
            ok = ok && wait.one(smem_u32(&S.q_full[t]), 0);
            begun |= 1u << t;
        }
        if (!ok) return;
        tc_fence_after();
        mma_scores<DH>(tm + t * kTile, base + t * C::TILE, ring + k * C::TILE, steps);
        mma_commit(smem_u32(&S.scores[t]));
    };
    auto pass = [&](unsigned act, bool safe) {
        const bool on[2] = {(act & 1u) != 0, (act & 2u) != 0};
        const int last[2] = {on[0] ? w.at[0].last() : -1, on[1] ? w.at[1].last() : -1};
        bool out[2] = {false, false};            // the output has been written
        uint32_t k = 0, v = 0;
        int i = 0;
        while (i < w.blocks.n && !w.used(i, act)) ++i;
        if (i == w.blocks.n || !arrive_tile(k)) return;
        for (int t = 0; t < 2; ++t)
            if (on[t] && w.at[t].sees(i)) scores(t, k);
        if (!ok) return;
        mma_commit(smem_u32(&S.empty[k]));
        while (i < w.blocks.n) {
            int next = i + 1;
            while (next < w.blocks.n && !w.used(next, act)) ++next;
            const bool more = next < w.blocks.n;
            const bool check = safe && on[0] && on[1] && w.at[0].sees(i) && w.at[1].sees(i);
            if (!arrive_tile(v)) return;
            bool have_next = false;
            for (int t = 0; t < 2; ++t) {
                if (!on[t]) continue;
                if (w.at[t].sees(i)) {
                    const uint32_t phase = (probs >> t) & 1u;
                    ok = wait.one(smem_u32(&S.probs[t][0]), phase);
                    probs ^= 1u << t;
                    // Both tiles' threads have looked at their part of the values. (The first tile's have if its P is there; awaited
                    // here all the same, as its next scores could take them on to the next block.)
                    if (ok && check && t == 0) {
                        for (int u = 0; u < 2; ++u) ok = ok && wait.one(smem_u32(&S.sane[u]), (sane >> u) & 1u);
                        sane ^= 3u;
                    }
                    if (!ok) return;
                    tc_fence_after();
                    mma_rows<64>(tm + 2 * kTile + t * kTile, tm + t * kTile, ring + v * C::TILE, n, out[t]);
                    out[t] = true;
                    ok = wait.one(smem_u32(&S.probs[t][1]), phase);
                    if (!ok) return;
                    tc_fence_after();
                    mma_rows<64>(tm + 2 * kTile + t * kTile, tm + t * kTile + 32, ring + v * C::TILE + 64 * 128, n, true);
                    if (i == last[t]) mma_commit(smem_u32(&S.done[t]));
                }
                if (more && w.at[t].sees(next)) {
                    if (!have_next && !arrive_tile(k)) return;
                    have_next = true;
                    scores(t, k);
                    if (!ok) return;
                }
            }
            mma_commit(smem_u32(&S.empty[v]));
            if (more) mma_commit(smem_u32(&S.empty[k]));
            i = next;
        }
    };
    for (int again = 0; again < 2 && ok; ++again) pass(again ? done_again(S, wait) : w.seeing(), again != 0);
}

// Adds the values that make_finite took out to the rows that see them: those of blocks that are seen in part key by key.
__device__ __noinline__ void add_taken(const AttnParams &p, const Work &w, const NotFinite &whole, int t, uint32_t out, int position)
{
    for (int c = 0; c < p.D; c += 8) {
        uint32_t o[8];
        detg::tmem_ld8(out + c, o);
        tmem_wait_ld();
        detg::reg_fence8(o);
        for (int i = 0; i < w.blocks.n && !all_nan(o); ++i) {
            const int b = w.blocks.at(i);
            if (!w.at[t].sees(i) || w.at[t].whole(i)) continue;
            for (int j = b * kTile; j < (b + 1) * kTile && j <= position; ++j) {
                if (!sees(p, position, j)) continue;
                const uint4 v = *reinterpret_cast<const uint4 *>(p.v.row(w.s.k0 + j, w.kv) + c);
                float f[8];
                unpack8(v, f);
                for (int e = 0; e < 8; ++e)
                    if (!isfinite(f[e])) o[e] = __float_as_uint(__uint_as_float(o[e]) + f[e]);
            }
        }
        whole.add_to(o, c);
        __syncwarp();
        detg::tmem_st8(out + c, o);
        tmem_wait_st();
    }
}

template <int DH>
__device__ void softmax_role(const AttnParams &p, const AttnMaps &maps, Shared &S, uint32_t base, const Waits &wait, int t, int warp, int lane)
{
    using C = Cfg<DH>;
    const Work &w = S.work;
    const int row = warp * 32 + lane;                                  // of the tile
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t ts = S.tmem + lanes + t * kTile, to = S.tmem + lanes + 2 * kTile + t * kTile;
    const int rows = w.rows[t], position = w.pos[t].lo + row;          // (of a row past the tile's: never stored)
    const int warp_lo = w.pos[t].lo + warp * 32, warp_hi = warp_lo + 31;
    const Places at = w.at[t];
    const float c = p.scale * kLog2e;
    float m = -INFINITY, l = 0.0f;               // m: what the row is scaled by, log2
    uint32_t phase = 0;
    int tile = 0;                                // of the ring, of the next block's keys
    // All blocks that the tile sees; `safe`: what is not finite is taken out of the values.
    auto pass = [&](unsigned act, bool safe) {
        bool out = false;
        m = -INFINITY;
        l = 0.0f;
        for (int i = 0; i < w.blocks.n; ++i) {
            if (!at.sees(i)) {
                if (w.used(i, act)) tile += 2;
                continue;
            }
            const int v_tile = tile + 1;
            tile += 2;
            if (!wait.warp(smem_u32(&S.scores[t]), phase)) return false;
            phase ^= 1u;
            if (safe) {
                // The scores wait for every tile of the ring before these values, so that their slot's barrier is in the phase before.
                const bool both = act == 3u && w.at[1 - t].sees(i);
                const int slot = v_tile % C::SLOTS;
                if (!wait.warp(smem_u32(&S.full[slot]), (v_tile / C::SLOTS) & 1)) return false;
                const int live = min(kTile, w.s.keys() - w.blocks.at(i) * kTile);
                if (make_finite<DH>(base + C::OFF_RING + slot * C::TILE, both ? 2 * row + t : row, live, w.whole(i, 0, act) ? &S.whole[0] : nullptr, w.whole(i, 1, act) ? &S.whole[1] : nullptr))
                    S.taken = 1;
                __syncwarp();
                if (both && lane == 0) mbar_arrive(smem_u32(&S.sane[t]));
            }
            tc_fence_after();
            uint32_t s[4][32];
#pragma unroll
            for (int x = 0; x < 4; ++x) tmem_ld32(ts + 32 * x, s[x]);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 4; ++x) reg_fence(s[x]);
            unsigned hidden = 0;                 // 32 keys (a bit each) that no row of the warp sees
            if (!at.whole(i)) {
                const int a = w.blocks.at(i) * kTile, last = position - a, first = first_seen(p, position, a), sink = p.sinks - a;
                const int first_lo = first_seen(p, warp_lo, a), first_hi = first_seen(p, warp_hi, a);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int k = 32 * x;
                    if (k > warp_hi - a || (k + 31 < first_lo && k >= sink)) {
                        hidden |= 1u << x;
                    } else if (k + 31 > warp_lo - a || (k < first_hi && k + 31 >= sink)) {
                        const uint32_t seen = seen_bits(k, first, last, sink);
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (!(seen & (1u << j))) s[x][j] = __float_as_uint(-INFINITY);
                    }
                }
            }
            float top[4];
            auto largest = [&](int x) {
                float v = fmaxf(__uint_as_float(s[x][0]), __uint_as_float(s[x][1]));
#pragma unroll
                for (int j = 2; j < 32; j += 2) v = max3(v, __uint_as_float(s[x][j]), __uint_as_float(s[x][j + 1]));
                return v;
            };
            if (hidden == 0) {                   // (the four go side by side)
#pragma unroll
                for (int x = 0; x < 4; ++x) top[x] = largest(x);
            } else {
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    top[x] = -INFINITY;
                    if (!((hidden >> x) & 1u)) top[x] = largest(x);
                }
            }
            const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * c;
            const bool grown = mx > m + kSlack;
            if (__any_sync(kWarp, grown)) {
                const float old = grown ? (m == -INFINITY ? 0.0f : exp2_fast(m - mx)) : 1.0f;
                l *= old;
                if (grown) m = mx;
                if (out) {
                    const uint64_t f = pair(old, old);
#pragma unroll 1
                    for (int x = 0; x < DH / 32; ++x) {
                        uint32_t o[32];
                        tmem_ld32(to + 32 * x, o);
                        tmem_wait_ld();
                        reg_fence(o);
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            float lo, hi;
                            unpair(mul2(pair(__uint_as_float(o[2 * j]), __uint_as_float(o[2 * j + 1])), f), lo, hi);
                            o[2 * j] = __float_as_uint(lo);
                            o[2 * j + 1] = __float_as_uint(hi);
                        }
                        tmem_st32(to + 32 * x, o);
                    }
                }
            }
            const float off = m == -INFINITY ? 0.0f : -m;
            const uint64_t c2 = pair(c, c), off2 = pair(off, off);
            uint64_t sum[4] = {0, 0, 0, 0};
            // The first half of P goes to its product while the second is made.
            auto arrive = [&](int half) {
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&S.probs[t][half]));
            };
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                if ((hidden >> x) & 1u) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) s[x >> 1][16 * (x & 1) + j] = 0u;
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float lo, hi;
                        unpair(fma2(pair(__uint_as_float(s[x][2 * j]), __uint_as_float(s[x][2 * j + 1])), c2, off2), lo, hi);
                        lo = exp2_fast(lo);
                        hi = exp2_fast(hi);
                        sum[j & 3] = add2(sum[j & 3], pair(lo, hi));
                        s[x >> 1][16 * (x & 1) + j] = pack_bf16(lo, hi);
                    }
                }
                if (x == 1) {
                    tmem_st32(ts, s[0]);
                    arrive(0);
                }
                if (x == 3) tmem_st32(ts + 32, s[1]);
            }
            float lo, hi;
            unpair(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), lo, hi);
            l += lo + hi;
            arrive(1);
            out = true;
        }
        return true;
    };
    const bool some = at.last() >= 0;            // the tile sees something
    uint32_t o[DH / 32][32];
    if (!some && lane == 0) mbar_arrive(smem_u32(&S.verdict[t]));
    unsigned act = w.seeing();
    for (int again = 0; some; ++again) {
        if (!pass(act, again != 0) || !wait.warp(smem_u32(&S.done[t]), again)) return;
        tc_fence_after();
        if (again && *reinterpret_cast<volatile int *>(&S.taken)) add_taken(p, w, S.whole[t], t, to, row < rows ? position : -1);
#pragma unroll
        for (int x = 0; x < DH / 32; ++x) tmem_ld32(to + 32 * x, o[x]);
        tmem_wait_ld();
#pragma unroll
        for (int x = 0; x < DH / 32; ++x) reg_fence(o[x]);
        if (again) break;
        if (__any_sync(kWarp, row < rows && not_finite(o, written(p)))) S.again[t] = 1;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&S.verdict[t]));
        if (!wait.warp(smem_u32(&S.verdict[t]), 0)) return;
        if (!*reinterpret_cast<volatile int *>(&S.again[t])) break;
        // (The other tile's verdict says which blocks come.)
        if (!wait.warp(smem_u32(&S.verdict[1 - t]), 0)) return;
        act = 1u << t | (*reinterpret_cast<volatile int *>(&S.again[1 - t]) ? 2u >> t : 0u);
    }
    // ---- the rows' end
    const bool seen = l != 0.0f;
    const float inv = seen ? 1.0f / l : 0.0f;
    // Through the tile's query rows (its own warp's part; the scores are done with them), so that rows leave in whole lines.
    const uint32_t mine = base + t * C::TILE;
#pragma unroll
    for (int chunk = 0; chunk < DH / 8; ++chunk) {
        uint32_t y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            y[e] = seen ? pack_bf16(__uint_as_float(o[chunk >> 2][8 * (chunk & 3) + 2 * e]) * inv, __uint_as_float(o[chunk >> 2][8 * (chunk & 3) + 2 * e + 1]) * inv) : 0u;
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(mine + (chunk >> 3) * (kTile * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) * 16)),
                     "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3])
                     : "memory");
    }
    const int token = w.row0 + t * kTile;
    if (row < rows) p.lse[static_cast<long long>(w.head) * p.T + token + row] = seen ? (m + log2f(l)) * kLn2 : -INFINITY;
    write_rows<DH>(&maps.out, p.out, mine, w.head, token, warp, lane, rows, p.D);
}

// Rows that no sequence owns, and the report of bad bounds: the two warps without another task.
__device__ void outside(const AttnParams &p, int thread)
{
    if (!p.qb) return;
    report_bounds(p, thread, 64);
    const int lo = p.N > 0 ? clamped(p.qb, 0, p.T) : 0, hi = p.N > 0 ? max(lo, clamped(p.qb, p.N, p.T)) : 0;
    const long long rows = static_cast<long long>(lo + p.T - hi) * p.H;
    for (long long i = blockIdx.x; i < rows; i += gridDim.x) {
        const int r = static_cast<int>(i / p.H), h = static_cast<int>(i % p.H), t = r < lo ? r : hi + r - lo;
        if (thread * 8 < p.D) *reinterpret_cast<uint4 *>(p.out.row(t, h) + thread * 8) = make_uint4(0, 0, 0, 0);
        if (thread == 0) p.lse[static_cast<long long>(h) * p.T + t] = -INFINITY;
    }
}

template <int DH>
__global__ void __launch_bounds__(kThreads, 1) attn_fwd_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ AttnMaps maps, const int slots)
{
    using C = Cfg<DH>;
    extern __shared__ uint8_t attn_smem[];
    const uint32_t raw = smem_u32(attn_smem), base = (raw + 1023u) & ~1023u;
    Shared &S = *reinterpret_cast<Shared *>(attn_smem + (base - raw) + C::OFF_SHARED);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        S.abort_flag = 0;
        S.copies = InFlight{0, 0};
        S.again[0] = S.again[1] = S.taken = 0;
        S.whole[0] = S.whole[1] = NotFinite{};
        for (int i = 0; i < C::SLOTS; ++i) {
            mbar_init(smem_u32(&S.full[i]), 1);
            mbar_init(smem_u32(&S.empty[i]), 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(smem_u32(&S.q_full[t]), 1);
            mbar_init(smem_u32(&S.scores[t]), 1);
            mbar_init(smem_u32(&S.probs[t][0]), 4);
            mbar_init(smem_u32(&S.probs[t][1]), 4);
            mbar_init(smem_u32(&S.sane[t]), 4);
            mbar_init(smem_u32(&S.done[t]), 1);
            mbar_init(smem_u32(&S.verdict[t]), 4);
        }
        mbar_init(smem_u32(&S.drain), 1);
        mbar_init(smem_u32(&S.never), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 8 && lane == 0 && p.S > 0) {
        tmap_prefetch(&maps.q);
        tmap_prefetch(&maps.k);
        tmap_prefetch(&maps.v);
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&S.tmem)), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    begin();
    if (threadIdx.x == 32) {
        Work w;
        S.some = find_work(p, blockIdx.x, slots, w);
        if (S.some) S.work = w;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const Waits wait{&S.abort_flag, p.status, p.timeout_ns};
    const bool some = S.some;
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        if (some) softmax_role<DH>(p, maps, S, base, wait, warp >> 2, warp & 3, lane);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kServiceRegs));
        if (some && warp == 8 && elect_one()) copy_role<DH>(p, maps, S, base, wait);
        else if (some && warp == 9 && elect_one()) issue_role<DH>(p, S, base, wait);
        __syncwarp();
        if (warp >= 10) outside(p, threadIdx.x - 320);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (*wait.abort_flag) {
        if (warp == 8 && elect_one()) drain_copies(S.q_full, S.copies, wait);
        if (warp == 9 && elect_one()) drain_products(smem_u32(&S.drain), wait);
        __syncwarp();
        __syncthreads();
    }
    if (warp == 9) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(S.tmem), "r"(512) : "memory");
}

template <int DH>
cudaError_t run(const AttnParams &p, const AttnMaps &maps, cudaStream_t s)
{
    using C = Cfg<DH>;
    auto fn = attn_fwd_kernel<DH>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = once_per_device(done, [&] {
        cudaFuncAttributes at;
        cudaError_t x = cudaFuncGetAttributes(&at, fn);
        if (x != cudaSuccess) return x;
        // setmaxnreg shares out exactly the registers of the launch.
        if (at.numRegs != kLaunchRegs) return cudaErrorInvalidDeviceFunction;
        return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    });
    if (e != cudaSuccess) return e;
    const int slots = p.qb ? tile_slots(p.T, p.N, 2 * kTile) : (p.T + 2 * kTile - 1) / (2 * kTile);
    return launch_early(fn, static_cast<long long>(slots) * p.H, kThreads, C::SMEM, 1, s, p, maps, slots);
}

}  // namespace

cudaError_t launch_attn(const AttnParams &p, const AttnMaps &maps, cudaStream_t s)
{
    return p.D <= 64 ? run<64>(p, maps, s) : run<128>(p, maps, s);
}

}  // namespace deto
