// Attention of packed sequences, forward.
//
//   m_i = max_j s_ij, p_ij = 2^(s_ij - m_i), out_i = sum_j p_ij v_j / sum_j p_ij,
//   lse_i = ln 2 (m_i + log2 sum_j p_ij),  s_ij = scale log2(e) q_i.k_j
//
// A CTA takes 256 queries of one head as two tiles of 128 and walks the blocks
// of 128 keys that they see in ascending order. Scores and outputs stay in
// TMEM (128 columns each for two tiles: all of it); a row is one TMEM lane and
// one thread, so its maximum and sum need no exchange:
//   warps 0-3, 4-7   a tile's softmax: scores out of TMEM, P back in their place
//   warp 8           copies (TMA): both query tiles, then key and value blocks
//                    through a ring of tiles
//   warp 9           issues the products from one thread: P V of a tile, then its
//                    next scores, while the other tile's softmax runs
// P is rounded to BF16, as the tensor core wants it beside BF16 values; the sum
// takes the unrounded ones.
//
// The output is rescaled only when a row's maximum has grown by more than
// 2^8 since: until then P is at most 256 and nothing is lost. The decision is
// the row's own (others in its warp are multiplied by one), so a row's bits are
// a function of its own query and keys, and blocks begin at fixed places of
// the sequence: batch, packing and chunks do not enter.
//
// What is masked does not reach the output: masked scores are replaced, and in
// blocks where some row sees only some keys, values that are not finite are
// taken out before the product (zero times infinity) and added afterwards to
// the rows that see them.
#include "attn_tile.cuh"

#include <atomic>
#include <cmath>

namespace deto {
namespace {

// The softmax warps keep a row's 128 scores in registers; the third warpgroup hands over what it does not need.
constexpr int kThreads = 384, kLaunchRegs = 168, kSoftmaxRegs = 208, kServiceRegs = 88;
static_assert(kSoftmaxRegs * 256 + kServiceRegs * 128 <= kLaunchRegs * kThreads, "register split");
constexpr float kSlack = 8.0f;       // how far (log2) a row's maximum may be above what it is scaled by

template <int DH>
struct Cfg {
    static constexpr int TILE = kTile * DH * 2;      // bytes
    static constexpr int SLOTS = DH == 128 ? 5 : 8;  // ring of key and value tiles
    static constexpr int OFF_RING = 2 * TILE;
    static constexpr int OFF_SHARED = OFF_RING + SLOTS * TILE;
    static constexpr int SMEM = OFF_SHARED + 384 + 1024;
    static_assert(SMEM <= 232448, "shared memory");
};

// What a CTA works on.
struct Work {
    Seq s;
    int head, kv, row0;              // first query row
    int rows[2];                     // queries of each tile
    Positions pos[2];
    Blocks blocks;                   // of both tiles
};

struct Shared {
    uint64_t q_full[2], full[8], empty[8], scores[2], probs[2], sane[2], done[2], drain, never;
    uint32_t tmem;
    int abort_flag;
    int poison;                      // some value of a partly masked block is not finite
    int some;                        // there is something to do
    Work work;
};
static_assert(sizeof(Shared) <= 384, "shared state");

__device__ __forceinline__ bool find_work(const AttnParams &p, int unit, int slots, Work &w)
{
    w.head = unit % p.H;
    w.kv = w.head / p.G;
    if (p.qb && p.N == 0) return false;
    int tile;
    const int n = tile_sequence(p.qb, p.N, p.T, 2 * kTile, slots - 1 - unit / p.H, tile);
    w.s = seq_at(p, n);
    const long long row0 = w.s.q0 + 2ll * kTile * tile;
    if (row0 >= w.s.q1) return false;
    w.row0 = static_cast<int>(row0);
    w.pos[0] = w.pos[1] = Positions{0, -1};
    for (int t = 0; t < 2; ++t) {
        w.rows[t] = max(0, min(kTile, w.s.q1 - w.row0 - t * kTile));
        const int first = w.s.position(w.row0 + t * kTile);
        if (w.rows[t] > 0) w.pos[t] = Positions{first, first + w.rows[t] - 1};
    }
    w.blocks = blocks_of(p, Positions{w.pos[0].lo, max(w.pos[0].hi, w.pos[1].hi)});
    return true;
}

// Some row sees some key of the block and not all: its values are looked at before the product.
__device__ __forceinline__ bool partly(const AttnParams &p, const Work &w, int b)
{
    return (sees_any(p, w.pos[0], b) && !sees_all(p, w.pos[0], b)) || (sees_any(p, w.pos[1], b) && !sees_all(p, w.pos[1], b));
}

// ---- roles

template <int DH>
__device__ void copy_role(const AttnParams &p, const AttnMaps &maps, Shared &S, uint32_t base, const Waits &wait)
{
    const Work w = S.work;
    using C = Cfg<DH>;
    if (p.force_timeout && !wait.one(smem_u32(&S.never), 0)) return;
    bool tile[2];
    for (int t = 0; t < 2; ++t) {
        tile[t] = w.pos[t].hi >= 0 && w.blocks.n > 0;
        if (!tile[t]) continue;
        mbar_arrive_expect_tx(smem_u32(&S.q_full[t]), C::TILE);
        load_tile<DH>(base + t * C::TILE, &maps.q, smem_u32(&S.q_full[t]), w.head, w.row0 + t * kTile);
    }
    int slot = 0;
    uint32_t round = 0;
    bool ok = true;
    uint32_t loaded = 0, parity = 0;
    for (int i = 0; ok && i < 2 * w.blocks.n; ++i) {
        if (!wait.one(smem_u32(&S.empty[slot]), round ^ 1u)) {
            ok = false;
            break;
        }
        const uint32_t bar = smem_u32(&S.full[slot]);
        mbar_arrive_expect_tx(bar, C::TILE);
        load_tile<DH>(base + C::OFF_RING + slot * C::TILE, (i & 1) ? &maps.v : &maps.k, bar, w.kv, w.s.k0 + w.blocks.at(i >> 1) * kTile);
        loaded |= 1u << slot;
        parity = (parity & ~(1u << slot)) | (round << slot);
        if (++slot == C::SLOTS) {
            slot = 0;
            round ^= 1u;
        }
    }
    // Nothing may land after the CTA's end; when all went well the last blocks' products have waited for them.
    if (!ok || *wait.abort_flag) {
        for (int t = 0; t < 2; ++t)
            if (tile[t]) wait.drain(smem_u32(&S.q_full[t]), 0);
        for (int i = 0; i < C::SLOTS; ++i)
            if (loaded & (1u << i)) wait.drain(smem_u32(&S.full[i]), (parity >> i) & 1u);
    }
}

template <int DH>
__device__ void issue_role(const AttnParams &p, Shared &S, uint32_t base, const Waits &wait)
{
    const Work w = S.work;
    using C = Cfg<DH>;
    const uint32_t ring = base + C::OFF_RING, tm = S.tmem;
    const int steps = (p.D + 15) / 16, n = steps * 16;
    int slot = 0;                    // of the next tile in the ring
    uint32_t round = 0, probs = 0, sane = 0;     // phases (a bit a tile)
    bool ok = true, issued = false, begun[2] = {false, false};
    auto arrive_tile = [&](uint32_t &at) {       // waits for the next tile of the ring
        at = slot;
        ok = ok && wait.one(smem_u32(&S.full[slot]), round);
        if (++slot == C::SLOTS) {
            slot = 0;
            round ^= 1u;
        }
        return ok;
    };
    auto scores = [&](int t, uint32_t k) {
        mma_scores<DH>(tm + t * kTile, base + t * C::TILE, ring + k * C::TILE, steps);
        mma_commit(smem_u32(&S.scores[t]));
        issued = true;
    };
    uint32_t k = 0, v = 0;
    if (w.blocks.n > 0 && arrive_tile(k)) {
        for (int t = 0; ok && t < 2; ++t) {
            if (!sees_any(p, w.pos[t], w.blocks.at(0))) continue;
            ok = wait.one(smem_u32(&S.q_full[t]), 0);
            if (!ok) break;
            tc_fence_after();
            begun[t] = true;
            scores(t, k);
        }
        if (ok) mma_commit(smem_u32(&S.empty[k]));
    }
    bool out[2] = {false, false};                // the output has been written
    for (int i = 0; ok && i < w.blocks.n; ++i) {
        const int b = w.blocks.at(i), next = i + 1 < w.blocks.n ? w.blocks.at(i + 1) : -1;
        const bool both = sees_any(p, w.pos[0], b) && sees_any(p, w.pos[1], b);
        const bool edge = partly(p, w, b);
        if (!arrive_tile(v)) break;
        bool have_next = false;
        for (int t = 0; t < 2; ++t) {
            if (sees_any(p, w.pos[t], b)) {
                if (!wait.one(smem_u32(&S.probs[t]), (probs >> t) & 1u)) { ok = false; break; }
                probs ^= 1u << t;
                if (both && edge) {              // the other tile's threads have looked at their part of the values
                    if (!wait.one(smem_u32(&S.sane[1 - t]), (sane >> (1 - t)) & 1u)) { ok = false; break; }
                    sane ^= 1u << (1 - t);
                }
                tc_fence_after();
                mma_rows(tm + 2 * kTile + t * kTile, tm + t * kTile, ring + v * C::TILE, n, out[t]);
                out[t] = issued = true;
            }
            if (next >= 0 && sees_any(p, w.pos[t], next)) {
                if (!have_next) {
                    if (!arrive_tile(k)) break;
                    have_next = true;
                }
                if (!begun[t]) {
                    if (!wait.one(smem_u32(&S.q_full[t]), 0)) { ok = false; break; }
                    begun[t] = true;
                }
                tc_fence_after();
                scores(t, k);
            }
        }
        if (!ok) break;
        mma_commit(smem_u32(&S.empty[v]));
        if (next >= 0) {
            if (!have_next && !arrive_tile(k)) break;        // (a block that neither tile sees does not occur)
            mma_commit(smem_u32(&S.empty[k]));
        }
    }
    if (ok) {
        mma_commit(smem_u32(&S.done[0]));
        mma_commit(smem_u32(&S.done[1]));
    } else if (issued) {
        mma_commit(smem_u32(&S.drain));
        wait.drain(smem_u32(&S.drain), 0);
    }
}

// Adds the values that make_finite took out to the rows that see them.
__device__ __noinline__ void add_taken(const AttnParams &p, const Work &w, int t, uint32_t out, int position)
{
    for (int c = 0; c < p.D; c += 8) {
        uint32_t o[8];
        detg::tmem_ld8(out + c, o);
        tmem_wait_ld();
        detg::reg_fence8(o);
        for (int i = 0; i < w.blocks.n; ++i) {
            const int b = w.blocks.at(i);
            if (!sees_any(p, w.pos[t], b) || !partly(p, w, b)) continue;
            for (int j = b * kTile; j < (b + 1) * kTile && j <= position; ++j) {
                if (!sees(p, position, j)) continue;
                const uint4 v = *reinterpret_cast<const uint4 *>(p.v.row(w.s.k0 + j, w.kv) + c);
                float f[8];
                unpack8(v, f);
                for (int e = 0; e < 8; ++e)
                    if (!isfinite(f[e])) o[e] = __float_as_uint(__uint_as_float(o[e]) + f[e]);
            }
        }
        __syncwarp();
        detg::tmem_st8(out + c, o);
        tmem_wait_st();
    }
}

template <int DH>
__device__ void softmax_role(const AttnParams &p, Shared &S, uint32_t base, const Waits &wait, int t, int warp, int lane)
{
    const Work &w = S.work;
    using C = Cfg<DH>;
    const int row = warp * 32 + lane;                                  // of the tile
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t ts = S.tmem + lanes + t * kTile, to = S.tmem + lanes + 2 * kTile + t * kTile;
    const int position = row < w.rows[t] ? w.pos[t].lo + row : -1;
    const float c = p.scale * kLog2e;
    float m = -INFINITY, l = 0.0f;               // m: what the row is scaled by, log2
    bool ok = true, out = false;
    uint32_t phase = 0;
    int v_slot = 1;                              // ring slot of block i's values: 2 i + 1
    for (int i = 0; ok && i < w.blocks.n; ++i, v_slot = (v_slot + 2) % C::SLOTS) {
        const int b = w.blocks.at(i);
        if (!sees_any(p, w.pos[t], b)) continue;
        ok = wait.warp(smem_u32(&S.scores[t]), phase);
        if (!ok) break;
        phase ^= 1u;
        if (partly(p, w, b)) {
            // The scores wait for every tile of the ring before block i's values, so that their slot's barrier is in the
            // phase before: slot (2 i + 1) % SLOTS for the ((2 i + 1) / SLOTS)th time.
            const bool both = sees_any(p, w.pos[1 - t], b);
            ok = wait.warp(smem_u32(&S.full[v_slot]), ((2 * i + 1) / C::SLOTS) & 1);
            if (!ok) break;
            const int live = min(kTile, w.s.keys() - b * kTile);
            if (make_finite<DH>(base + C::OFF_RING + v_slot * C::TILE, both ? 2 * row + t : row, live)) S.poison = 1;
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
        if (!sees_all(p, w.pos[t], b)) {
            const int a = b * kTile, last = position - a;              // keys [.., last] of the block, from `first` on or below `sink`
            const int first = first_seen(p, position, a), sink = p.sinks - a;
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const int k = 32 * x + j;
                    if (k > last || (k < first && k >= sink)) s[x][j] = __float_as_uint(-INFINITY);
                }
        }
        float top[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            top[x] = __uint_as_float(s[x][0]);
#pragma unroll
            for (int j = 1; j < 32; ++j) top[x] = fmaxf(top[x], __uint_as_float(s[x][j]));
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
#pragma unroll
        for (int x = 0; x < 4; ++x) {
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
        tmem_st32(ts, s[0]);
        tmem_st32(ts + 32, s[1]);
        float lo, hi;
        unpair(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), lo, hi);
        l += lo + hi;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&S.probs[t]));
        out = true;
    }
    // ---- the rows' end
    if (ok) ok = wait.warp(smem_u32(&S.done[t]), 0);
    if (!ok) return;
    tc_fence_after();
    if (out && *reinterpret_cast<volatile int *>(&S.poison)) add_taken(p, w, t, to, position);
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const bool seen = l != 0.0f;
    // Through the tile's query rows (its own warp's part; the scores are done with them), so that rows leave in whole lines.
    const uint32_t mine = base + t * C::TILE;
#pragma unroll 1
    for (int x = 0; x < DH / 32; ++x) {
        uint32_t o[32];
        if (out) {
            tmem_ld32(to + 32 * x, o);
            tmem_wait_ld();
            reg_fence(o);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                y[e] = seen && out ? pack_bf16(__uint_as_float(o[8 * q + 2 * e]) * inv, __uint_as_float(o[8 * q + 2 * e + 1]) * inv) : 0u;
            const int chunk = 4 * x + q;
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(mine + (chunk >> 3) * (kTile * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) * 16)),
                         "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3])
                         : "memory");
        }
    }
    __syncwarp();
    constexpr int CH = DH / 8, RW = 32 / CH;     // 16-byte chunks of a row; rows of one store instruction
#pragma unroll 4
    for (int r0 = 0; r0 < 32; r0 += RW) {
        const int r = warp * 32 + r0 + lane / CH, chunk = lane % CH;
        uint4 y;
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(y.x), "=r"(y.y), "=r"(y.z), "=r"(y.w)
                     : "r"(mine + (chunk >> 3) * (kTile * 128) + r * 128 + (((chunk & 7) ^ (r & 7)) * 16))
                     : "memory");
        if (r < w.rows[t] && chunk * 8 < p.D) *reinterpret_cast<uint4 *>(p.out.row(w.row0 + t * kTile + r, w.head) + chunk * 8) = y;
    }
    if (row < w.rows[t]) p.lse[static_cast<long long>(w.head) * p.T + w.row0 + t * kTile + row] = seen ? (m + log2f(l)) * kLn2 : -INFINITY;
}

// Rows that no sequence owns, and the report of bad bounds: the two warps without another task.
__device__ void outside(const AttnParams &p, int thread)
{
    if (!p.qb) return;
    if (blockIdx.x == 0) {
        bool bad = false;
        for (int n = thread; n < p.N; n += 64) {
            const Seq s = seq_at(p, n);
            bad |= s.q0 != p.qb[n] || s.q1 != p.qb[n + 1] || s.k0 != p.kb[n] || s.k1 != p.kb[n + 1];
        }
        if (bad) atomicExch(p.status, kStatusInvalid);
    }
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
        S.poison = 0;
        for (int i = 0; i < C::SLOTS; ++i) {
            mbar_init(smem_u32(&S.full[i]), 1);
            mbar_init(smem_u32(&S.empty[i]), 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(smem_u32(&S.q_full[t]), 1);
            mbar_init(smem_u32(&S.scores[t]), 1);
            mbar_init(smem_u32(&S.probs[t]), 4);
            mbar_init(smem_u32(&S.sane[t]), 4);
            mbar_init(smem_u32(&S.done[t]), 1);
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
        if (some) softmax_role<DH>(p, S, base, wait, warp >> 2, warp & 3, lane);
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
