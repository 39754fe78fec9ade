// Attention of one new token a sequence over a paged key-value cache.
//
//   out = sum_j p_j v_j / sum_j p_j,  p_j = 2^(s_j - m),  s_j = scale log2(e) q.k_j,  m = max_j s_j
//
// The launch is bound by reading keys and values once, so they come by TMA
// through a ring of tiles of 128 tokens (one copy a page and 64 columns), and
// everything else has to fit beside that. The tokens are the product's wide
// side: scores [128 tokens, heads] = K Q^T, outputs [D, heads] = V^T P^T, both
// from the tiles as they lie, so 16 (or 32) query heads that share a KV head
// cost one pass over its keys and no lane is wasted on a single query.
//
// The bits of a sequence do not depend on the batch: its keys are cut in chunks
// of 256 at fixed places, each with a maximum and a sum of its own, and chunks
// are joined in a fixed order: four to a block, 16 blocks to a super block, those
// one after the other. Where the work is cut between CTAs is about time alone:
// all CTAs take equally long runs of units (chunks, blocks or super blocks, the
// largest of which there are four for every CTA), and what one CTA does not
// see whole it leaves as its units' sums for a second launch, which joins them
// in the same order with the same arithmetic. Which those are is found on the
// device from the lengths, so a captured launch serves any.
//
//   warps 0-3, 4-7   scores of even and odd chunks to P (a lane a token), P to
//                    shared memory as the next product's operand
//   warps 8-11       join the chunks' sums (a lane a column of the output)
//   warps 12, 14     copies of keys and of values
//   warp 13          issues the products
//   warp 15          looks up the pages, some chunks ahead; sequences without tokens
// 64 contexts up to 8192 (32 heads of 128 on 8) 211 us, 6.3 TB/s; two of 262,144
// 257 us; one of 1021 12.8 us, of which three trips to memory in a row (lengths, page
// table, keys) are half; 96 windows of 1024 in eight heads of 64 66.6 us, where
// three chunks in flight are what bounds. With more than eight query heads to a KV head
// the softmax warps bound: 16 heads on one take 262 us for the 64 contexts (128 heads
// on 8), 32 heads 461 (256 on 8), where the bytes take 170. The instances for 17 to 32
// spill 730 to 870 bytes a thread: the softmax warps hold two tiles' scores and the
// maxima of 32 heads in 128 registers, as the joining warps need 208.
//
// A chunk's way through one warpgroup is latency (barriers, TMEM, the maximum
// over 256 tokens), about as long as its bytes take, so two take turns. P is
// rounded to BF16 beside BF16 values, and the sum is that of the rounded ones:
// the weights add up to one.
#include "attn_tile.cuh"

#include <algorithm>
#include <atomic>
#include <cmath>

namespace deto {
namespace {

constexpr int kThreads = 512;
constexpr int kLaunchRegs = 128;
constexpr int kSums = 2;             // chunks whose sums wait to be joined (four: 78 instead of 74 us for 96 windows of 1024)

// HE: query heads that are computed, 4 to 32; the products take at least 16.
template <int DH, int HE>
struct Cfg {
    static constexpr int NT = HE < 16 ? 16 : HE;
    static constexpr int TILE = kTile * DH * 2;
    // Tiles of keys and of values in rings of their own: keys leave with their scores, values a chunk's softmax later.
    static constexpr int KEYS = (NT == 16 ? 3 : 2) * (DH == 128 ? 1 : 2), VALUES = 3 * (DH == 128 ? 1 : 2), SLOTS = KEYS + VALUES;
    // A tile that its products have read goes back to the copies by a commit, at once, or (which spares the issuing thread
    // about 100 cycles each) by those who wait for the products. Tiles of 64 columns are half as long a wait, in twice as many
    // slots.
    static constexpr bool COMMIT = DH == 128;
    static constexpr int Q_BYTES = NT * DH * 2, P_BYTES = NT * kChunk * 2;
    // The ring is followed by more than the 16 KB that a tile of 64 columns' product reads past its end (128 lanes, of which
    // 64 are used).
    static constexpr int OFF_P = SLOTS * TILE;       // [2]
    static constexpr int OFF_Q = OFF_P + 2 * P_BYTES;               // [2]
    static constexpr int OFF_SHARED = OFF_Q + 2 * Q_BYTES;
    static constexpr int SMEM = OFF_SHARED + 7168 + 1024;
    static_assert(OFF_SHARED - OFF_P >= (DH == 64 ? 16384 : 0), "reads past the ring stay inside");
    static_assert(SMEM <= 232448, "shared memory");
    // TMEM columns: scores [2][2 tiles][NT], weighted values of a chunk [kSums][NT], states of the levels above a block [2]
    // (values, sum and maximum [HE]).
    static constexpr int T_SCORES = 0, T_CHUNK = 4 * NT, T_LEVEL = T_CHUNK + kSums * NT, STATE = 3 * HE;
    static_assert(T_LEVEL + 2 * STATE <= 512, "TMEM");
    // The joining warps hold two states of up to 96 registers; the service warps hand over what they can do without.
    static constexpr int JOIN_REGS = HE == 32 ? 208 : 152, SERVICE_REGS = HE == 32 ? 48 : 104;
    static_assert(JOIN_REGS + SERVICE_REGS <= 2 * kLaunchRegs, "register split");
};

struct Shared {
    uint64_t full[12], empty[12], q_full[2], q_empty[2], scores[2], probs[2], sums[kSums], joined[kSums], pages_full[8], pages_empty[8], drain, never;
    uint32_t tmem;
    int abort_flag;
    InFlight copies[2];              // of keys and of values: barriers from full[0] on
    int queries;                     // segments whose queries have been copied
    int page[8][32];                 // of the chunks ahead: the page of each eight tokens, -1 for hidden ones
    unsigned loaded[16];             // which of them have one
    alignas(16) float top[2][2][4][32];   // each warp's maxima of a chunk: of even and odd ones, the last two of each
    // The chunk's maxima, and each warp's sums of P: of twice as many chunks as wait to be joined, so that those who write them know
    // of arrivals behind the use of the last ones, not behind their loads alone.
    alignas(16) float most[2 * kSums][32];
    alignas(16) float sum[2 * kSums][4][32];
    long long first, last;           // the CTA's units
    unsigned scan[16];
    int start, start_list, start_unit;           // sequence of the first unit, its list, and its place there
    int unit;                        // chunks a unit
    long long list_unit;                         // units before the list
    long long sums_of[3][16];
};
static_assert(sizeof(Shared) <= 7168, "shared state");

__device__ __forceinline__ void prefetch_l2(const void *x) { asm volatile("prefetch.global.L2 [%0];" ::"l"(x)); }

// ---- the key axis

__device__ __forceinline__ int tokens_of(const DecodeParams &p, int b)
{
    const long long room = static_cast<long long>(p.max_pages) * p.page_size;
    const int n = p.lengths[b];
    return n < 0 ? 0 : n > room ? static_cast<int>(room) : n;
}
// The chunks that n tokens' last one sees: [0, ns) and from w0 on.
struct Chunks {
    int ns, w0, n;
    __device__ int at(int i) const { return i < ns ? i : w0 + i - ns; }
};
__device__ __forceinline__ Chunks chunks_of(const DecodeParams &p, int n)
{
    if (n == 0) return Chunks{0, 0, 0};
    Chunks c;
    c.w0 = max(0, n - p.window) / kChunk;
    c.ns = min((p.sinks + kChunk - 1) / kChunk, c.w0);
    c.n = c.ns + (n - 1) / kChunk - c.w0 + 1;
    return c;
}
__device__ __forceinline__ bool sees(const DecodeParams &p, int n, int j) { return j < n && (n - 1 - j < p.window || j < p.sinks); }
// Some, or every, of the tokens [a, a + len) is seen.
__device__ __forceinline__ bool sees_some(const DecodeParams &p, int n, int a, int len)
{
    return a < n && (n - 1 - (a + len - 1) < p.window || a < p.sinks);
}
__device__ __forceinline__ bool sees_every(const DecodeParams &p, int n, int a, int len)
{
    return a + len <= n && (n - 1 - a < p.window || a + len - 1 < p.sinks);
}

// A part of one sequence's chunks for one KV head (and part of its query heads), within a CTA's run.
struct Segment {
    int b, kv, part, tokens;
    Chunks chunks;
    int c0, c1;                      // chunks (of the list) to take
    long long unit0;                 // number of the list's first unit
    bool whole;
};

// Walks a CTA's run, segment by segment; every role walks it by itself.
struct Walk {
    const DecodeParams &p;
    long long left, unit0;           // units of the run still to come; number of the current list's first unit
    int b, list, u0, unit, units, tokens;
    Chunks chunks;
    __device__ Walk(const DecodeParams &p, const Shared &S)
        : p(p), left(S.last - S.first), unit0(S.list_unit), b(S.start - 1), list(S.start_list), u0(S.start_unit), unit(S.unit), units(0), tokens(0), chunks{0, 0, 0}
    {
        if (left > 0) sequence();
    }
    // The next sequence with something to see.
    __device__ void sequence()
    {
        do {
            if (++b == p.B) {
                b = 0;
                ++list;
            }
            tokens = tokens_of(p, b);
            chunks = chunks_of(p, tokens);
        } while (chunks.n == 0);
        units = (chunks.n + unit - 1) / unit;
    }
    __device__ bool next(Segment &s)
    {
        if (left <= 0) return false;
        if (u0 == units) {
            sequence();
            u0 = 0;
        }
        const int u1 = static_cast<int>(min(static_cast<long long>(units), u0 + left));
        s.b = b;
        s.kv = p.parts == 1 ? list : list / p.parts;
        s.part = list - s.kv * p.parts;
        s.tokens = tokens;
        s.chunks = chunks;
        s.c0 = u0 * unit;
        s.c1 = min(u1 * unit, chunks.n);
        s.unit0 = unit0;
        s.whole = u0 == 0 && u1 == units;
        left -= u1 - u0;
        unit0 += units;
        u0 = units;
        return true;
    }
};

// Which of a chunk's two tiles are needed.
__device__ __forceinline__ unsigned tiles_of(const DecodeParams &p, int n, int chunk)
{
    const int a = chunk * kChunk;
    return (sees_some(p, n, a, kTile) ? 1u : 0u) | (sees_some(p, n, a + kTile, kTile) ? 2u : 0u);
}

__device__ __forceinline__ long long quotient(long long x, long long y)
{
    return (x | y) >> 32 ? x / y : static_cast<long long>(static_cast<unsigned>(x) / static_cast<unsigned>(y));
}
// The CTA's run: how many units there are, of which size, and where its part begins. All threads. Units are numbered KV head
// by KV head, so that CTAs that go through different heads of a sequence, whose rows lie side by side, do it about the same time
// (sequence by sequence: 218.6 instead of 212.9 us for 64 contexts up to 8192, 266 instead of 258 for two of 262,144).
__device__ void plan(const DecodeParams &p, Shared &S)
{
    const int thread = threadIdx.x, warp = thread >> 5, lane = thread & 31, warps = min(kThreads / 32, (p.B + 31) / 32);
    const unsigned heads = p.KV * p.parts, ctas = gridDim.x;
    long long sum[3] = {0, 0, 0};
    int first_chunks = 0;            // of sequence `thread`
    for (int b0 = warp * 32; b0 < p.B; b0 += kThreads) {
        const int b = b0 + lane;
        unsigned c = 0;              // less than 2^23: a warp's sum fits
        if (b < p.B) {
            const int n = tokens_of(p, b);
            c = chunks_of(p, n).n;
            if (blockIdx.x == 0 && n != p.lengths[b]) atomicExch(p.status, kStatusInvalid);
        }
        if (b0 == warp * 32) first_chunks = c;
        sum[0] += __reduce_add_sync(kWarp, c);
        sum[1] += __reduce_add_sync(kWarp, (c + kBlockChunks - 1) / kBlockChunks);
        sum[2] += __reduce_add_sync(kWarp, (c + kSuperChunks - 1) / kSuperChunks);
    }
    if (warp < warps && lane < 3) S.sums_of[lane][warp] = lane == 0 ? sum[0] : lane == 1 ? sum[1] : sum[2];
    __syncthreads();
    long long total[3] = {0, 0, 0};
    for (int w = 0; w < warps; ++w)
#pragma unroll
        for (int i = 0; i < 3; ++i) total[i] += S.sums_of[i][w];
    const long long enough = static_cast<long long>(kUnitsEach) * ctas;
    const int level = total[2] * heads >= enough ? 2 : total[1] * heads >= enough ? 1 : 0;
    const int unit = level == 2 ? kSuperChunks : level == 1 ? kBlockChunks : 1;
    const long long round = level == 2 ? total[2] : level == 1 ? total[1] : total[0], units = round * heads;
    // Run i of the CTAs' is [units * i / ctas, units * (i + 1) / ctas).
    const long long each = quotient(units, ctas);
    const unsigned rest = static_cast<unsigned>(units - each * ctas);
    auto begin = [&](unsigned i) { return each * i + rest * i / ctas; };
    const long long first = begin(blockIdx.x), last = begin(blockIdx.x + 1);
    const long long list = first < units ? quotient(first, round) : 0, place = first - list * round;
    if (thread == 0) {
        S.first = first;
        S.last = last;
        S.unit = unit;
        if (first == units) p.cuts[blockIdx.x] = Cut{0, 0, 0, 0, unit};
    }
    long long carry = 0;
    for (int b0 = 0; b0 < p.B && carry <= place; b0 += kThreads) {
        const int b = b0 + thread;
        const int n = b >= p.B ? 0 : ((b0 ? chunks_of(p, tokens_of(p, b)).n : first_chunks) + unit - 1) / unit;
        unsigned up = n;
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned x = __shfl_up_sync(kWarp, up, o);
            if (lane >= o) up += x;
        }
        if (b0) __syncthreads();
        if (lane == 31) S.scan[warp] = up;
        __syncthreads();
        long long before = carry + up - n;
        for (int w = 0; w < warps; ++w) {
            const unsigned x = S.scan[w];
            if (w < warp) before += x;
            carry += x;
        }
        if (first < units && place >= before && place < before + n) {
            const long long lo = list * round + before;
            S.start = b;
            S.start_list = static_cast<int>(list);
            S.start_unit = static_cast<int>(place - before);
            S.list_unit = lo;
            // The cut at the run's begin, for the second launch: the list that it goes through, if it is the first inside.
            const bool cut = blockIdx.x > 0 && first > lo && begin(blockIdx.x - 1) <= lo;
            p.cuts[blockIdx.x] = cut ? Cut{lo, n, b, static_cast<int>(list), unit} : Cut{0, 0, 0, 0, unit};
        }
    }
}

// ---- roles

constexpr int kPagesAhead = 8, kLoaded = 16;

// One warp: the page of each eight tokens of a chunk (a lane each), kPagesAhead chunks ahead of the copies.
__device__ void page_role(const DecodeParams &p, Shared &S, const Waits &wait, int lane)
{
    Walk walk(p, S);
    Segment s;
    bool bad = false, more = walk.next(s);
    int c = more ? s.c0 : 0;
    // Four chunks' look-ups at once: each is a trip to memory that is busy.
    constexpr int kAtOnce = 4;
    for (int n = 0; more; n += kAtOnce) {
        int page[kAtOnce], count = 0;
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            page[j] = -2;
            if (!more) continue;
            const int token = s.chunks.at(c) * kChunk + lane * 8;
            if (sees_some(p, s.tokens, token, 8)) page[j] = p.table[s.b * p.ldt + token / p.page_size];
            ++count;
            if (++c == s.c1) {
                more = walk.next(s);
                c = more ? s.c0 : 0;
            }
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            if (j >= count) break;
            const int at = n + j;
            const bool have = page[j] >= 0 && page[j] < p.pages;
            bad |= page[j] != -2 && !have;
            const unsigned got = __ballot_sync(kWarp, have);
            if (!wait.warp(smem_u32(&S.pages_empty[at % kPagesAhead]), ((at / kPagesAhead) & 1) ^ 1)) return;
            S.page[at % kPagesAhead][lane] = have ? page[j] : -1;
            // (Read with the scores, when the copies cannot be as far as the chunk kLoaded further on.)
            if (lane == 0) S.loaded[at % kLoaded] = got;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&S.pages_full[at % kPagesAhead]));
        }
    }
    if (bad) atomicExch(p.status, kStatusInvalid);
}

// One warp for the queries and the keys' tiles (kind 0), one for the values' (kind 1): a copy of a page of 16 tokens is 2 KB, and
// issuing them is work enough for two. A lane is eight tokens (lanes 16-31: their second 64 columns); those at a box's begin
// copy it.
template <int DH, int HE>
__device__ void copy_role(const DecodeParams &p, const DecodeMaps &maps, Shared &S, uint32_t base, const Waits &wait, int kind, int lane)
{
    using C = Cfg<DH, HE>;
    Walk walk(p, S);
    Segment s;
    const CUtensorMap *map = kind ? &maps.v : &maps.k;
    const int g = lane & 15, half = lane >> 4;
    const unsigned in_box = p.box >= 128 ? 0xFFFFu : (1u << (p.box / 8)) - 1u;
    const bool begins_box = ((g * 8) & (p.box - 1)) == 0;
    const int slots = kind ? C::VALUES : C::KEYS, slot0 = kind ? C::KEYS : 0;
    int seq = 0, n = 0, queries = 0;
    InFlight copies{0, 0};           // slots that this warp has filled
    bool ok = !p.force_timeout || kind || wait.warp(smem_u32(&S.never), 0);
    for (int seg = 0; ok && walk.next(s); ++seg) {
        if (kind == 0) {
            const uint32_t qb = smem_u32(&S.q_full[seg & 1]);
            ok = wait.warp(smem_u32(&S.q_empty[seg & 1]), ((seg >> 1) & 1) ^ 1);
            if (!ok) break;
            ++queries;
            if (lane == 0) {
                mbar_arrive_expect_tx(qb, C::Q_BYTES);
                for (int h = 0; h < DH / 64; ++h)
                    load_rows(base + C::OFF_Q + (seg & 1) * C::Q_BYTES + h * C::NT * 128, &maps.q, qb, h * 64, s.kv * p.G + s.part * p.heads, s.b);
            }
        }
        for (int c = s.c0; ok && c < s.c1; ++c, ++n) {
            const int chunk = s.chunks.at(c);
            const unsigned tiles = tiles_of(p, s.tokens, chunk);
            ok = wait.warp(smem_u32(&S.pages_full[n % kPagesAhead]), (n / kPagesAhead) & 1);
            if (!ok) break;
            const int page[2] = {S.page[n % kPagesAhead][g], S.page[n % kPagesAhead][16 + g]};
            // Groups with a page, of either tile. (The vote needs the pages, which an arrival behind their loads would not wait for.)
            const unsigned pages[2] = {__ballot_sync(kWarp, page[0] >= 0) & 0xFFFFu, __ballot_sync(kWarp, page[1] >= 0) & 0xFFFFu};
            if (lane == 0) mbar_arrive(smem_u32(&S.pages_empty[n % kPagesAhead]));
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (!((tiles >> t) & 1u)) continue;
                // Boxes with a token to copy. Its page: of any of its groups (they share it).
                const unsigned mine = begins_box ? (pages[t] >> g) & in_box : 0;
                const int box_page = __shfl_sync(kWarp, page[t], mine ? (g + __ffs(mine) - 1) & 15 : g);
                const unsigned boxes = __popc(__ballot_sync(kWarp, mine != 0) & 0xFFFFu);
                const int slot = slot0 + seq % slots, token = chunk * kChunk + t * kTile + g * 8;
                ok = ok && wait.warp(smem_u32(&S.empty[slot]), ((seq / slots) & 1) ^ 1);
                if (!ok) break;
                copies.add(slot, (seq / slots) & 1);
                const uint32_t bar = smem_u32(&S.full[slot]);
                if (lane == 0) mbar_arrive_expect_tx(bar, boxes * p.box * (DH / 64) * 128);
                __syncwarp();
                if (mine && half < DH / 64)
                    asm volatile(
                        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(base + slot * C::TILE + half * kTile * 128 + g * 1024),
                        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(half * 64), "r"(s.kv), "r"(token % p.page_size), "r"(box_page)
                        : "memory");
                __syncwarp();
                ++seq;
            }
        }
    }
    // Copies in flight are of the last phases that were begun; older ones are over. (What another role's end asks for is at the
    // kernel's end. Without the waits here as well the loop above is compiled to something slower: 68.5 instead of 66.6 us for 96
    // windows of 1024 in eight heads of 64.)
    if (!ok || *wait.abort_flag) {
        for (int i = max(0, queries - 2); i < queries; ++i) wait.drain(smem_u32(&S.q_full[i & 1]), (i >> 1) & 1);
        for (int i = 0; i < C::SLOTS; ++i)
            if ((copies.begun >> i) & 1u) wait.drain(smem_u32(&S.full[i]), (copies.parity >> i) & 1u);
    }
    if (lane == 0) {
        S.copies[kind] = copies;
        if (kind == 0) S.queries = queries;
    }
}

// What the issuer keeps of a chunk whose scores have been made. 
struct Ahead {
    int value;                       // number of its first tile of values
    unsigned tiles;
};

template <int DH, int HE>
__device__ void issue_role(const DecodeParams &p, Shared &S, uint32_t base, const Waits &wait)
{
    using C = Cfg<DH, HE>;
    constexpr int NT = C::NT;
    constexpr uint32_t SC = idesc_bf16(kTile, NT, 0, 0), PV = idesc_bf16(kTile, NT, 1, 0);
    const uint32_t tm = S.tmem;
    const int steps = (p.D + 15) / 16;
    Walk walk(p, S);
    Segment s;
    bool ok = true, more = walk.next(s);
    int keys = 0, value = 0, seg = 0, c = more ? s.c0 : 0, n = 0;      // n: chunks whose scores were issued
    auto full = [&](int slot, int round) {
        ok = ok && wait.one(smem_u32(&S.full[slot]), round & 1);
        return ok;
    };
    // The scores of the run's next chunk.
    auto scores = [&](Ahead &a) {
        if (c == s.c0) ok = ok && wait.one(smem_u32(&S.q_full[seg & 1]), (seg >> 1) & 1);
        a = Ahead{value, tiles_of(p, s.tokens, s.chunks.at(c))};
        int q = keys;
        for (int t = 0; t < 2; ++t) {
            if (!((a.tiles >> t) & 1u)) continue;
            if (!full(q % C::KEYS, q / C::KEYS)) return;
            tc_fence_after();
            const uint64_t k = sdesc(base + q % C::KEYS * C::TILE, 16u, 1024u), x = sdesc(base + C::OFF_Q + (seg & 1) * C::Q_BYTES, 16u, 1024u);
            const uint32_t d = tm + C::T_SCORES + ((n & 1) * 2 + t) * NT;
#pragma unroll
            for (int i = 0; i < DH / 16; ++i)
                if (i < steps) mma_bf16(d, k + (i >> 2) * (kTile * 128 / 16) + (i & 3) * 2, x + (i >> 2) * (NT * 128 / 16) + (i & 3) * 2, SC, i != 0);
            ++q;
        }
        mma_commit(smem_u32(&S.scores[n & 1]));
        for (int i = keys; C::COMMIT && i < q; ++i) mma_commit(smem_u32(&S.empty[i % C::KEYS]));
        value += q - keys;
        keys = q;
        ++n;
        if (++c == s.c1) {
            more = walk.next(s);
            ++seg;
            c = more ? s.c0 : 0;
        }
    };
    // The weighted values of chunk i.
    auto values = [&](const Ahead &a, int i) {
        ok = ok && wait.one(smem_u32(&S.probs[i & 1]), (i >> 1) & 1);
        if (!ok) return;
        const uint32_t d = tm + C::T_CHUNK + i % kSums * NT;
        int q = a.value, first = 1;
        for (int t = 0; t < 2; ++t) {
            if (!((a.tiles >> t) & 1u)) continue;
            if (!full(C::KEYS + q % C::VALUES, q / C::VALUES)) return;
            tc_fence_after();
            const uint64_t v = sdesc(base + (C::KEYS + q % C::VALUES) * C::TILE, kTile * 128u, 1024u);
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k) {
                const int key = t * kTile + k * 16;
                const uint64_t pr = sdesc(base + C::OFF_P + (i & 1) * C::P_BYTES + (key >> 6) * NT * 128, 16u, 1024u) + ((key >> 4) & 3) * 2;
                mma_bf16(d, v + k * (2048 / 16), pr, PV, !first);
                first = 0;
            }
            ++q;
        }
        mma_commit(smem_u32(&S.sums[i % kSums]));
        for (int j = a.value; C::COMMIT && j < q; ++j) mma_commit(smem_u32(&S.empty[C::KEYS + j % C::VALUES]));
    };
    Ahead cur{}, next{};
    bool have = more;
    if (more) scores(cur);
    for (int i = 0; ok && have; ++i) {
        const bool have_next = more;
        if (have_next) scores(next);
        if (ok) values(cur, i);
        cur = next;
        have = have_next;
    }
}

__device__ __forceinline__ float redux_max(float v)
{
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// Whether one of a warpgroup's warps says so; they wait for one another (named barrier `id`).
__device__ __forceinline__ bool any_of_four(bool v, int id)
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "bar.red.or.pred p, %2, 128, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(v)), "r"(id)
        : "memory");
    return r != 0;
}

// N TMEM columns of this thread's lane.
template <int N>
__device__ __forceinline__ void ld(uint32_t at, uint32_t (&r)[N])
{
    if constexpr (N == 4) detg::tmem_ld4(at, r);
    else if constexpr (N == 8) detg::tmem_ld8(at, r);
    else if constexpr (N == 16) detg::tmem_ld16(at, r);
    else tmem_ld32(at, r);
}
template <int N>
__device__ __forceinline__ void st(uint32_t at, const uint32_t (&r)[N])
{
    if constexpr (N == 4) detg::tmem_st4(at, r);
    else if constexpr (N == 8) detg::tmem_st8(at, r);
    else if constexpr (N == 16) detg::tmem_st16(at, r);
    else tmem_st32(at, r);
}
template <int N>
__device__ __forceinline__ void fence(uint32_t (&r)[N])
{
    if constexpr (N == 4) detg::reg_fence4(r);
    else if constexpr (N == 8) detg::reg_fence8(r);
    else if constexpr (N == 16) detg::reg_fence16(r);
    else reg_fence(r);
}

// v[0] of lane i: the sum over all lanes of v[i / (32 / N)]. Each step halves the values and doubles the lanes that they are of.
template <int N>
__device__ __forceinline__ void sum_lanes(float (&v)[N], int lane)
{
#pragma unroll
    for (int n = N / 2, o = 16; n >= 1; n /= 2, o /= 2) {
        const bool high = lane & o;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float give = high ? v[i] : v[i + n], keep = high ? v[i + n] : v[i];
            v[i] = keep + __shfl_xor_sync(kWarp, give, o);
        }
    }
#pragma unroll
    for (int o = 16 / N; o >= 1; o /= 2) v[0] += __shfl_xor_sync(kWarp, v[0], o);
}

// One of two warpgroups: the chunks n with n % 2 == group.
template <int DH, int HE>
__device__ void softmax_role(const DecodeParams &p, Shared &S, uint32_t base, const Waits &wait, int group, int warp, int lane)
{
    using C = Cfg<DH, HE>;
    constexpr int NT = C::NT;
    const int row = warp * 32 + lane;                // token of a tile
    const uint32_t tm = S.tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const float c = p.scale * kLog2e;
    Walk walk(p, S);
    Segment s;
    bool ok = true;
    int n = 0, value = 0;
    for (int seg = 0; walk.next(s); ++seg) {
        for (int ch = s.c0; ch < s.c1; ++ch, ++n) {
            const int chunk = s.chunks.at(ch), token = chunk * kChunk + row;
            const unsigned tiles = tiles_of(p, s.tokens, chunk);
            int v = value;
            const int k = value;     // keys' tiles have the values' numbers
            value += __popc(tiles);
            if ((n & 1) != group) continue;
            const uint32_t phase = (n >> 1) & 1;
            uint32_t x[2][HE];
            float top[HE];
            float *shared_top = &S.top[group][phase][0][0];
            ok = ok && wait.warp(smem_u32(&S.scores[group]), phase);
            if (ok) {
                if (!C::COMMIT && warp == 0 && lane < value - k) mbar_arrive(smem_u32(&S.empty[(k + lane) % C::KEYS]));
                if (warp == 1 && lane == 0 && ch + 1 == s.c1) mbar_arrive(smem_u32(&S.q_empty[seg & 1]));
                tc_fence_after();
                const unsigned loaded = S.loaded[n % kLoaded];
                bool seen[2], edge = false;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    seen[t] = false;
                    if ((tiles >> t) & 1u) {
                        const unsigned have = (loaded >> (16 * t)) & 0xFFFFu;
                        seen[t] = sees(p, s.tokens, token + t * kTile) && ((have >> (row >> 3)) & 1u);
                        edge |= have != 0xFFFFu || !sees_every(p, s.tokens, chunk * kChunk + t * kTile, kTile);
                        ld<HE>(tm + C::T_SCORES + (group * 2 + t) * NT, x[t]);
                    }
                }
                tmem_wait_ld();
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    fence<HE>(x[t]);
#pragma unroll
                    for (int h = 0; h < HE; ++h) x[t][h] = __float_as_uint(seen[t] ? __uint_as_float(x[t][h]) * c : -INFINITY);
                }
#pragma unroll
                for (int h = 0; h < HE; ++h) top[h] = redux_max(fmaxf(__uint_as_float(x[0][h]), __uint_as_float(x[1][h])));
                if (lane == 0) {
#pragma unroll
                    for (int h = 0; h < HE; h += 4) *reinterpret_cast<float4 *>(shared_top + warp * 32 + h) = make_float4(top[h], top[h + 1], top[h + 2], top[h + 3]);
                }
                // The chunk two before has been joined: its values have been weighted and make room for P, and its sums for new ones.
                static_assert(kSums == 2, "P and sums are of the same chunks");
                ok = ok && wait.warp(smem_u32(&S.joined[n % kSums]), ((n / kSums) & 1) ^ 1);
                // Values of hidden tokens are whatever was there: zeros, for the product. What was in these values' slots
                // before has been used, so that their barriers are in the phase before: it was a chunk's two before or older,
                // or (a ring of less than two chunks) of the one before, whose sums are awaited.
                if (edge) {
                    if (C::VALUES < 4 && n > 0) ok = ok && wait.warp(smem_u32(&S.sums[(n - 1) % kSums]), ((n - 1) / kSums) & 1);
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (!((tiles >> t) & 1u)) continue;
                        ok = ok && wait.warp(smem_u32(&S.full[C::KEYS + v % C::VALUES]), (v / C::VALUES) & 1);
                        if (ok && !seen[t]) {
                            const uint32_t at = base + (C::KEYS + v % C::VALUES) * C::TILE + row * 128;
#pragma unroll
                            for (int h = 0; h < DH / 64; ++h)
#pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at + h * kTile * 128 + ((e ^ row) & 7) * 16), "r"(0) : "memory");
                        }
                        ++v;
                    }
                }
            }
            // All four warps leave here together, if one has to: none waits below for another that is gone.
            if (any_of_four(!ok, 1 + group)) return;
#pragma unroll
            for (int h = 0; h < HE; h += 4) {
                float4 y = *reinterpret_cast<const float4 *>(shared_top + h);
#pragma unroll
                for (int w = 1; w < 4; ++w) {
                    const float4 z = *reinterpret_cast<const float4 *>(shared_top + w * 32 + h);
                    y = make_float4(fmaxf(y.x, z.x), fmaxf(y.y, z.y), fmaxf(y.z, z.z), fmaxf(y.w, z.w));
                }
                if (row == 0) *reinterpret_cast<float4 *>(&S.most[n % (2 * kSums)][h]) = y;
                top[h] = y.x;
                top[h + 1] = y.y;
                top[h + 2] = y.z;
                top[h + 3] = y.w;
            }
            const uint32_t pr = base + C::OFF_P + group * C::P_BYTES;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (!((tiles >> t) & 1u)) continue;
                const int key = t * kTile + row;
                const uint32_t at = pr + (key >> 6) * NT * 128 + (key & 7) * 2;
#pragma unroll
                for (int h = 0; h < HE; ++h) {
                    const uint32_t y = pack_bf16(exp2_fast(__uint_as_float(x[t][h]) - (top[h] == -INFINITY ? 0.0f : top[h])), 0.0f);
                    x[t][h] = y << 16;
                    asm volatile("st.shared.u16 [%0], %1;" ::"r"(at + (h >> 3) * 1024 + (h & 7) * 128 + ((((key >> 3) & 7) ^ (h & 7)) * 16)),
                                 "h"(static_cast<uint16_t>(y))
                                 : "memory");
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
#pragma unroll
            for (int h = 0; h < HE; ++h) {
                const float a = (tiles & 1u) ? __uint_as_float(x[0][h]) : 0.0f, b = (tiles & 2u) ? __uint_as_float(x[1][h]) : 0.0f;
                top[h] = a + b;
            }
            sum_lanes<HE>(top, lane);
            if (lane % (32 / HE) == 0) S.sum[n % (2 * kSums)][warp][lane / (32 / HE)] = top[0];
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&S.probs[group]));
        }
    }
}

// Joins (m, l, o) of two neighbours, the earlier first: each scaled to the larger maximum.
struct Factors {
    float a, b, m;
};
__device__ __forceinline__ Factors factors(float ma, float mb)
{
    const float m = fmaxf(ma, mb), off = m == -INFINITY ? 0.0f : m;
    return Factors{exp2_fast(ma - off), exp2_fast(mb - off), m};
}
__device__ __forceinline__ float join(float a, float b, const Factors &f) { return __fmaf_rn(a, f.a, __fmul_rn(b, f.b)); }

// The output: zero where nothing was seen. (The quotient is off by 2^-22 at most, and rounded to BF16.)
__device__ __forceinline__ float weighted(float o, float l) { return l == 0.0f ? 0.0f : __fdividef(o, l); }

// Column `row` of the sums of every head, their l and m.
template <int HE>
struct Sums {
    uint32_t o[HE], l[HE], m[HE];
    // This, then `next`: into this.
    __device__ __forceinline__ void join_next(const Sums &next)
    {
#pragma unroll
        for (int i = 0; i < HE; ++i) {
            const Factors f = factors(__uint_as_float(m[i]), __uint_as_float(next.m[i]));
            o[i] = __float_as_uint(join(__uint_as_float(o[i]), __uint_as_float(next.o[i]), f));
            l[i] = __float_as_uint(join(__uint_as_float(l[i]), __uint_as_float(next.l[i]), f));
            m[i] = __float_as_uint(f.m);
        }
    }
    __device__ __forceinline__ void load(uint32_t at)
    {
        ld<HE>(at, o);
        ld<HE>(at + HE, l);
        ld<HE>(at + 2 * HE, m);
        tmem_wait_ld();
        fence<HE>(o);
        fence<HE>(l);
        fence<HE>(m);
    }
    __device__ __forceinline__ void store(uint32_t at) const
    {
        st<HE>(at, o);
        st<HE>(at + HE, l);
        st<HE>(at + 2 * HE, m);
        tmem_wait_st();
    }
};

// One warpgroup: the chunks' sums in order. A block's are kept in registers, those of a super block and of all in TMEM.
template <int DH, int HE>
__device__ void join_role(const DecodeParams &p, Shared &S, const Waits &wait, int warp, int lane)
{
    using C = Cfg<DH, HE>;
    constexpr int NT = C::NT;
    const int row = warp * 32 + lane, unit = S.unit;
    const uint32_t tm = S.tmem + (static_cast<uint32_t>(warp * 32) << 16);
    Walk walk(p, S);
    Segment s;
    int n = 0, value = 0;
    Sums<HE> sums;
    while (walk.next(s)) {
        const int head0 = s.kv * p.G + s.part * p.heads, heads = min(p.heads, p.G - s.part * p.heads);
        for (int ch = s.c0; ch < s.c1; ++ch, ++n) {
            const int at = n % kSums, of = n % (2 * kSums);
            if (!wait.warp(smem_u32(&S.sums[at]), (n / kSums) & 1)) return;
            const int count = __popc(tiles_of(p, s.tokens, s.chunks.at(ch)));
            if (!C::COMMIT && warp == 0 && lane < count) mbar_arrive(smem_u32(&S.empty[C::KEYS + (value + lane) % C::VALUES]));
            value += count;
            tc_fence_after();
            Sums<HE> x;
            ld<HE>(tm + C::T_CHUNK + at * NT, x.o);
#pragma unroll
            for (int h = 0; h < HE; h += 4) {
                const float4 y = *reinterpret_cast<const float4 *>(&S.most[of][h]);
                x.m[h] = __float_as_uint(y.x);
                x.m[h + 1] = __float_as_uint(y.y);
                x.m[h + 2] = __float_as_uint(y.z);
                x.m[h + 3] = __float_as_uint(y.w);
                const float4 a = *reinterpret_cast<const float4 *>(&S.sum[of][0][h]), b = *reinterpret_cast<const float4 *>(&S.sum[of][1][h]);
                const float4 c = *reinterpret_cast<const float4 *>(&S.sum[of][2][h]), d = *reinterpret_cast<const float4 *>(&S.sum[of][3][h]);
                x.l[h] = __float_as_uint((a.x + b.x) + (c.x + d.x));
                x.l[h + 1] = __float_as_uint((a.y + b.y) + (c.y + d.y));
                x.l[h + 2] = __float_as_uint((a.z + b.z) + (c.z + d.z));
                x.l[h + 3] = __float_as_uint((a.w + b.w) + (c.w + d.w));
            }
            tmem_wait_ld();
            fence<HE>(x.o);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&S.joined[at]));
            const bool end = ch + 1 == s.c1;
            // A unit that is one chunk of a list that others have parts of goes as it is; a block begins with its first.
            if ((unit == 1 && !s.whole) || ch % kBlockChunks == 0) {
                sums = x;
            } else {
                sums.join_next(x);
            }
            if (s.whole || unit > kBlockChunks) {
                // The block is over: into its super block, which is over as well at its end or the list's.
                if (!end && (ch + 1) % kBlockChunks != 0) continue;
                const bool super_end = end || (ch + 1) % kSuperChunks == 0;
                if (ch / kBlockChunks * kBlockChunks != ch / kSuperChunks * kSuperChunks) {
                    Sums<HE> before;
                    before.load(tm + C::T_LEVEL);
                    before.join_next(sums);
                    sums = before;
                }
                if (!super_end) {
                    sums.store(tm + C::T_LEVEL);
                    continue;
                }
                if (s.whole) {
                    if (ch >= kSuperChunks) {
                        Sums<HE> before;
                        before.load(tm + C::T_LEVEL + C::STATE);
                        before.join_next(sums);
                        sums = before;
                    }
                    if (!end) {
                        sums.store(tm + C::T_LEVEL + C::STATE);
                        continue;
                    }
                }
            } else if (!end && (ch + 1) % unit != 0) {
                continue;
            }
            if (s.whole && row < p.D) {
                uint16_t *out = p.out.row(s.b, head0) + row;
#pragma unroll
                for (int h = 0; h < HE; ++h, out += p.out.h)
                    if (h < heads) *out = static_cast<uint16_t>(pack_bf16(weighted(__uint_as_float(sums.o[h]), __uint_as_float(sums.l[h])), 0.0f));
            } else if (row < p.D) {
                float *part = p.partials + (s.unit0 + ch / unit) * static_cast<long long>(p.heads) * (p.D + 2);
#pragma unroll
                for (int h = 0; h < HE; ++h)
                    if (h < heads) {
                        part[h * p.D + row] = __uint_as_float(sums.o[h]);
                        if (row == 0) {
                            part[p.heads * p.D + h] = __uint_as_float(sums.l[h]);
                            part[p.heads * (p.D + 1) + h] = __uint_as_float(sums.m[h]);
                        }
                    }
            }
            __syncwarp();
        }
    }
}

template <int DH, int HE>
__global__ void __launch_bounds__(kThreads, 1) attn_decode_kernel(const __grid_constant__ DecodeParams p, const __grid_constant__ DecodeMaps maps)
{
    using C = Cfg<DH, HE>;
    extern __shared__ uint8_t attn_smem[];
    const uint32_t raw = smem_u32(attn_smem), base = (raw + 1023u) & ~1023u;
    uint8_t *smem = attn_smem + (base - raw);
    Shared &S = *reinterpret_cast<Shared *>(smem + C::OFF_SHARED);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        S.abort_flag = 0;
        S.copies[0] = S.copies[1] = InFlight{0, 0};
        S.queries = 0;
        for (int i = 0; i < C::SLOTS; ++i) {
            mbar_init(smem_u32(&S.full[i]), 1);
            mbar_init(smem_u32(&S.empty[i]), 1);
        }
        for (int i = 0; i < kSums; ++i) {
            mbar_init(smem_u32(&S.sums[i]), 1);
            mbar_init(smem_u32(&S.joined[i]), 4);
        }
        for (int i = 0; i < kPagesAhead; ++i) {
            mbar_init(smem_u32(&S.pages_full[i]), 1);
            mbar_init(smem_u32(&S.pages_empty[i]), 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&S.q_full[i]), 1);
            mbar_init(smem_u32(&S.q_empty[i]), 1);
            mbar_init(smem_u32(&S.scores[i]), 1);
            mbar_init(smem_u32(&S.probs[i]), 4);
        }
        mbar_init(smem_u32(&S.drain), 1);
        mbar_init(smem_u32(&S.never), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 12 && lane == 0) {
        tmap_prefetch(&maps.q);
        if (p.pages > 0) {
            tmap_prefetch(&maps.k);
            tmap_prefetch(&maps.v);
        }
    }
    if (warp == 13) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&S.tmem)), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    wait_for_last();
    if (warp == 14) {
        // The look-ups come after the lengths: the table's lines (of small ones all, else the first) are on their way to L2 by then.
        const int lines = (p.max_pages + 31) / 32, i = blockIdx.x * 32 + lane;
        if (lines > 0 && i / lines < p.B) prefetch_l2(p.table + i / lines * p.ldt + i % lines * 32);
    }
    plan(p, S);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const Waits wait{&S.abort_flag, p.status, p.timeout_ns};
    if (warp < 8) {
        softmax_role<DH, HE>(p, S, base, wait, warp >> 2, warp & 3, lane);
    } else if (warp < 12) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::JOIN_REGS));
        join_role<DH, HE>(p, S, wait, warp & 3, lane);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::SERVICE_REGS));
        if (warp == 12 || warp == 14) {
            copy_role<DH, HE>(p, maps, S, base, wait, warp == 14, lane);
        } else if (warp == 13) {
            if (elect_one()) issue_role<DH, HE>(p, S, base, wait);
        } else {
            page_role(p, S, wait, lane);
            for (int b = blockIdx.x; b < p.B; b += gridDim.x)
                if (tokens_of(p, b) == 0)
                    for (int i = lane * 8; i < p.H * p.D; i += 256) *reinterpret_cast<uint4 *>(p.out.row(b, i / p.D) + i % p.D) = make_uint4(0, 0, 0, 0);
        }
    }
    // (Every CTA: the next launch may be the join, which waits for all of this one at its start in any case.)
    let_next_begin();
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (*wait.abort_flag) {
        if ((warp == 12 || warp == 14) && elect_one()) {
            for (int i = max(0, S.queries - 2); i < S.queries; ++i) wait.drain(smem_u32(&S.q_full[i & 1]), (i >> 1) & 1);
            drain_copies(S.full, S.copies[warp == 14], wait);
        }
        if (warp == 13 && elect_one()) drain_products(smem_u32(&S.drain), wait);
        __syncwarp();
        __syncthreads();
    }
    if (warp == 13) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(S.tmem), "r"(512) : "memory");
}

// ------------------------------------------- joining what was cut
//
// For each CTA whose run begins inside a list (a sequence, KV head and part), the first of those: the list's units are joined.
// Threads of a warpgroup are the columns. Where no list is longer than a super block, a warpgroup is a query head (blocks of
// the grid: eight heads), or if there is one head a block of the list in turn; else a warpgroup is a super block in turn, and
// each head has blocks of its own. (With a block of the grid for each head throughout, 96 windows of 1024 took 20 us to join.)

constexpr int kJoinGroups = 8;

struct State {
    float o, l, m;
};
__device__ __forceinline__ void join(State &a, const State &b, bool first)
{
    if (first) {
        a = b;
        return;
    }
    const Factors f = factors(a.m, b.m);
    a.o = join(a.o, b.o, f);
    a.l = join(a.l, b.l, f);
    a.m = f.m;
}

__global__ void __launch_bounds__(128 * kJoinGroups) attn_join_kernel(const DecodeParams p, const bool short_lists)
{
    wait_for_last();
    __shared__ State at[kSuperChunks / kBlockChunks][128];
    const Cut cut = p.cuts[blockIdx.x + 1];
    const int group = threadIdx.x >> 7, d = threadIdx.x & 127, column = min(d, p.D - 1);
    const bool by_head = short_lists && p.heads > 1;
    const int n = cut.n, unit = cut.unit, h = by_head ? blockIdx.y * kJoinGroups + group : blockIdx.y;
    if (n == 0) return;
    const int kv = cut.list / p.parts, part = cut.list % p.parts, heads = min(p.heads, p.G - part * p.heads);
    if (h >= heads) return;          // (whole blocks, or groups that none waits for)
    const long long pitch = static_cast<long long>(p.heads) * (p.D + 2);
    const float *mine = p.partials + cut.first * pitch;
    auto load = [&](int i) {
        const float *x = mine + i * pitch;
        return State{x[h * p.D + column], x[p.heads * p.D + h], x[p.heads * (p.D + 1) + h]};
    };
    const int per_block = max(1, kBlockChunks / unit), per_super = kSuperChunks / unit, supers = (n + per_super - 1) / per_super;
    // Super block s, eight loads in flight.
    auto super_block = [&](int s) {
        State super{}, block{};
        const int end = min(n, (s + 1) * per_super);
        int i = s * per_super;
        while (i < end) {
            State x[8];
            const int count = min(8, end - i);
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = load(min(i + k, end - 1));
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (k >= count) break;
                join(block, x[k], (i + k) % per_block == 0);
                if ((i + k + 1) % per_block == 0 || i + k + 1 == end) join(super, block, (i + k) / per_block * per_block == s * per_super);
            }
            i += count;
        }
        return super;
    };
    State all{};
    if (by_head) {
        all = super_block(0);
    } else if (short_lists) {
        const int blocks = (n + per_block - 1) / per_block;
        for (int i = group; i < blocks; i += kJoinGroups) {
            State x[kBlockChunks], block{};
#pragma unroll
            for (int k = 0; k < kBlockChunks; ++k) x[k] = load(min(i * per_block + min(k, per_block - 1), n - 1));
#pragma unroll
            for (int k = 0; k < kBlockChunks; ++k)
                if (k < per_block && i * per_block + k < n) join(block, x[k], k == 0);
            at[i][d] = block;
        }
        __syncthreads();
        if (group == 0)
            for (int i = 0; i < blocks; ++i) join(all, at[i][d], i == 0);
    } else {
        for (int s0 = 0; s0 < supers; s0 += kJoinGroups) {
            if (s0 + group < supers) at[group][d] = super_block(s0 + group);
            __syncthreads();
            if (group == 0)
                for (int k = 0; k < kJoinGroups && s0 + k < supers; ++k) join(all, at[k][d], s0 + k == 0);
            __syncthreads();
        }
    }
    if ((by_head || group == 0) && d < p.D) {
        const float y = weighted(all.o, all.l);
        p.out.row(cut.b, kv * p.G + part * p.heads + h)[d] = static_cast<uint16_t>(pack_bf16(y, 0.0f));
    }
}

template <int DH, int HE>
cudaError_t run(const DecodeParams &p, const DecodeMaps &maps, int ctas, cudaStream_t s)
{
    using C = Cfg<DH, HE>;
    auto fn = attn_decode_kernel<DH, HE>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = once_per_device(done, [&] {
        cudaFuncAttributes a;
        const cudaError_t x = cudaFuncGetAttributes(&a, fn);
        if (x != cudaSuccess) return x;
        // setmaxnreg shares out exactly the registers of the launch.
        if (a.numRegs != kLaunchRegs) return cudaErrorInvalidDeviceFunction;
        return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    });
    if (e != cudaSuccess) return e;
    e = launch_early(fn, ctas, kThreads, C::SMEM, 1, s, p, maps);
    if (e != cudaSuccess || ctas < 2) return e;
    // The chunks of the longest list: the cache's, or its first and the window's.
    const long long room = (static_cast<long long>(p.max_pages) * p.page_size + kChunk - 1) / kChunk;
    const long long kept = (static_cast<long long>(p.sinks) + kChunk - 1) / kChunk + (static_cast<long long>(p.window) - 1) / kChunk + 2;
    const bool short_lists = std::min(room, kept) <= kSuperChunks;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas - 1), static_cast<unsigned>(short_lists ? (p.heads + kJoinGroups - 1) / kJoinGroups : p.heads));
    cfg.blockDim = dim3(128 * kJoinGroups);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, attn_join_kernel, p, short_lists);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

template <int DH>
cudaError_t run(const DecodeParams &p, const DecodeMaps &maps, int ctas, cudaStream_t s)
{
    if (p.heads <= 4) return run<DH, 4>(p, maps, ctas, s);
    if (p.heads <= 8) return run<DH, 8>(p, maps, ctas, s);
    return p.heads <= 16 ? run<DH, 16>(p, maps, ctas, s) : run<DH, 32>(p, maps, ctas, s);
}

}  // namespace

cudaError_t launch_attn_decode(const DecodeParams &p, const DecodeMaps &maps, int ctas, cudaStream_t s)
{
    return p.D <= 64 ? run<64>(p, maps, ctas, s) : run<128>(p, maps, ctas, s);
}

}  // namespace deto
