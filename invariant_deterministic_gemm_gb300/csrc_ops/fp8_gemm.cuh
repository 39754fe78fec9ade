// 8-bit block-scaled matrix products for sm_103a.
//
//   out[r, c] = sum over blocks b of sa(r, b) * sb(c, b) * P_b,
//   P_b = sum over the 128 contraction elements of block b of A[r, k] * B[c, k]
//
// P_b is one tcgen05 accumulation in FP32 (four K = 32 steps, products of
// two e4m3 values are exact); the blocks are added in ascending order by one
// FP32 fused multiply-add each, acc = fma(P_b, sa * sb, acc), the scales'
// product rounded once. Tiles, batch size and the choice of kernel never
// enter: an element's bits depend on its row of A and its row of B only.
//
// The tensor core cannot apply FP32 scales, so every block's accumulator
// leaves TMEM and is added in registers. For a 128 x 192 tile the four MMAs
// take about 390 cycles (98 each); what has to fit beside them is the TMEM
// read, whose latency (about 200 cycles) is the long part, and 192
// multiply-adds a row, done two at a time (fma.f32x2).
//
// Plain tile (BN / 64 epilogue warps per quadrant and four service warps,
// one CTA per SM, persistent over tiles):
//   epilogue   warp w: TMEM lane quadrant w % 4 (32 rows), columns
//              64 (w / 4).. of the tile; a thread keeps 64 sums of one row
//   service 0  copies A and B blocks in with TMA
//   service 1, 2  issue the MMAs of alternate blocks, each from one thread:
//              a block's waits, four MMAs and two commits take one thread
//              about 700 cycles, the MMAs themselves 390
//   service 3  allocates and frees TMEM
// Both accumulators of 192 columns alternate. 64 columns a thread let one
// wait cover a whole block's TMEM read; with eight warps of 128 columns (a
// 128 x 256 tile) a thread's four waits for TMEM were the bound, 1190 cycles
// a block where the MMAs take 520.
//
// Transposed tile (few rows: decode): the weight is the MMA's row side, its
// 32, 64 or 128 rows are TMEM lanes, and the tokens its 16 to 64 columns.
// The launch is bound by reading the weight once, and a tile walks its
// blocks one after the other, so what a block costs each role counts: copies
// come two blocks a stage, accumulators go round four blocks at a time (one
// wait and release for the four), two threads issue the MMAs of alternate
// stages, and a warp of its own brings the scales' products. Up to 96 KB of
// copies are in flight a CTA and two CTAs share an SM (192 KB and one for 64
// tokens). A tile of 32 or 64 weight rows still issues 128-row MMAs: the other
// lanes multiply whatever the following shared memory holds and are never
// read. Three rows on [12288, 4096] take 10.3 us, 4.9 TB/s of weights; 34 rows of
// eight experts on [1792, 4096] 9.8 us.
//
// Weight gradient: both operands are scaled per row of theirs. The scales come
// by TMA with the operands' copies, and each element takes one more
// multiplication (55 of a block's 395 ns). With scales copied by the epilogue's
// own threads, their ring took the room of a fifth stage: 413 ns.
//
// [8192, 4096] x [14336, 4096] takes 385 us (2.50 PFLOP/s), its weight gradient 498
// us. A block of a 128 x 192 tile takes 315 ns (weight gradient 395); 285 without
// the epilogue's reads and sums, 262 with operands from few lines of L2 too.
// The MMAs alone are 196. What holds the 262 is not known: 40 KB a block and SM
// in them are 156 bytes a ns, and the 128 x 128 tile's 32 KB in 217 ns are 151, so
// it may be what an SM takes in. A tile's end adds 2 us, half of it stores that
// all CTAs issue at once: a third of a tile of 14 blocks.
//
// Waits are bounded as in det_gemm's kernels (a timeout sets the status
// word, every role leaves, copies and MMAs in flight are drained).
#pragma once

#include "det_gemm_kernel.cuh"
#include "launch.cuh"
#include "ops_internal.h"
#include "vec.cuh"

namespace deto {

using detg::elect_one;
using detg::mbar_arrive_expect_tx;
using detg::mbar_arrive_if;
using detg::mbar_init;
using detg::mma_commit;
using detg::reg_fence;
using detg::reg_fence16;
using detg::smem_u32;
using detg::tc_fence_after;
using detg::tc_fence_before;
using detg::tma_load_2d;
using detg::tmap_prefetch;
using detg::tmem_ld16;
using detg::tmem_ld32;
using detg::tmem_wait_ld;
using detg::wait_bounded;
using detg::mbar_wait_inline;

constexpr unsigned kFull = 0xFFFFFFFFu;

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x, int y, int z)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// Instruction descriptor, kind::f8f6f4: e4m3 x e4m3 -> FP32, both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int m, int n)
{
    return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// The four K = 32 steps of one block (32 bytes along a 128-byte row each).
__device__ __forceinline__ void mma_block(uint32_t d, uint32_t a_smem, uint32_t b_smem, uint32_t idesc)
{
    const uint64_t a = detg::sdesc(a_smem, 16u, 1024u), b = detg::sdesc(b_smem, 16u, 1024u);
#pragma unroll
    for (int k = 0; k < 4; ++k) mma_e4m3(d, a + 2 * k, b + 2 * k, idesc, k != 0);
}

// Two FP32 operations at once, each rounded to nearest like the scalar one.
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi)
{
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
    return d;
}
__device__ __forceinline__ uint64_t pair(float lo, float hi) { return pair(__float_as_uint(lo), __float_as_uint(hi)); }
__device__ __forceinline__ void unpair(uint64_t v, float &lo, float &hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
// sum += v * scale for four columns, the scales read from shared memory. One volatile block: apart, the compiler loads a
// whole block's scales ahead of their use and spills.
__device__ __forceinline__ void add4(uint64_t &sum0, uint64_t &sum1, uint64_t v0, uint64_t v1, uint32_t at)
{
    asm volatile(
        "{\n\t.reg .b64 s0, s1;\n\t"
        "ld.shared.v2.b64 {s0, s1}, [%4];\n\t"
        "fma.rn.f32x2 %0, %2, s0, %0;\n\t"
        "fma.rn.f32x2 %1, %3, s1, %1;\n\t}"
        : "+l"(sum0), "+l"(sum1)
        : "l"(v0), "l"(v1), "r"(at)
        : "memory");
}
// 16 TMEM lanes x 64 columns: r[4 j + 2 h + e] is lane (thread / 4 + 8 h),
// column 8 j + 2 (thread % 4) + e. A thread then has few distinct columns
// (16 of 64) and a few rows, so few distinct scales.
__device__ __forceinline__ void tmem_ld_16x64(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, "
        "%20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float lds1(uint32_t at)
{
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint64_t lds2(uint32_t at)
{
    uint64_t v;
    asm volatile("ld.shared.b64 %0, [%1];" : "=l"(v) : "r"(at) : "memory");
    return v;
}

// A CTA's shared state besides the operand ring.
struct Fp8Shared {
    uint64_t full[16], empty[16], accf[8], acce[8], scale[12], drain[2], never;
    uint32_t tmem;
    int abort_flag;
    int first[kMaxExperts + 1];      // first work unit of each group; weight gradient: first contraction block
};

struct Unit {
    int group, row0, rows_end, col0, kblk0, nblk;    // rows_end: first row past the group
};

__device__ __forceinline__ int group_lo(const Fp8Params &p, int limit, int g) { return min(max(p.offsets[g], 0), limit); }

// Fills first[] from the group bounds; one warp, then a barrier.
// Bounds that leave [0, limit] are clamped and reported. Rows' bounds that go down
// are reported and leave no work, so that no row has two owners and the units
// are never more than the host has counted: the outputs become zeros. (Weight
// gradients have an output a group and blocks that are counted for any bounds.)
template <int KIND>
__device__ __forceinline__ void setup_groups(const Fp8Params &p, Fp8Shared &S, int tile_rows, int lane)
{
    if (!p.offsets) {
        if (lane == 0) {
            S.first[0] = 0;
            S.first[1] = KIND == kFp8Rows ? p.m_tiles * p.n_tiles : (p.kc + kBlock - 1) / kBlock;
        }
        return;
    }
    wait_for_last();
    const int limit = KIND == kFp8Rows ? p.rows : p.kc;
    int units = 0;
    bool bad = false, down = false;
    for (int g0 = 0; g0 < p.groups; g0 += 32) {
        const int g = g0 + lane;
        int u = 0;
        if (g < p.groups) {
            const int lo = group_lo(p, limit, g), hi = max(lo, group_lo(p, limit, g + 1));
            bad |= p.offsets[g] != lo || p.offsets[g + 1] != hi;
            if constexpr (KIND == kFp8Rows) down |= p.offsets[g + 1] < p.offsets[g];
            u = KIND == kFp8Rows ? (hi - lo + tile_rows - 1) / tile_rows * p.n_tiles : (hi - lo + kBlock - 1) / kBlock;
        }
        int us = u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(kFull, us, o);
            if (lane >= o) us += x;
        }
        if (g < p.groups) S.first[g] = units + us - u;
        units += __shfl_sync(kFull, us, 31);
    }
    if (lane == 0) S.first[p.groups] = units;
    if (KIND == kFp8Rows && __any_sync(kFull, down)) {
        __syncwarp();
        for (int g = lane; g <= p.groups; g += 32) S.first[g] = 0;
    }
    if (bad) atomicExch(p.status, kStatusInvalid);
}

// Work unit u: row tiles vary fastest, sixteen at a time, so that the CTAs
// of one moment share few panels of either operand (all in L2).
template <int KIND>
__device__ __forceinline__ Unit unit_of(const Fp8Params &p, const Fp8Shared &S, int u, int tile_rows, int tile_cols)
{
    constexpr int kSpan = 16;
    int g = 0;
    if (KIND == kFp8Wgrad) {
        g = u / (p.m_tiles * p.n_tiles);
        u -= g * (p.m_tiles * p.n_tiles);
    } else {
        if (p.offsets) {
            int a = 0, b = p.groups;
            while (b - a > 1) {
                const int mid = (a + b) >> 1;
                if (S.first[mid] <= u) a = mid;
                else b = mid;
            }
            g = a;
        }
        u -= S.first[g];
    }
    Unit r;
    r.group = g;
    int lo = 0, hi = p.rows, mt = p.m_tiles;
    if (KIND == kFp8Rows && p.offsets) {
        lo = group_lo(p, p.rows, g);
        hi = max(lo, group_lo(p, p.rows, g + 1));
        mt = (hi - lo + tile_rows - 1) / tile_rows;
    }
    const int span = kSpan * p.n_tiles;
    const int s = u / span;
    const int m0 = s * kSpan, mw = min(kSpan, mt - m0);
    const int w = u - s * span;
    const int n = w / mw;
    r.row0 = lo + (m0 + (w - n * mw)) * tile_rows;
    r.rows_end = hi;
    r.col0 = n * tile_cols;
    r.kblk0 = KIND == kFp8Rows ? 0 : S.first[g];
    // Never past the operands, whatever the bounds say.
    r.nblk = KIND == kFp8Rows ? p.max_blocks : max(0, min(S.first[g + 1], p.max_blocks) - r.kblk0);
    return r;
}

template <int KIND>
__device__ __forceinline__ int unit_count(const Fp8Params &p, const Fp8Shared &S)
{
    return KIND == kFp8Rows ? S.first[p.groups] : p.groups * p.m_tiles * p.n_tiles;
}

template <bool F32>
__device__ __forceinline__ void store_cols8(const Fp8Params &p, long long at, int c, const float (&f)[8])
{
    if constexpr (F32) store8f(static_cast<float *>(p.out) + at, c, p.cols, f);
    else store8(static_cast<uint16_t *>(p.out) + at, c, p.cols, pack8(f));
}

// Sixteen bytes of the output at element `at`, column c, clipped to the columns.
template <bool F32>
__device__ __forceinline__ void store_chunk(const Fp8Params &p, long long at, int c, const uint32_t (&v)[4])
{
    constexpr int N = F32 ? 4 : 8;
    if (c + N <= p.cols) {
        if constexpr (F32) *reinterpret_cast<uint4 *>(static_cast<float *>(p.out) + at) = make_uint4(v[0], v[1], v[2], v[3]);
        else *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + at) = make_uint4(v[0], v[1], v[2], v[3]);
        return;
    }
#pragma unroll
    for (int e = 0; e < N; ++e) {
        if (c + e >= p.cols) break;
        if constexpr (F32) static_cast<uint32_t *>(p.out)[at + e] = v[e];
        else static_cast<uint16_t *>(p.out)[at + e] = static_cast<uint16_t>(v[e / 2] >> (16 * (e & 1)));
    }
}

// 32 rows x 64 bytes of the output from one warp: lane l's row as 16 words.
// Through `buf` (16 rows at a time, 16-byte chunks swizzled by row), so that a
// store instruction writes 64 contiguous bytes of eight rows.
template <bool F32>
__device__ __forceinline__ void store_rows64(const Fp8Params &p, uint32_t buf, const uint32_t (&w)[16], int row0, int rows_end,
                                             long long base, int col, int lane)
{
    constexpr int EPW = F32 ? 1 : 2;                 // elements a word
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        __syncwarp();                                // the last use of buf is over
        if ((lane >> 4) == h) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(buf + (lane & 15) * 64 + ((k ^ (lane >> 1)) & 3) * 16),
                             "r"(w[4 * k]), "r"(w[4 * k + 1]), "r"(w[4 * k + 2]), "r"(w[4 * k + 3])
                             : "memory");
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 8 * i + (lane >> 2), k = lane & 3;
            uint32_t v[4];
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                         : "r"(buf + r * 64 + ((k ^ (r >> 1)) & 3) * 16)
                         : "memory");
            const int c = col + k * 4 * EPW, row = row0 + 16 * h + r;
            if (row < rows_end) store_chunk<F32>(p, base + row * p.ldo + c, c, v);
        }
    }
}

// The same for sums in the fragment layout (sum[16 g + 2 j + h]: row lane / 4
// + 16 g + 8 h, columns 8 j + 2 (lane % 4) + {0, 1}), 64 bytes of columns at a
// time: words are put where store_rows64 would have put them.
template <bool F32>
__device__ __forceinline__ void store_fragment(const Fp8Params &p, uint32_t buf, const uint64_t (&sum)[32], int row0, int rows_end,
                                               long long base, int col, int lane)
{
    constexpr int J = F32 ? 2 : 4;                   // groups of 8 columns in 64 bytes
    constexpr int EPW = F32 ? 1 : 2;
#pragma unroll
    for (int x = 0; x < 16 / J; ++x) {
        const int g = x & 1, j0 = (x >> 1) * J;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = (lane >> 2) + 8 * h;
                const uint64_t v = sum[16 * g + 2 * (j0 + j) + h];
                float lo, hi;
                unpair(v, lo, hi);
                const int word = F32 ? 8 * j + 2 * (lane & 3) : 4 * j + (lane & 3);
                const uint32_t at = buf + r * 64 + (((word >> 2) ^ (r >> 1)) & 3) * 16 + (word & 3) * 4;
                if constexpr (F32) asm volatile("st.shared.b64 [%0], %1;" ::"r"(at), "l"(v) : "memory");
                else asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(pack_bf16(lo, hi)) : "memory");
            }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 8 * i + (lane >> 2), k = lane & 3, row = row0 + 16 * g + r;
            const int c = col + 8 * j0 + k * 4 * EPW;
            uint32_t v[4];
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                         : "r"(buf + r * 64 + ((k ^ (r >> 1)) & 3) * 16)
                         : "memory");
            if (row < rows_end) store_chunk<F32>(p, base + row * p.ldo + c, c, v);
        }
    }
}

// Rows of the output that no group owns become zero (grouped launches): those in
// front of the first group and behind the last, or all.
template <bool F32>
__device__ __forceinline__ void zero_unowned(const Fp8Params &p, int units, int thread, int threads)
{
    if (!p.offsets) return;
    const int lo = group_lo(p, p.rows, 0), hi = units ? max(lo, group_lo(p, p.rows, p.groups)) : lo;
    const float z[8] = {};
    for (int i = blockIdx.x; i < lo + p.rows - hi; i += gridDim.x) {
        const long long r = i < lo ? i : hi + (i - lo);
        for (int c = thread * 8; c < p.cols; c += threads * 8) store_cols8<F32>(p, r * p.ldo, c, z);
    }
}

// ------------------------------------------------------------- plain tile

template <int KIND, int BN>
struct PlainCfg {
    static constexpr int BM = 128;
    static constexpr int COLS = 64;                  // columns of a thread
    static constexpr int EPI_WARPS = BN / COLS * 4;
    static constexpr int THREADS = 32 * (EPI_WARPS + 4);
    static constexpr int STAGES = BN == 128 ? 6 : 5;
    static constexpr int A_STAGE = BM * kBlock, B_STAGE = BN * kBlock;
    static constexpr int NACC = BN == 192 ? 2 : 4;
    static constexpr int OFF_B = STAGES * A_STAGE;
    // Scales. A weight's product reads a row's and a weight tile's into
    // registers, kAhead blocks before they are used (an L2 read takes about as
    // long as two blocks). The weight gradient's come with the operands'
    // copies, the tile's rows' and then its columns', into a ring of slots of
    // their own: a block's copies begin when the MMAs STAGES blocks before it
    // are done, so when the epilogue has let go of the block STAGES + NACC
    // before it, and so has read the scales of the one before that.
    static constexpr int kAhead = 2, SLOTS = STAGES + NACC + 1, SLOT = (BM + BN) * 4;
    static constexpr int OFF_SCALE = OFF_B + STAGES * B_STAGE;
    // A finished tile goes out through shared memory, 64 bytes of OUT_ROWS rows
    // a time and warp: written straight from the registers, every store
    // touches 32 lines and a 192-wide tile takes 3000 cycles to leave. (32
    // rows a time leave no room for a fifth stage: 356 instead of 315 ns a block.)
    static constexpr int OUT_ROWS = 16;
    static constexpr int OUT = OUT_ROWS * 64;
    static constexpr int OFF_OUT = OFF_SCALE + (KIND == kFp8Wgrad ? SLOTS * SLOT : 0);
    static constexpr int OFF_SHARED = OFF_OUT + EPI_WARPS * OUT;
    static constexpr int BYTES = OFF_SHARED + static_cast<int>(sizeof(Fp8Shared));
    static constexpr int SMEM = BYTES + 1024;
    // Registers: a thread's sums, its TMEM words and addresses take about
    // 160. 384 threads have that (168); 512 are launched with 128 and the
    // service warps hand theirs over.
    static constexpr bool SPLIT = THREADS > 384;
    static constexpr int LAUNCH_REGS = (65536 / THREADS) & ~7;
    static constexpr int SERVICE_REGS = 24, EPI_REGS = 160;
    static_assert(!SPLIT || SERVICE_REGS * 128 + EPI_REGS * 32 * EPI_WARPS <= LAUNCH_REGS * THREADS, "register split");
    static_assert(SMEM <= 232448, "shared memory");
    static_assert(NACC * BN <= 512, "TMEM");
    static_assert(NACC % 2 == 0 && (STAGES % 2 == 0 || NACC <= STAGES), "every issuer sees each barrier phase it waits for begin");
};

template <int KIND, bool F32, int BN>
__device__ __forceinline__ void plain_epilogue(const Fp8Params &p, Fp8Shared &S, uint32_t base, int warp, int lane)
{
    using C = PlainCfg<KIND, BN>;
    const int q = warp & 3, part = warp >> 2;
    const uint32_t t0 = S.tmem + (static_cast<uint32_t>(q * 32) << 16) + part * C::COLS;
    const uint32_t out = base + C::OFF_OUT + warp * C::OUT;
    const int units = unit_count<KIND>(p, S);
    wait_for_last();
    const uint32_t abort_s = smem_u32(&S.abort_flag);
    int acc = 0;
    uint32_t phase = 0;
    bool ok = true;
    // The current tile and where its scales are.
    Unit w{};
    const float *sa = p.sa, *sb = p.sb;
    // A weight's product: the row's scale and the weight tile's (one for all
    // the thread's columns), of the next kAhead blocks.
    float ra[C::kAhead], rb[C::kAhead];
    bool live = false, in0 = false;
    // Weight gradient: the slot of the next block's scales, and where in one
    // the thread's rows' and (as far on) its columns' begin.
    int slot = 0;
    uint32_t slot_phase = 0;
    const uint32_t scales = base + C::OFF_SCALE + q * 128 + (lane >> 2) * 4;
    const uint32_t to_cols = C::BM * 4 - q * 128 - (lane >> 2) * 4 + part * (C::COLS * 4) + (lane & 3) * 8;
    auto load = [&](int b, int j) {
        const bool more = b < w.nblk;
        ra[j] = more && live ? *sa : 0.0f;
        rb[j] = more && in0 ? *sb : 0.0f;
        sa += p.sa_blk;
        sb += p.sb_blk;
    };
    auto begin = [&](int u) {
        if (u >= units) return;
        w = unit_of<KIND>(p, S, u, C::BM, BN);
        if constexpr (KIND == kFp8Rows) {
            const int row0 = w.row0 + q * 32, col = w.col0 + part * C::COLS;
            live = row0 + lane < w.rows_end;
            in0 = col < p.cols;
            sa = p.sa + (live ? (row0 + lane) * p.sa_row : 0);
            sb = p.sb + (in0 ? w.group * p.sb_grp + static_cast<long long>(col / kBlock) * p.sb_row : 0);
#pragma unroll
            for (int j = 0; j < C::kAhead; ++j) load(j, j);
        }
    };
    begin(static_cast<int>(blockIdx.x));
    for (int u = static_cast<int>(blockIdx.x); u < units; u += static_cast<int>(gridDim.x)) {
        uint64_t sum[C::COLS / 2];
#pragma unroll
        for (int i = 0; i < C::COLS / 2; ++i) sum[i] = 0;
        // Waits for the next block's accumulator; hands it back when its words are in registers.
        auto arrived = [&]() {
            ok &= mbar_wait_inline(smem_u32(&S.accf[acc]), phase, abort_s, p.status, p.timeout_ns) != 0;
            tc_fence_after();
        };
        auto release = [&]() {
            tc_fence_before();
            __syncwarp();
            mbar_arrive_if(smem_u32(&S.acce[acc]), lane == 0);
            if (++acc == C::NACC) {
                acc = 0;
                phase ^= 1u;
            }
        };
        auto block = [&](int b, int j) {
            if constexpr (KIND == kFp8Rows) {
                const float rs = ra[j] * rb[j];
                const uint64_t r2 = pair(rs, rs);
                load(b + C::kAhead, j);
                arrived();
                uint32_t v0[32], v1[32];
                tmem_ld32(t0 + acc * BN, v0);
                tmem_ld32(t0 + acc * BN + 32, v1);
                tmem_wait_ld();
                reg_fence(v0);
                reg_fence(v1);
                release();
#pragma unroll
                for (int i = 0; i < 16; ++i) sum[i] = fma2(pair(v0[2 * i], v0[2 * i + 1]), r2, sum[i]);
#pragma unroll
                for (int i = 0; i < 16; ++i) sum[16 + i] = fma2(pair(v1[2 * i], v1[2 * i + 1]), r2, sum[16 + i]);
            } else {
                // sum[16 g + 2 i + h]: row lane / 4 + 16 g + 8 h, columns 8 i + 2 (lane % 4) + {0, 1}.
                // The accumulator goes back before the scales are looked at.
                arrived();
                uint32_t v[2][32];
                tmem_ld_16x64(t0 + acc * BN, v[0]);
                tmem_ld_16x64(t0 + acc * BN + (16u << 16), v[1]);
                tmem_wait_ld();
                reg_fence(v[0]);
                reg_fence(v[1]);
                release();
                ok &= mbar_wait_inline(smem_u32(&S.scale[slot]), slot_phase, abort_s, p.status, p.timeout_ns) != 0;
                const uint32_t at = scales + slot * C::SLOT;
                if (++slot == C::SLOTS) {
                    slot = 0;
                    slot_phase ^= 1u;
                }
                uint64_t rs[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float r = lds1(at + i * 32);
                    rs[i] = pair(r, r);
                }
#pragma unroll
                for (int i0 = 0; i0 < 8; i0 += 4) {
                    uint64_t cs[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) cs[i] = lds2(at + to_cols + (i0 + i) * 32);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const int e = 2 * (i0 + i) + (x & 1);    // of row group x / 2
                            sum[16 * (x >> 1) + e] =
                                fma2(pair(v[x >> 1][2 * e], v[x >> 1][2 * e + 1]), mul2(rs[x], cs[i]), sum[16 * (x >> 1) + e]);
                        }
                }
            }
        };
        if constexpr (KIND == kFp8Rows) {
            // Whole rounds of the scales' registers, then the rest: with a test after
            // every block the compiler moves the sums about at each (333 instead of
            // 315 ns a block).
            int b = 0;
#pragma unroll 1
            for (; b + C::kAhead <= w.nblk; b += C::kAhead) {
#pragma unroll
                for (int j = 0; j < C::kAhead; ++j) block(b + j, j);
            }
#pragma unroll
            for (int j = 0; j < C::kAhead - 1; ++j) {
                if (b + j >= w.nblk) break;
                block(b + j, j);
            }
        } else {
#pragma unroll 2
            for (int b = 0; b < w.nblk; ++b) block(b, 0);
        }
        if (!ok) return;             // a wait of this tile failed: the launch is aborting
        // The next tile's first scales are under way while this one is stored.
        const Unit done = w;
        begin(u + static_cast<int>(gridDim.x));
        const int row0 = done.row0 + q * 32, col = done.col0 + part * C::COLS;
        if constexpr (KIND == kFp8Rows) {
            constexpr int N = F32 ? 16 : 32;         // columns of 64 bytes
#pragma unroll
            for (int i = 0; i < C::COLS; i += N) {
                uint32_t o[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    float lo, hi;
                    if constexpr (F32) {
                        unpair(sum[(i + e) / 2], lo, hi);
                        o[e] = __float_as_uint((e & 1) ? hi : lo);
                    } else {
                        unpair(sum[i / 2 + e], lo, hi);
                        o[e] = pack_bf16(lo, hi);
                    }
                }
                if (col + i < p.cols) store_rows64<F32>(p, out, o, row0, done.rows_end, 0, col + i, lane);
            }
        } else {
            store_fragment<F32>(p, out, sum, row0, done.rows_end, done.group * p.og, col, lane);
        }
    }
    if constexpr (KIND == kFp8Rows) zero_unowned<F32>(p, units, warp * 32 + lane, C::EPI_WARPS * 32);
}

// One thread: the whole loop of TMA copies.
template <int KIND, int BN>
__device__ __forceinline__ void plain_copy(const Fp8Params &p, Fp8Shared &S, uint32_t base)
{
    using C = PlainCfg<KIND, BN>;
    const int units = unit_count<KIND>(p, S);
    volatile int *abort_flag = &S.abort_flag;
    const uint32_t tx = static_cast<uint32_t>(p.a_box + p.b_box) * kBlock;
    int s = 0;
    uint32_t round = 0, loaded = 0, parity = 0;
    int slot = 0;                        // of the weight gradient's scales
    uint32_t slot_round = 0, slot_loaded = 0, slot_parity = 0;
    wait_for_last();
    bool ok = !p.force_timeout || wait_bounded(smem_u32(&S.never), 0, abort_flag, p.status, p.timeout_ns, true);
    for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
        const Unit w = unit_of<KIND>(p, S, u, C::BM, BN);
        for (int b = 0; b < w.nblk; ++b) {
            if (!wait_bounded(smem_u32(&S.empty[s]), round ^ 1u, abort_flag, p.status, p.timeout_ns, true)) {
                ok = false;
                break;
            }
            const uint32_t full = smem_u32(&S.full[s]);
            mbar_arrive_expect_tx(full, tx);
            const int k = (w.kblk0 + b) * kBlock;
            if constexpr (KIND == kFp8Wgrad) {
                const uint32_t bar = smem_u32(&S.scale[slot]), at = base + C::OFF_SCALE + slot * C::SLOT;
                mbar_arrive_expect_tx(bar, static_cast<uint32_t>(p.sa_box + p.sb_box) * 4);
                tma_load_2d(at, &p.tmap_sa, bar, w.row0, w.kblk0 + b);
                tma_load_2d(at + C::BM * 4, &p.tmap_sb, bar, w.col0, w.kblk0 + b);
                slot_loaded |= 1u << slot;
                slot_parity = (slot_parity & ~(1u << slot)) | (slot_round << slot);
                if (++slot == C::SLOTS) {
                    slot = 0;
                    slot_round ^= 1u;
                }
            }
            tma_load_2d(base + s * C::A_STAGE, &p.tmap_a, full, k, w.row0);
            tma_load_3d(base + C::OFF_B + s * C::B_STAGE, &p.tmap_b, full, k, w.col0, KIND == kFp8Rows ? w.group : 0);
            loaded |= 1u << s;
            parity = (parity & ~(1u << s)) | (round << s);
            if (++s == C::STAGES) {
                s = 0;
                round ^= 1u;
            }
        }
    }
    if (!ok) {
        for (int i = 0; i < C::STAGES; ++i)
            if (loaded & (1u << i))
                wait_bounded(smem_u32(&S.full[i]), (parity >> i) & 1u, abort_flag, p.status, p.timeout_ns, false);
        for (int i = 0; KIND == kFp8Wgrad && i < C::SLOTS; ++i)
            if (slot_loaded & (1u << i))
                wait_bounded(smem_u32(&S.scale[i]), (slot_parity >> i) & 1u, abort_flag, p.status, p.timeout_ns, false);
    }
}

// One thread of each of the two issuing warps: issuer i takes the blocks g
// of the CTA's sequence with g % 2 == i.
template <int KIND, int BN>
__device__ __forceinline__ void plain_issue(const Fp8Params &p, Fp8Shared &S, uint32_t base, int issuer)
{
    using C = PlainCfg<KIND, BN>;
    constexpr uint32_t IDESC = idesc_e4m3(C::BM, BN);
    const int units = unit_count<KIND>(p, S);
    volatile int *abort_flag = &S.abort_flag;
    const uint32_t tmem = S.tmem;
    int s = issuer, acc = issuer;        // of this issuer's next block
    uint32_t round = 0, phase = 0;
    int b = issuer;                      // its position in the current tile
    bool ok = true, issued = false;
    wait_for_last();                     // the bounded waits' time begins after it
    for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
        const int nblk = KIND == kFp8Rows || !p.offsets ? p.max_blocks : unit_of<KIND>(p, S, u, C::BM, BN).nblk;
        for (; b < nblk; b += 2) {
            // The accumulator first: with an odd number of stages the block before
            // in this stage was the other issuer's, and a wait for a phase that a
            // barrier has not begun passes at once. The accumulator is free when
            // the epilogue has taken the block NACC before, so when that older
            // block's MMAs are done and its phase is over.
            if (!wait_bounded(smem_u32(&S.acce[acc]), phase ^ 1u, abort_flag, p.status, p.timeout_ns, true) ||
                !wait_bounded(smem_u32(&S.full[s]), round, abort_flag, p.status, p.timeout_ns, true)) {
                ok = false;
                break;
            }
            tc_fence_after();
            mma_block(tmem + acc * BN, base + s * C::A_STAGE, base + C::OFF_B + s * C::B_STAGE, IDESC);
            mma_commit(smem_u32(&S.accf[acc]));
            mma_commit(smem_u32(&S.empty[s]));
            issued = true;
            s += 2;
            if (s >= C::STAGES) {
                s -= C::STAGES;
                round ^= 1u;
            }
            acc += 2;
            if (acc >= C::NACC) {
                acc -= C::NACC;
                phase ^= 1u;
            }
        }
        b -= nblk;
    }
    if (!ok && issued) {
        mma_commit(smem_u32(&S.drain[issuer]));
        wait_bounded(smem_u32(&S.drain[issuer]), 0, abort_flag, p.status, p.timeout_ns, false);
    }
}

template <int KIND, bool F32, int BN>
__global__ void __launch_bounds__(PlainCfg<KIND, BN>::THREADS, 1) fp8_plain_kernel(const __grid_constant__ Fp8Params p)
{
    using C = PlainCfg<KIND, BN>;
    // Barriers, TMEM and, without group bounds, the tiles are set up before the wait for the launch in front.
    extern __shared__ uint8_t fp8_smem[];
    const uint32_t raw = smem_u32(fp8_smem);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *smem = fp8_smem + (base - raw);
    Fp8Shared &S = *reinterpret_cast<Fp8Shared *>(smem + C::OFF_SHARED);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        S.abort_flag = 0;
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(smem_u32(&S.full[s]), 1);
            mbar_init(smem_u32(&S.empty[s]), 1);
        }
        for (int a = 0; a < C::NACC; ++a) {
            mbar_init(smem_u32(&S.accf[a]), 1);
            mbar_init(smem_u32(&S.acce[a]), C::EPI_WARPS);
        }
        for (int i = 0; KIND == kFp8Wgrad && i < C::SLOTS; ++i) mbar_init(smem_u32(&S.scale[i]), 1);
        mbar_init(smem_u32(&S.drain[0]), 1);
        mbar_init(smem_u32(&S.drain[1]), 1);
        mbar_init(smem_u32(&S.never), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) setup_groups<KIND>(p, S, C::BM, lane);
    if (warp == C::EPI_WARPS && lane == 0) {
        tmap_prefetch(&p.tmap_a);
        tmap_prefetch(&p.tmap_b);
    }
    if (warp == C::EPI_WARPS + 3) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&S.tmem)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp < C::EPI_WARPS) {
        if constexpr (C::SPLIT) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::EPI_REGS));
        plain_epilogue<KIND, F32, BN>(p, S, base, warp, lane);
    } else {
        if constexpr (C::SPLIT) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::SERVICE_REGS));
        if (warp == C::EPI_WARPS && elect_one()) plain_copy<KIND, BN>(p, S, base);
        else if ((warp == C::EPI_WARPS + 1 || warp == C::EPI_WARPS + 2) && elect_one())
            plain_issue<KIND, BN>(p, S, base, warp - C::EPI_WARPS - 1);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == C::EPI_WARPS + 3)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(S.tmem), "r"(512) : "memory");
}

// -------------------------------------------------------- transposed tile

template <int NT>
struct SwapCfg {
    static constexpr int THREADS = 256;
    static constexpr int PER_STAGE = 2;              // blocks of a ring stage
    static constexpr int PER_SLOT = 4;               // blocks of an accumulator slot: two stages
    static constexpr int SLOTS = NT == 16 ? 4 : 2;
    static constexpr int TMEM_COLS = SLOTS * PER_SLOT * NT;
    static constexpr int MAX_STAGES = 16;
    // 64 columns of sums leave registers for one CTA an SM only.
    static constexpr int CTAS = NT == 64 ? 1 : 2;
    static constexpr int RING = (CTAS == 1 ? 192 : 96) * 1024;       // bytes of the operand ring
    static constexpr int OFF_SCALE = RING;           // [SLOTS][PER_SLOT][NT] floats
    static constexpr int OFF_SHARED = OFF_SCALE + SLOTS * PER_SLOT * NT * 4;
    static constexpr int BYTES = OFF_SHARED + static_cast<int>(sizeof(Fp8Shared));
    static constexpr int SMEM = BYTES + 1024;
    static_assert(CTAS * SMEM <= 232448, "the CTAs of an SM share its memory");
    static_assert(TMEM_COLS * CTAS <= 512, "the CTAs of an SM share its TMEM");
    __host__ __device__ static int stages(int tile_rows)
    {
        // The ring's weight part comes first and a 128-row MMA reads 16 KB
        // from its block's start: that stays inside the ring.
        // An even number, so that a stage is always the same issuer's: a wait
        // for a phase that a barrier has not begun would pass at once.
        const int n = (RING - (128 - tile_rows) * kBlock) / (PER_STAGE * (tile_rows + NT) * kBlock) & ~1;
        return n < MAX_STAGES ? n : MAX_STAGES;
    }
};

template <bool F32, int NT>
__device__ __forceinline__ void swap_epilogue(const Fp8Params &p, Fp8Shared &S, const float *scale_smem, int tile_rows,
                                              int warp, int lane)
{
    using C = SwapCfg<NT>;
    const uint32_t t0 = S.tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const int units = S.first[p.groups];
    wait_for_last();
    const uint32_t abort_s = smem_u32(&S.abort_flag);
    int slot = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
        const Unit w = unit_of<kFp8Rows>(p, S, u, NT, tile_rows);
        uint64_t sum[NT / 2];
#pragma unroll
        for (int i = 0; i < NT / 2; ++i) sum[i] = 0;
        for (int b = 0; b < w.nblk; b += C::PER_SLOT) {
            ok &= mbar_wait_inline(smem_u32(&S.accf[slot]), phase, abort_s, p.status, p.timeout_ns) != 0;
            tc_fence_after();
            const uint32_t t = t0 + slot * C::PER_SLOT * NT;
            const float *sc = scale_smem + slot * C::PER_SLOT * NT;
            if constexpr (NT == 16) {
                // All four blocks at once (a block past the contraction's end
                // has words of an earlier turn and is left out).
                uint32_t v[4][16];
#pragma unroll
                for (int j = 0; j < 4; ++j) tmem_ld16(t + j * NT, v[j]);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 4; ++j) reg_fence16(v[j]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (b + j >= w.nblk) break;
                    const ulonglong2 *c = reinterpret_cast<const ulonglong2 *>(sc + j * NT);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const ulonglong2 s = c[i];
                        sum[2 * i] = fma2(pair(v[j][4 * i], v[j][4 * i + 1]), s.x, sum[2 * i]);
                        sum[2 * i + 1] = fma2(pair(v[j][4 * i + 2], v[j][4 * i + 3]), s.y, sum[2 * i + 1]);
                    }
                }
            } else {
#pragma unroll 1
                for (int j = 0; j < C::PER_SLOT; ++j) {
                    if (b + j >= w.nblk) break;
#pragma unroll
                    for (int h = 0; h < NT / 32; ++h) {
                        uint32_t v[32];
                        tmem_ld32(t + j * NT + 32 * h, v);
                        tmem_wait_ld();
                        reg_fence(v);
                        const uint32_t c = smem_u32(sc + j * NT + 32 * h);
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            add4(sum[16 * h + i / 2], sum[16 * h + i / 2 + 1], pair(v[i], v[i + 1]), pair(v[i + 2], v[i + 3]), c + 4 * i);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            mbar_arrive_if(smem_u32(&S.acce[slot]), lane == 0);
            if (++slot == C::SLOTS) {
                slot = 0;
                phase ^= 1u;
            }
        }
        if (!ok) return;             // a wait of this tile failed: the launch is aborting
        const int n = w.col0 + warp * 32 + lane;     // this lane's output column (a weight row)
        if (n < p.cols && warp * 32 < tile_rows) {
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const long long r = w.row0 + i;
                float lo, hi;
                unpair(sum[i / 2], lo, hi);
                const float v = (i & 1) ? hi : lo;
                if (r < w.rows_end) {
                    if constexpr (F32) static_cast<float *>(p.out)[r * p.ldo + n] = v;
                    else static_cast<__nv_bfloat16 *>(p.out)[r * p.ldo + n] = __float2bfloat16_rn(v);
                }
            }
        }
    }
    zero_unowned<F32>(p, units, warp * 32 + lane, 128);
}

// One warp: the products of the scales, token by token, of a slot's blocks.
// The loads of the next slot are under way while one is handed out.
template <int NT>
__device__ __forceinline__ void swap_scales(const Fp8Params &p, Fp8Shared &S, float *scale_smem, int tile_rows, int lane)
{
    using C = SwapCfg<NT>;
    constexpr int SL = NT < 32 ? 1 : NT / 32;        // tokens of a lane
    const int units = S.first[p.groups];
    wait_for_last();
    const uint32_t abort_s = smem_u32(&S.abort_flag);
    int slot = 0;
    uint32_t phase = 0;
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
        const Unit w = unit_of<kFp8Rows>(p, S, u, NT, tile_rows);
        const float *sw = p.sb + w.group * p.sb_grp + static_cast<long long>(w.col0 / kBlock) * p.sb_row;
        float t[C::PER_SLOT][SL], wv[C::PER_SLOT];
        auto load = [&](int b0) {
#pragma unroll
            for (int j = 0; j < C::PER_SLOT; ++j) {
                const bool in = b0 + j < w.nblk;
                wv[j] = in ? sw[(b0 + j) * p.sb_blk] : 0.0f;
#pragma unroll
                for (int i = 0; i < SL; ++i) {
                    const int r = w.row0 + 32 * i + lane;
                    t[j][i] = (in && 32 * i + lane < NT && r < w.rows_end) ? p.sa[r * p.sa_row + (b0 + j) * p.sa_blk] : 0.0f;
                }
            }
        };
        load(0);
        for (int b0 = 0; b0 < w.nblk; b0 += C::PER_SLOT) {
            float c[C::PER_SLOT][SL];
#pragma unroll
            for (int j = 0; j < C::PER_SLOT; ++j)
#pragma unroll
                for (int i = 0; i < SL; ++i) c[j][i] = t[j][i] * wv[j];
            load(b0 + C::PER_SLOT);
            if (!__all_sync(kFull, mbar_wait_inline(smem_u32(&S.acce[slot]), phase ^ 1u, abort_s, p.status, p.timeout_ns) != 0))
                return;
#pragma unroll
            for (int j = 0; j < C::PER_SLOT; ++j)
#pragma unroll
                for (int i = 0; i < SL; ++i)
                    if (32 * i + lane < NT) scale_smem[(slot * C::PER_SLOT + j) * NT + 32 * i + lane] = c[j][i];
            __syncwarp();
            mbar_arrive_if(smem_u32(&S.accf[slot]), lane == 0);
            if (++slot == C::SLOTS) {
                slot = 0;
                phase ^= 1u;
            }
        }
    }
}

// One thread: the copies. tmap_b is the weight (b_box rows), tmap_a the
// tokens (a_box rows).
template <int NT>
__device__ __forceinline__ void swap_copy(const Fp8Params &p, Fp8Shared &S, uint32_t base, int tile_rows)
{
    using C = SwapCfg<NT>;
    const int stages = C::stages(tile_rows);
    const uint32_t w_blk = static_cast<uint32_t>(tile_rows) * kBlock;
    const uint32_t base_t = base + stages * C::PER_STAGE * w_blk;
    const uint32_t tx = static_cast<uint32_t>(p.a_box + p.b_box) * kBlock;
    const int units = S.first[p.groups];
    volatile int *abort_flag = &S.abort_flag;
    int s = 0;
    uint32_t round = 0, loaded = 0, parity = 0;
    wait_for_last();
    bool ok = !p.force_timeout || wait_bounded(smem_u32(&S.never), 0, abort_flag, p.status, p.timeout_ns, true);
    for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
        const Unit w = unit_of<kFp8Rows>(p, S, u, NT, tile_rows);
        for (int b = 0; b < w.nblk; b += C::PER_STAGE) {
            if (!wait_bounded(smem_u32(&S.empty[s]), round ^ 1u, abort_flag, p.status, p.timeout_ns, true)) {
                ok = false;
                break;
            }
            const uint32_t full = smem_u32(&S.full[s]);
            const int n = min(C::PER_STAGE, w.nblk - b);
            mbar_arrive_expect_tx(full, tx * n);
            for (int j = 0; j < n; ++j) {
                const int at = s * C::PER_STAGE + j;
                tma_load_3d(base + at * w_blk, &p.tmap_b, full, (b + j) * kBlock, w.col0, w.group);
                tma_load_2d(base_t + at * NT * kBlock, &p.tmap_a, full, (b + j) * kBlock, w.row0);
            }
            loaded |= 1u << s;
            parity = (parity & ~(1u << s)) | (round << s);
            if (++s == stages) {
                s = 0;
                round ^= 1u;
            }
        }
    }
    let_next_begin();                    // the last copies are under way
    if (!ok) {
        for (int i = 0; i < stages; ++i)
            if (loaded & (1u << i))
                wait_bounded(smem_u32(&S.full[i]), (parity >> i) & 1u, abort_flag, p.status, p.timeout_ns, false);
    }
}

// One thread of each of the two issuing warps: issuer i takes the stages s
// with s % 2 == i, so about half of every slot's blocks.
template <int NT>
__device__ __forceinline__ void swap_issue(const Fp8Params &p, Fp8Shared &S, uint32_t base, int tile_rows, int issuer)
{
    using C = SwapCfg<NT>;
    constexpr uint32_t IDESC = idesc_e4m3(128, NT);
    const int stages = C::stages(tile_rows);
    const uint32_t w_blk = static_cast<uint32_t>(tile_rows) * kBlock;
    const uint32_t base_t = base + stages * C::PER_STAGE * w_blk;
    const int units = S.first[p.groups];
    volatile int *abort_flag = &S.abort_flag;
    const uint32_t tmem = S.tmem;
    int s = 0, slot = 0;                 // all stages are counted, its own are issued
    uint32_t round = 0, phase = 0;
    bool ok = true, issued = false;
    wait_for_last();                     // the bounded waits' time begins after it
    for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
        const int nblk = p.max_blocks;
        for (int b = 0; b < nblk; b += C::PER_SLOT) {
            if (!wait_bounded(smem_u32(&S.acce[slot]), phase ^ 1u, abort_flag, p.status, p.timeout_ns, true)) {
                ok = false;
                break;
            }
            for (int h = 0; h < C::PER_SLOT && b + h < nblk; h += C::PER_STAGE) {
                if ((s & 1) == issuer) {
                    if (!wait_bounded(smem_u32(&S.full[s]), round, abort_flag, p.status, p.timeout_ns, true)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
#pragma unroll
                    for (int j = 0; j < C::PER_STAGE; ++j) {
                        if (b + h + j >= nblk) break;
                        const int at = s * C::PER_STAGE + j;
                        mma_block(tmem + (slot * C::PER_SLOT + h + j) * NT, base + at * w_blk, base_t + at * NT * kBlock, IDESC);
                    }
                    mma_commit(smem_u32(&S.empty[s]));
                    issued = true;
                }
                if (++s == stages) {
                    s = 0;
                    round ^= 1u;
                }
            }
            if (!ok) break;
            mma_commit(smem_u32(&S.accf[slot]));
            if (++slot == C::SLOTS) {
                slot = 0;
                phase ^= 1u;
            }
        }
    }
    if (!ok && issued) {
        mma_commit(smem_u32(&S.drain[issuer]));
        wait_bounded(smem_u32(&S.drain[issuer]), 0, abort_flag, p.status, p.timeout_ns, false);
    }
}

template <bool F32, int NT>
__global__ void __launch_bounds__(256, SwapCfg<NT>::CTAS) fp8_swap_kernel(const __grid_constant__ Fp8Params p, const int tile_rows)
{
    using C = SwapCfg<NT>;
    // Barriers, TMEM and, without group bounds, the tiles are set up before the wait for the launch in front.
    extern __shared__ uint8_t fp8_smem[];
    const uint32_t raw = smem_u32(fp8_smem);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *smem = fp8_smem + (base - raw);
    Fp8Shared &S = *reinterpret_cast<Fp8Shared *>(smem + C::OFF_SHARED);
    float *scale_smem = reinterpret_cast<float *>(smem + C::OFF_SCALE);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        S.abort_flag = 0;
        for (int s = 0; s < C::MAX_STAGES; ++s) {
            mbar_init(smem_u32(&S.full[s]), 1);
            mbar_init(smem_u32(&S.empty[s]), 1);
        }
        for (int a = 0; a < C::SLOTS; ++a) {
            mbar_init(smem_u32(&S.accf[a]), 3);      // both issuers' commits and the scales
            mbar_init(smem_u32(&S.acce[a]), 4);
        }
        mbar_init(smem_u32(&S.drain[0]), 1);
        mbar_init(smem_u32(&S.drain[1]), 1);
        mbar_init(smem_u32(&S.never), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) setup_groups<kFp8Rows>(p, S, NT, lane);
    if (warp == 4 && lane == 0) {
        tmap_prefetch(&p.tmap_a);
        tmap_prefetch(&p.tmap_b);
    }
    if (warp == 7) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&S.tmem)),
                     "r"(C::TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp < 4) swap_epilogue<F32, NT>(p, S, scale_smem, tile_rows, warp, lane);
    else if (warp == 4 && elect_one()) swap_copy<NT>(p, S, base, tile_rows);
    else if ((warp == 5 || warp == 6) && elect_one()) swap_issue<NT>(p, S, base, tile_rows, warp - 5);
    else if (warp == 7) swap_scales<NT>(p, S, scale_smem, tile_rows, lane);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 7)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(S.tmem), "r"(C::TMEM_COLS) : "memory");
}

template <int KIND, bool F32, int BN>
cudaError_t run_plain(const Fp8Params &p, int sms, cudaStream_t s)
{
    using C = PlainCfg<KIND, BN>;
    auto fn = fp8_plain_kernel<KIND, F32, BN>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = once_per_device(done, [&] {
        cudaFuncAttributes at;
        cudaError_t x = cudaFuncGetAttributes(&at, fn);
        if (x != cudaSuccess) return x;
        // setmaxnreg shares out exactly the registers of the launch.
        if (C::SPLIT && at.numRegs != C::LAUNCH_REGS) return cudaErrorInvalidDeviceFunction;
        return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    });
    if (e != cudaSuccess) return e;
    return launch_early(fn, sms, C::THREADS, C::SMEM, 1, s, p);
}

template <bool F32, int NT>
cudaError_t run_swap(const Fp8Params &p, int tile_rows, int sms, cudaStream_t s)
{
    using C = SwapCfg<NT>;
    auto fn = fp8_swap_kernel<F32, NT>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = once_per_device(
        done, [&] { return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM); });
    if (e != cudaSuccess) return e;
    return launch_early(fn, C::CTAS * sms, C::THREADS, C::SMEM, 1, s, p, tile_rows);
}

}  // namespace deto
