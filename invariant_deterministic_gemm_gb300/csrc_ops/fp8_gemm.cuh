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
// leaves TMEM and is added in registers. For a 128 x 256 tile the four MMAs
// take 512 cycles at the dense e4m3 rate, the TMEM reads 256 and the
// multiply-adds 256 on other pipes, so the tensor core stays the bound as
// long as the reads overlap the next block's MMAs: two accumulators of 256
// columns fill TMEM and alternate.
//
// Plain tile (384 threads, one CTA per SM, persistent over tiles):
//   warps 0-7  epilogue: TMEM lane quadrant w % 4 (32 rows), column half w / 4;
//              a thread keeps BN / 2 sums of one row in registers
//   warp 8     copies A and B blocks in with TMA (ring of 4 stages)
//   warp 9     issues the MMAs
//   warp 10    allocates and frees TMEM
// A block of a stage is 128 bytes of contraction for 128 rows of A and BN of
// B, in 128-byte swizzle. Why 256 columns: a 128 x 128 tile reads 32 KB from
// L2 for 256 MMA cycles, 128 B a cycle and SM; 128 x 256 reads 96.
//
// Transposed tile (few rows: decode): the weight is the MMA's row side, its
// 32, 64 or 128 rows are TMEM lanes, and the tokens its 16 to 64 columns.
// The launch is bound by reading the weight once; a CTA keeps up to 96 KB of
// copies in flight and two CTAs share an SM. A tile of 32 or 64 weight rows
// still issues 128-row MMAs: the other lanes multiply whatever the following
// shared memory holds and are never read.
//
// Weight gradient: both operands are scaled per row of theirs, so the
// columns' scales go through shared memory and each element takes one more
// multiplication.
//
// Waits are bounded as in det_gemm's kernels (a timeout sets the status
// word, every role leaves, copies and MMAs in flight are drained).
#pragma once

#include "det_gemm_kernel.cuh"
#include "ops_internal.h"
#include "vec.cuh"

#include <atomic>

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
using detg::warp_wait;

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

// A CTA's shared state besides the operand ring.
struct Fp8Shared {
    uint64_t full[16], empty[16], accf[4], acce[4], drain, never;
    uint32_t tmem;
    int abort_flag;
    int first[kMaxExperts + 1];      // first work unit of each group
    int blk0[kMaxExperts + 1];       // weight gradient: first contraction block of each group
};

struct Unit {
    int group, row0, rows_end, col0, kblk0, nblk;    // rows_end: first row past the group
};

__device__ __forceinline__ int group_lo(const Fp8Params &p, int limit, int g) { return min(max(p.offsets[g], 0), limit); }

// Fills first[] (and blk0[]) from the group bounds; one warp, then a barrier.
// Bounds that decrease or leave [0, limit] are clamped and reported.
template <int KIND>
__device__ __forceinline__ void setup_groups(const Fp8Params &p, Fp8Shared &S, int tile_rows, int lane)
{
    if (!p.offsets) {
        if (lane == 0) {
            S.first[0] = 0;
            S.first[1] = p.m_tiles * p.n_tiles;
            S.blk0[0] = 0;
            S.blk0[1] = (p.kc + kBlock - 1) / kBlock;
        }
        return;
    }
    const int limit = KIND == kFp8Rows ? p.rows : p.kc;
    int units = 0, blocks = 0;
    bool bad = false;
    for (int g0 = 0; g0 < p.groups; g0 += 32) {
        const int g = g0 + lane;
        int u = 0, b = 0;
        if (g < p.groups) {
            const int lo = group_lo(p, limit, g), hi = max(lo, group_lo(p, limit, g + 1));
            bad |= p.offsets[g] != lo || p.offsets[g + 1] != hi;
            b = (hi - lo + kBlock - 1) / kBlock;
            u = KIND == kFp8Rows ? (hi - lo + tile_rows - 1) / tile_rows * p.n_tiles : p.m_tiles * p.n_tiles;
        }
        int us = u, bs = b;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(kFull, us, o), y = __shfl_up_sync(kFull, bs, o);
            if (lane >= o) {
                us += x;
                bs += y;
            }
        }
        if (g < p.groups) {
            S.first[g] = units + us - u;
            S.blk0[g] = blocks + bs - b;
        }
        units += __shfl_sync(kFull, us, 31);
        blocks += __shfl_sync(kFull, bs, 31);
    }
    if (lane == 0) {
        S.first[p.groups] = units;
        S.blk0[p.groups] = blocks;
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
    if (p.offsets) {
        int a = 0, b = p.groups;
        while (b - a > 1) {
            const int mid = (a + b) >> 1;
            if (S.first[mid] <= u) a = mid;
            else b = mid;
        }
        g = a;
    }
    Unit r;
    r.group = g;
    u -= S.first[g];
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
    r.kblk0 = KIND == kFp8Rows ? 0 : S.blk0[g];
    // Never past the operands, whatever the bounds say (bounds that go down can claim rows twice).
    r.nblk = KIND == kFp8Rows ? p.max_blocks : max(0, min(S.blk0[g + 1], p.max_blocks) - r.kblk0);
    return r;
}

template <bool F32>
__device__ __forceinline__ void store_cols8(const Fp8Params &p, long long at, int c, const float (&f)[8])
{
    if constexpr (F32) store8f(static_cast<float *>(p.out) + at, c, p.cols, f);
    else store8(static_cast<uint16_t *>(p.out) + at, c, p.cols, pack8(f));
}

// Rows of the output that no group owns become zero (grouped launches).
template <bool F32>
__device__ __forceinline__ void zero_unowned(const Fp8Params &p, int thread, int threads)
{
    if (!p.offsets) return;
    const int lo = group_lo(p, p.rows, 0), hi = max(lo, group_lo(p, p.rows, p.groups));
    const float z[8] = {};
    for (int i = blockIdx.x; i < lo + p.rows - hi; i += gridDim.x) {
        const long long r = i < lo ? i : hi + (i - lo);
        for (int c = thread * 8; c < p.cols; c += threads * 8) store_cols8<F32>(p, r * p.ldo, c, z);
    }
}

// ------------------------------------------------------------- plain tile

template <int BN>
struct PlainCfg {
    static constexpr int BM = 128;
    static constexpr int EPI_WARPS = 8;
    static constexpr int THREADS = 384;
    static constexpr int STAGES = BN == 256 ? 4 : 6;
    static constexpr int A_STAGE = BM * kBlock, B_STAGE = BN * kBlock;
    static constexpr int NACC = BN == 256 ? 2 : 4;
    static constexpr int COLS = BN / 2;              // columns of a thread
    static constexpr int OFF_B = STAGES * A_STAGE;
    static constexpr int OFF_SCALE = OFF_B + STAGES * B_STAGE;       // [EPI_WARPS][2][COLS] floats
    static constexpr int OFF_SHARED = OFF_SCALE + EPI_WARPS * 2 * COLS * 4;
    static constexpr int BYTES = OFF_SHARED + static_cast<int>(sizeof(Fp8Shared));
    static constexpr int SMEM = BYTES + 1024;
    // 65536 registers: 168 a thread at launch; the four service warps keep 40, the epilogue warps take 232.
    static constexpr int LAUNCH_REGS = 168;
    static constexpr int SERVICE_REGS = 40, EPI_REGS = 232;
    static_assert(SERVICE_REGS * 128 + EPI_REGS * 256 <= LAUNCH_REGS * THREADS, "register split");
    static_assert(SMEM <= 232448, "shared memory");
    static_assert(NACC * BN <= 512, "TMEM");
};

template <int KIND, bool F32, int BN>
__device__ __forceinline__ void plain_epilogue(const Fp8Params &p, Fp8Shared &S, float *scale_smem, int warp, int lane)
{
    using C = PlainCfg<BN>;
    const int q = warp & 3, half = warp >> 2;
    const uint32_t t0 = S.tmem + (static_cast<uint32_t>(q * 32) << 16) + half * C::COLS;
    float *sc = scale_smem + warp * 2 * C::COLS;
    const int units = S.first[p.groups];
    int acc = 0;
    uint32_t phase = 0;
    int flip = 0;
    volatile int *abort_flag = &S.abort_flag;
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
        const Unit w = unit_of<KIND>(p, S, u, C::BM, BN);
        const int row = w.row0 + q * 32 + lane;
        const int col = w.col0 + half * C::COLS;
        const bool live = row < w.rows_end;
        const float *sa = p.sa + row * p.sa_row + w.kblk0 * p.sa_blk;
        // The thread's column scales: one for all its columns (a weight's
        // tile), or its lane's share of the warp's columns.
        const float *sb;
        constexpr int SB = KIND == kFp8Rows ? 1 : C::COLS / 32;
        float sbv[SB], sav = 0.0f;
        bool cl[SB];
        if constexpr (KIND == kFp8Rows) {
            sb = p.sb + w.group * p.sb_grp + static_cast<long long>(col / kBlock) * p.sb_row;
            cl[0] = col < p.cols;
        } else {
            sb = p.sb + w.kblk0 * p.sb_blk + static_cast<long long>(col + lane) * p.sb_row;
#pragma unroll
            for (int i = 0; i < SB; ++i) cl[i] = col + lane + 32 * i < p.cols;
        }
        auto load_scales = [&](int b) {
            sav = live ? __ldg(sa + b * p.sa_blk) : 0.0f;
#pragma unroll
            for (int i = 0; i < SB; ++i) sbv[i] = cl[i] ? __ldg(sb + b * p.sb_blk + 32 * i * p.sb_row) : 0.0f;
        };
        float sum[C::COLS];
#pragma unroll
        for (int i = 0; i < C::COLS; ++i) sum[i] = 0.0f;
        if (w.nblk > 0) load_scales(0);
        for (int b = 0; b < w.nblk; ++b) {
            float rs = sav;
            const float4 *cs = reinterpret_cast<const float4 *>(sc + flip * C::COLS);
            if constexpr (KIND == kFp8Rows) {
                rs = sav * sbv[0];
            } else {
#pragma unroll
                for (int i = 0; i < SB; ++i) sc[flip * C::COLS + lane + 32 * i] = sbv[i];
                __syncwarp();
                flip ^= 1;
            }
            if (b + 1 < w.nblk) load_scales(b + 1);
            if (!warp_wait(smem_u32(&S.accf[acc]), phase, abort_flag, p.status, p.timeout_ns)) return;
            tc_fence_after();
            const uint32_t t = t0 + acc * BN;
            uint32_t v[2][32];
            tmem_ld32(t, v[0]);
#pragma unroll
            for (int h = 0; h < C::COLS / 32; ++h) {
                tmem_wait_ld();
                reg_fence(v[h & 1]);
                if (h + 1 < C::COLS / 32) {
                    tmem_ld32(t + 32 * (h + 1), v[(h + 1) & 1]);
                } else {
                    tc_fence_before();
                    __syncwarp();
                    mbar_arrive_if(smem_u32(&S.acce[acc]), lane == 0);
                }
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    float s[4] = {rs, rs, rs, rs};
                    if constexpr (KIND == kFp8Wgrad) {
                        const float4 c4 = cs[(32 * h + i) / 4];
                        s[0] = rs * c4.x;
                        s[1] = rs * c4.y;
                        s[2] = rs * c4.z;
                        s[3] = rs * c4.w;
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sum[32 * h + i + e] = fmaf(__uint_as_float(v[h & 1][i + e]), s[e], sum[32 * h + i + e]);
                }
            }
            if (++acc == C::NACC) {
                acc = 0;
                phase ^= 1u;
            }
        }
        if (live) {
            const long long at = row * p.ldo + (KIND == kFp8Wgrad ? w.group * p.og : 0);
#pragma unroll
            for (int i = 0; i < C::COLS; i += 8) {
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = sum[i + e];
                if (col + i < p.cols) store_cols8<F32>(p, at, col + i, f);
            }
        }
    }
    if constexpr (KIND == kFp8Rows) zero_unowned<F32>(p, warp * 32 + lane, C::EPI_WARPS * 32);
}

template <int KIND, int BN>
__device__ __forceinline__ void plain_copy(const Fp8Params &p, Fp8Shared &S, uint32_t base)
{
    using C = PlainCfg<BN>;
    const bool leader = elect_one();
    const int units = S.first[p.groups];
    volatile int *abort_flag = &S.abort_flag;
    const uint32_t tx = static_cast<uint32_t>(p.a_box + p.b_box) * kBlock;
    int s = 0;
    uint32_t round = 0, loaded = 0, parity = 0;
    bool ok = true;
    if (p.force_timeout)
        ok = __all_sync(kFull, wait_bounded(smem_u32(&S.never), 0, abort_flag, p.status, p.timeout_ns, true));
    for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
        const Unit w = unit_of<KIND>(p, S, u, C::BM, BN);
        for (int b = 0; b < w.nblk; ++b) {
            if (!warp_wait(smem_u32(&S.empty[s]), round ^ 1u, abort_flag, p.status, p.timeout_ns)) {
                ok = false;
                break;
            }
            if (leader) {
                const uint32_t full = smem_u32(&S.full[s]);
                mbar_arrive_expect_tx(full, tx);
                const int k = (w.kblk0 + b) * kBlock;
                tma_load_2d(base + s * C::A_STAGE, &p.tmap_a, full, k, w.row0);
                tma_load_3d(base + C::OFF_B + s * C::B_STAGE, &p.tmap_b, full, k, w.col0, KIND == kFp8Rows ? w.group : 0);
            }
            __syncwarp();
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
    }
}

template <int KIND, int BN>
__device__ __forceinline__ void plain_issue(const Fp8Params &p, Fp8Shared &S, uint32_t base)
{
    using C = PlainCfg<BN>;
    constexpr uint32_t IDESC = idesc_e4m3(C::BM, BN);
    const bool leader = elect_one();
    const int units = S.first[p.groups];
    volatile int *abort_flag = &S.abort_flag;
    int s = 0, acc = 0;
    uint32_t round = 0, phase = 0;
    bool ok = true, issued = false;
    for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
        const int nblk = unit_of<KIND>(p, S, u, C::BM, BN).nblk;
        for (int b = 0; b < nblk; ++b) {
            if (!warp_wait(smem_u32(&S.acce[acc]), phase ^ 1u, abort_flag, p.status, p.timeout_ns) ||
                !warp_wait(smem_u32(&S.full[s]), round, abort_flag, p.status, p.timeout_ns)) {
                ok = false;
                break;
            }
            tc_fence_after();
            if (leader) {
                mma_block(S.tmem + acc * BN, base + s * C::A_STAGE, base + C::OFF_B + s * C::B_STAGE, IDESC);
                mma_commit(smem_u32(&S.empty[s]));
                mma_commit(smem_u32(&S.accf[acc]));
            }
            __syncwarp();
            issued = true;
            if (++s == C::STAGES) {
                s = 0;
                round ^= 1u;
            }
            if (++acc == C::NACC) {
                acc = 0;
                phase ^= 1u;
            }
        }
    }
    if (!ok && issued) {
        if (leader) mma_commit(smem_u32(&S.drain));
        __syncwarp();
        wait_bounded(smem_u32(&S.drain), 0, abort_flag, p.status, p.timeout_ns, false);
    }
}

template <int KIND, bool F32, int BN>
__global__ void __launch_bounds__(384, 1) fp8_plain_kernel(const __grid_constant__ Fp8Params p)
{
    using C = PlainCfg<BN>;
    extern __shared__ uint8_t fp8_smem[];
    const uint32_t raw = smem_u32(fp8_smem);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *smem = fp8_smem + (base - raw);
    Fp8Shared &S = *reinterpret_cast<Fp8Shared *>(smem + C::OFF_SHARED);
    float *scale_smem = reinterpret_cast<float *>(smem + C::OFF_SCALE);
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
        mbar_init(smem_u32(&S.drain), 1);
        mbar_init(smem_u32(&S.never), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) setup_groups<KIND>(p, S, C::BM, lane);
    if (warp == 8 && lane == 0) {
        tmap_prefetch(&p.tmap_a);
        tmap_prefetch(&p.tmap_b);
    }
    if (warp == 10) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&S.tmem)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp < C::EPI_WARPS) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::EPI_REGS));
        plain_epilogue<KIND, F32, BN>(p, S, scale_smem, warp, lane);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::SERVICE_REGS));
        if (warp == 8) plain_copy<KIND, BN>(p, S, base);
        else if (warp == 9) plain_issue<KIND, BN>(p, S, base);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 10)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(S.tmem), "r"(512) : "memory");
}

// -------------------------------------------------------- transposed tile

template <int NT>
struct SwapCfg {
    static constexpr int THREADS = 256;
    static constexpr int NACC = 4;
    static constexpr int TMEM_COLS = NACC * NT < 32 ? 32 : NACC * NT;
    static constexpr int B_STAGE = NT * kBlock;
    static constexpr int MAX_STAGES = 16;
    static constexpr int RING = 96 * 1024;           // bytes of the operand ring
    static constexpr int OFF_SCALE = RING;           // [4 warps][2][NT] floats
    static constexpr int OFF_SHARED = OFF_SCALE + 4 * 2 * NT * 4;
    static constexpr int BYTES = OFF_SHARED + static_cast<int>(sizeof(Fp8Shared));
    static constexpr int SMEM = BYTES + 1024;
    static_assert(2 * SMEM <= 232448, "two CTAs share an SM");
    static_assert(TMEM_COLS * 2 <= 512, "two CTAs share an SM's TMEM");
    __host__ __device__ static int stages(int tile_rows)
    {
        // The ring's weight part comes first and a 128-row MMA reads up to
        // 16 KB from its slot's start: that stays inside the allocation.
        const int n = (RING - (128 - tile_rows) * kBlock) / (tile_rows * kBlock + B_STAGE);
        return n < MAX_STAGES ? n : MAX_STAGES;
    }
};

template <bool F32, int NT>
__device__ __forceinline__ void swap_epilogue(const Fp8Params &p, Fp8Shared &S, float *scale_smem, int tile_rows, int warp,
                                              int lane)
{
    using C = SwapCfg<NT>;
    constexpr int SL = NT < 32 ? 1 : NT / 32;        // token scales of a lane
    const uint32_t t0 = S.tmem + (static_cast<uint32_t>(warp * 32) << 16);
    float *sc = scale_smem + warp * 2 * NT;
    const int units = S.first[p.groups];
    volatile int *abort_flag = &S.abort_flag;
    int acc = 0;
    uint32_t phase = 0;
    int flip = 0;
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
        const Unit w = unit_of<kFp8Rows>(p, S, u, NT, tile_rows);
        const int n = w.col0 + warp * 32 + lane;     // this lane's output column (a weight row)
        const float *sw = p.sb + w.group * p.sb_grp + static_cast<long long>(w.col0 / kBlock) * p.sb_row;
        float tv[SL], wv = 0.0f;
        auto load_scales = [&](int b) {
            wv = __ldg(sw + b * p.sb_blk);
#pragma unroll
            for (int i = 0; i < SL; ++i) {
                const int r = w.row0 + 32 * i + lane;
                tv[i] = (32 * i + lane < NT && r < w.rows_end) ? __ldg(p.sa + r * p.sa_row + b * p.sa_blk) : 0.0f;
            }
        };
        float sum[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) sum[i] = 0.0f;
        if (w.nblk > 0) load_scales(0);
        for (int b = 0; b < w.nblk; ++b) {
            float *cs = sc + flip * NT;
#pragma unroll
            for (int i = 0; i < SL; ++i)
                if (32 * i + lane < NT) cs[32 * i + lane] = tv[i] * wv;
            __syncwarp();
            flip ^= 1;
            if (b + 1 < w.nblk) load_scales(b + 1);
            if (!warp_wait(smem_u32(&S.accf[acc]), phase, abort_flag, p.status, p.timeout_ns)) return;
            tc_fence_after();
            const uint32_t t = t0 + acc * NT;
            if constexpr (NT == 16) {
                uint32_t v[16];
                tmem_ld16(t, v);
                tmem_wait_ld();
                reg_fence16(v);
                tc_fence_before();
                __syncwarp();
                mbar_arrive_if(smem_u32(&S.acce[acc]), lane == 0);
#pragma unroll
                for (int i = 0; i < 16; ++i) sum[i] = fmaf(__uint_as_float(v[i]), cs[i], sum[i]);
            } else {
#pragma unroll
                for (int h = 0; h < NT / 32; ++h) {
                    uint32_t v[32];
                    tmem_ld32(t + 32 * h, v);
                    tmem_wait_ld();
                    reg_fence(v);
                    if (h + 1 == NT / 32) {
                        tc_fence_before();
                        __syncwarp();
                        mbar_arrive_if(smem_u32(&S.acce[acc]), lane == 0);
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i) sum[32 * h + i] = fmaf(__uint_as_float(v[i]), cs[32 * h + i], sum[32 * h + i]);
                }
            }
            if (++acc == C::NACC) {
                acc = 0;
                phase ^= 1u;
            }
        }
        if (n < p.cols && warp * 32 < tile_rows) {
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const long long r = w.row0 + i;
                if (r < w.rows_end) {
                    if constexpr (F32) static_cast<float *>(p.out)[r * p.ldo + n] = sum[i];
                    else static_cast<__nv_bfloat16 *>(p.out)[r * p.ldo + n] = __float2bfloat16_rn(sum[i]);
                }
            }
        }
    }
    zero_unowned<F32>(p, warp * 32 + lane, 128);
}

template <bool F32, int NT>
__global__ void __launch_bounds__(256, 2) fp8_swap_kernel(const __grid_constant__ Fp8Params p, const int tile_rows)
{
    using C = SwapCfg<NT>;
    extern __shared__ uint8_t fp8_smem[];
    const uint32_t raw = smem_u32(fp8_smem);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *smem = fp8_smem + (base - raw);
    Fp8Shared &S = *reinterpret_cast<Fp8Shared *>(smem + C::OFF_SHARED);
    float *scale_smem = reinterpret_cast<float *>(smem + C::OFF_SCALE);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int stages = C::stages(tile_rows);
    const uint32_t w_stage = static_cast<uint32_t>(tile_rows) * kBlock;
    const uint32_t base_t = base + stages * w_stage;         // token slots
    if (threadIdx.x == 0) {
        S.abort_flag = 0;
        for (int s = 0; s < stages; ++s) {
            mbar_init(smem_u32(&S.full[s]), 1);
            mbar_init(smem_u32(&S.empty[s]), 1);
        }
        for (int a = 0; a < C::NACC; ++a) {
            mbar_init(smem_u32(&S.accf[a]), 1);
            mbar_init(smem_u32(&S.acce[a]), 4);
        }
        mbar_init(smem_u32(&S.drain), 1);
        mbar_init(smem_u32(&S.never), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) setup_groups<kFp8Rows>(p, S, NT, lane);
    if (warp == 4 && lane == 0) {
        tmap_prefetch(&p.tmap_a);
        tmap_prefetch(&p.tmap_b);
    }
    if (warp == 6) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&S.tmem)),
                     "r"(C::TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const int units = S.first[p.groups];
    volatile int *abort_flag = &S.abort_flag;
    if (warp < 4) {
        swap_epilogue<F32, NT>(p, S, scale_smem, tile_rows, warp, lane);
    } else if (warp == 4) {
        const bool leader = elect_one();
        // tmap_b is the weight (b_box rows of it), tmap_a the tokens (a_box)
        const uint32_t tx = static_cast<uint32_t>(p.a_box + p.b_box) * kBlock;
        int s = 0;
        uint32_t round = 0, loaded = 0, parity = 0;
        bool ok = true;
        if (p.force_timeout)
            ok = __all_sync(kFull, wait_bounded(smem_u32(&S.never), 0, abort_flag, p.status, p.timeout_ns, true));
        for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
            const Unit w = unit_of<kFp8Rows>(p, S, u, NT, tile_rows);
            for (int b = 0; b < w.nblk; ++b) {
                if (!warp_wait(smem_u32(&S.empty[s]), round ^ 1u, abort_flag, p.status, p.timeout_ns)) {
                    ok = false;
                    break;
                }
                if (leader) {
                    const uint32_t full = smem_u32(&S.full[s]);
                    mbar_arrive_expect_tx(full, tx);
                    tma_load_3d(base + s * w_stage, &p.tmap_b, full, b * kBlock, w.col0, w.group);
                    tma_load_2d(base_t + s * C::B_STAGE, &p.tmap_a, full, b * kBlock, w.row0);
                }
                __syncwarp();
                loaded |= 1u << s;
                parity = (parity & ~(1u << s)) | (round << s);
                if (++s == stages) {
                    s = 0;
                    round ^= 1u;
                }
            }
        }
        if (!ok) {
            for (int i = 0; i < stages; ++i)
                if (loaded & (1u << i))
                    wait_bounded(smem_u32(&S.full[i]), (parity >> i) & 1u, abort_flag, p.status, p.timeout_ns, false);
        }
    } else if (warp == 5) {
        const bool leader = elect_one();
        constexpr uint32_t IDESC = idesc_e4m3(128, NT);
        int s = 0, acc = 0;
        uint32_t round = 0, phase = 0;
        bool ok = true, issued = false;
        for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
            const int nblk = unit_of<kFp8Rows>(p, S, u, NT, tile_rows).nblk;
            for (int b = 0; b < nblk; ++b) {
                if (!warp_wait(smem_u32(&S.acce[acc]), phase ^ 1u, abort_flag, p.status, p.timeout_ns) ||
                    !warp_wait(smem_u32(&S.full[s]), round, abort_flag, p.status, p.timeout_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (leader) {
                    mma_block(S.tmem + acc * NT, base + s * w_stage, base_t + s * C::B_STAGE, IDESC);
                    mma_commit(smem_u32(&S.empty[s]));
                    mma_commit(smem_u32(&S.accf[acc]));
                }
                __syncwarp();
                issued = true;
                if (++s == stages) {
                    s = 0;
                    round ^= 1u;
                }
                if (++acc == C::NACC) {
                    acc = 0;
                    phase ^= 1u;
                }
            }
        }
        if (!ok && issued) {
            if (leader) mma_commit(smem_u32(&S.drain));
            __syncwarp();
            wait_bounded(smem_u32(&S.drain), 0, abort_flag, p.status, p.timeout_ns, false);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 6)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(S.tmem), "r"(C::TMEM_COLS) : "memory");
}

// Runs `set_up` once per device for one kernel instance (its state in `done`).
template <typename F>
cudaError_t once_per_device(std::atomic<uint64_t> &done, F set_up)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = set_up();
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

template <int KIND, bool F32, int BN>
cudaError_t run_plain(const Fp8Params &p, int sms, cudaStream_t s)
{
    using C = PlainCfg<BN>;
    auto fn = fp8_plain_kernel<KIND, F32, BN>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = once_per_device(done, [&] {
        cudaFuncAttributes at;
        cudaError_t x = cudaFuncGetAttributes(&at, fn);
        if (x != cudaSuccess) return x;
        // setmaxnreg shares out exactly the registers of the launch.
        if (at.numRegs != C::LAUNCH_REGS) return cudaErrorInvalidDeviceFunction;
        return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    });
    if (e != cudaSuccess) return e;
    fn<<<sms, C::THREADS, C::SMEM, s>>>(p);
    return cudaGetLastError();
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
    fn<<<2 * sms, C::THREADS, C::SMEM, s>>>(p, tile_rows);
    return cudaGetLastError();
}

}  // namespace deto
