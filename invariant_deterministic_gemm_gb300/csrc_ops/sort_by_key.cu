// Stable sort of small integer keys by one thread-block cluster: tokens by
// expert (dispatch), tokens by vocabulary row (embedding gradient).
//
// A stable sort's result is unique, so no order of execution can show in
// it. Each pass is a counting sort by one digit. CTA c of the cluster owns
// the c-th contiguous part of the items and each of its warps the w-th
// contiguous part of that, so "items before mine" is: smaller digits
// anywhere, the same digit in earlier CTAs, in earlier warps of the CTA,
// earlier in the warp's part.
//   1. every warp counts its digits into its own shared-memory row (the
//      lanes with one digit find each other with match.any; one of them
//      adds their number, so no atomics);
//   2. the CTA turns the 32 rows into exclusive sums over its warps;
//   3. the CTAs read each other's totals through distributed shared memory
//      and form the digits' first positions;
//   4. every warp walks its items again and writes each to its place.
// Expert ids take one pass with the id as the digit; vocabulary rows take
// 9-bit digits (two passes up to 262143 rows).
//
// What bounds it is latency: a pass is two walks over the items and two
// cluster barriers, and the whole sort is one launch: 34 items 3.2 us, 49152
// expert ids 15.7 us (both out of a graph). Beyond that its eight SMs bound it:
// 524288 ids 150 us. A warp loads its keys
// eight steps (256 items) at a time, and keeps them for the second walk when
// that is all of them (up to 65536 items over the cluster): loading them step
// by step, 8192 tokens took 33 us. Parts are sized for up to 8 CTAs (the
// portable cluster size) of 1024 threads; small inputs take one CTA and no
// cluster barrier crosses SMs.
//
// The first rows of the gradient's dense output are zeroed by the launch's
// other clusters meanwhile.
#include "launch.cuh"
#include "ops_internal.h"

#include <cooperative_groups.h>

#include <algorithm>

namespace cg = cooperative_groups;

namespace deto {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kDigitBits = 9;
constexpr int kMaxBins = 1 << 10;
static_assert((1 << kDigitBits) <= kMaxExperts + 1, "the larger histogram is the experts'");
constexpr int kBatch = 8;            // steps of 32 items whose keys are loaded at once
constexpr unsigned kAll = 0xFFFFFFFFu;

struct Smem {
    uint32_t base[kMaxBins];         // first position of each digit's items of this CTA
    uint32_t total[kMaxBins];        // this CTA's items of each digit (read by the other CTAs)
    uint32_t warp_sum[kWarps];
    int edge;                        // last run head of this CTA's part, or -1 (read by the other CTAs)
};

__device__ __forceinline__ int key_at(const SortParams &p, int i)
{
    long long k;
    if (p.keys64) k = static_cast<const long long *>(p.keys)[i];
    else k = static_cast<const int *>(p.keys)[i];
    if (k < 0 || k >= p.range) {
        if (p.flag_bad) atomicExch(p.status, kStatusInvalid);
        return p.range;
    }
    return k == p.skip_key ? p.range : static_cast<int>(k);
}

// Inclusive sum over the block's threads of one value each.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t *warp_sum, int warp, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(kAll, v, o);
        if (lane >= o) v += u;
    }
    if (lane == 31) warp_sum[warp] = v;
    __syncthreads();
    if (warp == 0) {
        uint32_t s = warp_sum[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(kAll, s, o);
            if (lane >= o) s += u;
        }
        warp_sum[lane] = s;
    }
    __syncthreads();
    if (warp > 0) v += warp_sum[warp - 1];
    return v;
}

// Rows [0, rows) of the output become zero: a warp's lanes write 16 bytes each.
__device__ __forceinline__ void zero_rows(const SortParams &p, int block, int blocks)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long bytes = p.zero_cols;             // of a row
    for (long long r = static_cast<long long>(block) * kWarps + warp; r < p.zero_rows; r += static_cast<long long>(blocks) * kWarps) {
        uint8_t *row = static_cast<uint8_t *>(p.zero) + r * p.zero_pitch;
        for (long long c = lane * 16; c < bytes; c += 512) {
            if (c + 16 <= bytes) *reinterpret_cast<uint4 *>(row + c) = make_uint4(0, 0, 0, 0);
            else
                for (long long i = c; i < bytes; i += 2) *reinterpret_cast<uint16_t *>(row + i) = 0;
        }
    }
}

template <bool RUNS>
__global__ void __launch_bounds__(kThreads) sort_kernel(const SortParams p)
{
    begin();
    extern __shared__ uint32_t hist[];               // [kWarps][bins]
    __shared__ Smem sm;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    if constexpr (RUNS) {
        if (static_cast<int>(blockIdx.x) >= C) {
            zero_rows(p, blockIdx.x - C, gridDim.x - C);
            return;
        }
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int bins = RUNS ? (1 << kDigitBits) : p.range + 1;
    // This warp's items, a contiguous part in whole 32s.
    const long long per = (static_cast<long long>(p.n) + C * kWarps * 32 - 1) / (C * kWarps * 32) * 32;
    const int lo = static_cast<int>(min(static_cast<long long>(p.n), (static_cast<long long>(rank) * kWarps + warp) * per));
    const int hi = static_cast<int>(min(static_cast<long long>(p.n), lo + per));
    const bool single = per <= kBatch * 32;          // one batch is all of them
    uint32_t *mine = hist + warp * bins;

    if constexpr (RUNS) {
        // (`seen` has room for a whole 16 bytes at its end)
        for (int i = (rank * kThreads + threadIdx.x) * 16; i < p.range; i += C * kThreads * 16)
            *reinterpret_cast<uint4 *>(p.seen + i) = make_uint4(0, 0, 0, 0);
    }
    int key[kBatch], idx[kBatch];
    for (int pass = 0; pass < p.passes; ++pass) {
        const int shift = pass * kDigitBits;
        const int32_t *ksrc = pass == 0 ? nullptr : p.kbuf[(pass - 1) & 1];
        const int32_t *isrc = pass == 0 ? nullptr : p.ibuf[(pass - 1) & 1];
        auto load = [&](int i0) {
#pragma unroll
            for (int s = 0; s < kBatch; ++s) {
                const int i = i0 + s * 32 + lane;
                key[s] = 0;
                idx[s] = i;
                if (i < hi) {
                    if (RUNS && pass > 0) {
                        key[s] = __ldcg(ksrc + i);
                        idx[s] = __ldcg(isrc + i);
                    } else {
                        key[s] = key_at(p, i);
                    }
                }
            }
        };
        auto digit = [&](int k) { return RUNS ? (k >> shift) & ((1 << kDigitBits) - 1) : k; };
        if (single) load(lo);
        for (int b = threadIdx.x; b < kWarps * bins; b += kThreads) hist[b] = 0;
        __syncthreads();
        for (int i0 = lo; i0 < hi; i0 += kBatch * 32) {
            if (!single) load(i0);
#pragma unroll
            for (int s = 0; s < kBatch; ++s) {
                if (i0 + s * 32 >= hi) break;
                const bool in = i0 + s * 32 + lane < hi;
                const int d = in ? digit(key[s]) : -1;
                const unsigned same = __match_any_sync(kAll, d);
                if (in && lane == __ffs(static_cast<int>(same)) - 1) mine[d] += __popc(same);
                __syncwarp();
            }
        }
        __syncthreads();
        for (int b = threadIdx.x; b < bins; b += kThreads) {
            uint32_t run = 0;
#pragma unroll 8
            for (int w = 0; w < kWarps; ++w) {
                const uint32_t c = hist[w * bins + b];
                hist[w * bins + b] = run;
                run += c;
            }
            sm.total[b] = run;
        }
        cluster.sync();
        uint32_t all = 0, before = 0;
        if (static_cast<int>(threadIdx.x) < bins) {
            for (int c = 0; c < C; ++c) {
                const uint32_t v = cluster.map_shared_rank(&sm.total[0], c)[threadIdx.x];
                all += v;
                if (c < rank) before += v;
            }
        }
        const uint32_t first = block_scan(all, sm.warp_sum, warp, lane) - all;
        if (static_cast<int>(threadIdx.x) < bins) {
            sm.base[threadIdx.x] = first + before;
            if (!RUNS && rank == 0) p.offsets[threadIdx.x] = static_cast<int32_t>(first);
        }
        __syncthreads();
        for (int i0 = lo; i0 < hi; i0 += kBatch * 32) {
            if (!single) load(i0);
#pragma unroll
            for (int s = 0; s < kBatch; ++s) {
                if (i0 + s * 32 >= hi) break;
                const bool in = i0 + s * 32 + lane < hi;
                const int k = key[s], i = idx[s];
                const int d = in ? digit(k) : -1;
                const unsigned same = __match_any_sync(kAll, d);
                if (in) {
                    const uint32_t pos = sm.base[d] + mine[d] + __popc(same & ((1u << lane) - 1u));
                    if constexpr (RUNS) {
                        p.kbuf[pass & 1][pos] = k;
                        p.ibuf[pass & 1][pos] = i;
                    } else {
                        p.rows[pos] = k < p.range ? i : -1;
                        p.slots[i] = k < p.range ? static_cast<int32_t>(pos) : -1;
                    }
                }
                __syncwarp();
                if (in && lane == __ffs(static_cast<int>(same)) - 1) mine[d] += __popc(same);
                __syncwarp();
            }
        }
        // The totals may be overwritten, and the other CTAs' writes read, only after this.
        cluster.sync();
    }

    if constexpr (RUNS) {
        // Each sorted position's run head (the first position with its key).
        const int32_t *sorted = p.kbuf[(p.passes - 1) & 1];
        auto load = [&](int i0) {                    // key: a position's key, idx: the one before it
#pragma unroll
            for (int s = 0; s < kBatch; ++s) {
                const int i = i0 + s * 32 + lane;
                key[s] = i < hi ? __ldcg(sorted + i) : 0;
                idx[s] = i < hi && i > 0 ? __ldcg(sorted + i - 1) : -1;
            }
        };
        if (single) load(lo);
        int last = -1;                               // last head of this warp's part
        for (int i0 = lo; i0 < hi; i0 += kBatch * 32) {
            if (!single) load(i0);
#pragma unroll
            for (int s = 0; s < kBatch; ++s) {
                const int i = i0 + s * 32 + lane;
                const bool head = i < hi && key[s] != idx[s];
                if (head && key[s] < p.range) p.seen[key[s]] = 1;
                const unsigned heads = __ballot_sync(kAll, head);
                if (heads) last = i0 + s * 32 + 31 - __clz(static_cast<int>(heads));
            }
        }
        if (lane == 0) sm.warp_sum[warp] = static_cast<uint32_t>(last);
        __syncthreads();
        if (threadIdx.x == 0) {
            int e = -1;
            for (int w = 0; w < kWarps; ++w) e = max(e, static_cast<int>(sm.warp_sum[w]));
            sm.edge = e;
        }
        cluster.sync();
        int carry = -1;
        for (int c = 0; c < rank; ++c) carry = max(carry, *cluster.map_shared_rank(&sm.edge, c));
        for (int w = 0; w < warp; ++w) carry = max(carry, static_cast<int>(sm.warp_sum[w]));
        for (int i0 = lo; i0 < hi; i0 += kBatch * 32) {
            if (!single) load(i0);
#pragma unroll
            for (int s = 0; s < kBatch; ++s) {
                const int i = i0 + s * 32 + lane;
                const unsigned heads = __ballot_sync(kAll, i < hi && key[s] != idx[s]);
                const unsigned upto = heads & (0xFFFFFFFFu >> (31 - lane));
                if (i < hi) p.head[i] = upto ? i0 + s * 32 + 31 - __clz(static_cast<int>(upto)) : carry;
                if (heads) carry = i0 + s * 32 + 31 - __clz(static_cast<int>(heads));
            }
        }
        cluster.sync();              // no CTA may exit while another reads its shared memory
    }
}

}  // namespace

cudaError_t launch_sort(const SortParams &p, bool runs, cudaStream_t s)
{
    const int bins = runs ? (1 << kDigitBits) : p.range + 1;
    const size_t smem = sizeof(uint32_t) * kWarps * bins;
    // CTAs: about two 32-item steps for each warp, at most 8.
    int C = 1;
    while (C < 8 && static_cast<long long>(C) * kThreads * 2 < p.n) C *= 2;
    auto fn = runs ? sort_kernel<true> : sort_kernel<false>;
    static std::atomic<uint64_t> done[2];
    const cudaError_t e = once_per_device(done[runs], [&] {
        return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(sizeof(uint32_t)) * kWarps * (kMaxExperts + 1));
    });
    if (e != cudaSuccess) return e;
    // Zeroing: whole clusters beside the sorting one, about two CTAs an SM.
    const int zero = runs && p.zero_rows > 0 ? static_cast<int>((std::min<long long>(2 * p.sms, (p.zero_rows + kWarps - 1) / kWarps) + C - 1) / C * C) : 0;
    return launch_early(fn, C + zero, kThreads, smem, C, s, p);
}

}  // namespace deto
