// Token rows to their experts' contiguous rows and back, with gradients.
//   gather:   xs[r] = x[rows[r] / k]                      (zero where rows[r] < 0)
//   combine:  y[t] = sum over j of w[t, j] * ys[slots[t, j]], FP32, ascending j
//   backward: dys[r] = w[t, j] * dy[t], dw[t, j] = dy[t] . ys[slots[t, j]]
// Every output row has one owner that reads its terms in a fixed order, so
// there are no atomics and a token's bits do not depend on the batch.
//
// Bytes bound all three: each row is read and written once, 16 bytes a
// thread, several rows' loads in flight per thread. 8192 tokens of six experts
// each, rows of 4096: gather 90 us (5.2 TB/s), combine 78 us (6.0), backward
// 135 us (6.4); a copy of this card reaches 6.8. The gather's rows leave by
// streaming stores, so that the six uses of a token's row find it in L2 (98 us
// without).
#include "launch.cuh"
#include "ops_internal.h"
#include "vec.cuh"

namespace deto {
namespace {

constexpr int kThreads = 128;        // 1024 columns of a row
constexpr int kCols = kThreads * 8;
constexpr int kRows = 4;             // gathered rows of a block: loads in flight per thread
constexpr unsigned kAll = 0xFFFFFFFFu;

__global__ void __launch_bounds__(kThreads) gather_kernel(const GatherParams p, int col_blocks)
{
    begin();
    const int cb = blockIdx.x % col_blocks;
    const long long r0 = static_cast<long long>(blockIdx.x / col_blocks) * kRows;
    const int c = cb * kCols + threadIdx.x * 8;
    if (c >= p.cols) return;
    uint4 v[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        v[i] = make_uint4(0, 0, 0, 0);
        if (r0 + i < p.n) {
            const int f = p.rows[r0 + i];
            if (f >= 0 && f / p.k < p.src_rows) v[i] = load8(p.src + (f / p.k) * p.lds, c, p.cols);
        }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i)
        if (r0 + i < p.n) store8_streaming(p.dst + (r0 + i) * p.ldd, c, p.cols, v[i]);
}

__global__ void __launch_bounds__(kThreads) combine_kernel(const CombineParams p, int col_blocks)
{
    begin();
    const int cb = blockIdx.x % col_blocks;
    const long long t = blockIdx.x / col_blocks;
    const int c = cb * kCols + threadIdx.x * 8;
    if (c >= p.cols) return;
    float acc[8] = {};
    for (int j0 = 0; j0 < p.k; j0 += 4) {
        uint4 v[4];
        float w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = make_uint4(0, 0, 0, 0);
            w[i] = 0.0f;
            if (j0 + i < p.k) {
                const int r = p.slots[t * p.k + j0 + i];
                if (r >= 0 && r < p.rows_n) {
                    v[i] = load8(p.ys + r * p.ldys, c, p.cols);
                    w[i] = p.weights ? p.weights[t * p.k + j0 + i] : 1.0f;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float f[8];
            unpack8(v[i], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = fmaf(w[i], f[e], acc[e]);
        }
    }
    store8(p.y + t * p.ldy, c, p.cols, pack8(acc));
}

// One CTA owns a token: it reads dy[t] once for each of its experts (from
// L1 after the first), the experts' rows once, and writes their gradients.
// The dot products are summed per thread in ascending columns, then by a
// fixed tree over the CTA's threads.
constexpr int kBwdThreads = 256;

__global__ void __launch_bounds__(kBwdThreads) combine_bwd_kernel(const CombineParams p)
{
    begin();
    __shared__ float part[kBwdThreads / 32][kMaxTopK];
    const long long t = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint16_t *dy = p.dy + t * p.lddy;
    for (int j = 0; j < p.k; ++j) {
        const int r = p.slots[t * p.k + j];
        const bool in = r >= 0 && r < p.rows_n;
        const float w = in ? p.weights[t * p.k + j] : 0.0f;
        float dot = 0.0f;
        if (in) {
            const uint16_t *ys = p.ys + r * p.ldys;
            uint16_t *dys = p.dys + r * p.lddys;
            for (int c = threadIdx.x * 8; c < p.cols; c += kBwdThreads * 8) {
                float a[8], b[8], o[8];
                unpack8(load8(dy, c, p.cols), a);
                unpack8(load8(ys, c, p.cols), b);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    dot = fmaf(a[e], b[e], dot);
                    o[e] = w * a[e];
                }
                store8_streaming(dys, c, p.cols, pack8(o));
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(kAll, dot, o);
        if (lane == 0) part[warp][j] = dot;
        // Rows no token owns (after the last expert's) get zero gradients.
        const long long tail = t * p.k + j;
        if (p.rows[tail] < 0) {
            for (int c = threadIdx.x * 8; c < p.cols; c += kBwdThreads * 8)
                store8(p.dys + tail * p.lddys, c, p.cols, make_uint4(0, 0, 0, 0));
        }
    }
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < p.k) {
        float s = 0.0f;
        for (int w = 0; w < kBwdThreads / 32; ++w) s += part[w][threadIdx.x];
        p.dw[t * p.k + threadIdx.x] = s;
    }
}

}  // namespace

cudaError_t launch_gather(const GatherParams &p, cudaStream_t s)
{
    const int cb = (p.cols + kCols - 1) / kCols;
    const long long blocks = static_cast<long long>(cb) * ((p.n + kRows - 1) / kRows);
    return launch_early(gather_kernel, blocks, kThreads, 0, 1, s, p, cb);
}

cudaError_t launch_combine(const CombineParams &p, cudaStream_t s)
{
    const int cb = (p.cols + kCols - 1) / kCols;
    return launch_early(combine_kernel, static_cast<long long>(cb) * p.tokens, kThreads, 0, 1, s, p, cb);
}

cudaError_t launch_combine_bwd(const CombineParams &p, cudaStream_t s)
{
    return launch_early(combine_bwd_kernel, p.tokens, kBwdThreads, 0, 1, s, p);
}

}  // namespace deto
