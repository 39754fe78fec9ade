// Quantisers to e4m3 with one FP32 scale for each block of 128.
//   amax = max(max |x| over the block, 2^-100)
//   s = amax / 448,  q = e4m3(x * 448 / amax)     (nearest, ties to even)
// A block holding an infinity or a NaN gets s = NaN and q = 0, so that every
// product it enters is NaN.
//
// The quotient decides a rounding, so it is formed exactly enough to never
// decide it wrongly: t = 448 x is exact in FP32 (11 significant bits), and
// y0 = t * (1 / amax) is corrected once by its residual t - y0 * amax, which
// one fused multiply-add forms exactly (Newton's correction of a quotient).
// y is then exact whenever the quotient has few bits, which every e4m3
// midpoint has; and a quotient of two BF16 values that is not a midpoint is
// at least 2^-20 of its size away from one, far more than y's error.
//
// Bytes bound these kernels: the input is read once (BF16) and one byte an
// element is written.
#include "ops_internal.h"
#include "vec.cuh"

namespace deto {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;

__device__ __forceinline__ float block_scale(float amax)     // amax already floored; inf or NaN: NaN
{
    return amax < __int_as_float(0x7f800000) ? __fdiv_rn(amax, kE4M3Max) : __int_as_float(0x7fc00000);
}

// x * 448 / amax for one element (r = 1 / amax; 0 when amax is not finite).
__device__ __forceinline__ float quotient(float x, float amax, float r)
{
    const float t = x * kE4M3Max;
    const float y = t * r;
    return fmaf(fmaf(-y, amax, t), r, y);
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

// |x| ordered as an integer (NaN above infinity), so that a maximum keeps NaN.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

__device__ __forceinline__ float floor_amax(uint32_t bits)
{
    const uint32_t lo = __float_as_uint(kAmaxMin);
    return __uint_as_float(bits < lo ? lo : bits);
}

// Eight elements of one block -> eight e4m3 bytes.
__device__ __forceinline__ uint2 quantize8(const float (&f)[8], float amax)   // amax floored
{
    if (!(amax < __int_as_float(0x7f800000))) return make_uint2(0, 0);
    // Blocks near the top of the range are divided by 2^40 first, where 448 x would overflow.
    const float down = amax > 1.2676506e30f ? 9.094947e-13f : 1.0f;
    amax *= down;
    const float r = __frcp_rn(amax);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = quotient(f[i] * down, amax, r);
    return make_uint2(e4m3x2(y[0], y[1]) | (e4m3x2(y[2], y[3]) << 16), e4m3x2(y[4], y[5]) | (e4m3x2(y[6], y[7]) << 16));
}

__device__ __forceinline__ void store_q8(uint8_t *row, int c, int cols, const uint2 &v)
{
    if (c + 8 <= cols) {
        *reinterpret_cast<uint2 *>(row + c) = v;
        return;
    }
    const uint32_t w[2] = {v.x, v.y};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c + i < cols) row[c + i] = static_cast<uint8_t>(w[i >> 2] >> (8 * (i & 3)));
}

// ---- along rows: 16 lanes own a block of 128 columns, 8 columns each; a
// warp takes kUnroll pairs of blocks of one row.
constexpr int kRowThreads = 128;
constexpr int kUnroll = 2;
constexpr int kWarpCols = 256 * kUnroll;

__global__ void __launch_bounds__(kRowThreads) quantize_rows_kernel(const QuantParams p, int col_parts)
{
    const int lane = threadIdx.x & 31;
    const long long w = static_cast<long long>(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5);
    const long long m = w / col_parts;
    if (m >= p.n) return;
    const int c0 = static_cast<int>(w % col_parts) * kWarpCols + lane * 8;
    const uint16_t *src = nullptr;
    if (p.rows) {
        const int f = __ldg(p.rows + m);
        if (f >= 0 && f / p.k < p.src_rows) src = p.x + (f / p.k) * p.ldx;
    } else {
        src = p.x + m * p.ldx;
    }
    uint4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        v[u] = make_uint4(0, 0, 0, 0);
        if (src && c0 + u * 256 < p.cols) v[u] = load8(src, c0 + u * 256, p.cols);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int c = c0 + u * 256;
        float f[8];
        unpack8(v[u], f);
        uint32_t a = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) a = max(a, abs_bits(f[i]));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(kAll, a, o));
        const float amax = floor_amax(a);
        if (c >= p.cols) continue;
        store_q8(p.q + m * p.ldq, c, p.cols, quantize8(f, amax));
        if ((lane & 15) == 0) p.s[(c / kBlock) * p.lds + m] = block_scale(amax);
    }
}

// ---- along columns (the contraction is the token dimension): a CTA owns a
// block of 128 rows and 64 columns. It reads 128 bytes of each row, keeps
// the tile in shared memory, and writes 128 bytes for each column: out row
// = column, out column = the block's place. With group bounds a block holds
// rows of one group only, and the rows past the group's end are zeros.
constexpr int kColThreads = 256;
constexpr int kColTile = 64;

__global__ void __launch_bounds__(kColThreads) quantize_cols_kernel(const QuantParams p, int col_tiles)
{
    __shared__ float tile[kBlock][kColTile + 1];
    __shared__ int sb[kMaxExperts + 1];
    __shared__ uint32_t part[4][kColTile];
    const int blk = blockIdx.x / col_tiles;
    const int c0 = (blockIdx.x % col_tiles) * kColTile;
    int r0, r1;
    if (p.offsets) {
        // First block of each group, by one warp (a running sum over the groups).
        if (threadIdx.x < 32) {
            int run = 0;
            for (int g0 = 0; g0 < p.groups; g0 += 32) {
                const int g = g0 + threadIdx.x;
                int nb = 0;
                if (g < p.groups) {
                    const int lo = min(max(p.offsets[g], 0), p.n), hi = min(max(p.offsets[g + 1], lo), p.n);
                    nb = (hi - lo + kBlock - 1) / kBlock;
                }
                int v = nb;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int u = __shfl_up_sync(kAll, v, o);
                    if (static_cast<int>(threadIdx.x) >= o) v += u;
                }
                if (g < p.groups) sb[g] = run + v - nb;
                run += __shfl_sync(kAll, v, 31);
            }
            if (threadIdx.x == 0) sb[p.groups] = run;
        }
        __syncthreads();
        if (blk >= sb[p.groups]) return;
        int a = 0, b = p.groups;                     // last group whose first block is <= blk
        while (b - a > 1) {
            const int mid = (a + b) / 2;
            if (sb[mid] <= blk) a = mid;
            else b = mid;
        }
        const int lo = min(max(p.offsets[a], 0), p.n), hi = min(max(p.offsets[a + 1], lo), p.n);
        r0 = lo + (blk - sb[a]) * kBlock;
        r1 = min(hi, r0 + kBlock);
    } else {
        r0 = blk * kBlock;
        r1 = min(p.n, r0 + kBlock);
    }
    {
        // 8 threads a row, 32 rows at a time
        const int c = c0 + (threadIdx.x & 7) * 8;
        for (int r = threadIdx.x >> 3; r < kBlock; r += kColThreads / 8) {
            float f[8] = {};
            if (r0 + r < r1 && c < p.cols) unpack8(load8(p.x + (r0 + r) * p.ldx, c, p.cols), f);
#pragma unroll
            for (int i = 0; i < 8; ++i) tile[r][(threadIdx.x & 7) * 8 + i] = f[i];
        }
    }
    __syncthreads();
    // Thread: column col, quarter qr of the rows (32 of them).
    const int col = threadIdx.x & 63, qr = threadIdx.x >> 6;
    uint32_t a = 0;
#pragma unroll 8
    for (int r = 0; r < 32; ++r) a = max(a, abs_bits(tile[qr * 32 + r][col]));
    part[qr][col] = a;
    __syncthreads();
    a = max(max(part[0][col], part[1][col]), max(part[2][col], part[3][col]));
    if (c0 + col >= p.cols) return;
    const float amax = floor_amax(a);
    uint8_t *dst = p.q + static_cast<long long>(c0 + col) * p.ldq + static_cast<long long>(blk) * kBlock + qr * 32;
    uint32_t w[8];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = tile[qr * 32 + b * 8 + i][col];
        const uint2 q = quantize8(f, amax);
        w[2 * b] = q.x;
        w[2 * b + 1] = q.y;
    }
    *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4 *>(dst + 16) = make_uint4(w[4], w[5], w[6], w[7]);
    if (qr == 0) p.s[blk * p.lds + c0 + col] = block_scale(amax);
}

// ---- 128 x 128 tiles (weights), written as they lie, transposed, or both.
constexpr int kTileThreads = 256;

__global__ void __launch_bounds__(kTileThreads) quantize_tiles_kernel(const QuantParams p, int row_tiles, int col_tiles)
{
    __shared__ uint8_t tq[kBlock][kBlock + 4];
    __shared__ uint32_t wmax[kTileThreads / 32];
    const int ct = blockIdx.x % col_tiles;
    const int rt = blockIdx.x / col_tiles % row_tiles;
    const long long g = blockIdx.x / col_tiles / row_tiles;
    const uint16_t *x = p.x + g * p.xg;
    const int c = ct * kBlock + (threadIdx.x & 15) * 8;
    uint4 v[8];
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = rt * kBlock + i * 16 + (threadIdx.x >> 4);
        v[i] = make_uint4(0, 0, 0, 0);
        if (r < p.n && c < p.cols) v[i] = load8(x + r * p.ldx, c, p.cols);
        float f[8];
        unpack8(v[i], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) a = max(a, abs_bits(f[e]));
    }
    a = __reduce_max_sync(kAll, a);
    if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = a;
    __syncthreads();
    a = 0;
#pragma unroll
    for (int w = 0; w < kTileThreads / 32; ++w) a = max(a, wmax[w]);
    const float amax = floor_amax(a);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int rl = i * 16 + (threadIdx.x >> 4), r = rt * kBlock + rl;
        float f[8];
        unpack8(v[i], f);
        const uint2 q = quantize8(f, amax);
        if (p.q && r < p.n && c < p.cols) store_q8(p.q + g * p.qg + r * p.ldq, c, p.cols, q);
        uint32_t *t = reinterpret_cast<uint32_t *>(&tq[rl][(threadIdx.x & 15) * 8]);
        t[0] = q.x;
        t[1] = q.y;
    }
    if (threadIdx.x == 0) {
        const float s = block_scale(amax);
        if (p.s) p.s[g * p.sg + rt * p.lds + ct] = s;
        if (p.st) p.st[g * p.stg + ct * p.ldst + rt] = s;
    }
    if (!p.qt) return;
    __syncthreads();
    // Transposed: thread = (column, half of the rows).
    const int col = threadIdx.x >> 1, half = threadIdx.x & 1;
    if (ct * kBlock + col >= p.cols) return;
    uint8_t *dst = p.qt + g * p.qtg + static_cast<long long>(ct * kBlock + col) * p.ldqt + rt * kBlock;
    const int n = p.n - rt * kBlock;                 // rows of this tile
    for (int b = half * 64; b < half * 64 + 64 && b < n; b += 16) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = tq[b + 4 * i][col] | (tq[b + 4 * i + 1][col] << 8) | (tq[b + 4 * i + 2][col] << 16) |
                   (static_cast<uint32_t>(tq[b + 4 * i + 3][col]) << 24);
        if (b + 16 <= n) {
            *reinterpret_cast<uint4 *>(dst + b) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            for (int i = 0; i < 16 && b + i < n; ++i) dst[b + i] = static_cast<uint8_t>(w[i >> 2] >> (8 * (i & 3)));
        }
    }
}

}  // namespace

cudaError_t launch_quantize_rows(const QuantParams &p, cudaStream_t s)
{
    const int parts = (p.cols + kWarpCols - 1) / kWarpCols;
    const long long warps = static_cast<long long>(parts) * p.n;
    const long long blocks = (warps + kRowThreads / 32 - 1) / (kRowThreads / 32);
    quantize_rows_kernel<<<static_cast<unsigned>(blocks), kRowThreads, 0, s>>>(p, parts);
    return cudaGetLastError();
}

cudaError_t launch_quantize_cols(const QuantParams &p, cudaStream_t s)
{
    const int ct = (p.cols + kColTile - 1) / kColTile;
    const long long blocks = static_cast<long long>(ct) * p.max_blocks;
    quantize_cols_kernel<<<static_cast<unsigned>(blocks), kColThreads, 0, s>>>(p, ct);
    return cudaGetLastError();
}

cudaError_t launch_quantize_tiles(const QuantParams &p, cudaStream_t s)
{
    const int rt = (p.n + kBlock - 1) / kBlock, ct = (p.cols + kBlock - 1) / kBlock;
    const long long blocks = static_cast<long long>(rt) * ct * p.groups;
    quantize_tiles_kernel<<<static_cast<unsigned>(blocks), kTileThreads, 0, s>>>(p, rt, ct);
    return cudaGetLastError();
}

}  // namespace deto
