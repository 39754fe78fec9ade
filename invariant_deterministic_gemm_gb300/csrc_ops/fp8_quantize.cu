// Quantisers to e4m3 with one FP32 scale for each block of 128.
//   amax = max(max |x| over the block, 2^-100)
//   s = amax / 448,  q = e4m3(x * 448 / amax)     (nearest, ties to even)
// A block holding an infinity or a NaN gets s = NaN and q = 0, so that every
// product it enters is NaN.
//
// The quotient decides a rounding, so it is formed exactly enough to never
// decide it wrongly: t = 448 x is exact in FP32 (11 significant bits), and
// y0 = t * r, r = 1 / amax within a unit in the last place, is corrected once
// by its residual t - y0 * amax, which one fused multiply-add forms exactly
// (Newton's correction of a quotient). y is then exact whenever the quotient
// has few bits, which every e4m3 midpoint has; and a quotient of two BF16
// values that is not a midpoint is at least 2^-20 of its size away from one,
// far more than y's error. Two elements at a time (f32x2 operations). The
// scale amax / 448 is corrected the same way and is correctly rounded.
//
// The input is read once (BF16) and one byte an element is written, and what
// is done to an element in between counts about as much as its bytes: a warp's
// instructions are kept few (a lane has 16 elements of a block along rows, 32
// of two columns along columns; tests for edges only in tiles that have one).
// [8192, 14336] along rows 52.6 us (6.7 TB/s; 61 us with eight elements a lane and
// a 64-bit division a warp), along columns 65 us (5.4 TB/s; 78 us with tests at
// every load); [8192, 4096] 16 and 20 us. Gathered, 49152 rows of 4096 from 8192:
// 85 us, where the gather alone takes 89. Weight tiles, [14336, 4096]: 44 us (4.0
// TB/s), transposed 51 (3.4), where the bytes would take 26: a CTA loads its 32 KB,
// waits for the tile's maximum and stores, and five CTAs an SM (48 registers) are
// few to have loads under way meanwhile: warps wait for memory, and half of the
// issue slots are empty.
#include "launch.cuh"
#include "ops_internal.h"
#include "vec.cuh"

namespace deto {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;

__device__ __forceinline__ float block_scale(float amax)     // amax already floored; inf or NaN: NaN
{
    if (!(amax < __int_as_float(0x7f800000))) return __int_as_float(0x7fc00000);
    constexpr float r = 1.0f / kE4M3Max;
    const float y = amax * r;
    return fmaf(fmaf(-y, kE4M3Max, amax), r, y);
}

__device__ __forceinline__ uint64_t pair(float lo, float hi)
{
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
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
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// What a block's elements are divided by: amax (floored, and at most 2^100)
// and its reciprocal; `down` is what the elements are multiplied by first.
struct Divisor {
    float amax, r, down;
    bool fine;
};
__device__ __forceinline__ Divisor divisor(float amax)
{
    Divisor d;
    d.fine = amax < __int_as_float(0x7f800000);
    // Near the top of the range, where 448 x would overflow, by 2^-40 first.
    const bool large = amax > 1.2676506e30f;
    d.down = large ? 448.0f * 9.094947e-13f : 448.0f;
    d.amax = large ? amax * 9.094947e-13f : amax;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(d.r) : "f"(d.amax));
    return d;
}

// Two elements' quotients. a: (amax, amax'), r: reciprocals, s: factors.
__device__ __forceinline__ uint64_t quotient2(uint64_t x, uint64_t neg_a, uint64_t r, uint64_t s)
{
    const uint64_t t = mul2(x, s);
    const uint64_t y = mul2(t, r);
    return fma2(fma2(y, neg_a, t), r, y);
}

// Four values to four bytes, in one block so that the second conversion
// merges into the first one's register.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d)
{
    uint32_t w;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(w)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return w;
}

// The larger magnitudes of two pairs of BF16 values; a NaN stays one.
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("{\n\t.reg .b32 x, y;\n\t"
        "abs.bf16x2 x, %1;\n\t"
        "abs.bf16x2 y, %2;\n\t"
        "max.NaN.bf16x2 %0, x, y;\n\t}"
        : "=r"(d)
        : "r"(a), "r"(b));
    return d;
}

// A BF16 bit pattern (magnitude) as a floored FP32 maximum.
__device__ __forceinline__ float floor_amax(uint32_t bf16_bits)
{
    const uint32_t lo = __float_as_uint(kAmaxMin), b = bf16_bits << 16;
    return __uint_as_float(b < lo ? lo : b);
}

// Eight elements of one block (BF16 pairs) -> eight e4m3 bytes.
__device__ __forceinline__ uint2 quantize8(const uint4 &v, const Divisor &d)
{
    if (!d.fine) return make_uint2(0, 0);
    const uint64_t na = pair(-d.amax, -d.amax), r = pair(d.r, d.r), s = pair(d.down, d.down);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) unpair(quotient2(pair(bf_lo(w[i]), bf_hi(w[i])), na, r, s), f[2 * i], f[2 * i + 1]);
    return make_uint2(e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7]));
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

// ---- along rows: 8 lanes own a block of 128 columns, 8 columns of either half
// each (whole lines an access); a warp takes kUnroll times four blocks of one
// row, all loads in flight at once.
constexpr int kRowThreads = 128;
constexpr int kUnroll = 2;
constexpr int kStepCols = 4 * kBlock;
constexpr int kWarpCols = kStepCols * kUnroll;

__global__ void __launch_bounds__(kRowThreads) quantize_rows_kernel(const QuantParams p, int col_parts)
{
    begin();
    const int lane = threadIdx.x & 31;
    // (rows x parts stay below 2^32: the rows are below 2^31, and a part more is a kilobyte of input)
    const unsigned w = blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
    const unsigned row = w / static_cast<unsigned>(col_parts);
    if (row >= static_cast<unsigned>(p.n)) return;
    const long long m = row;
    const int w0 = static_cast<int>(w - row * col_parts) * kWarpCols;
    const int c0 = w0 + (lane >> 3) * kBlock + (lane & 7) * 8;
    const uint16_t *src = nullptr;
    if (p.rows) {
        const int f = p.rows[m];
        if (f >= 0 && f / p.k < p.src_rows) src = p.x + (f / p.k) * p.ldx;
    } else {
        src = p.x + m * p.ldx;
    }
    uint4 v[kUnroll][2];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = c0 + u * kStepCols + h * (kBlock / 2);
            v[u][h] = make_uint4(0, 0, 0, 0);
            if (src && c < p.cols) v[u][h] = load8(src, c, p.cols);
        }
    uint8_t *q = p.q + m * p.ldq;
    float own = 0.0f;                                // maximum of the block whose scale this lane writes
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        if (w0 + u * kStepCols >= p.cols) break;     // the whole warp
        const int c = c0 + u * kStepCols;
        uint32_t a = max2(max2(max2(v[u][0].x, v[u][0].y), max2(v[u][0].z, v[u][0].w)),
                          max2(max2(v[u][1].x, v[u][1].y), max2(v[u][1].z, v[u][1].w)));
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) a = max2(a, __shfl_xor_sync(kAll, a, o));
        const float amax = floor_amax(max(a & 0xFFFFu, a >> 16));
        if ((lane & 7) == u) own = amax;
        if (c >= p.cols) continue;
        const Divisor d = divisor(amax);
        store_q8(q, c, p.cols, quantize8(v[u][0], d));
        if (c + kBlock / 2 < p.cols) store_q8(q, c + kBlock / 2, p.cols, quantize8(v[u][1], d));
    }
    const int b = w0 / kBlock + (lane & 7) * (kStepCols / kBlock) + (lane >> 3);
    if ((lane & 7) < kUnroll && b * kBlock < p.cols) p.s[b * p.lds + m] = block_scale(own);
}

// ---- along columns (the contraction is the token dimension): a CTA owns a
// block of 128 rows and 64 columns. A warp reads 16 of the rows, a lane two
// neighbouring columns of each (whole lines), so a lane ends up with 16
// consecutive bytes of either column's output; they go out through shared
// memory as 128 bytes a column. With group bounds a block holds rows of one
// group only, and the rows past the group's end are zeros.
constexpr int kColThreads = 256;
constexpr int kColTile = 64;
constexpr int kPitch = kBlock + 16;  // bytes between columns in shared memory: 16-byte accesses without conflicts

__global__ void __launch_bounds__(kColThreads) quantize_cols_kernel(const QuantParams p, int col_tiles)
{
    begin();
    __shared__ __align__(16) uint8_t out[kColTile * kPitch];
    __shared__ uint32_t part[kColThreads / 32][32];
    const int blk = blockIdx.x / col_tiles;
    const int c0 = (blockIdx.x - blk * col_tiles) * kColTile;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int r0, r1;
    if (p.offsets) {
        // The group this block belongs to: a running sum of the groups'
        // blocks, 32 groups a step, by every warp for itself.
        int run = 0;
        bool bad = false;
        r0 = r1 = -1;
        for (int g0 = 0; g0 < p.groups; g0 += 32) {
            const int g = g0 + lane;
            int lo = 0, hi = 0;
            if (g < p.groups) {
                lo = min(max(p.offsets[g], 0), p.n);
                hi = min(max(p.offsets[g + 1], lo), p.n);
                bad |= p.offsets[g] != lo || p.offsets[g + 1] != hi;
            }
            const int nb = (hi - lo + kBlock - 1) / kBlock;
            int v = nb;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(kAll, v, o);
                if (lane >= o) v += u;
            }
            const int first = run + v - nb;
            const unsigned who = __ballot_sync(kAll, blk >= first && blk < first + nb && blk + 1 < p.max_blocks);
            if (who) {
                const int at = __ffs(static_cast<int>(who)) - 1;
                const int l = __shfl_sync(kAll, lo, at), h = __shfl_sync(kAll, hi, at), f = __shfl_sync(kAll, first, at);
                r0 = l + (blk - f) * kBlock;
                r1 = min(h, r0 + kBlock);
                break;
            }
            run += __shfl_sync(kAll, v, 31);
        }
        if (r0 < 0) {
            // Past the last group's blocks (the whole CTA), as the last block always is
            // for bounds in order: it has seen all of them. Where bounds made no
            // sense a product may count a block here that no group filled: it finds
            // zeros.
            if (!__any_sync(kAll, bad)) return;
            if (threadIdx.x == 0) atomicExch(p.status, kStatusInvalid);
            for (int i = threadIdx.x; i < kColTile * (kBlock / 16); i += kColThreads) {
                const int col = c0 + i / (kBlock / 16);
                if (col < p.cols)
                    *reinterpret_cast<uint4 *>(p.q + col * p.ldq + static_cast<long long>(blk) * kBlock + i % (kBlock / 16) * 16) =
                        make_uint4(0, 0, 0, 0);
            }
            if (threadIdx.x < kColTile && c0 + static_cast<int>(threadIdx.x) < p.cols) p.s[blk * p.lds + c0 + threadIdx.x] = 0.0f;
            return;
        }
    } else {
        r0 = blk * kBlock;
        r1 = min(p.n, r0 + kBlock);
    }
    const int c = c0 + 2 * lane;
    uint32_t v[16];
    {
        const uint16_t *x = p.x + (r0 + warp * 16) * p.ldx + c;
        const int rows = r1 - r0 - warp * 16;
        if (rows >= 16 && c0 + kColTile <= p.cols) {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = *reinterpret_cast<const uint32_t *>(x + i * p.ldx);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                v[i] = 0;
                if (i < rows) {
                    if (c + 1 < p.cols) v[i] = *reinterpret_cast<const uint32_t *>(x + i * p.ldx);
                    else if (c < p.cols) v[i] = x[i * p.ldx];
                }
            }
        }
    }
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) a = __vmaxu2(a, v[i] & 0x7FFF7FFFu);
    part[warp][lane] = a;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kColThreads / 32; ++w) a = __vmaxu2(a, part[w][lane]);
    const float a0 = floor_amax(a & 0xFFFFu), a1 = floor_amax(a >> 16);
    const Divisor d0 = divisor(a0), d1 = divisor(a1);
    const uint64_t na = pair(-d0.amax, -d1.amax), r = pair(d0.r, d1.r), s = pair(d0.down, d1.down);
    uint32_t q0[4], q1[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float y0[4], y1[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t w = v[4 * i + e];
            unpair(quotient2(pair(bf_lo(w), bf_hi(w)), na, r, s), y0[e], y1[e]);
        }
        q0[i] = d0.fine ? e4m3x4(y0[0], y0[1], y0[2], y0[3]) : 0;
        q1[i] = d1.fine ? e4m3x4(y1[0], y1[1], y1[2], y1[3]) : 0;
    }
    *reinterpret_cast<uint4 *>(out + (2 * lane) * kPitch + warp * 16) = make_uint4(q0[0], q0[1], q0[2], q0[3]);
    *reinterpret_cast<uint4 *>(out + (2 * lane + 1) * kPitch + warp * 16) = make_uint4(q1[0], q1[1], q1[2], q1[3]);
    if (warp == 0) {
        float *sc = p.s + blk * p.lds + c;
        if (c < p.cols) sc[0] = block_scale(a0);
        if (c + 1 < p.cols) sc[1] = block_scale(a1);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int col = i * 32 + (threadIdx.x >> 3), k = threadIdx.x & 7;
        if (c0 + col < p.cols)
            *reinterpret_cast<uint4 *>(p.q + static_cast<long long>(c0 + col) * p.ldq + static_cast<long long>(blk) * kBlock + k * 16) =
                *reinterpret_cast<const uint4 *>(out + col * kPitch + k * 16);
    }
}

// ---- 128 x 128 tiles (weights), written as they lie, transposed, or both.
constexpr int kTileThreads = 256;

__global__ void __launch_bounds__(kTileThreads) quantize_tiles_kernel(const QuantParams p, int row_tiles, int col_tiles)
{
    begin();
    __shared__ __align__(4) uint8_t tq[kBlock][kBlock + 4];      // (also stored to four bytes at a time)
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
        a = max2(a, max2(max2(v[i].x, v[i].y), max2(v[i].z, v[i].w)));
    }
    a = __reduce_max_sync(kAll, max(a & 0xFFFFu, a >> 16));
    if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = a;
    __syncthreads();
    a = 0;
#pragma unroll
    for (int w = 0; w < kTileThreads / 32; ++w) a = max(a, wmax[w]);
    const float amax = floor_amax(a);
    const Divisor d = divisor(amax);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int rl = i * 16 + (threadIdx.x >> 4), r = rt * kBlock + rl;
        const uint2 q = quantize8(v[i], d);
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
    return launch_early(quantize_rows_kernel, blocks, kRowThreads, 0, 1, s, p, parts);
}

cudaError_t launch_quantize_cols(const QuantParams &p, cudaStream_t s)
{
    const int ct = (p.cols + kColTile - 1) / kColTile;
    const long long blocks = static_cast<long long>(ct) * p.max_blocks;
    return launch_early(quantize_cols_kernel, blocks, kColThreads, 0, 1, s, p, ct);
}

cudaError_t launch_quantize_tiles(const QuantParams &p, cudaStream_t s)
{
    const int rt = (p.n + kBlock - 1) / kBlock, ct = (p.cols + kBlock - 1) / kBlock;
    const long long blocks = static_cast<long long>(rt) * ct * p.groups;
    return launch_early(quantize_tiles_kernel, blocks, kTileThreads, 0, 1, s, p, rt, ct);
}

}  // namespace deto
