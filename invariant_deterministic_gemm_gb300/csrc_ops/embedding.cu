// Embedding lookup with scaling, and its gradient by sorted tokens.
//   out[t] = bf16(scale * table[tok[t]])
//   dtable[v] = scale * sum over t with tok[t] = v of dy[t]
// The gradient's terms are added in FP32 in a fixed order: the occurrences
// of a token in ascending t, in chunks of 32 summed from +0, and the chunks
// in ascending order. A row's bits depend on its own occurrences alone.
//
// The stable sort (sort_by_key.cu) brings a token's occurrences together; one
// block of threads then owns each chunk. The dense output's rows that never
// occur are zeroed beside that, and its first 128 MB beside the sort, which
// leaves the memory idle otherwise (a gradient of 1.2 GB: 200 us; with 64 MB
// there 205, 256 MB 204, all of it 250, nothing 218). How much is best grows with
// the sort, so with the tokens, but slowly: 128 MB is within 2 % of the best of
// 32 MB to 1 GB for the same gradient from 333 evenly spread tokens (167 us; 256
// MB 172), 8192 (213; 216), 32768 (357; 350) and 131072 (894; 890, 512 MB 877).
// Tokens that occur more
// than 32 times (a few stand in every twentieth position of a text) leave their
// chunks' sums in a workspace, and a second launch adds them up; with one owner
// per run instead, the most frequent token alone would be a serial walk over
// thousands of rows.
//
// Bytes bound it: dy is read once and the dense gradient written once. 8192
// tokens, a BF16 gradient of 151936 x 4096: 200 us, the lookup 20 us (6.6 TB/s);
// 333 tokens, an FP32 gradient of 32003 x 1000: 27 us, of which 14 stay without
// zeros to write (the latency of the sort, the sums and their joining). Accumulated,
// those 8192 tokens (4200 different ones) take 66 us, 79 in FP32, where the bytes
// would take 20 and 30: three launches that need one another, with no zeros to
// write beside the first.
#include "launch.cuh"
#include "ops_internal.h"
#include "vec.cuh"

namespace deto {
namespace {

constexpr int kChunk = 32;
constexpr int kThreads = 128;
constexpr int kCols = kThreads * 8;  // columns of a block
constexpr unsigned kAll = 0xFFFFFFFFu;

__global__ void __launch_bounds__(kThreads) lookup_kernel(const EmbedParams p, int col_blocks)
{
    begin();
    const int cb = blockIdx.x % col_blocks;
    const long long t = blockIdx.x / col_blocks;
    const int c = cb * kCols + threadIdx.x * 8;
    if (c >= p.cols) return;
    long long v;
    if (p.tokens64) v = static_cast<const long long *>(p.tokens)[t];
    else v = static_cast<const int *>(p.tokens)[t];
    if (v < 0 || v >= p.vocab) {
        if (threadIdx.x == 0 && cb == 0) atomicExch(p.status, kStatusInvalid);
        store8(p.out + t * p.ldo, c, p.cols, make_uint4(0, 0, 0, 0));
        return;
    }
    float f[8];
    unpack8(load8(p.table + v * p.ldt, c, p.cols), f);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] *= p.scale;
    store8(p.out + t * p.ldo, c, p.cols, pack8(f));
}

// A finished row's eight columns: scaled, and added to what is there when
// accumulating (one more rounding).
__device__ __forceinline__ void finish(const EmbedGradParams &p, long long v, int c, const float (&acc)[8])
{
    float f[8];
    if (p.fp32) {
        float *row = static_cast<float *>(p.dtable) + v * p.ldd;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            f[i] = acc[i] * p.scale;
            if (p.accumulate && c + i < p.cols) f[i] += row[c + i];
        }
        store8f(row, c, p.cols, f);
    } else {
        uint16_t *row = static_cast<uint16_t *>(p.dtable) + v * p.ldd;
        float old[8] = {};
        if (p.accumulate) unpack8(load8(row, c, p.cols), old);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = fmaf(acc[i], p.scale, old[i]);
        store8(row, c, p.cols, pack8(f));
    }
}

// Blocks [0, n * col_blocks): a sorted position and 1024 columns; a position
// that starts a chunk sums it. The rest: vocabulary rows that never occur,
// kZeroRows of them and 1024 columns.
constexpr int kZeroRows = 8;

__global__ void __launch_bounds__(kThreads) grad_kernel(const EmbedGradParams p, int col_blocks)
{
    begin();
    const long long chunk_blocks = static_cast<long long>(p.n) * col_blocks;
    const int cb = blockIdx.x % col_blocks;
    const int c = cb * kCols + threadIdx.x * 8;
    if (blockIdx.x >= chunk_blocks) {
        const long long v0 = p.zero_from + (blockIdx.x - chunk_blocks) / col_blocks * kZeroRows;
        const float zero[8] = {};
        if (c >= p.cols) return;
        for (int i = 0; i < kZeroRows; ++i) {
            const long long v = v0 + i;
            if (v >= p.vocab || p.seen[v]) continue;
            if (p.fp32) store8f(static_cast<float *>(p.dtable) + v * p.ldd, c, p.cols, zero);
            else store8(static_cast<uint16_t *>(p.dtable) + v * p.ldd, c, p.cols, make_uint4(0, 0, 0, 0));
        }
        return;
    }
    const int i = static_cast<int>(blockIdx.x / col_blocks);
    const int head = p.head[i];
    if ((i - head) % kChunk != 0) return;
    const int key = p.keys[i];
    if (key >= p.vocab) return;                      // not a token
    // The chunk's length: how many of the next 32 positions hold this key.
    const int lane = threadIdx.x & 31;
    const bool same = i + lane < p.n && p.keys[i + lane] == key;
    const int len = __popc(__ballot_sync(kAll, same));       // the keys are sorted: a prefix
    const bool more = i + kChunk < p.n && p.keys[i + kChunk] == key;
    const int src = i + lane < p.n ? p.order[i + lane] : 0;
    const bool in = c < p.cols;
    float acc[8] = {};
    for (int r0 = 0; r0 < len; r0 += 4) {
        uint4 v[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            v[r] = make_uint4(0, 0, 0, 0);
            const int t = __shfl_sync(kAll, src, (r0 + r) & 31);
            if (r0 + r < len && in) v[r] = load8(p.dy + t * p.lddy, c, p.cols);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if (r0 + r >= len) break;
            float f[8];
            unpack8(v[r], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] += f[e];
        }
    }
    if (!in) return;
    if (head == i && !more) {
        finish(p, key, c, acc);
    } else {
        // Slot: in any 32 positions at most one chunk of a long run starts
        // besides the first chunk of one more run, so (window, first or
        // not) names it.
        float *slot = p.partials + (2ll * (i / kChunk) + (i == head)) * p.ldp;
        *reinterpret_cast<float4 *>(slot + c) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        *reinterpret_cast<float4 *>(slot + c + 4) = make_float4(acc[4], acc[5], acc[6], acc[7]);
    }
}

// One block per 32 positions and 1024 columns: the long run that starts
// among them, if any (a second one would have to start within its first 33
// positions).
__global__ void __launch_bounds__(kThreads) fold_kernel(const EmbedGradParams p, int col_blocks)
{
    begin();
    const int cb = blockIdx.x % col_blocks;
    const int i0 = static_cast<int>(blockIdx.x / col_blocks) * kChunk;
    const int lane = threadIdx.x & 31;
    const int i = i0 + lane;
    bool starts = false;
    if (i + kChunk < p.n && p.head[i] == i) {
        const int k = p.keys[i];
        starts = k < p.vocab && p.keys[i + kChunk] == k;
    }
    const unsigned who = __ballot_sync(kAll, starts);
    if (who == 0) return;
    const int head = i0 + __ffs(static_cast<int>(who)) - 1;
    const int key = p.keys[head];
    // The run's chunks after the first: 32 positions 32 apart at a time.
    int chunks = 0;
    for (;;) {
        const long long x = head + static_cast<long long>(chunks + lane + 1) * kChunk;
        const unsigned same = __ballot_sync(kAll, x < p.n && p.keys[x] == key);
        const int add = __popc(same);                // the keys are sorted: a prefix
        chunks += add;
        if (add < 32) break;
    }
    const int c = cb * kCols + threadIdx.x * 8;
    if (c >= p.cols) return;
    float acc[8];
    {
        const float *s = p.partials + (2ll * (head / kChunk) + 1) * p.ldp + c;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = s[e];
    }
    for (int c0 = 1; c0 <= chunks; c0 += 8) {
        float4 a[8], b[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            a[r] = b[r] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c0 + r <= chunks) {
                const float *s = p.partials + 2ll * (head / kChunk + c0 + r) * p.ldp + c;
                a[r] = *reinterpret_cast<const float4 *>(s);
                b[r] = *reinterpret_cast<const float4 *>(s + 4);
            }
        }
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            if (c0 + r > chunks) break;
            acc[0] += a[r].x; acc[1] += a[r].y; acc[2] += a[r].z; acc[3] += a[r].w;
            acc[4] += b[r].x; acc[5] += b[r].y; acc[6] += b[r].z; acc[7] += b[r].w;
        }
    }
    finish(p, key, c, acc);
}

}  // namespace

cudaError_t launch_embedding(const EmbedParams &p, cudaStream_t s)
{
    const int cb = (p.cols + kCols - 1) / kCols;
    return launch_early(lookup_kernel, static_cast<long long>(cb) * p.n, kThreads, 0, 1, s, p, cb);
}

cudaError_t launch_embedding_grad(const EmbedGradParams &p, cudaStream_t s)
{
    const int cb = (p.cols + kCols - 1) / kCols;
    const long long blocks = static_cast<long long>(cb) * (p.n + (p.vocab - p.zero_from + kZeroRows - 1) / kZeroRows);
    if (blocks == 0) return cudaSuccess;
    const cudaError_t e = launch_early(grad_kernel, blocks, kThreads, 0, 1, s, p, cb);
    if (e != cudaSuccess || p.n <= kChunk) return e;
    return launch_early(fold_kernel, static_cast<long long>(cb) * ((p.n + kChunk - 1) / kChunk), kThreads, 0, 1, s, p, cb);
}

}  // namespace deto
