// C entry points of include/det_ops.h: argument checks, tensor maps, the
// choice of tile, launches.
#include "det_ops.h"
#include "det_gemm_internal.h"
#include "ops_internal.h"

#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <initializer_list>
#include <mutex>

namespace deto {

// First problem a kernel saw since the last det_ops_check.
__device__ int g_ops_status[4];

namespace {

constexpr int64_t kMaxRows = (int64_t{1} << 31) - 4096;
constexpr int kMaxDevices = 64;

struct Device {
    bool init = false;
    det_gemm_status status = DET_GEMM_OK;
    int sms = 0;
    int *word = nullptr;
};
std::mutex g_mu;
Device g_dev[kMaxDevices];
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::atomic<int> g_force_timeout{0};

det_gemm_status fail(det_gemm_status st, cudaError_t e, const char *where)
{
    char msg[256];
    std::snprintf(msg, sizeof msg, "%s: %s (%s)", where, cudaGetErrorName(e), cudaGetErrorString(e));
    detg::record_detail(msg);
    cudaGetLastError();
    return st;
}

det_gemm_status device(Device **out)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return DET_GEMM_ERR_UNSUPPORTED_DEVICE;
    }
    if (dev < 0 || dev >= kMaxDevices) return DET_GEMM_ERR_UNSUPPORTED_DEVICE;
    std::lock_guard<std::mutex> lk(g_mu);
    Device &d = g_dev[dev];
    if (!d.init) {
        d.init = true;
        int major = 0, minor = 0;
        cudaDriverEntryPointQueryResult q;
        void *fn = nullptr;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || major != 10 ||
            minor != 3) {
            cudaGetLastError();
            d.status = DET_GEMM_ERR_UNSUPPORTED_DEVICE;
        } else if (cudaGetSymbolAddress(reinterpret_cast<void **>(&d.word), g_ops_status) != cudaSuccess ||
                   cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) !=
                       cudaSuccess ||
                   q != cudaDriverEntryPointSuccess || fn == nullptr) {
            cudaGetLastError();
            d.status = DET_GEMM_ERR_LAUNCH;
        } else {
            g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
        }
    }
    if (d.status != DET_GEMM_OK) return d.status;
    *out = &d;
    return DET_GEMM_OK;
}

// A strided array: `rows` rows of `cols` elements, pitch `ld`, element size
// `es`, in `mats` matrices `gap` elements apart. `align`: the base's and the
// pitch's alignment in bytes.
struct Arr {
    const void *p;
    int64_t rows, cols, ld;
    int es, align;
    int64_t mats = 1, gap = 0;
    int64_t bytes() const { return ((mats - 1) * gap + (rows - 1) * ld + cols) * es; }
    bool empty() const { return rows <= 0 || cols <= 0 || mats <= 0; }
};

// More bytes than there are addresses; what is below fits 64-bit arithmetic.
constexpr double kMaxBytes = 1ull << 57;

det_gemm_status check(const Arr &a)
{
    if (a.empty()) return DET_GEMM_OK;
    if (!a.p || a.ld < a.cols || a.ld > (int64_t{1} << 36)) return DET_GEMM_ERR_INVALID_ARG;
    if ((static_cast<double>(a.mats - 1) * a.gap + static_cast<double>(a.rows - 1) * a.ld + a.cols) * a.es > kMaxBytes)
        return DET_GEMM_ERR_INVALID_ARG;
    if (a.mats > 1 && (a.gap < (a.rows - 1) * a.ld + a.cols || a.gap > (int64_t{1} << 40))) return DET_GEMM_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(a.p) % a.align != 0 || a.ld * a.es % a.align != 0) return DET_GEMM_ERR_ALIGNMENT;
    if (a.mats > 1 && a.gap * a.es % a.align != 0) return DET_GEMM_ERR_ALIGNMENT;
    return DET_GEMM_OK;
}

bool overlap(const Arr &a, const Arr &b)
{
    if (a.empty() || b.empty() || !a.p || !b.p) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + static_cast<uintptr_t>(b.bytes()) && y < x + static_cast<uintptr_t>(a.bytes());
}

// All arrays well formed, and no output overlapping an input or another output.
det_gemm_status check_all(std::initializer_list<Arr> in, std::initializer_list<Arr> out)
{
    for (const Arr &a : in) {
        const det_gemm_status s = check(a);
        if (s != DET_GEMM_OK) return s;
    }
    for (const Arr *o = out.begin(); o != out.end(); ++o) {
        const det_gemm_status s = check(*o);
        if (s != DET_GEMM_OK) return s;
        for (const Arr &a : in)
            if (overlap(*o, a)) return DET_GEMM_ERR_INVALID_ARG;
        for (const Arr *b = out.begin(); b != o; ++b)
            if (overlap(*o, *b)) return DET_GEMM_ERR_INVALID_ARG;
    }
    return DET_GEMM_OK;
}

Arr bf16(const void *p, int64_t r, int64_t c, int64_t ld) { return Arr{p, r, c, ld, 2, 16}; }
Arr vec4(const void *p, int64_t n) { return Arr{p, 1, n, n, 4, 4}; }
Arr mat8(const void *p, int64_t r, int64_t c, int64_t ld, int64_t mats = 1, int64_t gap = 0)
{
    return Arr{p, r, c, ld, 1, 16, mats, gap};
}

bool ok_size(int64_t v) { return v >= 0 && v <= kMaxRows; }
bool launchable(int64_t blocks) { return blocks <= (int64_t{1} << 31) - 1; }
cudaStream_t cs(det_gemm_stream s) { return reinterpret_cast<cudaStream_t>(s); }
int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

unsigned long long timeout_ns()
{
    if (g_force_timeout.load()) return 50ull * 1000 * 1000;
    const char *s = std::getenv("DET_GEMM_TIMEOUT_MS");
    long long ms = s ? std::atoll(s) : 1000;
    return static_cast<unsigned long long>(ms < 1 ? 1 : ms) * 1000000ull;
}

// [mats] x [rows, k] e4m3 matrix -> map with boxes of 128 contraction bytes x box_rows.
bool encode(CUtensorMap *m, int rank, const void *p, int64_t k, int64_t rows, int64_t ld, int64_t mats, int64_t gap,
            int box_rows)
{
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(mats)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld), static_cast<cuuint64_t>(mats > 1 ? gap : ld * rows)};
    cuuint32_t box[3] = {kBlock, static_cast<cuuint32_t>(box_rows), 1};
    cuuint32_t es[3] = {1, 1, 1};
    return g_encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<void *>(p), dims, strides, box, es,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [blocks, n] scales -> map with boxes of `box` scales of one block.
bool encode_scales(CUtensorMap *m, const float *p, int64_t n, int64_t blocks, int64_t ld, int box)
{
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(n), static_cast<cuuint64_t>(blocks)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 4};
    cuuint32_t boxes[2] = {static_cast<cuuint32_t>(box), 1}, es[2] = {1, 1};
    return g_encode(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<float *>(p), dims, strides, boxes, es,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of a copied box: the operand's own when it has fewer than the tile
// (a box mostly outside its tensor is slow to copy).
int box_rows(int64_t rows, int tile) { return rows >= tile ? tile : static_cast<int>(std::max<int64_t>(16, up(rows, 8) * 8)); }

struct Fp8Args {
    const uint8_t *a;
    const float *sa;
    const uint8_t *b;
    const float *sb;
    const int32_t *offsets;
    void *out;
    int out_fp32;
    int64_t groups, rows, cols, kc;      // kc: the contraction's length as stored
    int64_t lda, ldb, gb, ldo, go;
    int64_t ldsa = 0, ldsb = 0;          // weight gradient: pitches of the scales
};

det_gemm_status enqueue(const Fp8Args &x, Fp8Params &p, const Fp8Plan &plan, Device *d, det_gemm_stream stream)
{
    const bool rows_kind = plan.kind == kFp8Rows;
    p.a_box = (rows_kind && x.offsets) ? plan.tile_m : box_rows(x.rows, plan.tile_m);
    p.b_box = box_rows(x.cols, plan.tile_n);
    p.sa_box = p.a_box;
    p.sb_box = p.b_box;
    if (!encode(&p.tmap_a, 2, x.a, x.kc, x.rows, x.lda, 1, 0, p.a_box) ||
        !encode(&p.tmap_b, 3, x.b, x.kc, x.cols, x.ldb, rows_kind ? x.groups : 1, x.gb, p.b_box) ||
        (!rows_kind && (!encode_scales(&p.tmap_sa, x.sa, x.rows, p.max_blocks, x.ldsa, p.sa_box) ||
                        !encode_scales(&p.tmap_sb, x.sb, x.cols, p.max_blocks, x.ldsb, p.sb_box)))) {
        detg::record_detail("tensor map");
        return DET_GEMM_ERR_LAUNCH;
    }
    p.sa = x.sa;
    p.sb = x.sb;
    p.out = x.out;
    p.ldo = x.ldo;
    p.og = x.go;
    p.offsets = x.offsets;
    p.groups = static_cast<int>(x.groups);
    p.rows = static_cast<int>(x.rows);
    p.cols = static_cast<int>(x.cols);
    p.n_tiles = static_cast<int>(up(x.cols, plan.tile_n));
    p.m_tiles = static_cast<int>(up(x.rows, plan.tile_m));
    p.out_fp32 = x.out_fp32;
    p.status = d->word;
    p.timeout_ns = timeout_ns();
    p.force_timeout = g_force_timeout.load();
    const cudaError_t e = launch_fp8(p, plan, d->sms, cs(stream));
    return e == cudaSuccess ? DET_GEMM_OK : fail(DET_GEMM_ERR_LAUNCH, e, "8-bit product launch");
}

// Width of a weight's product's plain tile: 192 columns, or 128 where the last
// round of one tile per SM would leave too many idle. Four rounds of 128-wide
// tiles take 0.72 of four of 192-wide ones' time with 112 blocks (122 and 170 us)
// and with 32 (36.0, 49.7), 0.74 with 14 and with 8, 0.76 with 4, 0.80 with 1 (9.4,
// 11.7); one round 0.69 with 112, 0.75 with 32, 0.80 with 14, 0.90 with 1. Nothing
// measured is chosen more than 2 % too slow for the one factor ([8192, 4096] from
// 1024: 128 wide 45.7 us, 192 wide 46.5).
int plain_width(int64_t row_tiles, int64_t cols, int sms)
{
    const int64_t wide = up(row_tiles * up(cols, 192), sms) * 100, narrow = up(row_tiles * up(cols, 128), sms) * 72;
    return narrow < wide ? 128 : 192;
}

// The tile of a product with a weight. Both tiles give the same bits; the
// choice is about time. Few rows (per expert): the transposed tile, which
// reads a weight once for up to 64 rows; otherwise the plain one. With weights
// from HBM (us, transposed of 16, 32 and 64 tokens, then plain):
//   [12288, 4096]  16 rows 12.0 15.3 13.3 13.1    64 rows 21 23 14.0 13.4
//   [4096, 14336]  16 rows 18.4 21.6 22.6 27.8    64 rows 42 32 23.5 28.6
//   [14336, 1024]  16 rows 6.5 7.2 7.9 6.6        64 rows 9.4 9.5 8.4 6.9
//   16 x [2048, 4096], as many rows an expert:    16 rows 25.4 25.8 27.1 33.4
//     64 rows 46 31 29.6 30.6, 65 rows 53 38 38 30.6
//   the same, uneven: 16 rows 31 25.9 27.4 33.4; 64 rows 45 39 33 30.3
//   the same, all but one row each on one expert: 16 rows 32 32.7 27 33.7;
//     64 rows 54 41 41 35
// From 65 rows on the plain tile is the faster one everywhere. Up to 64 it is in
// short contractions and where few experts have most rows (by up to a third: 8 x
// [1792, 4096] at 64 uneven rows 22.2 and 14.8), which the host cannot see.
Fp8Plan plan_rows(int64_t rows, int64_t cols, int64_t groups, bool grouped, int sms)
{
    Fp8Plan pl{kFp8Rows, false, 128, 192};
    const int64_t per = grouped ? up(rows, groups) : rows;
    if (per <= 64) {
        pl.swap = true;
        pl.tile_m = per <= (grouped ? 8 : 16) ? 16 : per <= (grouped ? 16 : 32) ? 32 : 64;
        // The narrowest weight tile whose units all run at once: a tile walks
        // the contraction block by block at the same pace whatever its width,
        // so a second round costs as much as the first.
        const int64_t used = grouped ? std::min(rows, groups) : 1, room = (pl.tile_m == 64 ? 1 : 2) * sms;
        pl.tile_n = 32;
        while (pl.tile_n < 128 && used * up(cols, pl.tile_n) > room) pl.tile_n *= 2;
        return pl;
    }
    pl.tile_n = plain_width(up(rows, 128) + (grouped ? groups / 2 : 0), cols, sms);
    return pl;
}

det_gemm_status fp8_rows(const uint8_t *A, const float *sa, const uint8_t *W, const float *sb, const int32_t *offsets,
                         void *C, int out_fp32, int64_t G, int64_t M, int64_t N, int64_t K, int64_t lda, int64_t sa_row,
                         int64_t sa_blk, int64_t ldw, int64_t gw, int64_t sb_row, int64_t gsb, int64_t ldc,
                         bool grouped, det_gemm_stream stream)
{
    if (!ok_size(M) || !ok_size(N) || !ok_size(K) || G < 0 || G > DET_MOE_MAX_EXPERTS) return DET_GEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return DET_GEMM_OK;
    if (!launchable((up(M, 16) + G) * up(N, 32))) return DET_GEMM_ERR_INVALID_ARG;    // more tiles than are counted
    const int es = out_fp32 ? 4 : 2;
    const Arr out{C, M, N, ldc, es, 16};
    const int64_t nb = up(K, kBlock);
    det_gemm_status s;
    if (K > 0 && G > 0) {
        if (!sa || !sb || sa_row < 0 || sa_blk < 0 || sb_row < nb ||
            (static_cast<double>(M - 1) * sa_row + static_cast<double>(nb - 1) * sa_blk) * 4 > kMaxBytes)
            return DET_GEMM_ERR_INVALID_ARG;
        if (grouped && !offsets) return DET_GEMM_ERR_INVALID_ARG;
        const Arr as{sa, 1, (M - 1) * sa_row + (nb - 1) * sa_blk + 1, int64_t{1} << 36, 4, 4};
        const Arr bs{sb, up(N, kBlock), nb, sb_row, 4, 4, G, gsb};
        if ((s = check_all({mat8(A, M, K, lda), mat8(W, N, K, ldw, G, gw), as, bs,
                            vec4(offsets, grouped ? G + 1 : 0)}, {out})) != DET_GEMM_OK)
            return s;
    } else if ((s = check(out)) != DET_GEMM_OK) {
        return s;
    }
    Device *d = nullptr;
    if ((s = device(&d)) != DET_GEMM_OK) return s;
    if (K == 0 || G == 0) {
        const cudaError_t e = cudaMemset2DAsync(C, static_cast<size_t>(ldc * es), 0, static_cast<size_t>(N * es),
                                                static_cast<size_t>(M), cs(stream));
        return e == cudaSuccess ? DET_GEMM_OK : fail(DET_GEMM_ERR_LAUNCH, e, "memset");
    }
    const Fp8Args x{A, sa, W, sb, offsets, C, out_fp32, G, M, N, K, lda, ldw, gw, ldc, 0};
    Fp8Params p;
    std::memset(&p, 0, sizeof p);
    p.sa_row = sa_row;
    p.sa_blk = sa_blk;
    p.sb_row = sb_row;
    p.sb_blk = 1;
    p.sb_grp = gsb;
    p.kc = static_cast<int>(K);
    p.max_blocks = static_cast<int>(nb);
    return enqueue(x, p, plan_rows(M, N, G, grouped, d->sms), d, stream);
}

constexpr int64_t kZeroBeside = 128 << 20;    // bytes of the dense gradient zeroed while the tokens are sorted

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

struct GradSpace {
    size_t key[2], idx[2], head, seen, partials, total;
    int64_t ldp;
};
GradSpace grad_space(int64_t T, int64_t V, int64_t H)
{
    GradSpace g;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t r = at;
        at += align256(bytes);
        return r;
    };
    for (int i = 0; i < 2; ++i) {
        g.key[i] = take(4 * T);
        g.idx[i] = take(4 * T);
    }
    g.head = take(4 * T);
    g.seen = take(V);
    g.ldp = up(H, 8) * 8;
    g.partials = take(T > 32 ? 2 * up(T, 32) * g.ldp * 4 : 0);
    g.total = at;
    return g;
}

}  // namespace
}  // namespace deto

using namespace deto;

extern "C" {

det_gemm_status det_moe_route(const void *logits, int logits_fp32, const float *bias, float *weights, int32_t *ids,
                              int64_t T, int64_t E, int64_t ldl, int top_k, int score, int n_groups, int top_groups,
                              int group_best, int renormalize, float scale, det_gemm_stream stream)
{
    if (!ok_size(T) || E < 1 || E > DET_MOE_MAX_EXPERTS || top_k < 1 || top_k > DET_MOE_MAX_TOP_K || top_k > E)
        return DET_GEMM_ERR_INVALID_ARG;
    if (score < 0 || score > 1 || n_groups < 1 || n_groups > DET_MOE_MAX_GROUPS || E % n_groups != 0 || top_groups < 1 ||
        top_groups > n_groups || group_best < 1 || group_best > 2 || E / n_groups * top_groups < top_k)
        return DET_GEMM_ERR_INVALID_ARG;
    if (T == 0) return DET_GEMM_OK;
    const int es = logits_fp32 ? 4 : 2;
    det_gemm_status s = check_all({Arr{logits, T, E, ldl, es, es}, vec4(bias, bias ? E : 0)},
                                  {vec4(weights, T * top_k), vec4(ids, T * top_k)});
    if (s != DET_GEMM_OK) return s;
    Device *d = nullptr;
    if ((s = device(&d)) != DET_GEMM_OK) return s;
    RouteParams p;
    std::memset(&p, 0, sizeof p);
    p.logits = logits;
    p.bias = bias;
    p.weights = weights;
    p.ids = ids;
    p.ldl = ldl;
    p.tokens = static_cast<int>(T);
    p.experts = static_cast<int>(E);
    p.k = top_k;
    p.groups = n_groups;
    p.top_groups = top_groups;
    p.group_mul = (1 << 18) / (static_cast<int>(E) / n_groups) + 1;
    p.group_best = group_best;
    p.renorm = renormalize != 0;
    p.sigmoid = score;
    p.scale = scale;
    const cudaError_t e = logits_fp32 ? launch_route_f32(p, cs(stream)) : launch_route_bf16(p, cs(stream));
    return e == cudaSuccess ? DET_GEMM_OK : fail(DET_GEMM_ERR_LAUNCH, e, "route launch");
}

det_gemm_status det_moe_route_bwd(const float *dweights, const void *logits, int logits_fp32, const int32_t *ids,
                                  void *dlogits, int64_t T, int64_t E, int64_t ldl, int64_t ldd, int top_k, int score,
                                  int renormalize, float scale, det_gemm_stream stream)
{
    if (!ok_size(T) || E < 1 || E > DET_MOE_MAX_EXPERTS || top_k < 1 || top_k > DET_MOE_MAX_TOP_K || top_k > E ||
        score < 0 || score > 1)
        return DET_GEMM_ERR_INVALID_ARG;
    if (T == 0) return DET_GEMM_OK;
    const int es = logits_fp32 ? 4 : 2;
    det_gemm_status s = check_all({Arr{logits, T, E, ldl, es, es}, vec4(dweights, T * top_k), vec4(ids, T * top_k)},
                                  {Arr{dlogits, T, E, ldd, es, es}});
    if (s != DET_GEMM_OK) return s;
    Device *d = nullptr;
    if ((s = device(&d)) != DET_GEMM_OK) return s;
    RouteParams p;
    std::memset(&p, 0, sizeof p);
    p.logits = logits;
    p.dw = dweights;
    p.ids = const_cast<int32_t *>(ids);
    p.dlogits = dlogits;
    p.ldl = ldl;
    p.ldd = ldd;
    p.tokens = static_cast<int>(T);
    p.experts = static_cast<int>(E);
    p.k = top_k;
    p.renorm = renormalize != 0;
    p.sigmoid = score;
    p.scale = scale;
    const cudaError_t e = logits_fp32 ? launch_route_bwd_f32(p, cs(stream)) : launch_route_bwd_bf16(p, cs(stream));
    return e == cudaSuccess ? DET_GEMM_OK : fail(DET_GEMM_ERR_LAUNCH, e, "route gradient launch");
}

det_gemm_status det_moe_dispatch(const int32_t *ids, int32_t *offsets, int32_t *rows, int32_t *slots, int64_t T,
                                 int64_t E, int top_k, det_gemm_stream stream)
{
    if (!ok_size(T) || E < 1 || E > DET_MOE_MAX_EXPERTS || top_k < 1 || top_k > DET_MOE_MAX_TOP_K || !ok_size(T * top_k))
        return DET_GEMM_ERR_INVALID_ARG;
    const int64_t n = T * top_k;
    det_gemm_status s = check_all({vec4(ids, n)}, {vec4(offsets, E + 1), vec4(rows, n), vec4(slots, n)});
    if (s != DET_GEMM_OK) return s;
    Device *d = nullptr;
    if ((s = device(&d)) != DET_GEMM_OK) return s;
    SortParams p;
    std::memset(&p, 0, sizeof p);
    p.keys = ids;
    p.n = static_cast<int>(n);
    p.range = static_cast<int>(E);
    p.passes = 1;
    p.offsets = offsets;
    p.rows = rows;
    p.slots = slots;
    p.skip_key = -1;
    p.status = d->word;
    const cudaError_t e = launch_sort(p, false, cs(stream));
    return e == cudaSuccess ? DET_GEMM_OK : fail(DET_GEMM_ERR_LAUNCH, e, "dispatch launch");
}

det_gemm_status det_moe_gather(const det_gemm_bf16 *x, const int32_t *rows, det_gemm_bf16 *xs, int64_t T, int64_t R,
                               int64_t H, int top_k, int64_t ldx, int64_t ldxs, det_gemm_stream stream)
{
    if (!ok_size(T) || !ok_size(R) || !ok_size(H) || top_k < 1 || !launchable(up(H, 1024) * up(R, 4)))
        return DET_GEMM_ERR_INVALID_ARG;
    if (R == 0 || H == 0) return DET_GEMM_OK;
    det_gemm_status s = check_all({bf16(x, T, H, ldx), vec4(rows, R)}, {bf16(xs, R, H, ldxs)});
    if (s != DET_GEMM_OK) return s;
    Device *d = nullptr;
    if ((s = device(&d)) != DET_GEMM_OK) return s;
    const GatherParams p{x, xs, rows, ldx, ldxs, static_cast<int>(R), static_cast<int>(T), static_cast<int>(H), top_k};
    const cudaError_t e = launch_gather(p, cs(stream));
    return e == cudaSuccess ? DET_GEMM_OK : fail(DET_GEMM_ERR_LAUNCH, e, "gather launch");
}

det_gemm_status det_moe_combine(const det_gemm_bf16 *ys, const int32_t *slots, const float *weights, det_gemm_bf16 *y,
                                int64_t T, int64_t R, int64_t H, int top_k, int64_t ldys, int64_t ldy,
                                det_gemm_stream stream)
{
    if (!ok_size(T) || !ok_size(R) || !ok_size(H) || top_k < 1 || top_k > DET_MOE_MAX_TOP_K ||
        !launchable(up(H, 1024) * T))
        return DET_GEMM_ERR_INVALID_ARG;
    if (T == 0 || H == 0) return DET_GEMM_OK;
    det_gemm_status s = check_all({bf16(ys, R, H, ldys), vec4(slots, T * top_k), vec4(weights, weights ? T * top_k : 0)},
                                  {bf16(y, T, H, ldy)});
    if (s != DET_GEMM_OK) return s;
    Device *d = nullptr;
    if ((s = device(&d)) != DET_GEMM_OK) return s;
    CombineParams p;
    std::memset(&p, 0, sizeof p);
    p.ys = ys;
    p.slots = slots;
    p.weights = weights;
    p.y = y;
    p.ldys = ldys;
    p.ldy = ldy;
    p.tokens = static_cast<int>(T);
    p.k = top_k;
    p.rows_n = static_cast<int>(R);
    p.cols = static_cast<int>(H);
    const cudaError_t e = launch_combine(p, cs(stream));
    return e == cudaSuccess ? DET_GEMM_OK : fail(DET_GEMM_ERR_LAUNCH, e, "combine launch");
}

det_gemm_status det_moe_combine_bwd(const det_gemm_bf16 *dy, const det_gemm_bf16 *ys, const int32_t *rows,
                                    const int32_t *slots, const float *weights, det_gemm_bf16 *dys, float *dweights,
                                    int64_t T, int64_t H, int top_k, int64_t lddy, int64_t ldys, int64_t lddys,
                                    det_gemm_stream stream)
{
    if (!ok_size(T) || !ok_size(H) || top_k < 1 || top_k > DET_MOE_MAX_TOP_K || !ok_size(T * top_k))
        return DET_GEMM_ERR_INVALID_ARG;
    const int64_t R = T * top_k;
    if (T == 0) return DET_GEMM_OK;
    det_gemm_status s = check_all({bf16(dy, T, H, lddy), bf16(ys, R, H, ldys), vec4(rows, R), vec4(slots, R), vec4(weights, R)},
                                  {bf16(dys, R, H, lddys), vec4(dweights, R)});
    if (s != DET_GEMM_OK) return s;
    Device *d = nullptr;
    if ((s = device(&d)) != DET_GEMM_OK) return s;
    CombineParams p;
    std::memset(&p, 0, sizeof p);
    p.ys = ys;
    p.dy = dy;
    p.rows = rows;
    p.slots = slots;
    p.weights = weights;
    p.dys = dys;
    p.dw = dweights;
    p.ldys = ldys;
    p.lddy = lddy;
    p.lddys = lddys;
    p.tokens = static_cast<int>(T);
    p.k = top_k;
    p.rows_n = static_cast<int>(R);
    p.cols = static_cast<int>(H);
    const cudaError_t e = launch_combine_bwd(p, cs(stream));
    return e == cudaSuccess ? DET_GEMM_OK : fail(DET_GEMM_ERR_LAUNCH, e, "combine gradient launch");
}

det_gemm_status det_fp8_quantize_rows(const det_gemm_bf16 *x, const int32_t *rows, uint8_t *q, float *s, int64_t T,
                                      int64_t M, int64_t K, int top_k, int64_t ldx, int64_t ldq, int64_t lds,
                                      det_gemm_stream stream)
{
    if (!ok_size(T) || !ok_size(M) || !ok_size(K) || top_k < 1 || (!rows && M != T) ||
        !launchable(up(up(K, 256) * M, 4)))
        return DET_GEMM_ERR_INVALID_ARG;
    if (M == 0 || K == 0) return DET_GEMM_OK;
    det_gemm_status st = check_all({bf16(x, T, K, ldx), vec4(rows, rows ? M : 0)},
                                   {mat8(q, M, K, ldq), Arr{s, up(K, kBlock), M, lds, 4, 4}});
    if (st != DET_GEMM_OK) return st;
    Device *d = nullptr;
    if ((st = device(&d)) != DET_GEMM_OK) return st;
    QuantParams p;
    std::memset(&p, 0, sizeof p);
    p.x = x;
    p.rows = rows;
    p.q = q;
    p.s = s;
    p.ldx = ldx;
    p.ldq = ldq;
    p.lds = lds;
    p.n = static_cast<int>(M);
    p.src_rows = static_cast<int>(T);
    p.cols = static_cast<int>(K);
    p.k = top_k;
    const cudaError_t e = launch_quantize_rows(p, cs(stream));
    return e == cudaSuccess ? DET_GEMM_OK : fail(DET_GEMM_ERR_LAUNCH, e, "quantiser launch");
}

det_gemm_status det_fp8_quantize_cols(const det_gemm_bf16 *x, const int32_t *offsets, uint8_t *qt, float *s, int64_t M,
                                      int64_t K, int64_t G, int64_t max_blocks, int64_t ldx, int64_t ldqt, int64_t lds,
                                      det_gemm_stream stream)
{
    if (!ok_size(M) || !ok_size(K) || G < 0 || G > DET_MOE_MAX_EXPERTS || max_blocks < up(M, kBlock) + (offsets ? G : 0) ||
        !launchable(up(K, 64) * max_blocks))
        return DET_GEMM_ERR_INVALID_ARG;
    if (M == 0 || K == 0) return DET_GEMM_OK;
    const int64_t blocks = offsets ? max_blocks : up(M, kBlock);
    det_gemm_status st = check_all({bf16(x, M, K, ldx), vec4(offsets, offsets ? G + 1 : 0)},
                                   {mat8(qt, K, blocks * kBlock, ldqt), Arr{s, blocks, K, lds, 4, 4}});
    if (st != DET_GEMM_OK) return st;
    Device *d = nullptr;
    if ((st = device(&d)) != DET_GEMM_OK) return st;
    QuantParams p;
    std::memset(&p, 0, sizeof p);
    p.x = x;
    p.offsets = offsets;
    p.q = qt;
    p.s = s;
    p.ldx = ldx;
    p.ldq = ldqt;
    p.lds = lds;
    p.n = static_cast<int>(M);
    p.cols = static_cast<int>(K);
    p.groups = static_cast<int>(G);
    p.max_blocks = static_cast<int>(blocks);
    p.status = d->word;
    const cudaError_t e = launch_quantize_cols(p, cs(stream));
    return e == cudaSuccess ? DET_GEMM_OK : fail(DET_GEMM_ERR_LAUNCH, e, "column quantiser launch");
}

det_gemm_status det_fp8_quantize_tiles(const det_gemm_bf16 *w, uint8_t *q, float *s, uint8_t *qt, float *st, int64_t G,
                                       int64_t N, int64_t K, int64_t ldw, int64_t gw, int64_t ldq, int64_t gq,
                                       int64_t ldqt, int64_t gqt, det_gemm_stream stream)
{
    if (!ok_size(N) || !ok_size(K) || G < 0 || G > kMaxRows || (q == nullptr) != (s == nullptr) ||
        (qt == nullptr) != (st == nullptr))
        return DET_GEMM_ERR_INVALID_ARG;
    if (N == 0 || K == 0 || G == 0 || (!q && !qt)) return DET_GEMM_OK;
    const int64_t rt = up(N, kBlock), ct = up(K, kBlock);
    if (!launchable(rt * ct) || !launchable(rt * ct * G)) return DET_GEMM_ERR_INVALID_ARG;
    Arr x = bf16(w, N, K, ldw);
    x.mats = G;
    x.gap = gw;
    det_gemm_status r = check_all({x}, {mat8(q, q ? N : 0, K, ldq, G, gq), Arr{s, q ? G : 0, rt * ct, rt * ct, 4, 4},
                                        mat8(qt, qt ? K : 0, N, ldqt, G, gqt), Arr{st, qt ? G : 0, rt * ct, rt * ct, 4, 4}});
    if (r != DET_GEMM_OK) return r;
    Device *d = nullptr;
    if ((r = device(&d)) != DET_GEMM_OK) return r;
    QuantParams p;
    std::memset(&p, 0, sizeof p);
    p.x = w;
    p.q = q;
    p.s = s;
    p.qt = qt;
    p.st = st;
    p.ldx = ldw;
    p.xg = gw;
    p.ldq = ldq;
    p.qg = gq;
    p.ldqt = ldqt;
    p.qtg = gqt;
    p.lds = ct;
    p.sg = rt * ct;
    p.ldst = rt;
    p.stg = rt * ct;
    p.n = static_cast<int>(N);
    p.cols = static_cast<int>(K);
    p.groups = static_cast<int>(G);
    const cudaError_t e = launch_quantize_tiles(p, cs(stream));
    return e == cudaSuccess ? DET_GEMM_OK : fail(DET_GEMM_ERR_LAUNCH, e, "tile quantiser launch");
}

det_gemm_status det_fp8_gemm(const uint8_t *A, const float *sa, const uint8_t *W, const float *sb, void *C,
                             int out_fp32, int64_t M, int64_t N, int64_t K, int64_t lda, int64_t sa_row,
                             int64_t sa_blk, int64_t ldw, int64_t sb_row, int64_t ldc, det_gemm_stream stream)
{
    return fp8_rows(A, sa, W, sb, nullptr, C, out_fp32, 1, M, N, K, lda, sa_row, sa_blk, ldw, 0, sb_row, 0, ldc, false,
                    stream);
}

det_gemm_status det_fp8_gemm_grouped(const uint8_t *A, const float *sa, const uint8_t *W, const float *sb,
                                     const int32_t *offsets, void *C, int out_fp32, int64_t G, int64_t M, int64_t N,
                                     int64_t K, int64_t lda, int64_t sa_row, int64_t sa_blk, int64_t ldw, int64_t gw,
                                     int64_t sb_row, int64_t gsb, int64_t ldc, det_gemm_stream stream)
{
    return fp8_rows(A, sa, W, sb, offsets, C, out_fp32, G, M, N, K, lda, sa_row, sa_blk, ldw, gw, sb_row, gsb, ldc, true,
                    stream);
}

det_gemm_status det_fp8_gemm_wgrad(const uint8_t *Yt, const float *sy, const uint8_t *Xt, const float *sx,
                                   const int32_t *offsets, void *dW, int out_fp32, int64_t G, int64_t M, int64_t N,
                                   int64_t K, int64_t max_blocks, int64_t ldyt, int64_t ldsy, int64_t ldxt,
                                   int64_t ldsx, int64_t lddw, int64_t gdw, det_gemm_stream stream)
{
    if (!ok_size(M) || !ok_size(N) || !ok_size(K) || G < 0 || G > DET_MOE_MAX_EXPERTS || (!offsets && G != 1) ||
        max_blocks < up(M, kBlock) + (offsets ? G : 0) || !ok_size(max_blocks * kBlock) || !launchable(G * (up(M, kBlock) + 1)))
        return DET_GEMM_ERR_INVALID_ARG;
    if (N == 0 || K == 0 || G == 0) return DET_GEMM_OK;
    if (!launchable(up(N, 128) * up(K, 128) * G)) return DET_GEMM_ERR_INVALID_ARG;
    const int64_t blocks = offsets ? max_blocks : up(M, kBlock);
    const int es = out_fp32 ? 4 : 2;
    const Arr out{dW, N, K, lddw, es, 16, G, gdw};
    det_gemm_status s;
    if (M > 0)
        s = check_all({mat8(Yt, N, blocks * kBlock, ldyt), Arr{sy, blocks, N, ldsy, 4, 16},
                       mat8(Xt, K, blocks * kBlock, ldxt), Arr{sx, blocks, K, ldsx, 4, 16},
                       vec4(offsets, offsets ? G + 1 : 0)}, {out});
    else
        s = check(out);
    if (s != DET_GEMM_OK) return s;
    Device *d = nullptr;
    if ((s = device(&d)) != DET_GEMM_OK) return s;
    if (M == 0) {
        for (int64_t g = 0; g < G; ++g) {
            const cudaError_t e = cudaMemset2DAsync(static_cast<uint8_t *>(dW) + g * gdw * es, static_cast<size_t>(lddw * es),
                                                    0, static_cast<size_t>(K * es), static_cast<size_t>(N), cs(stream));
            if (e != cudaSuccess) return fail(DET_GEMM_ERR_LAUNCH, e, "memset");
        }
        return DET_GEMM_OK;
    }
    const Fp8Args x{Yt, sy, Xt, sx, offsets, dW, out_fp32, G, N, K, blocks * kBlock, ldyt, ldxt, 0, lddw, gdw,
                    ldsy, ldsx};
    Fp8Params p;
    std::memset(&p, 0, sizeof p);
    p.kc = static_cast<int>(M);
    p.max_blocks = static_cast<int>(blocks);
    // Always the wide tile: a block takes an epilogue warp 395 ns whether the
    // tile has eight or twelve of them ([2432, 3648] from 8192 tokens: four rounds
    // of 128 columns 112 us, three of 192 columns 90; where one round is enough,
    // [1000, 1000] from 4096, 17.7 and 18.6).
    const Fp8Plan plan{kFp8Wgrad, false, 128, 192};
    return enqueue(x, p, plan, d, stream);
}

det_gemm_status det_embedding(const void *tokens, int tokens64, const det_gemm_bf16 *table, det_gemm_bf16 *out,
                              int64_t T, int64_t V, int64_t H, float scale, int64_t ldt, int64_t ldo,
                              det_gemm_stream stream)
{
    if (!ok_size(T) || !ok_size(V) || !ok_size(H) || !launchable(up(H, 1024) * T)) return DET_GEMM_ERR_INVALID_ARG;
    if (T == 0 || H == 0) return DET_GEMM_OK;
    const int es = tokens64 ? 8 : 4;
    det_gemm_status s = check_all({Arr{tokens, 1, T, T, es, es}, bf16(table, V, H, ldt)}, {bf16(out, T, H, ldo)});
    if (s != DET_GEMM_OK) return s;
    Device *d = nullptr;
    if ((s = device(&d)) != DET_GEMM_OK) return s;
    const EmbedParams p{tokens, tokens64 != 0, table, out, ldt, ldo, static_cast<int>(T), static_cast<int>(V),
                        static_cast<int>(H), scale, d->word};
    const cudaError_t e = launch_embedding(p, cs(stream));
    return e == cudaSuccess ? DET_GEMM_OK : fail(DET_GEMM_ERR_LAUNCH, e, "embedding launch");
}

int64_t det_embedding_grad_workspace(int64_t T, int64_t V, int64_t H)
{
    if (!ok_size(T) || !ok_size(V) || !ok_size(H)) return 0;
    return static_cast<int64_t>(grad_space(T, V, H).total);
}

det_gemm_status det_embedding_grad(const det_gemm_bf16 *dy, const void *tokens, int tokens64, void *dtable,
                                   int out_fp32, int64_t T, int64_t V, int64_t H, float scale, int64_t padding_idx,
                                   int accumulate, int64_t lddy, int64_t ldd, void *workspace, int64_t workspace_bytes,
                                   det_gemm_stream stream)
{
    if (!ok_size(T) || !ok_size(V) || !ok_size(H) || V > (int64_t{1} << 27) - 2 || padding_idx < -1 || padding_idx >= V ||
        !launchable(up(H, 1024) * (T + up(V, 8))))
        return DET_GEMM_ERR_INVALID_ARG;
    if (V == 0 || H == 0 || (T == 0 && accumulate)) return DET_GEMM_OK;
    const int es = tokens64 ? 8 : 4, ds = out_fp32 ? 4 : 2;
    const GradSpace g = grad_space(T, V, H);
    const Arr ws{workspace, 1, static_cast<int64_t>(g.total), static_cast<int64_t>(g.total + 255) / 256 * 256, 1, 256};
    det_gemm_status s = check_all({bf16(dy, T, H, lddy), Arr{tokens, 1, T, T, es, es}},
                                  {Arr{dtable, V, H, ldd, ds, 16}, ws});
    if (s != DET_GEMM_OK) return s;
    if (workspace_bytes < static_cast<int64_t>(g.total)) return DET_GEMM_ERR_INVALID_ARG;
    Device *d = nullptr;
    if ((s = device(&d)) != DET_GEMM_OK) return s;
    uint8_t *w = static_cast<uint8_t *>(workspace);
    SortParams p;
    std::memset(&p, 0, sizeof p);
    p.keys = tokens;
    p.keys64 = tokens64 != 0;
    p.n = static_cast<int>(T);
    p.range = static_cast<int>(V);
    p.passes = 1;
    while ((int64_t{1} << (9 * p.passes)) < V + 1) ++p.passes;
    for (int i = 0; i < 2; ++i) {
        p.kbuf[i] = reinterpret_cast<int32_t *>(w + g.key[i]);
        p.ibuf[i] = reinterpret_cast<int32_t *>(w + g.idx[i]);
    }
    p.head = reinterpret_cast<int32_t *>(w + g.head);
    if (!accumulate) {
        p.zero = dtable;
        p.zero_rows = std::min<int64_t>(V, kZeroBeside / (H * ds));
        p.zero_cols = H * ds;
        p.zero_pitch = ldd * ds;
    }
    p.sms = d->sms;
    p.seen = w + g.seen;
    p.skip_key = static_cast<int>(padding_idx);
    p.status = d->word;
    p.flag_bad = 1;
    cudaError_t e = launch_sort(p, true, cs(stream));
    if (e != cudaSuccess) return fail(DET_GEMM_ERR_LAUNCH, e, "sort launch");
    EmbedGradParams q;
    std::memset(&q, 0, sizeof q);
    q.dy = dy;
    q.dtable = dtable;
    q.lddy = lddy;
    q.ldd = ldd;
    q.n = static_cast<int>(T);
    q.vocab = static_cast<int>(V);
    q.cols = static_cast<int>(H);
    q.scale = scale;
    q.accumulate = accumulate != 0;
    q.fp32 = out_fp32 != 0;
    q.keys = p.kbuf[(p.passes - 1) & 1];
    q.order = p.ibuf[(p.passes - 1) & 1];
    q.head = p.head;
    q.seen = p.seen;
    q.zero_from = static_cast<int>(accumulate ? V : p.zero_rows);
    q.partials = reinterpret_cast<float *>(w + g.partials);
    q.ldp = g.ldp;
    e = launch_embedding_grad(q, cs(stream));
    return e == cudaSuccess ? DET_GEMM_OK : fail(DET_GEMM_ERR_LAUNCH, e, "embedding gradient launch");
}

det_gemm_status det_ops_check(det_gemm_stream stream)
{
    Device *d = nullptr;
    const det_gemm_status s = device(&d);
    if (s != DET_GEMM_OK) return s;
    int code = 0;
    const int zero = 0;
    if (cudaStreamSynchronize(cs(stream)) != cudaSuccess ||
        cudaMemcpyFromSymbol(&code, g_ops_status, sizeof code) != cudaSuccess ||
        (code != 0 && cudaMemcpyToSymbol(g_ops_status, &zero, sizeof zero) != cudaSuccess)) {
        cudaGetLastError();
        return DET_GEMM_ERR_CUDA;
    }
    return static_cast<det_gemm_status>(code);
}

det_gemm_status det_ops_debug_force_timeout(int enable)
{
    g_force_timeout.store(enable != 0);
    return DET_GEMM_OK;
}

}  // extern "C"
