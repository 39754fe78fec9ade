// C entry points of include/det_attn.h: argument checks and launches.
#include "det_attn.h"
#include "attn_internal.h"
#include "det_gemm_internal.h"
#include "ops_host.h"

#include <algorithm>
#include <cmath>
#include <cstring>

namespace deto {
namespace {

// An array of rows of D BF16 values with up to three strided axes.
struct Strided {
    const void *p;
    int64_t n[3], stride[3];
    int64_t D;
    bool empty() const { return n[0] <= 0 || n[1] <= 0 || n[2] <= 0; }
};

Strided heads(const void *p, int64_t T, int64_t H, int64_t D, int64_t t, int64_t h) { return Strided{p, {T, H, 1}, {t, h, 0}, D}; }

// Rows that do not overlap, on 16 bytes.
det_gemm_status check(const Strided &a)
{
    if (a.empty()) return DET_GEMM_OK;
    if (!a.p) return DET_GEMM_ERR_INVALID_ARG;
    int order[3] = {0, 1, 2};
    std::sort(order, order + 3, [&](int x, int y) { return a.stride[x] < a.stride[y]; });
    double span = static_cast<double>(a.D);
    for (int i : order) {
        if (a.n[i] == 1) continue;
        if (a.stride[i] > (int64_t{1} << 38) || static_cast<double>(a.stride[i]) < span) return DET_GEMM_ERR_INVALID_ARG;
        span += static_cast<double>(a.n[i] - 1) * static_cast<double>(a.stride[i]);
        if (span * 2 > kMaxBytes) return DET_GEMM_ERR_INVALID_ARG;
    }
    if (reinterpret_cast<uintptr_t>(a.p) % 16 != 0) return DET_GEMM_ERR_ALIGNMENT;
    for (int i = 0; i < 3; ++i)
        if (a.n[i] > 1 && a.stride[i] % 8 != 0) return DET_GEMM_ERR_ALIGNMENT;
    return DET_GEMM_OK;
}

struct Range {
    uintptr_t lo, hi;
};
Range range(const Strided &a)
{
    const uintptr_t p = reinterpret_cast<uintptr_t>(a.p);
    if (a.empty() || !a.p) return Range{0, 0};
    int64_t e = a.D;
    for (int i = 0; i < 3; ++i)
        if (a.n[i] > 1) e += (a.n[i] - 1) * a.stride[i];
    return Range{p, p + static_cast<uintptr_t>(e) * 2};
}
Range range(const Arr &a)
{
    const uintptr_t p = reinterpret_cast<uintptr_t>(a.p);
    return a.empty() || !a.p ? Range{0, 0} : Range{p, p + static_cast<uintptr_t>(a.bytes())};
}
bool overlap(const Range &a, const Range &b) { return a.lo < b.hi && b.lo < a.hi; }

// Whether two arrays of one shape and layout lie between one another, as keys and values do that share each page, token or head of
// a buffer: b begins in a place that an axis of a leaves free.
bool interleaved(const Strided &a, const Strided &b)
{
    if (a.D != b.D || !std::equal(a.n, a.n + 3, b.n) || !std::equal(a.stride, a.stride + 3, b.stride)) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    int64_t off = static_cast<int64_t>((x < y ? y - x : x - y) / 2), span = a.D, inner[3];
    int order[3] = {0, 1, 2};
    std::sort(order, order + 3, [&](int i, int j) { return a.stride[i] < a.stride[j]; });
    for (int i : order) {
        inner[i] = span;
        if (a.n[i] > 1) span += (a.n[i] - 1) * a.stride[i];
    }
    for (int k = 2; k >= 0; --k) {
        const int i = order[k];
        if (a.n[i] == 1) continue;
        off %= a.stride[i];
        if (off + inner[i] > a.stride[i]) return false;
        if (off >= inner[i]) return true;
    }
    return false;
}

// All arrays well formed, and no output overlapping an input or another output.
det_gemm_status check_all(std::initializer_list<Strided> in, std::initializer_list<Arr> flat_in, std::initializer_list<Strided> out,
                          std::initializer_list<Arr> flat_out)
{
    det_gemm_status s;
    Range ins[16], outs[8];
    int ni = 0, no = 0;
    for (const Strided &a : in) {
        if ((s = check(a)) != DET_GEMM_OK) return s;
        ins[ni++] = range(a);
    }
    for (const Arr &a : flat_in) {
        if ((s = check(a)) != DET_GEMM_OK) return s;
        ins[ni++] = range(a);
    }
    for (const Strided &a : out) {
        if ((s = check(a)) != DET_GEMM_OK) return s;
        outs[no++] = range(a);
    }
    for (const Arr &a : flat_out) {
        if ((s = check(a)) != DET_GEMM_OK) return s;
        outs[no++] = range(a);
    }
    for (int o = 0; o < no; ++o) {
        for (int i = 0; i < ni; ++i)
            if (overlap(outs[o], ins[i])) return DET_GEMM_ERR_INVALID_ARG;
        for (int i = 0; i < o; ++i)
            if (overlap(outs[o], outs[i]) && !(o < static_cast<int>(out.size()) && interleaved(out.begin()[o], out.begin()[i])))
                return DET_GEMM_ERR_INVALID_ARG;
    }
    return DET_GEMM_OK;
}

Heads on(const void *p, int64_t t, int64_t h) { return Heads{static_cast<uint16_t *>(const_cast<void *>(p)), t, h}; }
Cache on(const void *p, int64_t page, int64_t s, int64_t h) { return Cache{static_cast<uint16_t *>(const_cast<void *>(p)), page, s, h}; }
Arr table(const float *p, int64_t rows, int64_t cols, int64_t ld) { return Arr{p, rows, cols, ld, 4, 4}; }
Arr bytes(void *p, int64_t n) { return Arr{p, 1, n, up(n, 256) * 256, 1, 256}; }

bool ok_heads(int64_t H, int64_t KV, int64_t D)
{
    return KV >= 1 && H >= KV && H <= DET_ATTN_MAX_HEADS && H % KV == 0 && D >= 8 && D <= DET_ATTN_MAX_HEAD_DIM && D % 8 == 0;
}
// (The kernels' scores are in units of log2: scale times log2(e), which has to be a number too.)
bool ok_mask(float scale, int64_t window, int64_t sinks)
{
    return scale > 0.0f && std::isfinite(scale * 1.4426950408889634f) && window >= 0 && sinks >= 0;
}
int window_of(int64_t w) { return w == 0 || w > kMaxRows ? kNoWindow : static_cast<int>(w); }
int sinks_of(int64_t s) { return static_cast<int>(std::min(s, kMaxRows)); }

// Heads as (column, head, token), copied in boxes of 64 columns of one head and 128 tokens.
bool encode(CUtensorMap *m, const void *p, int64_t T, int64_t H, int64_t D, int64_t t, int64_t h, int box_heads = 1, int box_tokens = 128)
{
    std::memset(m, 0, sizeof *m);
    if (T == 0) return true;                   // nothing will be copied
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(T)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(H > 1 ? h : D) * 2, static_cast<cuuint64_t>(T > 1 ? t : H * D) * 2};
    cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_tokens)}, es[3] = {1, 1, 1};
    return tensor_map_encoder()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(p), dims, strides, box, es,
                                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
det_gemm_status no_map()
{
    detg::record_detail("tensor map");
    return DET_GEMM_ERR_LAUNCH;
}

// (The launch counts blocks of 256 items, at most 128 a head.)
bool ok_turn(int64_t T, int64_t heads, int64_t D, int64_t rot, int64_t P)
{
    if (!launchable(T * heads / 2 + 1)) return false;
    return D >= 8 && D <= DET_ATTN_MAX_HEAD_DIM && D % 8 == 0 && rot >= 2 && rot <= D && rot % 2 == 0 && ok_size(P);
}

// Device memory of the backward pass: delta [H, T], then the first keys' pieces.
struct BwdSpace {
    int64_t partials, total;
};
BwdSpace bwd_space(int64_t N, int64_t T, int64_t H, int64_t KV, int64_t D, int64_t window, int64_t sinks)
{
    const int64_t delta = up(std::max<int64_t>(4 * T * H, 1), 256) * 256;
    return BwdSpace{delta, delta + piece_slots(T, N, true) * sink_blocks(window, sinks) * KV * 2 * 128 * D * 4};
}

// Decode: the query heads of a KV head are taken up to 32 at once; device memory of the cuts between CTAs, and of what
// they leave in parts.
constexpr int64_t kMaxCtas = 160, kTokens = 128;
struct DecodeSpace {
    int64_t parts, heads, partials, total;
};
DecodeSpace decode_space(int64_t B, int64_t H, int64_t KV, int64_t D, int64_t tokens)
{
    DecodeSpace s;
    s.parts = up(H / KV, 32);
    s.heads = up(H / KV, s.parts);
    s.partials = up(kMaxCtas * static_cast<int64_t>(sizeof(Cut)), 256) * 256;
    s.total = s.partials + up(decode_slots(B * KV * s.parts, tokens, kMaxCtas) * s.heads * (D + 2) * 4, 256) * 256;
    return s;
}

// A cache as (column, head, token of a page, page), copied in boxes of 64 columns of one head and `box` tokens of a page. Where
// a head's row is 128 bytes, no more than that is fetched (256, with the next head's: 69.8 instead of 67.7 us, then, for 96 windows of
// 1024 in eight heads of 64; rows of 256 bytes by 128: 222 instead of 218 us for 64 contexts up to 8192).
bool encode(CUtensorMap *m, const void *p, int64_t pages, int64_t size, int64_t KV, int64_t D, int64_t page, int64_t s, int64_t h, int box)
{
    std::memset(m, 0, sizeof *m);
    if (pages == 0) return true;               // nothing will be copied
    cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(KV), static_cast<cuuint64_t>(size), static_cast<cuuint64_t>(pages)};
    cuuint64_t strides[3] = {static_cast<cuuint64_t>(KV > 1 ? h : D) * 2, static_cast<cuuint64_t>(size > 1 ? s : D) * 2,
                             static_cast<cuuint64_t>(pages > 1 ? page : D) * 2};
    cuuint32_t boxes[4] = {64, 1, static_cast<cuuint32_t>(box), 1}, es[4] = {1, 1, 1, 1};
    return tensor_map_encoder()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(p), dims, strides, boxes, es,
                                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, D <= 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace deto

using namespace deto;

extern "C" {

det_gemm_status det_rope(const det_gemm_bf16 *x, const float *cosine, const float *sine, const int32_t *positions,
                         det_gemm_bf16 *y, int64_t T, int64_t H, int64_t D, int64_t rot, int64_t P, int interleaved,
                         int inverse, int64_t xt, int64_t xh, int64_t ldt, int64_t yt, int64_t yh, det_gemm_stream stream)
{
    if (!ok_size(T) || H < 0 || H > DET_ATTN_MAX_HEADS || !ok_turn(T, H, D, rot, P)) return DET_GEMM_ERR_INVALID_ARG;
    if (T == 0 || H == 0) return DET_GEMM_OK;
    const Strided in = heads(x, T, H, D, xt, xh), out = heads(y, T, H, D, yt, yh);
    const bool place = x == y && (T == 1 || xt == yt) && (H == 1 || xh == yh);
    const Arr c = table(cosine, P, rot / 2, ldt), sn = table(sine, P, rot / 2, ldt), pos = vec4(positions, T);
    det_gemm_status s = place ? check_all({}, {c, sn, pos}, {out}, {}) : check_all({in}, {c, sn, pos}, {out}, {});
    if (s != DET_GEMM_OK) return s;
    Device *d = nullptr;
    if ((s = device(&d)) != DET_GEMM_OK) return s;
    RopeParams p;
    std::memset(&p, 0, sizeof p);
    p.q = on(x, xt, xh);
    p.out = on(y, yt, yh);
    p.cosine = cosine;
    p.sine = sine;
    p.pos = positions;
    p.ldt = ldt;
    p.T = static_cast<int>(T);
    p.H = static_cast<int>(H);
    p.D = static_cast<int>(D);
    p.rot = static_cast<int>(rot);
    p.P = static_cast<int>(P);
    p.sign = inverse ? -1.0f : 1.0f;
    p.status = d->word;
    const cudaError_t e = launch_rope(p, interleaved != 0, cs(stream));
    return e == cudaSuccess ? DET_GEMM_OK : fail(DET_GEMM_ERR_LAUNCH, e, "rotation launch");
}

det_gemm_status det_kv_append(const det_gemm_bf16 *q, const det_gemm_bf16 *k, const det_gemm_bf16 *v, const float *cosine,
                              const float *sine, const int32_t *positions, const int32_t *slots, det_gemm_bf16 *q_out,
                              det_gemm_bf16 *k_cache, det_gemm_bf16 *v_cache, int64_t T, int64_t H, int64_t KV, int64_t D,
                              int64_t rot, int64_t P, int64_t pages, int64_t page_size, int interleaved, int64_t qt,
                              int64_t qh, int64_t kt, int64_t kh, int64_t vt, int64_t vh, int64_t ldt, int64_t ot,
                              int64_t oh, int64_t kcp, int64_t kcs, int64_t kch, int64_t vcp, int64_t vcs, int64_t vch,
                              det_gemm_stream stream)
{
    if (!ok_size(T) || H < 0 || H > DET_ATTN_MAX_HEADS || KV < 1 || KV > DET_ATTN_MAX_HEADS || !ok_turn(T, H + 2 * KV, D, rot, P) ||
        !ok_size(pages) || page_size < 1 || !ok_size(page_size) || !ok_size(pages * page_size))
        return DET_GEMM_ERR_INVALID_ARG;
    if (T == 0) return DET_GEMM_OK;
    const int64_t hq = q ? H : 0;
    const Strided kc{k_cache, {pages, page_size, KV}, {kcp, kcs, kch}, D}, vc{v_cache, {pages, page_size, KV}, {vcp, vcs, vch}, D};
    det_gemm_status s = check_all({heads(q, T, hq, D, qt, qh), heads(k, T, KV, D, kt, kh), heads(v, T, KV, D, vt, vh)},
                                  {table(cosine, P, rot / 2, ldt), table(sine, P, rot / 2, ldt), vec4(positions, T), vec4(slots, T)},
                                  {heads(q_out, T, hq, D, ot, oh), kc, vc}, {});
    if (s != DET_GEMM_OK) return s;
    Device *d = nullptr;
    if ((s = device(&d)) != DET_GEMM_OK) return s;
    RopeParams p;
    std::memset(&p, 0, sizeof p);
    p.q = on(q, qt, qh);
    p.k = on(k, kt, kh);
    p.v = on(v, vt, vh);
    p.out = on(q_out, ot, oh);
    p.kc = on(k_cache, kcp, kcs, kch);
    p.vc = on(v_cache, vcp, vcs, vch);
    p.cosine = cosine;
    p.sine = sine;
    p.pos = positions;
    p.slots = slots;
    p.ldt = ldt;
    p.T = static_cast<int>(T);
    p.H = static_cast<int>(hq);
    p.KV = static_cast<int>(KV);
    p.D = static_cast<int>(D);
    p.rot = static_cast<int>(rot);
    p.P = static_cast<int>(P);
    p.pages = static_cast<int>(pages);
    p.page_size = static_cast<int>(page_size);
    p.sign = 1.0f;
    p.status = d->word;
    const cudaError_t e = launch_rope(p, interleaved != 0, cs(stream));
    return e == cudaSuccess ? DET_GEMM_OK : fail(DET_GEMM_ERR_LAUNCH, e, "append launch");
}

int64_t det_attn_decode_workspace(int64_t B, int64_t H, int64_t KV, int64_t D, int64_t max_tokens)
{
    if (!ok_size(B) || !ok_heads(H, KV, D) || !ok_size(B * H) || !ok_size(max_tokens)) return 0;
    return decode_space(B, H, KV, D, max_tokens).total;
}

det_gemm_status det_attn_decode(const det_gemm_bf16 *q, const det_gemm_bf16 *k_cache, const det_gemm_bf16 *v_cache,
                                const int32_t *table, const int32_t *lengths, det_gemm_bf16 *out, int64_t B, int64_t H,
                                int64_t KV, int64_t D, int64_t pages, int64_t page_size, int64_t max_pages, float scale,
                                int64_t window, int64_t sinks, int64_t qt, int64_t qh, int64_t kcp, int64_t kcs,
                                int64_t kch, int64_t vcp, int64_t vcs, int64_t vch, int64_t ldt, int64_t ot, int64_t oh,
                                void *workspace, int64_t workspace_bytes, det_gemm_stream stream)
{
    if (!ok_size(B) || !ok_heads(H, KV, D) || !ok_size(B * H) || H / KV > DET_ATTN_MAX_SHARED || !ok_size(pages) || page_size < 8 ||
        page_size % 8 != 0 || !ok_size(page_size) || !ok_size(pages * page_size) || !ok_size(max_pages) ||
        !ok_size(max_pages * page_size) || !ok_mask(scale, window, sinks))
        return DET_GEMM_ERR_INVALID_ARG;
    if (B == 0) return DET_GEMM_OK;
    const DecodeSpace space = decode_space(B, H, KV, D, max_pages * page_size);
    const int64_t need = space.total;
    const Strided kc{k_cache, {pages, page_size, KV}, {kcp, kcs, kch}, D}, vc{v_cache, {pages, page_size, KV}, {vcp, vcs, vch}, D};
    det_gemm_status s = check_all({heads(q, B, H, D, qt, qh), kc, vc}, {Arr{table, B, max_pages, ldt, 4, 4}, vec4(lengths, B)},
                                  {heads(out, B, H, D, ot, oh)}, {bytes(workspace, need)});
    if (s != DET_GEMM_OK) return s;
    if (workspace_bytes < need) return DET_GEMM_ERR_INVALID_ARG;
    Device *d = nullptr;
    if ((s = device(&d)) != DET_GEMM_OK) return s;
    DecodeParams p;
    std::memset(&p, 0, sizeof p);
    p.q = on(q, qt, qh);
    p.out = on(out, ot, oh);
    p.table = table;
    p.lengths = lengths;
    p.ldt = ldt;
    p.B = static_cast<int>(B);
    p.H = static_cast<int>(H);
    p.KV = static_cast<int>(KV);
    p.G = static_cast<int>(H / KV);
    p.D = static_cast<int>(D);
    p.pages = static_cast<int>(pages);
    p.page_size = static_cast<int>(page_size);
    p.max_pages = static_cast<int>(max_pages);
    p.scale = scale;
    p.window = window_of(window);
    p.sinks = sinks_of(sinks);
    p.parts = static_cast<int>(space.parts);
    p.heads = static_cast<int>(space.heads);
    p.box = static_cast<int>(std::min<int64_t>(page_size & -page_size, kTokens));
    p.cuts = static_cast<Cut *>(workspace);
    p.partials = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + space.partials);
    p.status = d->word;
    p.timeout_ns = timeout_ns();
    p.force_timeout = timeout_forced();
    DecodeMaps maps;
    if (!encode(&maps.q, q, B, H, D, qt, qh, space.heads <= 16 ? 16 : 32, 1) ||
        !encode(&maps.k, k_cache, pages, page_size, KV, D, kcp, kcs, kch, p.box) ||
        !encode(&maps.v, v_cache, pages, page_size, KV, D, vcp, vcs, vch, p.box))
        return no_map();
    const int64_t most = B * KV * space.parts * up(std::max<int64_t>(max_pages * page_size, 1), kChunk);
    const cudaError_t e = launch_attn_decode(p, maps, static_cast<int>(std::min({most, static_cast<int64_t>(d->sms), kMaxCtas})), cs(stream));
    return e == cudaSuccess ? DET_GEMM_OK : fail(DET_GEMM_ERR_LAUNCH, e, "decode attention launch");
}

static det_gemm_status ok_attn(const int32_t *q_bounds, const int32_t *k_bounds, int64_t N, int64_t T, int64_t S, int64_t H,
                               int64_t KV, int64_t D, float scale, int64_t window, int64_t sinks)
{
    if (!ok_size(N) || !ok_size(T) || !ok_size(S) || !ok_heads(H, KV, D) || !ok_mask(scale, window, sinks))
        return DET_GEMM_ERR_INVALID_ARG;
    if (!q_bounds && (k_bounds || N != 1)) return DET_GEMM_ERR_INVALID_ARG;
    if (q_bounds && !k_bounds && T != S) return DET_GEMM_ERR_INVALID_ARG;
    // Tiles and rows are counted in 32 bits.
    if (!ok_size(T + S + 256 * (N + 1)) || !launchable((T / 128 + N + 1) * H) || !launchable((S / 128 + N + 1) * KV)) return DET_GEMM_ERR_INVALID_ARG;
    return DET_GEMM_OK;
}

static AttnParams attn_params(const int32_t *q_bounds, const int32_t *k_bounds, int64_t N, int64_t T, int64_t S, int64_t H,
                              int64_t KV, int64_t D, float scale, int64_t window, int64_t sinks, const Device *d)
{
    AttnParams p;
    std::memset(&p, 0, sizeof p);
    p.qb = q_bounds;
    p.kb = k_bounds ? k_bounds : q_bounds;
    p.N = static_cast<int>(N);
    p.T = static_cast<int>(T);
    p.S = static_cast<int>(S);
    p.H = static_cast<int>(H);
    p.KV = static_cast<int>(KV);
    p.G = static_cast<int>(H / KV);
    p.D = static_cast<int>(D);
    p.scale = scale;
    p.window = window_of(window);
    p.sinks = sinks_of(sinks);
    p.status = d->word;
    p.timeout_ns = timeout_ns();
    p.force_timeout = timeout_forced();
    return p;
}

det_gemm_status det_attn(const det_gemm_bf16 *q, const det_gemm_bf16 *k, const det_gemm_bf16 *v, const int32_t *q_bounds,
                         const int32_t *k_bounds, det_gemm_bf16 *out, float *lse, int64_t N, int64_t T, int64_t S,
                         int64_t H, int64_t KV, int64_t D, float scale, int64_t window, int64_t sinks, int64_t qt,
                         int64_t qh, int64_t kt, int64_t kh, int64_t vt, int64_t vh, int64_t ot, int64_t oh,
                         det_gemm_stream stream)
{
    det_gemm_status s = ok_attn(q_bounds, k_bounds, N, T, S, H, KV, D, scale, window, sinks);
    if (s != DET_GEMM_OK) return s;
    if (T == 0) return DET_GEMM_OK;
    if ((s = check_all({heads(q, T, H, D, qt, qh), heads(k, S, KV, D, kt, kh), heads(v, S, KV, D, vt, vh)},
                       {vec4(q_bounds, q_bounds ? N + 1 : 0), vec4(k_bounds, k_bounds ? N + 1 : 0)},
                       {heads(out, T, H, D, ot, oh)}, {vec4(lse, H * T)})) != DET_GEMM_OK)
        return s;
    Device *d = nullptr;
    if ((s = device(&d)) != DET_GEMM_OK) return s;
    AttnParams p = attn_params(q_bounds, k_bounds, N, T, S, H, KV, D, scale, window, sinks, d);
    p.q = on(q, qt, qh);
    p.k = on(k, kt, kh);
    p.v = on(v, vt, vh);
    p.out = on(out, ot, oh);
    p.lse = lse;
    AttnMaps maps;
    if (!encode(&maps.q, q, T, H, D, qt, qh) || !encode(&maps.k, k, S, KV, D, kt, kh) || !encode(&maps.v, v, S, KV, D, vt, vh) ||
        !encode(&maps.out, out, T, H, D, ot, oh, 1, 32))
        return no_map();
    const cudaError_t e = launch_attn(p, maps, cs(stream));
    return e == cudaSuccess ? DET_GEMM_OK : fail(DET_GEMM_ERR_LAUNCH, e, "attention launch");
}

int64_t det_attn_bwd_workspace(int64_t N, int64_t T, int64_t S, int64_t H, int64_t KV, int64_t D, int64_t window, int64_t sinks)
{
    if (!ok_size(N) || !ok_size(T) || !ok_size(S) || !ok_heads(H, KV, D) || window < 0 || sinks < 0) return 0;
    return bwd_space(N, T, H, KV, D, window, sinks).total;
}

det_gemm_status det_attn_bwd(const det_gemm_bf16 *dout, const det_gemm_bf16 *q, const det_gemm_bf16 *k,
                             const det_gemm_bf16 *v, const det_gemm_bf16 *out, const float *lse, const int32_t *q_bounds,
                             const int32_t *k_bounds, det_gemm_bf16 *dq, det_gemm_bf16 *dk, det_gemm_bf16 *dv, int64_t N,
                             int64_t T, int64_t S, int64_t H, int64_t KV, int64_t D, float scale, int64_t window,
                             int64_t sinks, int64_t dot, int64_t doh, int64_t qt, int64_t qh, int64_t kt, int64_t kh,
                             int64_t vt, int64_t vh, int64_t ot, int64_t oh, int64_t dqt, int64_t dqh, int64_t dkt,
                             int64_t dkh, int64_t dvt, int64_t dvh, void *workspace, int64_t workspace_bytes,
                             det_gemm_stream stream)
{
    det_gemm_status s = ok_attn(q_bounds, k_bounds, N, T, S, H, KV, D, scale, window, sinks);
    if (s != DET_GEMM_OK) return s;
    if (T == 0 && S == 0) return DET_GEMM_OK;
    const BwdSpace space = bwd_space(N, T, H, KV, D, window, sinks);
    const int64_t need = space.total;
    if (!launchable((S / 128 + N + 1 + piece_slots(T, N, true) * sink_blocks(window, sinks)) * KV) ||
        !launchable(N * sink_blocks(window, sinks) * KV * 16))
        return DET_GEMM_ERR_INVALID_ARG;
    if ((s = check_all({heads(dout, T, H, D, dot, doh), heads(q, T, H, D, qt, qh), heads(k, S, KV, D, kt, kh),
                        heads(v, S, KV, D, vt, vh), heads(out, T, H, D, ot, oh)},
                       {vec4(lse, H * T), vec4(q_bounds, q_bounds ? N + 1 : 0), vec4(k_bounds, k_bounds ? N + 1 : 0)},
                       {heads(dq, T, H, D, dqt, dqh), heads(dk, S, KV, D, dkt, dkh), heads(dv, S, KV, D, dvt, dvh)},
                       {bytes(workspace, need)})) != DET_GEMM_OK)
        return s;
    if (workspace_bytes < need) return DET_GEMM_ERR_INVALID_ARG;
    Device *d = nullptr;
    if ((s = device(&d)) != DET_GEMM_OK) return s;
    AttnParams p = attn_params(q_bounds, k_bounds, N, T, S, H, KV, D, scale, window, sinks, d);
    p.dout = on(dout, dot, doh);
    p.q = on(q, qt, qh);
    p.k = on(k, kt, kh);
    p.v = on(v, vt, vh);
    p.out = on(out, ot, oh);
    p.lse = const_cast<float *>(lse);
    p.delta = static_cast<float *>(workspace);
    p.partials = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + space.partials);
    p.sink_blocks = sink_blocks(window, sinks);
    p.dq = on(dq, dqt, dqh);
    p.dk = on(dk, dkt, dkh);
    p.dv = on(dv, dvt, dvh);
    AttnMaps maps;
    if (!encode(&maps.q, q, T, H, D, qt, qh) || !encode(&maps.k, k, S, KV, D, kt, kh) || !encode(&maps.v, v, S, KV, D, vt, vh) ||
        !encode(&maps.dout, dout, T, H, D, dot, doh) || !encode(&maps.o, out, T, H, D, ot, oh) || !encode(&maps.out, dq, T, H, D, dqt, dqh, 1, 32) ||
        !encode(&maps.dk, dk, S, KV, D, dkt, dkh, 1, 32) || !encode(&maps.dv, dv, S, KV, D, dvt, dvh, 1, 32))
        return no_map();
    const cudaError_t e = launch_attn_bwd(p, maps, cs(stream));
    return e == cudaSuccess ? DET_GEMM_OK : fail(DET_GEMM_ERR_LAUNCH, e, "attention gradient launch");
}

}  // extern "C"
