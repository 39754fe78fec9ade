// Routing to experts: scores, the choice of the top k, their weights, and
// the gradient of the weights with respect to the logits.
//
//   p = softmax(l) or s = sigmoid(l); choice c = score + bias (without a
//   bias the order of the scores is the order of the logits, so c = l);
//   with groups, each group's value is the sum of its best one or two
//   choices and only the best groups' experts stay; the k largest choices
//   win, ties to the lower index; w = score[ids], over their sum when
//   renormalised, times `scale`. An expert whose logit is -inf or NaN is
//   masked; choices that are left over are -1 with weight 0.
//
// One warp owns a token, so a row's result is a function of that row alone:
// the logits are read once, and everything else lives in registers. Bytes
// bound it: T * E logits in, T * k ids and weights out.
//
// Which expert is chosen is a discrete question, so FP32 rounding must not
// decide it. Choices are compared in FP32, where each carries an error of a
// few units in the last place; when two neighbours of the chosen order (or
// the last kept and the first dropped group) are closer than FP32's
// error bound, the warp repeats the choice in FP64. Neighbours with equal
// logits and equal bias are exact ties and need no repeat. On 8192 tokens of
// 256 experts with random logits about one row in a thousand repeats (at
// 4e-6 for both scores, one in a hundred, and the FP64 units then took most
// of the launch's 45 us).
#include "ops_internal.h"
#include "vec.cuh"

namespace deto {
namespace {

constexpr int kWarps = 8;
// Bounds of the FP32 errors of two choices, relative to their scores' and
// biases' sizes. A sigmoid: one unit of expf, an addition, a division and the
// bias, below 8 * 2^-24 for both; a softmax adds its sum's rounding, common
// to all choices of a row but not to their biases, below 40 * 2^-24.
constexpr float kNearSigmoid = 6e-7f, kNearSoftmax = 4e-6f;
constexpr unsigned kAll = 0xFFFFFFFFu;

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

template <bool FP32>
__device__ __forceinline__ float logit_at(const RouteParams &p, int t, int e)
{
    if constexpr (FP32) return static_cast<const float *>(p.logits)[t * p.ldl + e];
    else return bf_at(static_cast<const uint16_t *>(p.logits) + t * p.ldl + e);
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
}

template <typename F>
__device__ __forceinline__ F warp_sum(F v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

__device__ __forceinline__ float sigmoid(float l) { return __fdiv_rn(1.0f, 1.0f + expf(-l)); }

// Order-preserving map of a float; 0 is left for "not a candidate".
__device__ __forceinline__ uint32_t order_key(float c)
{
    const uint32_t u = __float_as_uint(c + 0.0f);     // -0 -> +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// The lanes that look after group `lane / lanes_per_group`.
__device__ __forceinline__ int lanes_per_group(int groups)
{
    int l = 1;
    while (l * 2 * groups <= 32) l *= 2;
    return l;
}

// Best groups of a token: v[e] are the experts' values in shared memory
// (-inf: masked). Returns a bit mask of the kept groups; `near` is set when
// the border between kept and dropped groups is closer than rounding error.
template <typename F>
__device__ __forceinline__ uint32_t keep_groups(const RouteParams &p, const F *v, int lane, bool &near)
{
    const F ninf = static_cast<F>(neg_inf());
    const int size = p.experts / p.groups;
    const int lpg = lanes_per_group(p.groups);
    const int g = lane / lpg, sub = lane % lpg;
    F a = ninf, b = ninf;                             // best, second best
    if (g < p.groups) {
        for (int x = sub; x < size; x += lpg) {
            const F c = v[g * size + x];
            if (c > a) {
                b = a;
                a = c;
            } else if (c > b) {
                b = c;
            }
        }
    }
    for (int o = 1; o < lpg; o <<= 1) {
        const F a2 = __shfl_xor_sync(kAll, a, o), b2 = __shfl_xor_sync(kAll, b, o);
        const F lo = a < a2 ? a : a2;
        a = a < a2 ? a2 : a;
        b = b < b2 ? b2 : b;
        b = b < lo ? lo : b;
    }
    F val = a;
    if (p.group_best == 2 && b > ninf) val = a + b;
    int rank = 0;
    F next = ninf;                                    // best value ranked below this group
    for (int h = 0; h < p.groups; ++h) {
        const F o = __shfl_sync(kAll, val, h * lpg);
        const bool before = o > val || (o == val && h < g);
        rank += before ? 1 : 0;
        if (!before && h != g && o > next) next = o;
    }
    const bool kept = g < p.groups && sub == 0 && rank < p.top_groups && val > ninf;
    if (kept && rank == p.top_groups - 1 && next > ninf) {
        const F d = val - next;
        const F size2 = (val < 0 ? -val : val) + (next < 0 ? -next : next);
        // A value is at most the sum of two choices, each of a score of at
        // most 1 and a bias; the bias can cancel the score, hence the 1.
        const F bound = static_cast<F>(p.sigmoid ? kNearSigmoid : kNearSoftmax);
        if (!(d > bound * (p.bias ? size2 + static_cast<F>(1) : size2))) near = true;
    }
    const uint32_t lanes = __ballot_sync(kAll, kept);
    near = __any_sync(kAll, near);
    uint32_t mask = 0;
    for (int h = 0; h < p.groups; ++h) mask |= ((lanes >> (h * lpg)) & 1u) << h;
    return mask;
}

// The choice in FP64, for the few rows FP32 cannot decide. Returns the
// chosen expert of rank `lane` (-1: none).
template <bool FP32>
__device__ __noinline__ int choose_fp64(const RouteParams &p, int t, int lane, float top, double *v)
{
    const double ninf = static_cast<double>(neg_inf());
    double sum = 1.0;
    if (!p.sigmoid) {
        sum = 0.0;
        for (int e = lane; e < p.experts; e += 32) {
            const float l = logit_at<FP32>(p, t, e);
            if (l > neg_inf()) sum += exp(static_cast<double>(l) - static_cast<double>(top));
        }
        sum = warp_sum(sum);
    }
    for (int e = lane; e < p.experts; e += 32) {
        const float l = logit_at<FP32>(p, t, e);
        double c = ninf;
        if (l > neg_inf()) {
            c = p.sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(l)))
                          : exp(static_cast<double>(l) - static_cast<double>(top)) / sum;
            if (p.bias) c += static_cast<double>(p.bias[e]);
            if (!(c > ninf)) c = ninf;
        }
        v[e] = c;
    }
    __syncwarp();
    if (p.groups > 1) {
        bool near = false;
        const uint32_t kept = keep_groups<double>(p, v, lane, near);
        const int size = p.experts / p.groups;
        __syncwarp();
        for (int e = lane; e < p.experts; e += 32)
            if (!((kept >> (e / size)) & 1u)) v[e] = ninf;
        __syncwarp();
    }
    if (!p.bias) {                   // without a bias the logits give the order
        for (int e = lane; e < p.experts; e += 32)
            if (v[e] > ninf) v[e] = static_cast<double>(logit_at<FP32>(p, t, e));
        __syncwarp();
    }
    int mine = -1;
    for (int j = 0; j < p.k; ++j) {
        double best = ninf;
        int at = p.experts;
        for (int e = lane; e < p.experts; e += 32)
            if (v[e] > best) {
                best = v[e];
                at = e;
            }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const double b2 = __shfl_xor_sync(kAll, best, o);
            const int a2 = __shfl_xor_sync(kAll, at, o);
            if (b2 > best || (b2 == best && a2 < at)) {
                best = b2;
                at = a2;
            }
        }
        if (!(best > ninf)) break;
        if (lane == j) mine = at;
        if ((at & 31) == lane) v[at] = ninf;
        __syncwarp();
    }
    return mine;
}

// Shared memory per warp: `experts` doubles, used as floats for the group
// values and as doubles by the FP64 repeat.
template <bool FP32, int PER>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(const RouteParams p)
{
    extern __shared__ double route_smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = blockIdx.x * kWarps + warp;
    if (t >= p.tokens) return;
    double *vd = route_smem + warp * p.experts;
    float *vf = reinterpret_cast<float *>(vd);

    float l[PER];
    float top = neg_inf();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = i * 32 + lane;
        float x = e < p.experts ? logit_at<FP32>(p, t, e) : neg_inf();
        if (!(x > neg_inf())) x = neg_inf();          // NaN: masked
        l[i] = x;
        top = fmaxf(top, x);
    }
    top = warp_max(top);

    // Scores are needed for the choice only with a bias or groups.
    const bool scored = p.bias != nullptr || p.groups > 1;
    uint32_t key[PER];
    float total = 1.0f;
    if (!p.sigmoid && (scored || !p.renorm)) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) s += l[i] > neg_inf() ? expf(l[i] - top) : 0.0f;
        total = warp_sum(s);
    }
    bool near = false;
    if (scored) {
        float c[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = i * 32 + lane;
            c[i] = neg_inf();
            if (l[i] > neg_inf()) {
                c[i] = p.sigmoid ? sigmoid(l[i]) : __fdiv_rn(expf(l[i] - top), total);
                if (p.bias) c[i] += p.bias[e];
                if (!(c[i] > neg_inf())) {
                    c[i] = neg_inf();
                    l[i] = neg_inf();
                }
            }
        }
        uint32_t kept = kAll;
        const int size = p.experts / p.groups;
        if (p.groups > 1) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int e = i * 32 + lane;
                if (e < p.experts) vf[e] = c[i];
            }
            __syncwarp();
            kept = keep_groups<float>(p, vf, lane, near);
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = i * 32 + lane;
            const bool ok = l[i] > neg_inf() && (p.groups == 1 || ((kept >> (e / size)) & 1u));
            key[i] = ok ? order_key(p.bias ? c[i] : l[i]) : 0u;
        }
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) key[i] = l[i] > neg_inf() ? order_key(l[i]) : 0u;
    }

    // The k largest keys in order; with a bias one more, to see how close
    // the first that lost came.
    int mine = -1, lost = -1;
    uint32_t my_key = 0, lost_key = 0;
    const int take = p.bias ? p.k + 1 : p.k;
    for (int j = 0; j < take; ++j) {
        uint32_t best = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (key[i] > best) {
                best = key[i];
                at = i * 32 + lane;
            }
        const uint32_t m = __reduce_max_sync(kAll, best);
        if (m == 0) break;
        const int e = static_cast<int>(__reduce_min_sync(kAll, best == m ? static_cast<uint32_t>(at) : 0xFFFFFFFFu));
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (i * 32 + lane == e) key[i] = 0;
        if (j == p.k) {
            lost = e;
            lost_key = m;
        }
        if (j < p.k && lane == j) {
            mine = e;
            my_key = m;
        }
    }
    if (p.bias) {
        // Each choice against the next one (the last against the best that lost).
        int ne = __shfl_down_sync(kAll, mine, 1);
        uint32_t nk = __shfl_down_sync(kAll, my_key, 1);
        if (lane == p.k - 1) {
            ne = lost;
            nk = lost_key;
        }
        if (lane < p.k && mine >= 0 && ne >= 0) {
            const float hi = __uint_as_float((my_key & 0x80000000u) ? my_key & 0x7FFFFFFFu : ~my_key);
            const float lo = __uint_as_float((nk & 0x80000000u) ? nk & 0x7FFFFFFFu : ~nk);
            const float bh = p.bias[mine], bl = p.bias[ne];
            const float size = fabsf(bh) + fabsf(hi) + fabsf(bl) + fabsf(lo);   // >= the scores too
            if (!(hi - lo > (p.sigmoid ? kNearSigmoid : kNearSoftmax) * size) &&
                !(bh == bl && logit_at<FP32>(p, t, mine) == logit_at<FP32>(p, t, ne)))
                near = true;
        }
        near = __any_sync(kAll, near);
    }
    if (near) mine = choose_fp64<FP32>(p, t, lane, top, vd);

    // Weights, FP32: lane j holds choice j.
    const float lj = mine >= 0 ? logit_at<FP32>(p, t, mine) : neg_inf();
    float w = 0.0f;
    if (p.sigmoid) {
        if (mine >= 0) w = sigmoid(lj);
        if (p.renorm) w = __fdiv_rn(w, warp_sum(w) + 1e-20f);
    } else if (p.renorm) {
        // exp(l - top) of the chosen over their sum, shifted by their own maximum
        const float m = warp_max(lj);
        if (mine >= 0) w = expf(lj - m);
        const float s = warp_sum(w);
        if (mine >= 0) w = __fdiv_rn(w, s);
    } else if (mine >= 0) {
        w = __fdiv_rn(expf(lj - top), total);
    }
    if (lane < p.k) {
        p.ids[static_cast<long long>(t) * p.k + lane] = mine;
        p.weights[static_cast<long long>(t) * p.k + lane] = mine >= 0 ? w * p.scale : 0.0f;
    }
}

// Gradient with respect to the logits, g = scale * dw over the chosen:
//   softmax, renormalised: dl_j = q_j (g_j - sum q g), q = p_j / sum p
//   softmax:               dl_i = p_i (g_i - sum p g), every unmasked i
//   sigmoid, renormalised: dl_j = s_j (1 - s_j) (g_j - sum q g) / (S + 1e-20)
//   sigmoid:               dl_j = s_j (1 - s_j) g_j
// The row of chosen gradients is spread out in shared memory, one float for
// each expert, and read back with the logits' layout.
template <bool FP32, int PER>
__global__ void __launch_bounds__(kWarps * 32) route_bwd_kernel(const RouteParams p)
{
    extern __shared__ double route_smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = blockIdx.x * kWarps + warp;
    if (t >= p.tokens) return;
    float *d = reinterpret_cast<float *>(route_smem) + warp * (PER * 32);
#pragma unroll
    for (int i = 0; i < PER; ++i) d[i * 32 + lane] = 0.0f;
    __syncwarp();
    int id = -1;
    float g = 0.0f, lj = neg_inf();
    if (lane < p.k) {
        id = p.ids[static_cast<long long>(t) * p.k + lane];
        if (id < 0 || id >= p.experts) id = -1;
        if (id >= 0) {
            g = p.dw[static_cast<long long>(t) * p.k + lane] * p.scale;
            lj = logit_at<FP32>(p, t, id);
        }
    }
    float l[PER];
    float top = neg_inf(), total = 1.0f;
    const bool full = !p.sigmoid && !p.renorm;        // every expert's logit moves every weight
    if (full) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = i * 32 + lane;
            float x = e < p.experts ? logit_at<FP32>(p, t, e) : neg_inf();
            if (!(x > neg_inf())) x = neg_inf();
            l[i] = x;
            top = fmaxf(top, x);
        }
        top = warp_max(top);
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) s += l[i] > neg_inf() ? expf(l[i] - top) : 0.0f;
        total = warp_sum(s);
    }
    float dot = 0.0f, dj = 0.0f;
    if (p.sigmoid) {
        const float s = id >= 0 ? sigmoid(lj) : 0.0f;
        // 1 - s, without cancellation for large logits
        const float s1 = id >= 0 ? sigmoid(-lj) : 0.0f;
        if (p.renorm) {
            const float S = warp_sum(s) + 1e-20f;
            dot = warp_sum(__fdiv_rn(s, S) * g);
            dj = s * s1 * __fdiv_rn(g - dot, S);
        } else {
            dj = s * s1 * g;
        }
    } else if (p.renorm) {
        const float m = warp_max(lj);
        float q = id >= 0 ? expf(lj - m) : 0.0f;
        const float s = warp_sum(q);
        q = id >= 0 ? __fdiv_rn(q, s) : 0.0f;
        dot = warp_sum(q * g);
        dj = q * (g - dot);
    } else {
        const float pj = id >= 0 ? __fdiv_rn(expf(lj - top), total) : 0.0f;
        dot = warp_sum(pj * g);
        dj = g;
    }
    if (id >= 0) d[id] = dj;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = i * 32 + lane;
        if (e >= p.experts) continue;
        float v = d[e];
        if (full) v = l[i] > neg_inf() ? __fdiv_rn(expf(l[i] - top), total) * (v - dot) : 0.0f;
        if constexpr (FP32) static_cast<float *>(p.dlogits)[t * p.ldd + e] = v;
        else static_cast<__nv_bfloat16 *>(p.dlogits)[t * p.ldd + e] = __float2bfloat16_rn(v);
    }
}

template <bool FP32, int PER>
cudaError_t go(const RouteParams &p, bool bwd, cudaStream_t s)
{
    const int blocks = (p.tokens + kWarps - 1) / kWarps;
    if (bwd) {
        route_bwd_kernel<FP32, PER><<<blocks, kWarps * 32, kWarps * PER * 32 * 4, s>>>(p);
    } else {
        const bool scored = p.bias != nullptr || p.groups > 1;
        route_kernel<FP32, PER><<<blocks, kWarps * 32, scored ? kWarps * p.experts * 8 : 0, s>>>(p);
    }
    return cudaGetLastError();
}

template <bool FP32>
cudaError_t pick(const RouteParams &p, bool bwd, cudaStream_t s)
{
    if (p.experts <= 32) return go<FP32, 1>(p, bwd, s);
    if (p.experts <= 64) return go<FP32, 2>(p, bwd, s);
    if (p.experts <= 128) return go<FP32, 4>(p, bwd, s);
    if (p.experts <= 256) return go<FP32, 8>(p, bwd, s);
    return go<FP32, 16>(p, bwd, s);
}

}  // namespace

cudaError_t launch_route(const RouteParams &p, bool fp32, cudaStream_t s)
{
    return fp32 ? pick<true>(p, false, s) : pick<false>(p, false, s);
}

cudaError_t launch_route_bwd(const RouteParams &p, bool fp32, cudaStream_t s)
{
    return fp32 ? pick<true>(p, true, s) : pick<false>(p, true, s);
}

}  // namespace deto
