// Routing to experts: scores, the choice of the top k, their weights, and
// the gradient of the weights with respect to the logits.
//
//   p = softmax(l) or s = sigmoid(l); choice c = score + bias (without a
//   bias the order of the scores is the order of the logits, so c = l);
//   with groups, each group's value is the sum of its best one or two
//   choices and only the best groups' experts stay; the k largest choices
//   win, ties to the lower index; w = score[ids], over their sum when
//   renormalised, times `scale`. An expert whose logit is -inf or NaN is
//   masked; choices that are left over are -1 with weight 0. A logit of +inf
//   is chosen like the largest finite one; the softmax of its row, and so the
//   row's weights, are NaN.
//
// One warp owns a token, so a row's result is a function of that row alone:
// the logits are read once, and everything else lives in registers. Bytes
// bound it: T * E logits in, T * k ids and weights out.
//
// Which expert is chosen is a discrete question, so FP32 rounding must not
// decide it. Choices are compared in FP32, where each carries an error of a
// few units in the last place; when two neighbours of the chosen order, the last
// choice and any that lost (a large bias means a large error: not only the next
// one), or a kept and a dropped group, are closer than FP32's error bound,
// the warp decides again: the few candidates near the last choice in FP64, one
// a lane; the groups whose place is open with pairs of FP32 values (about 43
// bits), or in FP64 where a score is too small for those; and every expert so
// where many candidates are close. Neighbours with equal logits and equal
// bias are exact ties and need no repeat. On 8192 tokens of 256 experts with
// random logits about one row in a thousand decides again. The launch takes
// as long as its last row: repeating all experts' choices for a border of
// groups took 23.6 us in the mean over random inputs, the open groups alone
// 18.8.
//
// On those 8192 x 256 FP32 logits the kernel takes 5.6 us by the logits alone,
// 10.3 with sigmoid scores and a bias, 14.4 with eight groups besides, where the
// bytes would take 1.3: instructions bound it, mostly integer and comparisons.
// With groups a token takes 1270 of them; on 262144 tokens (330 us, 1.26 ns each)
// 81 % of the issue slots are used. 8192 tokens at that pace are 10.3 us: the
// rest is the start and the end, 2048 blocks on an SM's ten places being 1.35
// rounds (58 % of the slots). A lane holds neighbouring experts, so that it loads
// 16 bytes at a time and a group's best choices are found in registers (every
// 32nd expert, and groups through shared memory, cost 0.4, 1.0 and 1.9 us more).
// Four warps a block and 48 registers keep 40 warps on an SM to the end; 48 warps
// with 40 registers spill and take 1.2 us more.
#pragma once

#include "launch.cuh"
#include "ops_internal.h"
#include "vec.cuh"

namespace deto {
namespace {

constexpr int kWarps = 4;
// Bounds of the FP32 errors of two choices, relative to their scores' and
// biases' sizes. A sigmoid: one unit of expf, an addition, a reciprocal of one
// unit and the bias, below 8 * 2^-24; a softmax adds its sum's rounding, common
// to all choices of a row but not to their biases, and its argument's, 64 * 2^-24
// of a score whose logit is up to 128 below the row's largest: below 92 * 2^-24.
// Scores below FP32's normal numbers are off by units of 2^-149 besides.
constexpr float kNearSigmoid = 6e-7f, kNearSoftmax = 5.5e-6f, kNearTiny = 1e-44f;
constexpr unsigned kAll = 0xFFFFFFFFu;

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }
__device__ __forceinline__ float pos_inf() { return __int_as_float(0x7f800000); }

template <bool FP32>
__device__ __forceinline__ float logit_at(const RouteParams &p, int t, int e)
{
    if constexpr (FP32) return static_cast<const float *>(p.logits)[t * p.ldl + e];
    else return bf_at(static_cast<const uint16_t *>(p.logits) + t * p.ldl + e);
}

constexpr float kLargest = 3.402823466e38f;         // what +inf counts as in the choice

// A lane's PER neighbours from src[lane * PER] on, -inf past `experts`; in
// 16-byte loads where the row is full and aligned.
template <typename T, int PER>
__device__ __forceinline__ void load_own(const T *src, int experts, int lane, float (&v)[PER])
{
    constexpr int bytes = PER * static_cast<int>(sizeof(T)), N = bytes < 16 ? bytes : 16;   // of one load
    const T *own = src + lane * PER;
    if (N >= 4 && experts == 32 * PER && (reinterpret_cast<uintptr_t>(src) & (N - 1)) == 0) {
        alignas(16) uint32_t w[bytes / 4 > 0 ? bytes / 4 : 1];
#pragma unroll
        for (int i = 0; i < bytes / N; ++i) {
            if constexpr (N == 16) *reinterpret_cast<uint4 *>(w + 4 * i) = reinterpret_cast<const uint4 *>(own)[i];
            else if constexpr (N == 8) *reinterpret_cast<uint2 *>(w) = *reinterpret_cast<const uint2 *>(own);
            else w[0] = *reinterpret_cast<const uint32_t *>(own);
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if constexpr (sizeof(T) == 4) v[i] = __uint_as_float(w[i]);
            else v[i] = (i & 1) ? bf_hi(w[i / 2]) : bf_lo(w[i / 2]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            v[i] = neg_inf();
            if (lane * PER + i < experts) {
                if constexpr (sizeof(T) == 4) v[i] = own[i];
                else v[i] = bf_at(own + i);
            }
        }
    }
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

// The same within one more unit, for the choice (a reciprocal of one unit's error).
__device__ __forceinline__ float sigmoid_choice(float l)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + expf(-l)));
    return r;
}

// Order-preserving map of a float; 0 is left for "not a candidate".
__device__ __forceinline__ uint32_t order_key(float c)
{
    const int u = __float_as_int(c + 0.0f);           // -0 -> +0
    return static_cast<uint32_t>(u ^ ((u >> 31) | static_cast<int>(0x80000000u)));
}

__device__ __forceinline__ float key_value(uint32_t key)
{
    return __uint_as_float((key & 0x80000000u) ? key & 0x7FFFFFFFu : ~key);
}

// Group g is looked after by the lanes from g << lane_shift on; a set of
// groups is a mask of those first lanes.
__device__ __forceinline__ int lane_shift(int groups) { return __clz(groups - 1) - 27; }

// ---- pairs of FP32 values: hi + lo, |lo| at most half a unit of hi (the sums
// and products of Dekker and Knuth, each operation rounded on its own).
struct Df {
    float hi, lo;
};
__device__ __forceinline__ Df quick_sum(float a, float b)    // |a| >= |b|
{
    const float s = __fadd_rn(a, b);
    return Df{s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Df two_sum(float a, float b)
{
    const float s = __fadd_rn(a, b), bb = __fsub_rn(s, a);
    return Df{s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb))};
}
__device__ __forceinline__ Df operator+(const Df &a, const Df &b)
{
    Df s = two_sum(a.hi, b.hi);
    const Df t = two_sum(a.lo, b.lo);
    s = quick_sum(s.hi, __fadd_rn(s.lo, t.hi));
    return quick_sum(s.hi, __fadd_rn(s.lo, t.lo));
}
__device__ __forceinline__ Df operator*(const Df &a, const Df &b)
{
    const float p = __fmul_rn(a.hi, b.hi);
    const float e = __fmaf_rn(a.hi, b.hi, -p);
    return quick_sum(p, __fmaf_rn(a.hi, b.lo, __fmaf_rn(a.lo, b.hi, e)));
}
// Quotient by long division: each of three steps takes the quotient of the leading
// parts as the next digit and its product from the remainder, which stays a pair.
// No branches, so that independent ones overlap.
__device__ __forceinline__ Df operator/(const Df &a, const Df &b)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(b.hi));
    const float q1 = __fmul_rn(a.hi, r);
    Df d = a + Df{-q1, 0.0f} * b;
    const float q2 = __fmul_rn(d.hi, r);
    d = d + Df{-q2, 0.0f} * b;
    return quick_sum(q1, q2) + Df{__fmul_rn(d.hi, r), 0.0f};
}
__device__ __forceinline__ bool operator>(const Df &a, const Df &b) { return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo); }
__device__ __forceinline__ bool operator<(const Df &a, const Df &b) { return b > a; }
__device__ __forceinline__ bool operator==(const Df &a, const Df &b) { return a.hi == b.hi && a.lo == b.lo; }

constexpr Df split(double v)
{
    return Df{static_cast<float>(v), static_cast<float>(v - static_cast<double>(static_cast<float>(v)))};
}

// exp of N values in [-60, 60]: x = n ln 2 + r, |r| <= 0.347, and the
// exponential series of r up to r^12 / 12! (the next term is below 2^-52), its
// first terms in pairs and those below 2^-23 in FP32. Relative error about
// 2^-43. The N values go side by side, so that one's operations fill another's
// latency, and the terms are a loop, so that the code stays small.
__constant__ float g_series[6] = {1.0f / 479001600.0f, 1.0f / 39916800.0f, 1.0f / 3628800.0f, 1.0f / 362880.0f, 1.0f / 40320.0f,
                                  1.0f / 5040.0f};
__constant__ Df g_terms[7] = {split(1.0 / 720.0), split(1.0 / 120.0), split(1.0 / 24.0), split(1.0 / 6.0), Df{0.5f, 0.0f},
                              Df{1.0f, 0.0f}, Df{1.0f, 0.0f}};

template <int N>
__device__ __forceinline__ void exp_all(Df (&x)[N])
{
    constexpr Df ln2 = split(0.69314718055994530942);
    float n[N];
    Df r[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        n[i] = rintf(x[i].hi * 1.44269504f);
        r[i] = x[i] + Df{-n[i], 0.0f} * ln2;
        x[i] = Df{g_series[0], 0.0f};
    }
#pragma unroll 1
    for (int k = 1; k < 6; ++k) {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i].hi = __fmaf_rn(x[i].hi, r[i].hi, g_series[k]);
    }
#pragma unroll 1
    for (int k = 0; k < 7; ++k) {
        const Df c = g_terms[k];
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = x[i] * r[i] + c;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float scale = __int_as_float((static_cast<int>(n[i]) + 127) << 23);
        x[i] = Df{x[i].hi * scale, x[i].lo * scale};
    }
}
template <int N>
__device__ __forceinline__ void exp_all(double (&x)[N])
{
#pragma unroll 1
    for (int i = 0; i < N; ++i) x[i] = exp(x[i]);
}

// The value types the choice runs in.
template <typename F>
struct Num;
template <>
struct Num<double> {
    static __device__ __forceinline__ double of(float v) { return v; }
    static __device__ __forceinline__ double half(double v) { return 0.5 * v; }
    static __device__ __forceinline__ double shfl(double v, int l) { return __shfl_sync(kAll, v, l); }
    static __device__ __forceinline__ double shfl_xor(double v, int o) { return __shfl_xor_sync(kAll, v, o); }
    static __device__ __forceinline__ double diff(float a, float b) { return static_cast<double>(a) - static_cast<double>(b); }
};
template <>
struct Num<Df> {
    static __device__ __forceinline__ Df of(float v) { return Df{v, 0.0f}; }
    static __device__ __forceinline__ Df half(Df v) { return Df{0.5f * v.hi, 0.5f * v.lo}; }
    static __device__ __forceinline__ Df shfl(Df v, int l) { return Df{__shfl_sync(kAll, v.hi, l), __shfl_sync(kAll, v.lo, l)}; }
    static __device__ __forceinline__ Df shfl_xor(Df v, int o)
    {
        return Df{__shfl_xor_sync(kAll, v.hi, o), __shfl_xor_sync(kAll, v.lo, o)};
    }
    static __device__ __forceinline__ Df diff(float a, float b) { return two_sum(a, -b); }
};

// A score and its expert's bias. An infinite bias is the choice itself: beside an
// infinity the low part of a pair would be NaN.
template <typename F>
__device__ __forceinline__ F with_bias(const F &score, float bias)
{
    return bias < pos_inf() ? score + Num<F>::of(bias) : Num<F>::of(bias);
}

// The group of expert e, for e and experts up to 512: e / size by a product
// (size * (2^18 / size + 1) is above 2^18 by at most size, and e * size < 2^18).
__device__ __forceinline__ int group_of(const RouteParams &p, int e) { return (e * p.group_mul) >> 18; }
__device__ __forceinline__ bool in_groups(const RouteParams &p, uint32_t kept, int e)
{
    return (kept >> (group_of(p, e) << lane_shift(p.groups))) & 1u;
}

// The sum over the row of exp(l - top), in type F.
template <bool FP32, typename F>
__device__ __forceinline__ F exp_sum(const RouteParams &p, int t, int lane, float top)
{
    using N = Num<F>;
    constexpr int B = 4;             // experts of a lane side by side
    F sum = N::of(0.0f);
#pragma unroll 1
    for (int e0 = 0; e0 < p.experts; e0 += 32 * B) {
        F x[B];
        bool in[B];
#pragma unroll
        for (int i = 0; i < B; ++i) {
            const int e = e0 + 32 * i + lane;
            const float l = e < p.experts ? logit_at<FP32>(p, t, e) : neg_inf();
            in[i] = l > neg_inf();
            x[i] = N::diff(in[i] ? fminf(l, kLargest) : top, top);
        }
        exp_all(x);
#pragma unroll
        for (int i = 0; i < B; ++i)
            if (in[i]) sum = sum + x[i];
    }
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1) sum = sum + N::shfl_xor(sum, o);
    return sum;
}

// Of the groups in `doubt`, the `slots` best, with values of type F; two
// groups at a time, 32 experts of each at a time. Returns their mask.
template <bool FP32, typename F>
__device__ __forceinline__ uint32_t settle_groups(const RouteParams &p, int t, int lane, float top, uint32_t doubt, int slots)
{
    using N = Num<F>;
    const F ninf = N::of(neg_inf()), pinf = N::of(pos_inf()), one = N::of(1.0f);
    const int size = p.experts / p.groups;
    const int shift = lane_shift(p.groups);
    const F sum = p.sigmoid ? one : exp_sum<FP32, F>(p, t, lane, top);
    F val = ninf;                    // in a group's first lane: its value
#pragma unroll 1
    for (uint32_t left = doubt; left;) {
        int g[2];
        g[0] = __ffs(left) - 1;
        left &= left - 1;
        g[1] = left ? __ffs(left) - 1 : g[0];
        left &= left - 1;
        F a[2] = {ninf, ninf}, b[2] = {ninf, ninf};   // best, second best
#pragma unroll 1
        for (int x0 = 0; x0 < size; x0 += 32) {
            F c[2];
            float bias[2];
            bool in[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int x = x0 + lane, e = (g[i] >> shift) * size + x;
                const float l = x < size ? logit_at<FP32>(p, t, e) : neg_inf();
                bias[i] = p.bias && x < size ? p.bias[e] : 0.0f;
                in[i] = l > neg_inf() && bias[i] > neg_inf();
                c[i] = N::diff(p.sigmoid ? 0.0f : in[i] ? fminf(l, kLargest) : top, p.sigmoid ? (in[i] ? l : 0.0f) : top);
            }
            exp_all(c);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                c[i] = (p.sigmoid ? one : c[i]) / (p.sigmoid ? one + c[i] : sum);
                if (p.bias) c[i] = with_bias(c[i], in[i] ? bias[i] : 0.0f);
                if (!in[i]) c[i] = ninf;
                const F lo = c[i] > a[i] ? a[i] : c[i];
                a[i] = c[i] > a[i] ? c[i] : a[i];
                b[i] = lo > b[i] ? lo : b[i];
            }
        }
#pragma unroll 1
        for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const F a2 = N::shfl_xor(a[i], o), b2 = N::shfl_xor(b[i], o);
                const F lo = a2 > a[i] ? a[i] : a2;
                a[i] = a2 > a[i] ? a2 : a[i];
                b[i] = b2 > b[i] ? b2 : b[i];
                b[i] = lo > b[i] ? lo : b[i];
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (lane == g[i]) {
                val = N::half(a[i]);                  // as in keep_groups
                if (p.group_best == 2 && b[i] > ninf && a[i] < pinf) val = val + N::half(b[i]);
            }
    }
    int rank = 0;
    for (int h = 0; h < p.groups; ++h) {
        const F o = N::shfl(val, h << shift);
        rank += (o > val || (o == val && h << shift < lane)) ? 1 : 0;
    }
    return __ballot_sync(kAll, ((doubt >> lane) & 1u) && rank < slots);
}

// A lane's two best choices of its group, from the choices in shared memory: a lane takes every (1 << shift)-th of its group.
__device__ __forceinline__ void scan_group(const RouteParams &p, const float *v, int lane, float &a, float &b)
{
    const int size = p.experts / p.groups;
    const int shift = lane_shift(p.groups), lpg = 1 << shift;
    const int g = lane >> shift, sub = lane & (lpg - 1);
    if (g < p.groups) {
        // Each group begins elsewhere in its row: sizes of 32 keep to different banks.
        int x = sub + g * lpg;
        while (x >= size) x -= size;
#pragma unroll 4
        for (int i = sub; i < size; i += lpg) {
            const float c = v[g * size + x];
            b = fmaxf(b, fminf(a, c));
            a = fmaxf(a, c);
            x += lpg;
            if (x >= size) x -= size;
        }
    }
}

// Best groups of a token from the two best choices that each lane holds of its
// group's (a, b; -inf: none). Returns the mask of the kept groups. When FP32 cannot tell
// every kept group from every dropped one, `doubt` are the groups whose place is
// open and `slots` how many of them stay; the mask then holds the certain ones
// alone.
__device__ __forceinline__ uint32_t keep_groups(const RouteParams &p, float a, float b, int lane, uint32_t &doubt, int &slots)
{
    const int shift = lane_shift(p.groups), lpg = 1 << shift;
    const int g = lane >> shift, sub = lane & (lpg - 1);
    for (int o = 1; o < lpg; o <<= 1) {
        const float a2 = __shfl_xor_sync(kAll, a, o), b2 = __shfl_xor_sync(kAll, b, o);
        b = fmaxf(fmaxf(b, b2), fminf(a, a2));
        a = fmaxf(a, a2);
    }
    // Half of the group's value: two of the largest finite biases have a sum then.
    float val = 0.5f * a, amount = fabsf(val);
    if (p.group_best == 2 && b > neg_inf()) {
        val += 0.5f * b;
        amount += 0.5f * fabsf(b);
    }
    int rank = 0;
#pragma unroll 4
    for (int h = 0; h < p.groups; ++h) {
        const float o = __shfl_sync(kAll, val, h << shift);
        rank += (o > val || (o == val && h < g)) ? 1 : 0;
    }
    const bool leader = g < p.groups && sub == 0 && val > neg_inf();
    const bool kept = leader && rank < p.top_groups;
    // A value's FP32 error: that of its scores, which are at most 1 each (a
    // bias can cancel them, so the value does not tell their size), and of its
    // one or two additions; scores below 1e-20 only absolutely. A value of +inf
    // (from a bias) is exact.
    const float err = val < pos_inf() ? (p.sigmoid ? kNearSigmoid : kNearSoftmax) * (amount + (p.bias ? 1.0f : 0.0f)) + 1e-25f : 0.0f;
    // Every kept group against every dropped one: errors go with the size of a
    // group's choices, which its value, a sum, does not tell.
    const uint32_t low = __reduce_min_sync(kAll, kept ? order_key(val - err) : 0xFFFFFFFFu);
    const uint32_t high = __reduce_max_sync(kAll, leader && !kept ? order_key(val + err) : 0u);
    uint32_t lanes = __ballot_sync(kAll, kept);
    if (low <= high) {
        const uint32_t open = __ballot_sync(kAll, leader && order_key(val - err) <= high && order_key(val + err) >= low);
        lanes &= ~open;
        slots = p.top_groups - __popc(lanes);
        doubt = open;
    }
    return lanes;
}

// The choice with values of type F, for the few rows FP32 cannot decide (with a
// bias: without one the logits give the order).
// Returns the chosen expert of rank `lane` (-1: none).
template <bool FP32, typename F>
__device__ __forceinline__ int choose_again(const RouteParams &p, int t, int lane, float top, uint32_t kept, F *v)
{
    using N = Num<F>;
    const F ninf = N::of(neg_inf()), one = N::of(1.0f);
    const bool sig = p.sigmoid;
    constexpr int B = 4;             // experts of a lane side by side
    F sum = N::of(0.0f);
    // First the exponentials (exp(-l), or exp(l - top) and their sum), then the choices.
#pragma unroll 1
    for (int e0 = 0; e0 < p.experts; e0 += 32 * B) {
        F x[B];
        bool in[B];
#pragma unroll
        for (int i = 0; i < B; ++i) {
            const int e = e0 + 32 * i + lane;
            const float l = e < p.experts ? logit_at<FP32>(p, t, e) : neg_inf();
            in[i] = l > neg_inf();
            x[i] = N::diff(sig ? 0.0f : in[i] ? fminf(l, kLargest) : top, sig ? (in[i] ? l : 0.0f) : top);
        }
        exp_all(x);
#pragma unroll
        for (int i = 0; i < B; ++i) {
            const int e = e0 + 32 * i + lane;
            if (e < p.experts) v[e] = in[i] ? x[i] : ninf;
            if (in[i]) sum = sum + x[i];
        }
    }
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1) sum = sum + N::shfl_xor(sum, o);
#pragma unroll 1
    for (int e0 = 0; e0 < p.experts; e0 += 32 * B) {
#pragma unroll
        for (int i = 0; i < B; ++i) {
            const int e = e0 + 32 * i + lane;
            if (e >= p.experts) continue;
            const F x = v[e];
            const float bias = p.bias[e];
            const bool in = x > ninf && bias > neg_inf() && (p.groups == 1 || in_groups(p, kept, e));
            const F c = (sig ? one : x) / (sig ? one + x : sum);
            v[e] = in ? with_bias(c, bias) : ninf;
        }
    }
    __syncwarp();
    int mine = -1;
#pragma unroll 1
    for (int j = 0; j < p.k; ++j) {
        F best = ninf;
        int at = p.experts;
        for (int e = lane; e < p.experts; e += 32)
            if (v[e] > best) {
                best = v[e];
                at = e;
            }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const F b2 = N::shfl_xor(best, o);
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

// The order of a few candidates (one at least) in FP64, one for each of the first
// `count` lanes (list[lane].y). Leaves the chosen in list[0 .. min(count, k)).y.
template <bool FP32>
__device__ __forceinline__ void order_candidates(const RouteParams &p, int t, int lane, float top, uint2 *list, int count)
{
    double sum = 1.0;
    if (!p.sigmoid) {
        sum = 0.0;
        for (int e = lane; e < p.experts; e += 32) {
            const float l = logit_at<FP32>(p, t, e);
            if (l > neg_inf()) sum += exp(static_cast<double>(fminf(l, kLargest)) - static_cast<double>(top));
        }
        sum = warp_sum(sum);
    }
    const int e = static_cast<int>(list[min(lane, count - 1)].y);
    const double l = static_cast<double>(fminf(logit_at<FP32>(p, t, e), kLargest));
    const double c = (p.sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - static_cast<double>(top)) / sum) + static_cast<double>(p.bias[e]);
    int rank = 0;
    for (int o = 0; o < count; ++o) {
        const double d = __shfl_sync(kAll, c, o);
        const int f = __shfl_sync(kAll, e, o);
        rank += (d > c || (d == c && f < e)) ? 1 : 0;
    }
    __syncwarp();
    if (lane < count) list[rank].y = static_cast<uint32_t>(e);
    __syncwarp();
}

// Pairs of FP32 values hold what exp gives between -60 and 60: whether an
// argument of the row, -l or l - top, lies elsewhere. (Read again: the repeats
// are few, and their registers are the common path's.)
template <bool FP32>
__device__ __forceinline__ bool far_logits(const RouteParams &p, int t, int lane, float top)
{
    bool far = false;
    for (int e = lane; e < p.experts; e += 32) {
        const float l = logit_at<FP32>(p, t, e);
        if (l > neg_inf()) far |= !(fabsf(p.sigmoid ? l : fminf(l, kLargest) - top) < 60.0f);
    }
    return __any_sync(kAll, far);
}

// Shared memory per warp: `experts` doubles, used as floats for the group
// values and as doubles by the FP64 repeat.
// MODE: what the choice needs besides the logits. The repeats' registers are
// held down to the common path's, which then has 40 warps on an SM.
enum { kLogits, kBias, kGroups };    // kGroups: with or without a bias
template <bool FP32, int PER, int MODE>
__global__ void __launch_bounds__(kWarps * 32, PER <= 8 ? 10 : 6) route_kernel(const __grid_constant__ RouteParams p)
{
    begin();
    extern __shared__ double route_smem[];
    __shared__ uint2 gather_smem[kWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = blockIdx.x * kWarps + warp;
    if (t >= p.tokens) return;
    uint2 *gathered = gather_smem[warp];
    double *vd = route_smem + warp * p.experts;
    float *vf = reinterpret_cast<float *>(vd);

    // Lane `lane` holds experts lane * PER and on.
    float l[PER];
    float top = neg_inf();
    if constexpr (FP32) load_own(static_cast<const float *>(p.logits) + t * p.ldl, p.experts, lane, l);
    else load_own(static_cast<const uint16_t *>(p.logits) + t * p.ldl, p.experts, lane, l);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (!(l[i] > neg_inf())) l[i] = neg_inf();    // NaN: masked
        top = fmaxf(top, l[i]);
    }
    top = warp_max(top);

    // Scores are needed for the choice only with a bias or groups.
    constexpr bool scored = MODE != kLogits;
    const bool overflowed = scored && top == pos_inf();
    if (overflowed) {
        top = kLargest;
#pragma unroll
        for (int i = 0; i < PER; ++i) l[i] = fminf(l[i], kLargest);
    }
    const bool biased = MODE == kBias || (MODE == kGroups && p.bias != nullptr);
    uint32_t key[PER];
    float total = 1.0f;
    if (!p.sigmoid && (scored || !p.renorm)) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) s += l[i] > neg_inf() ? expf(l[i] - top) : 0.0f;
        total = warp_sum(s);
    }
    uint32_t kept = kAll;
    if constexpr (scored) {
        float c[PER], bias[PER];
        if (biased) load_own(p.bias, p.experts, lane, bias);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            c[i] = neg_inf();
            if (l[i] > neg_inf()) {
                c[i] = p.sigmoid ? sigmoid_choice(l[i]) : __fdiv_rn(expf(l[i] - top), total);
                if (biased) c[i] += bias[i];
                if (!(c[i] > neg_inf())) {
                    c[i] = neg_inf();
                    l[i] = neg_inf();
                }
            }
        }
        // A lane's experts are all of one group, and the group's lanes next to one another: no need of shared memory.
        bool whole = true, stays = true;
        if constexpr (MODE == kGroups) {
            const int shift = lane_shift(p.groups);
            whole = p.experts == (PER << shift) * p.groups;
            float a = neg_inf(), b = neg_inf();       // best, second best
            if (whole) {
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    b = fmaxf(b, fminf(a, c[i]));
                    a = fmaxf(a, c[i]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    if (lane * PER + i < p.experts) vf[lane * PER + i] = c[i];
                __syncwarp();
                scan_group(p, vf, lane, a, b);
                __syncwarp();
            }
            uint32_t doubt = 0;
            int slots = 0;
            kept = keep_groups(p, a, b, lane, doubt, slots);
            if (doubt)
                kept |= far_logits<FP32>(p, t, lane, top) ? settle_groups<FP32, double>(p, t, lane, top, doubt, slots)
                                              : settle_groups<FP32, Df>(p, t, lane, top, doubt, slots);
            stays = (kept >> (lane >> shift << shift)) & 1u;
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const bool ok = l[i] > neg_inf() && (whole ? stays : in_groups(p, kept, lane * PER + i));
            key[i] = ok ? order_key(biased ? c[i] : l[i]) : 0u;
        }
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) key[i] = l[i] > neg_inf() ? order_key(l[i]) : 0u;
    }

    // The k largest keys in order; with a bias one more, to see how close the
    // first that lost came. The take-th largest of the lanes' own maxima
    // bounds the take-th largest of all from below; the few keys that reach
    // it are gathered, one for each lane, and each counts those before it.
    // (One warp-wide maximum after the other over all keys took 60
    // instructions a choice.)
    int mine = -1, lost = -1;
    uint32_t my_key = 0, lost_key = 0;
    const int take = biased ? p.k + 1 : p.k;
    bool emptied = false;            // the keys have been used up
    uint32_t own = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) own = max(own, key[i]);
    uint32_t bound = 1;
    {
        uint32_t left = own;
        for (int j = 0; j < take; ++j) {
            const uint32_t m = __reduce_max_sync(kAll, left);
            if (m == 0) {
                bound = 1;
                break;
            }
            bound = m;
            if (left == m) left = 0;                  // equal maxima go together: the bound only gets lower
        }
    }
    int count = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const bool in = key[i] >= bound;
        const unsigned who = __ballot_sync(kAll, in);
        const int at = count + __popc(who & ((1u << lane) - 1u));
        if (in && at < 32) gathered[at] = make_uint2(key[i], static_cast<uint32_t>(lane * PER + i));
        count += __popc(who);
    }
    __syncwarp();
    if (count <= 32) {
        const uint2 c = lane < count ? gathered[lane] : make_uint2(0, 0);
        __syncwarp();
        int rank = 0;
        for (int o = 0; o < count; ++o) {
            const uint2 d = gathered[o];
            rank += (d.x > c.x || (d.x == c.x && d.y < c.y)) ? 1 : 0;
        }
        __syncwarp();
        if (lane < count && rank < 32) gathered[rank] = c;
        __syncwarp();
        const int n = min(count, p.k);
        if (lane < n) {
            my_key = gathered[lane].x;
            mine = static_cast<int>(gathered[lane].y);
        }
        if (biased && count > p.k) {
            lost_key = gathered[p.k].x;
            lost = static_cast<int>(gathered[p.k].y);
        }
    } else {
        // Many keys reach the bound (ties, or many choices): one after the other.
        emptied = true;
        for (int j = 0; j < take; ++j) {
            uint32_t best = 0;
            int at = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (key[i] > best) {
                    best = key[i];
                    at = lane * PER + i;
                }
            const uint32_t m = __reduce_max_sync(kAll, best);
            if (m == 0) break;
            const int e = static_cast<int>(__reduce_min_sync(kAll, best == m ? static_cast<uint32_t>(at) : 0xFFFFFFFFu));
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (lane * PER + i == e) key[i] = 0;
            if (j == p.k) {
                lost = e;
                lost_key = m;
            }
            if (j < p.k && lane == j) {
                mine = e;
                my_key = m;
            }
        }
    }
    if constexpr (scored) {
        bool close = false;              // two choices whose order matters cannot be told apart
        if (biased) {
            // Each choice against the next one (the last against the best that lost).
            const float rel = p.sigmoid ? kNearSigmoid : kNearSoftmax;
            int ne = __shfl_down_sync(kAll, mine, 1);
            uint32_t nk = __shfl_down_sync(kAll, my_key, 1);
            if (lane == p.k - 1) {
                ne = lost;
                nk = lost_key;
            }
            bool open = false;
            if (lane < p.k && mine >= 0 && ne >= 0) {
                const float hi = key_value(my_key), lo = key_value(nk);
                const float bh = p.bias[mine], bl = p.bias[ne];
                const float own = fabsf(bh) + fabsf(hi);              // >= the score too
                // (a choice of +inf is above every finite one and ties exactly with its like)
                close = hi < pos_inf() && !(hi - lo > rel * (own + fabsf(bl) + fabsf(lo)) + kNearTiny) &&
                        !(bh == bl && logit_at<FP32>(p, t, mine) == logit_at<FP32>(p, t, ne));
                // Farther back may lie one with a larger error (its bias is at most
                // 1 + |c| in size), or one behind exact ties of the last choice.
                open = lane == p.k - 1 && hi < pos_inf() && !(hi - lo > rel * (own + 2.0f * fabsf(lo) + 1.0f));
            }
            close = __any_sync(kAll, close);
            if (!close && __any_sync(kAll, open)) {
                const int last = __shfl_sync(kAll, mine, p.k - 1);
                const uint32_t lk = __shfl_sync(kAll, my_key, p.k - 1);
                const float c = key_value(lk), b = p.bias[last], x = fminf(logit_at<FP32>(p, t, last), kLargest);
                const float low = c - rel * (fabsf(b) + fabsf(c)) - kNearTiny;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int e = lane * PER + i;
                    if (key[i] == 0 || key[i] > lk || (key[i] == lk && e <= last)) continue;   // not one that lost
                    const float ce = key_value(key[i]), be = p.bias[e];
                    if (!(ce + rel * (fabsf(be) + fabsf(ce)) < low) && !(be == b && fminf(logit_at<FP32>(p, t, e), kLargest) == x)) close = true;
                }
                close = __any_sync(kAll, close);
            }
        }
        if (close && !emptied) {
            // The groups stand; whatever may lie above the last choice is put in
            // order again: c >= the last choice less both errors (a score is at
            // most 1, so the other's bias is at most 1 + |c| in size). The last
            // choice is finite: it is no larger than one whose neighbour was close.
            const int last = __shfl_sync(kAll, mine, p.k - 1);
            uint32_t bound2 = 1;
            if (last >= 0) {
                const uint32_t lk = __shfl_sync(kAll, my_key, p.k - 1);
                const float c = key_value(lk);
                bound2 = order_key(c - (p.sigmoid ? kNearSigmoid : kNearSoftmax) * (fabsf(p.bias[last]) + 3.0f * fabsf(c) + 2.0f));
            }
            int n = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const bool in = key[i] >= bound2 && key[i] != 0;
                const unsigned who = __ballot_sync(kAll, in);
                const int at = n + __popc(who & ((1u << lane) - 1u));
                if (in && at < 32) gathered[at] = make_uint2(key[i], static_cast<uint32_t>(lane * PER + i));
                n += __popc(who);
            }
            __syncwarp();
            if (n > 0 && n <= 32) {
                order_candidates<FP32>(p, t, lane, top, gathered, n);
                mine = lane < min(n, p.k) ? static_cast<int>(gathered[lane].y) : -1;
                close = false;
            }
        }
        if (close) {
            if (far_logits<FP32>(p, t, lane, top)) mine = choose_again<FP32, double>(p, t, lane, top, kept, vd);
            else mine = choose_again<FP32, Df>(p, t, lane, top, kept, reinterpret_cast<Df *>(vd));
        }
    }

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
    if (overflowed && !p.sigmoid) w = __int_as_float(0x7fc00000);     // inf - inf: the row has no softmax (by the logits alone w is one already)
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
    begin();
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
    if (bwd) return launch_early(route_bwd_kernel<FP32, PER>, blocks, kWarps * 32, kWarps * PER * 32 * 4, 1, s, p);
    const int smem = kWarps * p.experts * 8;
    if (p.groups > 1) return launch_early(route_kernel<FP32, PER, kGroups>, blocks, kWarps * 32, smem, 1, s, p);
    if (p.bias) return launch_early(route_kernel<FP32, PER, kBias>, blocks, kWarps * 32, smem, 1, s, p);
    return launch_early(route_kernel<FP32, PER, kLogits>, blocks, kWarps * 32, 0, 1, s, p);
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
}  // namespace deto
