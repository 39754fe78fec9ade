// Attention of packed sequences and its gradients: one warp for each row of
// the output, 32 keys (or queries) at a time, running maximum and sum.
//
//   out_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i.k_j - m_i),  lse_i = m_i + log sum_j p_ij
//   P = exp(scale q.k - lse), dS = P (dout.v - delta), delta_i = dout_i.out_i
//   dv_j = sum_i P_ij dout_i, dq_i = scale sum_j dS_ij k_j, dk_j = scale sum_i dS_ij q_i
//
// Everything in FP32; a lane holds four columns of the row's sums.
#include "attn_internal.h"
#include "launch.cuh"
#include "ops_internal.h"
#include "vec.cuh"

#include <cmath>

namespace deto {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kWarps = 4;

__device__ __forceinline__ float warp_max(float v)
{
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
}
__device__ __forceinline__ float warp_sum(float v)
{
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

__device__ __forceinline__ float dot(const float *a, const uint16_t *row, int D)
{
    float s = 0.0f;
    for (int c = 0; c < D; c += 8) {
        float f[8];
        unpack8(*reinterpret_cast<const uint4 *>(row + c), f);
        for (int i = 0; i < 8; ++i) s += a[c + i] * f[i];
    }
    return s;
}

// sum += w * row, four columns a lane.
__device__ __forceinline__ void add(float (&sum)[4], float w, const uint16_t *row, int D, int lane)
{
    for (int i = 0; i < 4; ++i)
        if (lane + 32 * i < D) sum[i] += w * bf_at(row + lane + 32 * i);
}

__device__ __forceinline__ void put(uint16_t *row, const float (&v)[4], int D, int lane)
{
    for (int i = 0; i < 4; ++i)
        if (lane + 32 * i < D) row[lane + 32 * i] = static_cast<uint16_t>(pack_bf16(v[i], 0.0f));
}

__device__ __forceinline__ void take(float *dst, const uint16_t *row, int D, int lane)
{
    for (int c = lane; c < D; c += 32) dst[c] = bf_at(row + c);
}

__global__ void __launch_bounds__(32 * kWarps) attn_delta(const AttnParams p)
{
    begin();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, h = blockIdx.y, t = blockIdx.x * kWarps + warp;
    if (t >= p.T) return;
    float d = 0.0f;
    for (int c = lane; c < p.D; c += 32) d += bf_at(p.dout.row(t, h) + c) * bf_at(p.out.row(t, h) + c);
    d = warp_sum(d);
    if (lane == 0) p.delta[static_cast<long long>(h) * p.T + t] = d;
}

__global__ void __launch_bounds__(32 * kWarps) attn_bwd_queries(const AttnParams p)
{
    begin();
    __shared__ float qs[kWarps][128], ds[kWarps][128];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, h = blockIdx.y, g = h / p.G;
    const int t = blockIdx.x * kWarps + warp;
    if (t >= p.T) return;
    const Seq s = seq_at(p, p.qb ? seq_of(p.qb, p.N, t) : 0);
    const int pos = t >= s.q0 && t < s.q1 ? s.position(t) : -1;
    take(qs[warp], p.q.row(t, h), p.D, lane);
    take(ds[warp], p.dout.row(t, h), p.D, lane);
    __syncwarp();
    const float lse = p.lse[static_cast<long long>(h) * p.T + t], delta = p.delta[static_cast<long long>(h) * p.T + t];
    float dq[4] = {};
    for (int j0 = 0; j0 <= pos; j0 += 32) {
        const int j = j0 + lane;
        const bool vis = sees(p, pos, j);
        if (!__any_sync(kFull, vis)) continue;
        float d = 0.0f;
        if (vis) {
            const float pr = expf(p.scale * dot(qs[warp], p.k.row(s.k0 + j, g), p.D) - lse);
            d = pr * (dot(ds[warp], p.v.row(s.k0 + j, g), p.D) - delta) * p.scale;
        }
        unsigned live = __ballot_sync(kFull, vis);
        for (; live; live &= live - 1) {
            const int i = __ffs(live) - 1;
            add(dq, __shfl_sync(kFull, d, i), p.k.row(s.k0 + j0 + i, g), p.D, lane);
        }
    }
    put(p.dq.row(t, h), dq, p.D, lane);
}

__global__ void __launch_bounds__(32 * kWarps) attn_bwd_keys(const AttnParams p)
{
    begin();
    __shared__ float ks[kWarps][128], vs[kWarps][128];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = blockIdx.y;
    const int r = blockIdx.x * kWarps + warp;
    if (r >= p.S) return;
    const Seq s = seq_at(p, p.kb ? seq_of(p.kb, p.N, r) : 0);
    const int j = r - s.k0, n = r >= s.k0 && r < s.k1 ? s.queries() : 0;
    take(ks[warp], p.k.row(r, g), p.D, lane);
    take(vs[warp], p.v.row(r, g), p.D, lane);
    __syncwarp();
    float dk[4] = {}, dv[4] = {};
    const int first = max(0, j - (s.keys() - s.queries())) & ~31;
    for (int i0 = first; i0 < n; i0 += 32) {
        const int t = s.q0 + i0 + lane;
        const bool vis = i0 + lane < n && sees(p, s.position(t), j);
        if (!__any_sync(kFull, vis)) continue;
        for (int h = g * p.G; h < (g + 1) * p.G; ++h) {
            float pr = 0.0f, d = 0.0f;
            if (vis) {
                const long long at = static_cast<long long>(h) * p.T + t;
                pr = expf(p.scale * dot(ks[warp], p.q.row(t, h), p.D) - p.lse[at]);
                d = pr * (dot(vs[warp], p.dout.row(t, h), p.D) - p.delta[at]) * p.scale;
            }
            unsigned live = __ballot_sync(kFull, vis);
            for (; live; live &= live - 1) {
                const int i = __ffs(live) - 1;
                add(dk, __shfl_sync(kFull, d, i), p.q.row(s.q0 + i0 + i, h), p.D, lane);
                add(dv, __shfl_sync(kFull, pr, i), p.dout.row(s.q0 + i0 + i, h), p.D, lane);
            }
        }
    }
    put(p.dk.row(r, g), dk, p.D, lane);
    put(p.dv.row(r, g), dv, p.D, lane);
}

// One warp for each sequence and head.
__global__ void __launch_bounds__(32 * kWarps) attn_decode_rows(const DecodeParams p)
{
    begin();
    __shared__ float qs[kWarps][128];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, h = blockIdx.y * kWarps + warp, b = blockIdx.x;
    if (h >= p.H) return;
    const int g = h / p.G;
    take(qs[warp], p.q.row(b, h), p.D, lane);
    __syncwarp();
    const long long room = static_cast<long long>(p.max_pages) * p.page_size;
    const int given = p.lengths[b];
    const int n = given < 0 ? 0 : given > room ? static_cast<int>(room) : given;
    bool bad = n != given;
    float m = -INFINITY, l = 0.0f, o[4] = {};
    for (int j0 = 0; j0 < n; j0 += 32) {
        const int j = j0 + lane;
        bool vis = j < n && (n - 1 - j < p.window || j < p.sinks);
        const int page = vis ? p.table[b * p.ldt + j / p.page_size] : -1;
        if (vis && (page < 0 || page >= p.pages)) {
            bad = true;
            vis = false;
        }
        if (!__any_sync(kFull, vis)) continue;
        const float x = vis ? p.scale * dot(qs[warp], p.kc.row(page, j % p.page_size, g), p.D) : -INFINITY;
        const float top = fmaxf(m, warp_max(x));
        const float old = m == -INFINITY ? 0.0f : expf(m - top);
        const float e = vis ? expf(x - top) : 0.0f;
        l = l * old + warp_sum(e);
        for (float &v : o) v *= old;
        m = top;
        unsigned live = __ballot_sync(kFull, vis);
        for (; live; live &= live - 1) {
            const int i = __ffs(live) - 1;
            add(o, __shfl_sync(kFull, e, i), p.vc.row(__shfl_sync(kFull, page, i), (j0 + i) % p.page_size, g), p.D, lane);
        }
    }
    if (bad) atomicExch(p.status, kStatusInvalid);
    for (float &v : o) v = m == -INFINITY ? 0.0f : v / l;
    put(p.out.row(b, h), o, p.D, lane);
}

dim3 grid(int rows, int y) { return dim3(static_cast<unsigned>((rows + kWarps - 1) / kWarps), static_cast<unsigned>(y)); }

}  // namespace

cudaError_t launch_attn_bwd(const AttnParams &p, int, cudaStream_t s)
{
    if (p.T > 0) {
        attn_delta<<<grid(p.T, p.H), 32 * kWarps, 0, s>>>(p);
        attn_bwd_queries<<<grid(p.T, p.H), 32 * kWarps, 0, s>>>(p);
    }
    if (p.S > 0) attn_bwd_keys<<<grid(p.S, p.KV), 32 * kWarps, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_attn_decode(const DecodeParams &p, int, cudaStream_t s)
{
    attn_decode_rows<<<dim3(p.B, (p.H + kWarps - 1) / kWarps), 32 * kWarps, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace deto
