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

}  // namespace

cudaError_t launch_attn_decode(const DecodeParams &p, int, cudaStream_t s)
{
    attn_decode_rows<<<dim3(p.B, (p.H + kWarps - 1) / kWarps), 32 * kWarps, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace deto
