// Loads, stores and conversions of eight BF16 values (16 bytes) at a time.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

namespace deto {

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ float bf_at(const uint16_t *p) { return __uint_as_float(static_cast<uint32_t>(*p) << 16); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8])
{
    f[0] = bf_lo(v.x); f[1] = bf_hi(v.x);
    f[2] = bf_lo(v.y); f[3] = bf_hi(v.y);
    f[4] = bf_lo(v.z); f[5] = bf_hi(v.z);
    f[6] = bf_lo(v.w); f[7] = bf_hi(v.w);
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8])
{
    return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}

// Columns [c, c + 8) of a row of `cols` BF16 values; the columns past the
// row's end read as zero and are never touched. c is a multiple of 8 and
// the row starts on a 16-byte boundary.
__device__ __forceinline__ uint4 load8(const uint16_t *row, int c, int cols)
{
    if (c + 8 <= cols) return *reinterpret_cast<const uint4 *>(row + c);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c + i < cols) w[i >> 1] |= static_cast<uint32_t>(row[c + i]) << (16 * (i & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void store8(uint16_t *row, int c, int cols, const uint4 &v)
{
    if (c + 8 <= cols) {
        *reinterpret_cast<uint4 *>(row + c) = v;
        return;
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c + i < cols) row[c + i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
}

// store8 for rows that this launch does not read again: they leave L2 first.
__device__ __forceinline__ void store8_streaming(uint16_t *row, int c, int cols, const uint4 &v)
{
    if (c + 8 <= cols) __stcs(reinterpret_cast<uint4 *>(row + c), v);
    else store8(row, c, cols, v);
}

__device__ __forceinline__ void store8f(float *row, int c, int cols, const float (&f)[8])
{
    if (c + 8 <= cols) {
        *reinterpret_cast<float4 *>(row + c) = make_float4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<float4 *>(row + c + 4) = make_float4(f[4], f[5], f[6], f[7]);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c + i < cols) row[c + i] = f[i];
}

}  // namespace deto
