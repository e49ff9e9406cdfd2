// rowvec.cuh -- eight consecutive elements of a row as fp32 registers, for kernels that walk
// rows of any width.  VEC: the width is a multiple of 8 and rows start on 16 bytes, so the
// eight elements move in 16-byte accesses; otherwise each element is checked against the
// row's end and moves by itself.
#pragma once

#include <cuda_bf16.h>

namespace hstu {

constexpr unsigned kFullMask = 0xffffffffu;

// Plain loads, not the read-only path: a caller may pass one tensor as input and output.

template <bool VEC>
__device__ __forceinline__ void load8(const __nv_bfloat16 *row, int i, int width, float (&f)[8])
{
    if constexpr (VEC) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (i < width) v = *reinterpret_cast<const uint4 *>(row + i);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f[2 * e] = __uint_as_float(u[e] << 16);
            f[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = i + e < width ? __bfloat162float(row[i + e]) : 0.f;
    }
}

template <bool VEC>
__device__ __forceinline__ void load8(const float *row, int i, int width, float (&f)[8])
{
    if constexpr (VEC) {
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
        if (i < width) {
            a = reinterpret_cast<const float4 *>(row + i)[0];
            b = reinterpret_cast<const float4 *>(row + i)[1];
        }
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = i + e < width ? row[i + e] : 0.f;
    }
}

template <bool VEC>
__device__ __forceinline__ void store8(__nv_bfloat16 *row, int i, int width, const float (&f)[8])
{
    if constexpr (VEC) {
        if (i >= width) return;
        uint32_t u[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
            u[e] = *reinterpret_cast<const uint32_t *>(&p);
        }
        *reinterpret_cast<uint4 *>(row + i) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (i + e < width) row[i + e] = __float2bfloat16_rn(f[e]);
    }
}

template <bool VEC>
__device__ __forceinline__ void store8(float *row, int i, int width, const float (&f)[8])
{
    if constexpr (VEC) {
        if (i >= width) return;
        reinterpret_cast<float4 *>(row + i)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4 *>(row + i)[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (i + e < width) row[i + e] = f[e];
    }
}

}  // namespace hstu
