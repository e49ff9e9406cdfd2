// rowvec.cuh -- 256 consecutive elements of a row per warp, 8 of them per lane as fp32 registers,
// for kernels that walk rows of any width.  VEC (the width is a multiple of 8 and rows start on
// 16 bytes): a lane holds 8 neighbours, moved in 16-byte accesses.  Otherwise a lane holds every
// 32nd element, each checked against the row's end, so that a warp's access is one run of
// neighbours whatever the row's alignment (8 neighbours per lane, one by one, took 2 to 4 times
// as long: every access touched as many sectors as a 16-byte one for an eighth of the data).
#pragma once

#include <cuda_bf16.h>

namespace hstu {

constexpr unsigned kFullMask = 0xffffffffu;

// Index of a lane's element e of the 256 that start at c0.
template <bool VEC>
__device__ __forceinline__ int elem8(int c0, int e)
{
    const int lane = threadIdx.x & 31;
    return VEC ? c0 + 8 * lane + e : c0 + 32 * e + lane;
}

__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8])
{
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        f[2 * e] = __uint_as_float(u[e] << 16);
        f[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
    }
}

// Plain loads, not the read-only path: a caller may pass one tensor as input and output.
// Elements past the row's end read as 0.  `row` may be in shared memory.
template <bool VEC>
__device__ __forceinline__ void load8(const __nv_bfloat16 *row, int c0, int width, float (&f)[8])
{
    if constexpr (VEC) {
        const int i = elem8<true>(c0, 0);
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (i < width) v = *reinterpret_cast<const uint4 *>(row + i);
        unpack8(v, f);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = elem8<false>(c0, e);
            f[e] = i < width ? __bfloat162float(row[i]) : 0.f;
        }
    }
}

template <bool VEC>
__device__ __forceinline__ void load8(const float *row, int c0, int width, float (&f)[8])
{
    if constexpr (VEC) {
        const int i = elem8<true>(c0, 0);
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
        if (i < width) {
            a = reinterpret_cast<const float4 *>(row + i)[0];
            b = reinterpret_cast<const float4 *>(row + i)[1];
        }
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = elem8<false>(c0, e);
            f[e] = i < width ? row[i] : 0.f;
        }
    }
}

template <bool VEC>
__device__ __forceinline__ void store8(__nv_bfloat16 *row, int c0, int width, const float (&f)[8])
{
    if constexpr (VEC) {
        const int i = elem8<true>(c0, 0);
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
        for (int e = 0; e < 8; ++e) {
            const int i = elem8<false>(c0, e);
            if (i < width) row[i] = __float2bfloat16_rn(f[e]);
        }
    }
}

template <bool VEC>
__device__ __forceinline__ void store8(float *row, int c0, int width, const float (&f)[8])
{
    if constexpr (VEC) {
        const int i = elem8<true>(c0, 0);
        if (i >= width) return;
        reinterpret_cast<float4 *>(row + i)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4 *>(row + i)[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = elem8<false>(c0, e);
            if (i < width) row[i] = f[e];
        }
    }
}

}  // namespace hstu
