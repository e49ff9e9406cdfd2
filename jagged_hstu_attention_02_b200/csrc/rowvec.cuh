// rowvec.cuh -- 256 consecutive elements of a row per warp, 8 neighbours per lane as fp32
// registers, for kernels that walk rows.
//
// VEC: the width is a multiple of 8, so every row starts on 16 bytes and a lane's 8 elements
// move in 16-byte accesses (the norm, and combine of such widths).  Otherwise rows start anywhere,
// and this is the norm's way, whose input and output rows have the same number and so lie alike in
// every tensor of the same type.  A warp's 256 elements then start `lead` elements in front of where
// they otherwise would, such that a lane's 8 lie on aligned addresses of the row: only its first and
// last piece are cut to single elements.  What lies otherwise (the weights, which start on 16 bytes)
// is read as the aligned pieces that cover it, and a lane puts its elements together from two of
// them (a shuffle and a funnel shift).
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace hstu {

constexpr unsigned kFullMask = 0xffffffffu;

// First element of a lane's 8 of the 256 that start at c0.
__device__ __forceinline__ int elem8(int c0) { return c0 + 8 * (int)(threadIdx.x & 31); }

__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8])
{
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        f[2 * e] = __uint_as_float(u[e] << 16);
        f[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack8_bf16(const float (&f)[8])
{
    uint32_t u[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
        u[e] = *reinterpret_cast<const uint32_t *>(&p);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// x[i] <- the 4 bytes at byte offset `off` + 4 i of x (off uniform in the warp, below 4 M).
template <int N, int M>
__device__ __forceinline__ void shift_words(uint32_t (&x)[N], int off)
{
    const int words = off >> 2, bits = (off & 3) * 8;
#pragma unroll
    for (int m = 1; m <= M; m <<= 1)
        if (words & m) {
#pragma unroll
            for (int i = 0; i + m < N; ++i) x[i] = x[i + m];
        }
    if (bits) {
#pragma unroll
        for (int i = 0; i + 1 < N; ++i) x[i] = __funnelshift_r(x[i], x[i + 1], bits);
    }
}

// The 16 bytes at the 16-byte-aligned p, where it lies in the tensor [begin, end): zeros
// outside (begin is on 16 bytes, end may cut the last piece).
__device__ __forceinline__ void load_piece(const uint8_t *p, const uint8_t *begin, const uint8_t *end,
                                           uint32_t *w)
{
    if (p >= begin && p + 16 <= end) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else if (p >= begin) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (p + i < end) w[i / 4] |= (uint32_t)p[i] << (8 * (i % 4));
    }
}

// NW words per lane from p on, wherever p lies: what [from, to) holds, other bytes arbitrary.
// All lanes of the warp together.
template <int NW>
__device__ __forceinline__ void load_words(const uint8_t *p, const uint8_t *from, const uint8_t *to,
                                           const uint8_t *begin, const uint8_t *end,
                                           uint32_t (&r)[NW])
{
    const int lane = threadIdx.x & 31;
    const int off = (int)(reinterpret_cast<uintptr_t>(p) & 15);
    const uint8_t *at = p - off + 4 * NW * lane;
    uint32_t x[NW + 4] = {};
    const uint8_t *first = p - off;                   // the pieces' span, against the row's
    if (first >= from && first + 128 * NW + 16 <= to) {
#pragma unroll
        for (int k = 0; k < NW; k += 4) {
            const uint4 v = *reinterpret_cast<const uint4 *>(at + 4 * k);
            x[k] = v.x; x[k + 1] = v.y; x[k + 2] = v.z; x[k + 3] = v.w;
        }
        if (off) {
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (lane == 31) v = *reinterpret_cast<const uint4 *>(at + 4 * NW);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t u = __shfl_down_sync(kFullMask, x[i], 1);
                x[NW + i] = lane == 31 ? w[i] : u;
            }
            shift_words<NW + 4, 2>(x, off);
        }
#pragma unroll
        for (int i = 0; i < NW; ++i) r[i] = x[i];
        return;
    }
#pragma unroll
    for (int k = 0; k < NW; k += 4)
        if (at + 4 * k < to && at + 4 * k + 16 > from) load_piece(at + 4 * k, begin, end, x + k);
    if (off) {
        uint32_t w[4] = {};
        if (lane == 31 && at + 4 * NW < to) load_piece(at + 4 * NW, begin, end, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t u = __shfl_down_sync(kFullMask, x[i], 1);
            x[NW + i] = lane == 31 ? w[i] : u;
        }
        shift_words<NW + 4, 2>(x, off);
    }
#pragma unroll
    for (int i = 0; i < NW; ++i) r[i] = x[i];
}

// The elements (of ES bytes) among the 4 PW bytes for address p that lie in [from, to).
template <int PW, int ES>
__device__ __forceinline__ void store_cut(uint8_t *p, const uint32_t *w, const uint8_t *from,
                                          const uint8_t *to)
{
#pragma unroll
    for (int i = 0; i < 4 * PW; i += ES)
        if (p + i >= from && p + i < to) {
            const uint32_t v = w[i / 4] >> (8 * (i % 4));
            if constexpr (ES == 4) *reinterpret_cast<uint32_t *>(p + i) = v;
            if constexpr (ES == 2) *reinterpret_cast<uint16_t *>(p + i) = (uint16_t)v;
            if constexpr (ES == 1) p[i] = (uint8_t)v;
        }
}

// NW words per lane to where p lies, aligned to them (at most 16 bytes), as far as [from, to)
// reaches; elements of ES bytes.
template <int NW, int ES>
__device__ __forceinline__ void store_words(uint8_t *p, const uint8_t *from, const uint8_t *to,
                                            const uint32_t (&r)[NW])
{
    uint8_t *at = p + 4 * NW * (int)(threadIdx.x & 31);
    if (at >= from && at + 4 * NW <= to) {
        if constexpr (NW == 2) *reinterpret_cast<uint2 *>(at) = make_uint2(r[0], r[1]);
        else {
#pragma unroll
            for (int k = 0; k < NW; k += 4)
                *reinterpret_cast<uint4 *>(at + 4 * k) = make_uint4(r[k], r[k + 1], r[k + 2], r[k + 3]);
        }
    } else if (at < to && at + 4 * NW > from) {
        store_cut<NW, ES>(at, r, from, to);
    }
}

// How far in front of its elements a warp's window starts, for rows of `width` elements.
template <bool VEC>
__device__ __forceinline__ int lead_of(int64_t row, int width)
{
    return VEC ? 0 : (int)(((uint32_t)row * (uint32_t)width) & 7u);
}

// 16 bytes of global memory if `yes`, else zeros.  (Inline, so that the compiler keeps a batch of these loads in
// front of the first use: it had sunk them into the uses, one latency after another.)
__device__ __forceinline__ void load16_if(const void *p, bool yes, uint32_t *v)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "@q ld.global.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=&r"(v[0]), "=&r"(v[1]), "=&r"(v[2]), "=&r"(v[3])
        : "l"(p), "r"((int)yes));
}

// A lane's 8 elements of the 256 from c0 on, as they lie in memory, fetched ahead of their use.
// Elements outside the row read as 0.  Plain loads, not the read-only path: a caller may pass
// one tensor as input and output.  [begin, end): the row's tensor (used where rows start
// anywhere).
template <typename T, bool VEC> struct Piece {
    static constexpr int NW = sizeof(T) == 2 ? 4 : 8;
    uint32_t v[NW];
    __device__ __forceinline__ void load(const T *row, int c0, int width, const T *begin, const T *end)
    {
        const int i = elem8(c0);
        if constexpr (VEC) {
#pragma unroll
            for (int k = 0; k < NW; k += 4)
                load16_if(reinterpret_cast<const uint4 *>(row + i) + k / 4, i < width, v + k);
        } else {
            // a window inside the row: nothing to cut (and, often, nothing to shift)
            const bool inside = c0 >= 0 && c0 + 256 <= width;
            if (inside && (reinterpret_cast<uintptr_t>(row + c0) & 15) == 0) {
#pragma unroll
                for (int k = 0; k < NW; k += 4) {
                    const uint4 u = reinterpret_cast<const uint4 *>(row + i)[k / 4];
                    v[k] = u.x; v[k + 1] = u.y; v[k + 2] = u.z; v[k + 3] = u.w;
                }
                return;
            }
            load_words<NW>(reinterpret_cast<const uint8_t *>(row + c0),
                           reinterpret_cast<const uint8_t *>(row),
                           reinterpret_cast<const uint8_t *>(row + width),
                           reinterpret_cast<const uint8_t *>(begin),
                           reinterpret_cast<const uint8_t *>(end), v);
            if (inside) return;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (i + e < 0 || i + e >= width) {
                    if constexpr (sizeof(T) == 4) v[e] = 0u;
                    else v[e / 2] &= e % 2 ? 0x0000FFFFu : 0xFFFF0000u;
                }
        }
    }
    __device__ __forceinline__ void get(float (&f)[8]) const
    {
        if constexpr (sizeof(T) == 2) {
            unpack8(make_uint4(v[0], v[1], v[2], v[3]), f);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(v[e]);
        }
    }
};

template <bool VEC, typename T>
__device__ __forceinline__ void load8(const T *row, int c0, int width, const T *begin, const T *end,
                                      float (&f)[8])
{
    if constexpr (VEC) {                     // (the row may be in shared memory)
        const int i = elem8(c0);
        uint4 v[sizeof(T) / 2] = {};
#pragma unroll
        for (int k = 0; k < (int)sizeof(T) / 2; ++k)
            if (i < width) v[k] = reinterpret_cast<const uint4 *>(row + i)[k];
        if constexpr (sizeof(T) == 2) {
            unpack8(v[0], f);
        } else {
            f[0] = __uint_as_float(v[0].x); f[1] = __uint_as_float(v[0].y);
            f[2] = __uint_as_float(v[0].z); f[3] = __uint_as_float(v[0].w);
            f[4] = __uint_as_float(v[1].x); f[5] = __uint_as_float(v[1].y);
            f[6] = __uint_as_float(v[1].z); f[7] = __uint_as_float(v[1].w);
        }
    } else {
        Piece<T, false> p;
        p.load(row, c0, width, begin, end);
        p.get(f);
    }
}

// Rows that start anywhere: row + c0 lies on a lane's boundary (lead_of).
template <bool VEC>
__device__ __forceinline__ void store8(__nv_bfloat16 *row, int c0, int width, const float (&f)[8])
{
    const uint4 v = pack8_bf16(f);
    if constexpr (VEC) {
        if (elem8(c0) < width) *reinterpret_cast<uint4 *>(row + elem8(c0)) = v;
    } else {
        if (c0 >= 0 && c0 + 256 <= width) {
            *reinterpret_cast<uint4 *>(row + elem8(c0)) = v;
            return;
        }
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
        store_words<4, 2>(reinterpret_cast<uint8_t *>(row + c0), reinterpret_cast<uint8_t *>(row),
                          reinterpret_cast<uint8_t *>(row + width), u);
    }
}

template <bool VEC>
__device__ __forceinline__ void store8(float *row, int c0, int width, const float (&f)[8])
{
    const int i = elem8(c0);
    if (VEC || (c0 >= 0 && c0 + 256 <= width)) {
        if (i >= width) return;
        reinterpret_cast<float4 *>(row + i)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4 *>(row + i)[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
        uint32_t u[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = __float_as_uint(f[e]);
        store_words<8, 4>(reinterpret_cast<uint8_t *>(row + c0), reinterpret_cast<uint8_t *>(row),
                          reinterpret_cast<uint8_t *>(row + width), u);
    }
}

}  // namespace hstu
