// rmsnorm.cu -- root-mean-square norm of rows with the residual's addition, output in the
// rows' type or in 8 bits (e4m3) with scales, and the gradients.
//
//   h = x + residual;  rstd = 1 / sqrt(mean(h^2) + eps);  y = h * rstd * weight
//   e4m3: per group of columns (or per row) scale = max|y| / 448, q = y / scale to nearest
//   backward at the stored h, with xh = h * rstd and g = dy * weight:
//     dx = rstd * (g - xh * mean(g * xh)) + dsum;   dweight = sum over rows of dy * xh
//
// Bound by memory: every tensor is read or written once, so a row stays in registers between
// the sum of squares and the output.  W warps share a row (each thread NC chunks of 8
// elements), and a block of several narrow rows or one wide row keeps 256 threads or more.
// The forward normalises the fp32 sum, before it is rounded to the stored h.
#include <cuda_fp8.h>

#include <type_traits>

#include "experts.h"
#include "kernels.h"
#include "lnrow.cuh"
#include "rowvec.cuh"

namespace hstu {

namespace {

constexpr float kE4m3Max = 448.f;

// The largest magnitude that a group's scale maps to 448: its own, kept away from where
// 448 / m overflows; 0 for a group of zeros, whose scale and values are then 0.
__device__ __forceinline__ float scale_top(float m)
{
    return m > 0.f ? fmaxf(m, 7.888609e-31f /* 2^-100 */) : 0.f;
}

// Sum over the W warps of each row group of the block; every thread gets its group's sum.
template <int W>
__device__ __forceinline__ float group_sum(float v, float *buf)
{
    v = warp_sum(v);
    if constexpr (W == 1) return v;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) buf[warp] = v;
    __syncthreads();
    float s = 0.f;
    const float *g = buf + warp / W * W;
#pragma unroll
    for (int i = 0; i < W; ++i) s += g[i];
    return s;
}

template <int W>
__device__ __forceinline__ float group_max(float v, float *buf)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFullMask, v, o));
    if constexpr (W == 1) return v;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) buf[warp] = v;
    __syncthreads();
    float s = 0.f;
    const float *g = buf + warp / W * W;
#pragma unroll
    for (int i = 0; i < W; ++i) s = fmaxf(s, g[i]);
    return s;
}

template <bool VEC>
__device__ __forceinline__ void store8_e4m3(uint8_t *row, int i, int width, const float (&f)[8])
{
    if constexpr (VEC) {
        if (i >= width) return;
        uint32_t u[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * e], f[4 * e + 1]),
                                                         __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * e + 2], f[4 * e + 3]),
                                                         __NV_SATFINITE, __NV_E4M3);
            u[e] = lo | hi << 16;
        }
        *reinterpret_cast<uint2 *>(row + i) = make_uint2(u[0], u[1]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (i + e < width) row[i + e] = __nv_cvt_float_to_fp8(f[e], __NV_SATFINITE, __NV_E4M3);
    }
}

template <int W> struct NormShape {
    static constexpr int kWarps = W < 8 ? 8 : W;
    static constexpr int kRows = kWarps / W;       // rows per block
};

template <typename T, int W, int NC, bool E4M3, bool VEC>
__global__ void __launch_bounds__(32 * NormShape<W>::kWarps)
    rms_norm_kernel(const __grid_constant__ RmsArgs a)
{
    constexpr int kRows = NormShape<W>::kRows;
    __shared__ float buf[2][NormShape<W>::kWarps];
    const int t = threadIdx.x % (32 * W);
    const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / (32 * W);
    const bool live = row < a.rows;
    const int width = live ? a.width : 0;
    const int64_t base = live ? row * a.width : 0;
    const T *x = reinterpret_cast<const T *>(a.x) + base;
    const T *r = reinterpret_cast<const T *>(a.resid) + base;
    float h[NC][8];
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c) load8<VEC>(x, (c * 32 * W + t) * 8, width, h[c]);
    if (a.resid) {
        float b[NC][8];
#pragma unroll
        for (int c = 0; c < NC; ++c) load8<VEC>(r, (c * 32 * W + t) * 8, width, b[c]);
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int e = 0; e < 8; ++e) h[c][e] += b[c][e];
    }
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(h[c][e], h[c][e], ss);
    ss = group_sum<W>(ss, buf[0]);
    const float rs = rsqrtf(ss / (float)a.width + a.eps);
    if (a.rstd && live && t == 0) a.rstd[row] = rs;
    if (a.sum) {
        T *s = reinterpret_cast<T *>(a.sum) + base;
#pragma unroll
        for (int c = 0; c < NC; ++c) store8<VEC>(s, (c * 32 * W + t) * 8, width, h[c]);
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        float w[8];
        if (a.weight) load8<VEC>(a.weight, (c * 32 * W + t) * 8, width, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[c][e] = a.weight ? h[c][e] * rs * w[e] : h[c][e] * rs;
    }
    if constexpr (!E4M3) {
        T *y = reinterpret_cast<T *>(a.y) + base;
#pragma unroll
        for (int c = 0; c < NC; ++c) store8<VEC>(y, (c * 32 * W + t) * 8, width, h[c]);
    } else {
        uint8_t *y = reinterpret_cast<uint8_t *>(a.y) + base;
        float m[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            m[c] = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) m[c] = fmaxf(m[c], fabsf(h[c][e]));
        }
        if (a.group == 0) {
            float mm = m[0];
#pragma unroll
            for (int c = 1; c < NC; ++c) mm = fmaxf(mm, m[c]);
            mm = scale_top(group_max<W>(mm, buf[1]));
#pragma unroll
            for (int c = 0; c < NC; ++c) m[c] = mm;
            if (live && t == 0) a.scales[row] = mm * (1.f / kE4m3Max);
        } else {
            const int lanes = a.group / 8;              // 4, 8 or 16 neighbouring threads
            const int groups = (a.width + a.group - 1) / a.group;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                for (int o = lanes / 2; o > 0; o >>= 1)
                    m[c] = fmaxf(m[c], __shfl_xor_sync(kFullMask, m[c], o));
                m[c] = scale_top(m[c]);
                const int i = (c * 32 * W + t) * 8;
                if (i < width && t % lanes == 0)
                    a.scales[row * groups + i / a.group] = m[c] * (1.f / kE4m3Max);
            }
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const float back = m[c] > 0.f ? kE4m3Max / m[c] : 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) h[c][e] *= back;
            store8_e4m3<VEC>(y, (c * 32 * W + t) * 8, width, h[c]);
        }
    }
}

// Each block walks rows with a stride of the grid and keeps its columns' part of the weight
// gradient in registers; the parts meet in shared memory and leave as one row of `part` per
// block, which rms_dweight_kernel adds in a fixed order.
template <typename T, int W, int NC, bool VEC>
__global__ void __launch_bounds__(32 * NormShape<W>::kWarps)
    rms_norm_bwd_kernel(const __grid_constant__ RmsBwdArgs a)
{
    constexpr int kRows = NormShape<W>::kRows;
    constexpr int kWarps = NormShape<W>::kWarps;
    __shared__ float buf[2][kWarps];
    extern __shared__ float dws[];                      // [kRows][width] when kRows > 1
    const int t = threadIdx.x % (32 * W);
    const int sub = threadIdx.x / (32 * W);
    float acc[NC][8];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[c][e] = 0.f;
    int parity = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * kRows; row0 < a.rows;
         row0 += (int64_t)gridDim.x * kRows, parity ^= 1) {
        const int64_t row = row0 + sub;
        const bool live = row < a.rows;
        const int width = live ? a.width : 0;
        const int64_t base = live ? row * a.width : 0;
        const T *dy = reinterpret_cast<const T *>(a.dy) + base;
        const T *hp = reinterpret_cast<const T *>(a.h) + base;
        const float rs = live ? a.rstd[row] : 0.f;
        float g[NC][8], h[NC][8];
        float dot = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            load8<VEC>(dy, (c * 32 * W + t) * 8, width, g[c]);
            load8<VEC>(hp, (c * 32 * W + t) * 8, width, h[c]);
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            float w[8];
            if (a.weight) load8<VEC>(a.weight, (c * 32 * W + t) * 8, width, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                h[c][e] *= rs;
                acc[c][e] = fmaf(g[c][e], h[c][e], acc[c][e]);
                if (a.weight) g[c][e] *= w[e];
                dot = fmaf(g[c][e], h[c][e], dot);
            }
        }
        dot = group_sum<W>(dot, buf[parity]) / (float)a.width;
        T *dx = reinterpret_cast<T *>(a.dx) + base;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            float o[8];
            if (a.dsum)
                load8<VEC>(reinterpret_cast<const T *>(a.dsum) + base, (c * 32 * W + t) * 8, width, o);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = rs * (g[c][e] - h[c][e] * dot);
                o[e] = a.dsum ? d + o[e] : d;
            }
            store8<VEC>(dx, (c * 32 * W + t) * 8, width, o);
        }
    }
    if (!a.dweight) return;
    float *part = a.part + (int64_t)blockIdx.x * a.width;
    if constexpr (kRows == 1) {
#pragma unroll
        for (int c = 0; c < NC; ++c) store8<VEC>(part, (c * 32 * W + t) * 8, a.width, acc[c]);
    } else {
#pragma unroll
        for (int c = 0; c < NC; ++c)
            store8<VEC>(dws + sub * a.width, (c * 32 * W + t) * 8, a.width, acc[c]);
        __syncthreads();
        for (int i = threadIdx.x; i < a.width; i += blockDim.x) {
            float s = 0.f;
#pragma unroll
            for (int q = 0; q < kRows; ++q) s += dws[q * a.width + i];
            part[i] = s;
        }
    }
}

// dweight[i] = sum of the blocks' parts, in block order within each of 8 strands, the
// strands in order: the same result every time.
__global__ void __launch_bounds__(256) rms_dweight_kernel(const float *__restrict__ part,
                                                          int blocks, int width,
                                                          float *__restrict__ dweight)
{
    __shared__ float s[8][32];
    grid_dep_wait();
    const int lane = threadIdx.x & 31, strand = threadIdx.x >> 5;
    const int i = blockIdx.x * 32 + lane;
    float v = 0.f;
    if (i < width) {
#pragma unroll 4
        for (int b = strand; b < blocks; b += 8) v += part[(int64_t)b * width + i];
    }
    s[strand][lane] = v;
    __syncthreads();
    if (strand == 0 && i < width) {
        float r = 0.f;
#pragma unroll
        for (int q = 0; q < 8; ++q) r += s[q][lane];
        dweight[i] = r;
    }
}

// Warps per row: two chunks of 8 elements per thread, so 512 columns per warp.
int warps_for(int width)
{
    int w = 1;
    while (w < 32 && w * 512 < width) w *= 2;
    return w;
}

template <typename T, bool E4M3, int W>
cudaError_t run_fwd(const RmsArgs &a, cudaStream_t st)
{
    constexpr int kRows = NormShape<W>::kRows;
    const unsigned grid = (unsigned)((a.rows + kRows - 1) / kRows);
    const unsigned thr = 32 * NormShape<W>::kWarps;
    if (a.width % 8 == 0)
        rms_norm_kernel<T, W, 2, E4M3, true><<<grid, thr, 0, st>>>(a);
    else
        rms_norm_kernel<T, W, 2, E4M3, false><<<grid, thr, 0, st>>>(a);
    return cudaGetLastError();
}

template <typename T, bool E4M3>
cudaError_t fwd_w(const RmsArgs &a, cudaStream_t st)
{
    switch (warps_for(a.width)) {
    case 1: return run_fwd<T, E4M3, 1>(a, st);
    case 2: return run_fwd<T, E4M3, 2>(a, st);
    case 4: return run_fwd<T, E4M3, 4>(a, st);
    case 8: return run_fwd<T, E4M3, 8>(a, st);
    case 16: return run_fwd<T, E4M3, 16>(a, st);
    default: return run_fwd<T, E4M3, 32>(a, st);
    }
}

template <typename T, int W>
cudaError_t run_bwd(const RmsBwdArgs &a, cudaStream_t st)
{
    constexpr int kRows = NormShape<W>::kRows;
    const unsigned thr = 32 * NormShape<W>::kWarps;
    const int blocks = rms_bwd_blocks(a.rows, a.width);
    const size_t smem = kRows > 1 && a.dweight ? (size_t)kRows * a.width * 4 : 0;
    if (a.width % 8 == 0)
        rms_norm_bwd_kernel<T, W, 2, true><<<blocks, thr, smem, st>>>(a);
    else
        rms_norm_bwd_kernel<T, W, 2, false><<<blocks, thr, smem, st>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !a.dweight) return e;
    return launch_pdl(rms_dweight_kernel, dim3((a.width + 31) / 32), dim3(256), 0, st,
                      (const float *)a.part, blocks, a.width, a.dweight);
}

template <typename T>
cudaError_t bwd_w(const RmsBwdArgs &a, cudaStream_t st)
{
    switch (warps_for(a.width)) {
    case 1: return run_bwd<T, 1>(a, st);
    case 2: return run_bwd<T, 2>(a, st);
    case 4: return run_bwd<T, 4>(a, st);
    case 8: return run_bwd<T, 8>(a, st);
    case 16: return run_bwd<T, 16>(a, st);
    default: return run_bwd<T, 32>(a, st);
    }
}

}  // namespace

int rms_bwd_blocks(int64_t rows, int width)
{
    const int w = warps_for(width), per = w < 8 ? 8 / w : 1;
    const int64_t need = (rows + per - 1) / per;
    const int64_t most = 296;
    return (int)(need < 1 ? 1 : need < most ? need : most);
}

cudaError_t launch_rms_norm(const RmsArgs &a, bool f32, bool e4m3, cudaStream_t st)
{
    if (a.rows <= 0) return cudaSuccess;
    if (f32) return e4m3 ? fwd_w<float, true>(a, st) : fwd_w<float, false>(a, st);
    return e4m3 ? fwd_w<__nv_bfloat16, true>(a, st) : fwd_w<__nv_bfloat16, false>(a, st);
}

cudaError_t launch_rms_norm_bwd(const RmsBwdArgs &a, bool f32, cudaStream_t st)
{
    if (a.rows <= 0)
        return a.dweight ? cudaMemsetAsync(a.dweight, 0, (size_t)a.width * 4, st) : cudaSuccess;
    return f32 ? bwd_w<float>(a, st) : bwd_w<__nv_bfloat16>(a, st);
}

}  // namespace hstu
