// rmsnorm.cu -- root-mean-square norm of rows with the residual's addition, output in the
// rows' type or in 8 bits (e4m3) with scales, and the gradients.
//
//   h = x + residual;  rstd = 1 / sqrt(mean(h^2) + eps);  y = h * rstd * weight
//   e4m3: per group of columns (or per row) scale = max|y| / 448, q = y / scale to nearest
//   backward at the stored h, with xh = h * rstd and g = dy * weight:
//     dx = rstd * (g - xh * mean(g * xh)) + dsum;   dweight = sum over rows of dy * xh
//
// Bound by memory: every tensor is read or written once.  W warps (a group) share a row, each
// thread 2 chunks of 8 elements, kept in registers between the sum of squares and the output.
// A group's chain per row (load, sum, scale, store) is all latency, so with more rows than
// groups the groups stay and their rows arrive ahead of them through a ring of bulk copies in
// shared memory (RING); with fewer they load directly.  Rows that start anywhere come with the rest
// of their first and last 16 bytes (SHIFTED_RING; 16384 x 1001 bf16, against direct loads: forward
// 41.7 -> 31.0 us, to e4m3 59.3 -> 47.4, backward 71.6 -> 38.1).
// The forward normalises the fp32 sum, before it is rounded to the stored h.
#include <cuda_fp8.h>
#include <math_constants.h>

#include <algorithm>

#include "experts.h"
#include "kernels.h"
#include "lnrow.cuh"
#include "rowvec.cuh"
#include "sm100.cuh"

namespace hstu {

namespace {

using sm100::mbar_arrive_expect_tx;
using sm100::mbar_init;
using sm100::mbar_try_wait;
using sm100::named_bar_sync;
using sm100::smem_u32;

constexpr int kMaxRing = 4;
constexpr float kE4m3Max = 448.f;

// How rows are read: through the ring or directly, rows that start on 16 bytes or anywhere.
enum Access { RING, DIRECT, SHIFTED_RING, SHIFTED };
constexpr bool on_pieces(Access a) { return a == RING || a == DIRECT; }
constexpr bool staged_rows(Access a) { return a == RING || a == SHIFTED_RING; }

// Chunks of 8 elements per thread.  Rows that start anywhere need up to 7 elements more.
template <int W, Access A>
constexpr int chunks() { return !on_pieces(A) && W == 32 ? 3 : 2; }

template <int W> struct NormShape {
    static constexpr int kGroups = W < 8 ? 8 / W : 1;      // per block
    static constexpr int kThreads = 32 * W * kGroups;
    // blocks that share an SM: the forward at 64 registers a thread, the backward at 128
    static constexpr int kFwdBlocks = 1024 / kThreads;
    static constexpr int kBwdBlocks = kThreads >= 512 ? 1 : 512 / kThreads;
    // (the forward of rows that start anywhere: their cuts, and e4m3's, take registers)
    static constexpr int shifted_blocks(bool e4m3) { return e4m3 ? kBwdBlocks * 3 / 2 : kFwdBlocks; }
};

// The largest magnitude that a group's scale maps to 448: its own, kept away from where
// 448 / m overflows; 0 for a group of zeros, whose scale and values are then 0.
__device__ __forceinline__ float scale_top(float m)
{
    return m > 0.f ? fmaxf(m, 7.888609e-31f /* 2^-100 */) : 0.f;
}

// 448 / m to 2 ulp, for m = 0 or from 2^-100 on.  (The fast division gives 0 for divisors above 2^126:
// both are taken by 4.)  Of 451 M values 302 come out one e4m3 step from those of exact arithmetic,
// 362 with every operation rounded to nearest; a step of Newton's here makes that 261 and
// 16384 x 4096 bf16 3 % slower.
__device__ __forceinline__ float scale_back(float m)
{
    return m > 0.f ? __fdividef(kE4m3Max * 0.25f, m * 0.25f) : 0.f;
}

// rs as a power of two times a factor in [1, 2).  The 8-bit values do not depend on the factor: it
// goes into the scales alone, and the values carry one rounding less.
__device__ __forceinline__ float power_of(float rs)
{
    return isnan(rs) ? rs : __uint_as_float(__float_as_uint(rs) & 0x7f800000u);
}
__device__ __forceinline__ float factor_of(float rs)
{
    return __uint_as_float((__float_as_uint(rs) & 0x007fffffu) | 0x3f800000u);
}

template <int W>
__device__ __forceinline__ void group_sync()
{
    if constexpr (W == 1) __syncwarp();
    else if constexpr (W >= 8) __syncthreads();
    else named_bar_sync(1 + threadIdx.x / (32 * W), 32 * W);
}

// Sum (or maximum) over the W warps of the row group; every thread gets it.
template <int W, bool MAX>
__device__ __forceinline__ float group_reduce(float v, float *buf)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float u = __shfl_xor_sync(kFullMask, v, o);
        v = MAX ? fmaxf(v, u) : v + u;
    }
    if constexpr (W > 1) {
        const int warp = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0) buf[warp] = v;
        group_sync<W>();
        const float *g = buf + warp / W * W;
        v = g[0];
#pragma unroll
        for (int i = 1; i < W; ++i) v = MAX ? fmaxf(v, g[i]) : v + g[i];
    }
    return v;
}

// A group's ring of `depth` stages, each one row of every input; `full` its barriers.
struct Ring {
    uint8_t *base;
    uint64_t *full;
    int depth, stage_bytes;
};

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}

// Bytes that a row takes in a stage.  A row that starts anywhere keeps the up to 7 elements in front
// of it that share its first piece, so its pieces are on 16 bytes there too.
template <Access A, typename T>
__host__ __device__ constexpr int row_slot(int width)
{
    return (on_pieces(A) ? width : (width + 14) / 8 * 8) * (int)sizeof(T);
}

// Copies row `row` of each tensor of `in` to the stage, from `skew` elements in front of it and to
// the end of its last 16 bytes; where the tensor ends before that, its last elements one by one.
template <Access A, typename T, int N>
__device__ __forceinline__ void ring_fill(const Ring &r, int stage, const T *const (&in)[N], int64_t row,
                                          int width, int skew, int64_t rows)
{
    uint8_t *dst = r.base + stage * r.stage_bytes;
    const uint32_t slot = (uint32_t)row_slot<A, T>(width);
    uint32_t bytes = slot, all = 0;
    const T *src[N];
#pragma unroll
    for (int n = 0; n < N; ++n) src[n] = in[n] ? in[n] + row * width - skew : nullptr;
    if constexpr (!on_pieces(A)) {
        const uint32_t need = (uint32_t)(skew + width) * sizeof(T);
        bytes = (need + 15) & ~15u;
        if (((rows - row) * width + skew) * (int64_t)sizeof(T) < bytes) {
            bytes = need & ~15u;
#pragma unroll
            for (int n = 0; n < N; ++n)
                for (uint32_t i = bytes / sizeof(T); src[n] && i < need / sizeof(T); ++i)
                    reinterpret_cast<T *>(dst + n * slot)[i] = src[n][i];
        }
    }
#pragma unroll
    for (int n = 0; n < N; ++n) all += in[n] ? bytes : 0u;
    mbar_arrive_expect_tx(&r.full[stage], all);
#pragma unroll
    for (int n = 0; n < N; ++n)
        if (in[n]) {
            if (on_pieces(A) || bytes) bulk_load(dst, src[n], bytes, &r.full[stage]);
            dst += slot;
        }
}

// A lane's 8 elements of a staged row that starts anywhere; zeros outside the row.
template <typename T>
__device__ __forceinline__ void load8_staged(const T *row, int c0, int width, float (&f)[8])
{
    const int i = elem8(c0);
    uint4 v[sizeof(T) / 2] = {};
#pragma unroll
    for (int k = 0; k < (int)sizeof(T) / 2; ++k)
        if (i + 8 > 0 && i < width) v[k] = reinterpret_cast<const uint4 *>(row + i)[k];
    if constexpr (sizeof(T) == 2) {
        unpack8(v[0], f);
    } else {
        f[0] = __uint_as_float(v[0].x); f[1] = __uint_as_float(v[0].y);
        f[2] = __uint_as_float(v[0].z); f[3] = __uint_as_float(v[0].w);
        f[4] = __uint_as_float(v[1].x); f[5] = __uint_as_float(v[1].y);
        f[6] = __uint_as_float(v[1].z); f[7] = __uint_as_float(v[1].w);
    }
    if (c0 >= 0 && c0 + 256 <= width) return;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (i + e < 0 || i + e >= width) f[e] = 0.f;
}

// 8 elements of a row as A reads it: `row` in a stage or in the tensor [begin, end).
template <Access A, typename T>
__device__ __forceinline__ void read8(const T *row, int c0, int width, const T *begin, const T *end,
                                      float (&f)[8])
{
    if constexpr (A == SHIFTED_RING) load8_staged(row, c0, width, f);
    else load8<on_pieces(A)>(row, c0, width, begin, end, f);
}

// Waits for a stage; false if its copies have not landed within the limit (of a sound device
// they always do), in which case the row's results are made NaN.
__device__ __forceinline__ bool ring_wait(const Ring &r, int stage, uint32_t parity)
{
    return sm100::mbar_wait(&r.full[stage], parity, sm100::kWaitLimitCycles);
}

// The group's part of the block's dynamic shared memory: barriers first, then the stages.
template <int W>
__device__ __forceinline__ Ring ring_of(uint8_t *smem, int depth, int stage_bytes)
{
    constexpr int kGroups = NormShape<W>::kGroups;
    const int group = threadIdx.x / (32 * W);
    Ring r;
    r.depth = depth;
    r.stage_bytes = stage_bytes;
    r.full = reinterpret_cast<uint64_t *>(smem) + group * kMaxRing;
    r.base = smem + kGroups * kMaxRing * 8 + (int64_t)group * depth * stage_bytes;
    return r;
}

template <bool VEC>
__device__ __forceinline__ void store8_e4m3(uint8_t *row, int c0, int width, const float (&f)[8])
{
    uint32_t u[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * e], f[4 * e + 1]),
                                                     __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * e + 2], f[4 * e + 3]),
                                                     __NV_SATFINITE, __NV_E4M3);
        u[e] = lo | hi << 16;
    }
    if constexpr (VEC) {
        if (elem8(c0) < width) *reinterpret_cast<uint2 *>(row + elem8(c0)) = make_uint2(u[0], u[1]);
    } else {
        store_words<2, 1>(row + c0, row, row + width, u);
    }
}

// y * (448 / max) and the scales of one chunk of 256 columns from c0, in groups of `group`
// columns (32, 64 or 128): group / 8 neighbouring lanes.
__device__ __forceinline__ void scale_groups(float (&h)[8], int c0, int width, int group,
                                             float factor, float *scales)
{
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(h[e]));
    for (int o = group / 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFullMask, m, o));
    m = scale_top(m);
    const int i = elem8(c0), shift = 31 - __clz(group);    // a power of two
    if (i < width && (i & (group - 1)) == 0) scales[i >> shift] = m * factor * (1.f / kE4m3Max);
    const float back = scale_back(m);
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] *= back;
}

// The same for a row that starts anywhere, all its chunks: a lane's elements may lie in two
// neighbouring groups, so the groups' maxima meet in shared memory (`gm`, one word per group;
// the order of maxima does not matter).
template <int W, int NC>
__device__ __forceinline__ void scale_groups_shifted(float (&h)[NC][8], int skew, int width, int group,
                                                     float factor, float *scales, uint32_t *gm)
{
    const int t = threadIdx.x % (32 * W), wg = (threadIdx.x / 32) % W;
    const int shift = 31 - __clz(group), groups = (width + group - 1) / group;
    for (int g = t; g < groups; g += 32 * W) gm[g] = 0u;
    group_sync<W>();
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int i = elem8((c * W + wg) * 256 - skew);
        const int lo = max(i, 0) >> shift, next = (lo + 1) << shift;
        float m0 = 0.f, m1 = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (i + e < next) m0 = fmaxf(m0, fabsf(h[c][e]));
            else m1 = fmaxf(m1, fabsf(h[c][e]));
        }
        if (i + 8 > 0 && i < width) {
            atomicMax(&gm[lo], __float_as_uint(m0));
            if (i + 8 > next && next < width) atomicMax(&gm[lo + 1], __float_as_uint(m1));
        }
    }
    group_sync<W>();
    for (int g = t; g < groups; g += 32 * W)
        scales[g] = scale_top(__uint_as_float(gm[g])) * factor * (1.f / kE4m3Max);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int i = elem8((c * W + wg) * 256 - skew);
        const int lo = min(max(i, 0) >> shift, groups - 1), next = (lo + 1) << shift;
        const float b0 = scale_back(scale_top(__uint_as_float(gm[lo])));
        const float b1 = scale_back(scale_top(__uint_as_float(gm[min(lo + 1, groups - 1)])));
#pragma unroll
        for (int e = 0; e < 8; ++e) h[c][e] *= i + e < next ? b0 : b1;
    }
    group_sync<W>();
}

template <typename T, int W, bool E4M3, Access A>
__global__ void __launch_bounds__(NormShape<W>::kThreads,
                                  on_pieces(A) ? NormShape<W>::kFwdBlocks
                                               : NormShape<W>::shifted_blocks(E4M3))
    rms_norm_kernel(const __grid_constant__ RmsArgs a, int depth)
{
    constexpr bool VEC = on_pieces(A), STAGED = staged_rows(A);
    constexpr int NC = chunks<W, A>();
    constexpr int kGroups = NormShape<W>::kGroups;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float buf[2][NormShape<W>::kThreads / 32];
    const int group = threadIdx.x / (32 * W), wg = (threadIdx.x / 32) % W;
    const bool lead = threadIdx.x % (32 * W) == 0;
    const int64_t stride = (int64_t)gridDim.x * kGroups;
    int64_t row = (int64_t)blockIdx.x * kGroups + group;
    const int width = a.width;
    // the same for all rows of a group: the stride is a multiple of 8 (or there is one row)
    const int skew = lead_of<VEC>(row, width);
    const T *const in[2] = {reinterpret_cast<const T *>(a.x), reinterpret_cast<const T *>(a.resid)};
    Ring ring;
    if constexpr (STAGED) {
        ring = ring_of<W>(smem, depth, (a.resid ? 2 : 1) * row_slot<A, T>(width));
        if (lead) {
            for (int s = 0; s < depth; ++s) mbar_init(&ring.full[s], 1);
            sm100::fence_mbar_init();
        }
        group_sync<W>();
    }
    grid_dep_wait();
    grid_dep_release();
    if (STAGED && lead)
        for (int s = 0; s < depth && row + s * stride < a.rows; ++s)
            ring_fill<A>(ring, s, in, row + s * stride, width, skew, a.rows);
    float w[NC][8];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        if (a.weight) {
            load8<VEC>(a.weight, (c * W + wg) * 256 - skew, width, a.weight, a.weight + width, w[c]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[c][e] = 1.f;
        }
    }
    const T *x_begin = reinterpret_cast<const T *>(a.x), *x_end = x_begin + a.rows * width;
    const T *r_begin = reinterpret_cast<const T *>(a.resid), *r_end = r_begin + a.rows * width;
    int stage = 0;
    uint32_t parity = 0;
    for (; row < a.rows; row += stride) {
        const int64_t base = row * width;
        const T *x = reinterpret_cast<const T *>(a.x) + base;
        const T *r = a.resid ? reinterpret_cast<const T *>(a.resid) + base : nullptr;
        bool landed = true;
        if constexpr (STAGED) {
            landed = ring_wait(ring, stage, parity);
            x = reinterpret_cast<const T *>(ring.base + stage * ring.stage_bytes) + skew;
            r = a.resid ? x + row_slot<A, T>(width) / sizeof(T) : nullptr;
        }
        float h[NC][8];
        float ss = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c) read8<A>(x, (c * W + wg) * 256 - skew, width, x_begin, x_end, h[c]);
        if (r) {
            float b[NC][8];
#pragma unroll
            for (int c = 0; c < NC; ++c) read8<A>(r, (c * W + wg) * 256 - skew, width, r_begin, r_end, b[c]);
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int e = 0; e < 8; ++e) h[c][e] += b[c][e];
        }
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(h[c][e], h[c][e], ss);
        ss = group_reduce<W, false>(ss, buf[0]);
        if constexpr (STAGED) {
            // every thread of the group has read the stage
            if constexpr (W == 1) __syncwarp();
            if (lead && row + depth * stride < a.rows)
                ring_fill<A>(ring, stage, in, row + depth * stride, width, skew, a.rows);
            if (++stage == depth) {
                stage = 0;
                parity ^= 1;
            }
        }
        const float rs = landed ? rsqrtf(ss / (float)width + a.eps) : CUDART_NAN_F;
        const float power = power_of(rs), factor = factor_of(rs);      // (8 bits only)
        if (a.rstd && lead) a.rstd[row] = rs;
        if (a.sum) {
#pragma unroll
            for (int c = 0; c < NC; ++c)
                store8<VEC>(reinterpret_cast<T *>(a.sum) + base, (c * W + wg) * 256 - skew, width, h[c]);
        }
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int e = 0; e < 8; ++e) h[c][e] *= (E4M3 ? power : rs) * w[c][e];
        if constexpr (!E4M3) {
#pragma unroll
            for (int c = 0; c < NC; ++c)
                store8<VEC>(reinterpret_cast<T *>(a.y) + base, (c * W + wg) * 256 - skew, width, h[c]);
            if constexpr (W > 1) group_sync<W>();          // buf is used again
        } else {
            if (a.group == 0) {
                float m = 0.f;
#pragma unroll
                for (int c = 0; c < NC; ++c)
#pragma unroll
                    for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(h[c][e]));
                m = scale_top(group_reduce<W, true>(m, buf[1]));
                if (lead) a.scales[row] = m * factor * (1.f / kE4m3Max);
                const float back = scale_back(m);
#pragma unroll
                for (int c = 0; c < NC; ++c)
#pragma unroll
                    for (int e = 0; e < 8; ++e) h[c][e] *= back;
            } else if constexpr (!VEC) {
                const int groups = (width + a.group - 1) / a.group;
                uint32_t *maxima = reinterpret_cast<uint32_t *>(smem);
                if constexpr (STAGED)                      // behind the stages of all groups
                    maxima += kGroups * (kMaxRing * 8 + depth * ring.stage_bytes) / 4;
                scale_groups_shifted<W, NC>(h, skew, width, a.group, factor, a.scales + row * groups,
                                            maxima + group * groups);
            } else {
                const int groups = (width + a.group - 1) / a.group;
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    scale_groups(h[c], (c * W + wg) * 256, width, a.group, factor,
                                 a.scales + row * groups);
                if constexpr (W > 1) group_sync<W>();
            }
#pragma unroll
            for (int c = 0; c < NC; ++c)
                store8_e4m3<VEC>(reinterpret_cast<uint8_t *>(a.y) + base, (c * W + wg) * 256 - skew, width, h[c]);
        }
    }
}

// Each group walks rows with a stride of the grid and keeps its columns' part of the weight
// gradient in registers; the parts of a block meet in shared memory and leave as one row of
// `part`, which rms_dweight_kernel adds in a fixed order.
template <typename T, int W, Access A>
__global__ void __launch_bounds__(NormShape<W>::kThreads, NormShape<W>::kBwdBlocks)
    rms_norm_bwd_kernel(const __grid_constant__ RmsBwdArgs a, int depth)
{
    constexpr bool VEC = on_pieces(A), STAGED = staged_rows(A);
    constexpr int NC = chunks<W, A>();
    constexpr int kGroups = NormShape<W>::kGroups;
    extern __shared__ __align__(128) uint8_t smem[];       // barriers, the ring; then [kGroups][width] floats
    __shared__ float buf[2][NormShape<W>::kThreads / 32];
    const int group = threadIdx.x / (32 * W), wg = (threadIdx.x / 32) % W;
    const bool lead = threadIdx.x % (32 * W) == 0;
    const int64_t stride = (int64_t)gridDim.x * kGroups;
    int64_t row = (int64_t)blockIdx.x * kGroups + group;
    const int width = a.width;
    const int skew = lead_of<VEC>(row, width);             // of all rows of the group
    const T *const in[3] = {reinterpret_cast<const T *>(a.dy), reinterpret_cast<const T *>(a.h),
                            reinterpret_cast<const T *>(a.dsum)};
    Ring ring;
    if constexpr (STAGED) {
        ring = ring_of<W>(smem, depth, (a.dsum ? 3 : 2) * row_slot<A, T>(width));
        if (lead) {
            for (int s = 0; s < depth; ++s) mbar_init(&ring.full[s], 1);
            sm100::fence_mbar_init();
        }
        group_sync<W>();
    }
    grid_dep_wait();
    grid_dep_release();
    if (STAGED && lead)
        for (int s = 0; s < depth && row + s * stride < a.rows; ++s)
            ring_fill<A>(ring, s, in, row + s * stride, width, skew, a.rows);
    // the weights stay in registers: with shared memory full of rows L1 keeps nothing, and
    // reading them again for every row took 127 us instead of 83 (8192 x 8192 bf16)
    float acc[NC][8], w[NC][8];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        if (a.weight) load8<VEC>(a.weight, (c * W + wg) * 256 - skew, width, a.weight, a.weight + width, w[c]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            acc[c][e] = 0.f;
            if (!a.weight) w[c][e] = 1.f;
        }
    }
    const T *dy_begin = reinterpret_cast<const T *>(a.dy), *dy_end = dy_begin + a.rows * width;
    const T *h_begin = reinterpret_cast<const T *>(a.h), *h_end = h_begin + a.rows * width;
    const T *ds_begin = reinterpret_cast<const T *>(a.dsum), *ds_end = ds_begin + a.rows * width;
    int stage = 0, flip = 0;
    uint32_t parity = 0;
    float rs_next = row < a.rows ? a.rstd[row] : 0.f;      // one row ahead
    for (; row < a.rows; row += stride, flip ^= 1) {
        const int64_t base = row * width;
        const T *dy = reinterpret_cast<const T *>(a.dy) + base;
        const T *hp = reinterpret_cast<const T *>(a.h) + base;
        const T *ds = a.dsum ? reinterpret_cast<const T *>(a.dsum) + base : nullptr;
        float rs = rs_next;
        if (row + stride < a.rows) rs_next = a.rstd[row + stride];
        if constexpr (STAGED) {
            if (!ring_wait(ring, stage, parity)) rs = CUDART_NAN_F;
            dy = reinterpret_cast<const T *>(ring.base + stage * ring.stage_bytes) + skew;
            hp = dy + row_slot<A, T>(width) / sizeof(T);
            ds = a.dsum ? hp + row_slot<A, T>(width) / sizeof(T) : nullptr;
        }
        float g[NC][8], h[NC][8];
        float dot = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            read8<A>(dy, (c * W + wg) * 256 - skew, width, dy_begin, dy_end, g[c]);
            read8<A>(hp, (c * W + wg) * 256 - skew, width, h_begin, h_end, h[c]);
        }
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                h[c][e] *= rs;
                acc[c][e] = fmaf(g[c][e], h[c][e], acc[c][e]);
                g[c][e] *= w[c][e];
                dot = fmaf(g[c][e], h[c][e], dot);
            }
        dot = group_reduce<W, false>(dot, buf[flip]) / (float)width;
        T *dx = reinterpret_cast<T *>(a.dx) + base;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            float o[8];
            if (ds) read8<A>(ds, (c * W + wg) * 256 - skew, width, ds_begin, ds_end, o);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = rs * (g[c][e] - h[c][e] * dot);
                o[e] = ds ? d + o[e] : d;
            }
            store8<VEC>(dx, (c * W + wg) * 256 - skew, width, o);
        }
        if constexpr (STAGED) {
            group_sync<W>();                               // the group has read the stage
            if (lead && row + depth * stride < a.rows)
                ring_fill<A>(ring, stage, in, row + depth * stride, width, skew, a.rows);
            if (++stage == depth) {
                stage = 0;
                parity ^= 1;
            }
        }
    }
    if (!a.dweight) return;
    float *part = a.part + (int64_t)blockIdx.x * width;
    if constexpr (kGroups == 1) {
        // (the parts' own rows start on 16 bytes where VEC)
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int i = elem8((c * W + wg) * 256 - skew);
            if constexpr (VEC) {
                store8<true>(part, (c * W + wg) * 256, width, acc[c]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (i + e >= 0 && i + e < width) part[i + e] = acc[c][e];
            }
        }
    } else {
        // The groups' stages are done with: their memory holds the groups' parts.  Not the barriers in
        // front of them: a word that has been a barrier may still change after the last wait on it
        // (parts of 5183 x 512 bf16 that lay there came out wrong in one call of six).
        float *dws = reinterpret_cast<float *>(smem + (STAGED ? kGroups * kMaxRing * 8 : 0));
        __syncthreads();
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int i = elem8((c * W + wg) * 256 - skew);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (i + e >= 0 && i + e < width) dws[group * width + i + e] = acc[c][e];
        }
        __syncthreads();
        for (int i = threadIdx.x; i < width; i += blockDim.x) {
            float s = 0.f;
#pragma unroll
            for (int q = 0; q < kGroups; ++q) s += dws[q * width + i];
            part[i] = s;
        }
    }
}

// dweight[i] = sum of the blocks' parts, in block order within each of 32 strands, the
// strands in order: the same result every time.
__global__ void __launch_bounds__(1024) rms_dweight_kernel(const float *__restrict__ part,
                                                           int blocks, int width,
                                                           float *__restrict__ dweight)
{
    __shared__ float s[32][33];
    grid_dep_wait();
    grid_dep_release();
    const int lane = threadIdx.x & 31, strand = threadIdx.x >> 5;
    const int i = blockIdx.x * 32 + lane;
    float v = 0.f;
    if (i < width) {
#pragma unroll 10
        for (int b = strand; b < blocks; b += 32) v += part[(int64_t)b * width + i];
    }
    s[strand][lane] = v;
    __syncthreads();
    const float r = warp_sum(s[lane][strand]);             // column blockIdx.x * 32 + strand
    if (lane == 0 && blockIdx.x * 32 + strand < width) dweight[blockIdx.x * 32 + strand] = r;
}

// Warps per row: 512 columns per warp, with room for the lead of rows that start anywhere.
int warps_for(int width)
{
    const int room = width % 8 ? width + 7 : width;
    int w = 1;
    while (w < 32 && w * 512 < room) w *= 2;
    return w;
}

// How many blocks share an SM and how deep their rings are: rows in flight of `flight` bytes per
// SM.  (Forward, 64 KB: 16384 x 4096 bf16 to e4m3 takes 79 us; with 128 KB in flight 82 and with
// 192 KB 88, as reads that run further ahead only crowd the writes; with half the warps 91.)
// The blocks' shared memory is sized to leave no room for more of them, or a kernel behind
// this one would place its blocks unevenly.
struct RingPlan {
    int blocks, depth;
    size_t smem;
};

template <int W>
RingPlan ring_plan(int blocks, int64_t stage_bytes, int64_t flight, int64_t extra = 0)
{
    constexpr int64_t kSmem = 227 * 1024, kGroups = NormShape<W>::kGroups;
    RingPlan p;
    p.blocks = blocks;
    while (p.blocks > 1 && p.blocks * kGroups * stage_bytes > flight) p.blocks /= 2;
    const int64_t room = kSmem / p.blocks - 2048 - extra;
    const int64_t most = std::min<int64_t>(kMaxRing, (room - kGroups * kMaxRing * 8) / (kGroups * stage_bytes));
    p.depth = (int)std::max<int64_t>(1, std::min(most, flight / (p.blocks * kGroups * stage_bytes)));
    p.smem = (size_t)(room + extra);
    return p;
}

template <auto Kern, typename Args>
cudaError_t launch_norm(const Args &a, int64_t blocks, int threads, size_t smem, int depth, cudaStream_t st)
{
    cudaError_t e = allow_smem<Kern>(smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(Kern, dim3((unsigned)blocks), dim3((unsigned)threads), smem, st, a, depth);
}

template <typename T, bool E4M3, int W>
cudaError_t run_fwd(const RmsArgs &a, cudaStream_t st)
{
    using S = NormShape<W>;
    const int64_t most = (int64_t)num_sms() * S::kFwdBlocks;
    const int64_t blocks = (a.rows + S::kGroups - 1) / S::kGroups;
    if (a.width % 8 != 0) {
        // groups keep their rows' alignment: a stride of a multiple of 8 rows
        const int64_t stay = (int64_t)num_sms() * S::shifted_blocks(E4M3) / 8 * 8;
        const size_t maxima = E4M3 && a.group ? (size_t)S::kGroups * ((a.width + a.group - 1) / a.group) * 4 : 0;
        if (blocks <= stay)
            return launch_norm<rms_norm_kernel<T, W, E4M3, SHIFTED>>(a, blocks, S::kThreads, maxima, 0, st);
        const int64_t stage = (int64_t)row_slot<SHIFTED_RING, T>(a.width) * (a.resid ? 2 : 1);
        const RingPlan p = ring_plan<W>(S::shifted_blocks(E4M3), stage, 64 * 1024, (int64_t)maxima);
        return launch_norm<rms_norm_kernel<T, W, E4M3, SHIFTED_RING>>(
            a, (int64_t)num_sms() * p.blocks / 8 * 8, S::kThreads, p.smem, p.depth, st);
    }
    if (blocks <= most)
        return launch_norm<rms_norm_kernel<T, W, E4M3, DIRECT>>(a, blocks, S::kThreads, 0, 0, st);
    const int64_t stage = (int64_t)a.width * sizeof(T) * (a.resid ? 2 : 1);
    const RingPlan p = ring_plan<W>(S::kFwdBlocks, stage, 64 * 1024);
    return launch_norm<rms_norm_kernel<T, W, E4M3, RING>>(a, (int64_t)num_sms() * p.blocks,
                       S::kThreads, p.smem, p.depth, st);
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
    using S = NormShape<W>;
    const int blocks = rms_bwd_blocks(a.rows, a.width);
    const size_t parts = S::kGroups > 1 && a.dweight ? (size_t)S::kGroups * a.width * 4 : 0;
    cudaError_t e;
    if (a.rows <= (int64_t)blocks * S::kGroups) {
        e = a.width % 8 != 0 ? launch_norm<rms_norm_bwd_kernel<T, W, SHIFTED>>(a, blocks, S::kThreads, parts, 0, st)
                             : launch_norm<rms_norm_bwd_kernel<T, W, DIRECT>>(a, blocks, S::kThreads, parts, 0, st);
    } else if (a.width % 8 != 0) {
        const int64_t stage = (int64_t)row_slot<SHIFTED_RING, T>(a.width) * (a.dsum ? 3 : 2);
        const RingPlan p = ring_plan<W>(S::kBwdBlocks, stage, 160 * 1024);
        e = launch_norm<rms_norm_bwd_kernel<T, W, SHIFTED_RING>>(a, blocks, S::kThreads, p.smem, p.depth, st);
    } else {
        const int64_t stage = (int64_t)a.width * sizeof(T) * (a.dsum ? 3 : 2);
        const RingPlan p = ring_plan<W>(S::kBwdBlocks, stage, 160 * 1024);
        e = launch_norm<rms_norm_bwd_kernel<T, W, RING>>(a, blocks, S::kThreads, p.smem, p.depth, st);
    }
    if (e != cudaSuccess || !a.dweight) return e;
    return launch_pdl(rms_dweight_kernel, dim3((a.width + 31) / 32), dim3(1024), 0, st,
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
    // 512 threads per SM; more blocks would only add rows of partial sums
    const int w = warps_for(width), per = w < 8 ? 8 / w : 1;
    const int64_t need = (rows + per - 1) / per;
    // (rows that start anywhere keep their alignment with a stride of a multiple of 8)
    const int64_t most = w < 16 ? 296 : width % 8 ? 144 : 148;
    return (int)std::max<int64_t>(1, std::min<int64_t>(need, most));
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
