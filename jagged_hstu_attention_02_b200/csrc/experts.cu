// experts.cu -- (token, choice) pairs sorted by expert, the tokens' rows moved to their sorted
// places and back, and the gradients of the way back.
//
// Sort: a stable counting sort of the n = tokens * choices pairs by expert.  Expert e's pairs
// take the places [offsets[e], offsets[e+1]), in the order of their pair number, so the sorted
// rows are a jagged tensor whose sequences are the experts.  Ids below 0 are pairs that no
// expert takes (place -1).
//
// Dispatch: token t's row goes to each place slots[t, j].  Combine, with out_t = resid_t +
// sum_j w_tj y[slot_tj] accumulated in fp32 in the order of j, is the way back, and without
// weights the gradient of dispatch.  Its own gradients are dy[slot_tj] = w_tj dout_t and
// dw_tj = <dout_t, y[slot_tj]>.
//
// All of them move rows: bound by memory.  A token's warps read its row (dispatch) or its
// gradient (combine backward) once for all choices; no atomics on floating-point values
// anywhere, so every result is the same each time.
#include "experts.h"
#include "kernels.h"
#include "lnrow.cuh"
#include "rowvec.cuh"

namespace hstu {

namespace {

// ------------------------------------------------------------------ sort

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortOneBlock = 8192;     // pairs that one block sorts by itself
constexpr int kSortMaxBlocks = 148;

// The expert of pair p, or -1 (reported when the id is not below `experts`).
template <typename I>
__device__ __forceinline__ int expert_of(const SortArgs &a, int64_t p, bool report)
{
    const I id = reinterpret_cast<const I *>(a.ids)[p];
    if (id < 0) return -1;
    if (id >= (I)a.experts) {
        if (report && a.status) atomicOr(a.status, HSTU_DEV_BAD_EXPERT);
        return -1;
    }
    return (int)id;
}

// Pairs [lo, hi) of the block are dealt to its warps in contiguous runs of whole 32s.
__device__ __forceinline__ void warp_run(int64_t lo, int64_t hi, int warp, int64_t &b, int64_t &e)
{
    const int64_t per = ((hi - lo + 32 * kSortWarps - 1) / (32 * kSortWarps)) * 32;
    b = min(hi, lo + warp * per);
    e = min(hi, b + per);
}

// Counts this warp's pairs per expert into its own row of shared memory.
template <typename I>
__device__ __forceinline__ void count_run(const SortArgs &a, int64_t b, int64_t e, int32_t *mine,
                                          bool report)
{
    const int lane = threadIdx.x & 31;
    for (int64_t p0 = b; p0 < e; p0 += 32) {
        const int64_t p = p0 + lane;
        const int x = p < e ? expert_of<I>(a, p, report) : -1;
        const unsigned same = __match_any_sync(kFullMask, x);
        if (x >= 0 && lane == __ffs(same) - 1) mine[x] += __popc(same);
        __syncwarp();
    }
}

// Exclusive prefix sum over the block's threads of one value each; *total their sum.
__device__ __forceinline__ int block_scan(int v, int *wsum, int *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kFullMask, s, o);
        if (lane >= o) s += u;
    }
    if (lane == 31) wsum[warp] = s;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
        const int u = wsum[w];
        if (w < warp) before += u;
        all += u;
    }
    __syncthreads();
    *total = all;
    return before + s - v;
}

// Places of this warp's pairs; mine[x]: the place of its next pair of expert x.
template <typename I>
__device__ __forceinline__ void place_run(const SortArgs &a, int64_t b, int64_t e, int32_t *mine)
{
    const int lane = threadIdx.x & 31;
    for (int64_t p0 = b; p0 < e; p0 += 32) {
        const int64_t p = p0 + lane;
        const int x = p < e ? expert_of<I>(a, p, false) : -1;
        const unsigned same = __match_any_sync(kFullMask, x);
        int at = -1;
        if (x >= 0) at = mine[x] + __popc(same & ((1u << lane) - 1u));
        __syncwarp();
        if (x >= 0 && lane == __ffs(same) - 1) mine[x] += __popc(same);
        __syncwarp();
        if (p < e) {
            a.slots[p] = at;
            if (at >= 0 && a.rows) a.rows[at] = p / a.choices;
        }
    }
}

// ONE: the whole sort in one block.  Otherwise the second launch of two: expert_count_kernel
// has left every block's counts in a.hist, and each block adds those of the blocks before it.
template <typename I, bool ONE>
__global__ void __launch_bounds__(kSortThreads) expert_place_kernel(const __grid_constant__ SortArgs a)
{
    extern __shared__ int32_t sh[];                  // [kSortWarps][experts]
    __shared__ int wsum[kSortWarps];
    const int tid = threadIdx.x, warp = tid >> 5;
    const int64_t chunk = (a.n + gridDim.x - 1) / gridDim.x;
    const int64_t lo = min(a.n, (int64_t)blockIdx.x * chunk), hi = min(a.n, lo + chunk);
    int64_t b, e;
    warp_run(lo, hi, warp, b, e);
    for (int x = tid; x < kSortWarps * a.experts; x += kSortThreads) sh[x] = 0;
    __syncthreads();
    count_run<I>(a, b, e, sh + warp * a.experts, ONE);
    if constexpr (!ONE) grid_dep_wait();
    __syncthreads();
    int base = 0;
    for (int x0 = 0; x0 < a.experts; x0 += kSortThreads) {
        const int x = x0 + tid;
        int all = 0, before = 0;
        if (x < a.experts) {
            if constexpr (ONE) {
                for (int w = 0; w < kSortWarps; ++w) all += sh[w * a.experts + x];
            } else {
#pragma unroll 8
                for (int q = 0; q < (int)gridDim.x; ++q) {
                    const int v = a.hist[(int64_t)q * a.experts + x];
                    all += v;
                    if (q < (int)blockIdx.x) before += v;
                }
            }
        }
        int total;
        const int at = base + block_scan(all, wsum, &total);
        if (x < a.experts) {
            if (blockIdx.x == 0) a.offsets[x] = at;
            int run = at + before;
            for (int w = 0; w < kSortWarps; ++w) {
                const int v = sh[w * a.experts + x];
                sh[w * a.experts + x] = run;
                run += v;
            }
        }
        base += total;
    }
    if (blockIdx.x == 0 && tid == 0) a.offsets[a.experts] = base;
    __syncthreads();
    place_run<I>(a, b, e, sh + warp * a.experts);
}

template <typename I>
__global__ void __launch_bounds__(kSortThreads) expert_count_kernel(const __grid_constant__ SortArgs a)
{
    extern __shared__ int32_t sh[];                  // [kSortWarps][experts]
    const int tid = threadIdx.x, warp = tid >> 5;
    const int64_t chunk = (a.n + gridDim.x - 1) / gridDim.x;
    const int64_t lo = min(a.n, (int64_t)blockIdx.x * chunk), hi = min(a.n, lo + chunk);
    int64_t b, e;
    warp_run(lo, hi, warp, b, e);
    grid_dep_release();
    for (int x = tid; x < kSortWarps * a.experts; x += kSortThreads) sh[x] = 0;
    __syncthreads();
    count_run<I>(a, b, e, sh + warp * a.experts, true);
    __syncthreads();
    for (int x = tid; x < a.experts; x += kSortThreads) {
        int all = 0;
        for (int w = 0; w < kSortWarps; ++w) all += sh[w * a.experts + x];
        a.hist[(int64_t)blockIdx.x * a.experts + x] = all;
    }
}

template <typename I>
cudaError_t run_sort(const SortArgs &a, cudaStream_t st)
{
    const int blocks = sort_blocks(a.n);
    const size_t smem = (size_t)kSortWarps * a.experts * sizeof(int32_t);
    cudaError_t e;
    if (blocks == 1) {
        auto k = expert_place_kernel<I, true>;
        e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        k<<<1, kSortThreads, smem, st>>>(a);
        return cudaGetLastError();
    }
    auto c = expert_count_kernel<I>;
    e = cudaFuncSetAttribute(c, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    c<<<blocks, kSortThreads, smem, st>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    auto k = expert_place_kernel<I, false>;
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(k, dim3(blocks), dim3(kSortThreads), smem, st, a);
}

// ------------------------------------------------------------------ rows of tokens

// Warps that share a token's row, and tokens per block, for rows of `chunks` 16-byte (or
// smaller) pieces: up to 4 pieces per thread, up to 8 warps.
constexpr int kRowWarps = 8;

int warps_per_row(int64_t chunks)
{
    int w = 1;
    while (w < kRowWarps && w * 128 < chunks) w *= 2;
    return w;
}

// A row's slots in the lanes of a warp: lane j holds slot j (-1 where there is none).
__device__ __forceinline__ int lane_slot(const int32_t *slots, int64_t t, int k, int64_t max_rows)
{
    const int lane = threadIdx.x & 31;
    int s = lane < k ? slots[t * k + lane] : -1;
    return s >= 0 && s < max_rows ? s : -1;
}

template <typename V>
__global__ void __launch_bounds__(32 * kRowWarps)
    expert_dispatch_kernel(const __grid_constant__ DispatchArgs a, int wpr)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * (kRowWarps / wpr) + warp / wpr;
    if (t >= a.tokens) return;
    const int part = warp % wpr;
    const int mine = lane_slot(a.slots, t, a.choices, a.max_rows);
    const int64_t per = a.row_bytes / (int64_t)sizeof(V);
    const V *src = reinterpret_cast<const V *>(a.x + t * a.row_bytes);
    for (int64_t c0 = part * 32 + lane; c0 - lane < per; c0 += 4 * 32 * wpr) {
        V v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t c = c0 + u * 32 * wpr;
            if (c < per) v[u] = src[c];
        }
        for (int j = 0; j < a.choices; ++j) {
            const int s = __shfl_sync(kFullMask, mine, j);
            if (s < 0) continue;
            V *dst = reinterpret_cast<V *>(a.out + (int64_t)s * a.row_bytes);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int64_t c = c0 + u * 32 * wpr;
                if (c < per) dst[c] = v[u];
            }
        }
    }
    if (part != 0 || !a.scales) return;
    for (int j = 0; j < a.choices; ++j) {
        const int s = __shfl_sync(kFullMask, mine, j);
        if (s < 0) continue;
        for (int g = lane; g < a.n_scales; g += 32)
            a.scales_out[(int64_t)s * a.n_scales + g] = a.scales[t * a.n_scales + g];
    }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(32 * kRowWarps)
    expert_combine_kernel(const __grid_constant__ CombineArgs a, int wpr)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * (kRowWarps / wpr) + warp / wpr;
    if (t >= a.tokens) return;
    const int mine = lane_slot(a.slots, t, a.choices, a.max_rows);
    float weight = 1.f;
    if (a.weights && lane < a.choices) weight = a.weights[t * a.choices + lane];
    const T *y = reinterpret_cast<const T *>(a.y);
    for (int i0 = (warp % wpr) * 256; i0 < a.width; i0 += 256 * wpr) {
        float acc[8];
        if (a.resid) {
            load8<VEC>(reinterpret_cast<const T *>(a.resid) + t * a.width, i0, a.width, acc);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = 0.f;
        }
        for (int j0 = 0; j0 < a.choices; j0 += 4) {
            float f[4][8];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                // lanes from `choices` up hold -1
                const int s = __shfl_sync(kFullMask, mine, j0 + u);
                load8<VEC>(y + (s < 0 ? 0 : (int64_t)s * a.width), i0, s < 0 ? 0 : a.width, f[u]);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int s = __shfl_sync(kFullMask, mine, j0 + u);
                const float w = __shfl_sync(kFullMask, weight, j0 + u);
                if (s >= 0) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[e] = fmaf(w, f[u][e], acc[e]);
                }
            }
        }
        store8<VEC>(reinterpret_cast<T *>(a.out) + t * a.width, i0, a.width, acc);
    }
}

// KM: the choices, rounded up to a power of two (their dot products stay in registers).
template <typename T, bool VEC, int KM>
__global__ void __launch_bounds__(32 * kRowWarps)
    expert_combine_bwd_kernel(const __grid_constant__ CombineArgs a, int wpr)
{
    __shared__ float dots[kRowWarps][KM];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * (kRowWarps / wpr) + warp / wpr;
    const bool live = t < a.tokens;
    const int mine = live ? lane_slot(a.slots, t, a.choices, a.max_rows) : -1;
    float weight = 1.f;
    if (a.weights && live && lane < a.choices) weight = a.weights[t * a.choices + lane];
    const T *y = reinterpret_cast<const T *>(a.y);
    T *dy = reinterpret_cast<T *>(a.dy);
    const int width = live ? a.width : 0;
    float dot[KM];
#pragma unroll
    for (int j = 0; j < KM; ++j) dot[j] = 0.f;
    for (int i0 = (warp % wpr) * 256; i0 < width; i0 += 256 * wpr) {
        float g[8];
        load8<VEC>(reinterpret_cast<const T *>(a.dout) + t * a.width, i0, width, g);
#pragma unroll
        for (int j = 0; j < KM; ++j) {
            const int s = __shfl_sync(kFullMask, mine, j);
            const float w = __shfl_sync(kFullMask, weight, j);
            if (s < 0) continue;                       // (warp-uniform)
            if (a.dweights) {
                float f[8];
                load8<VEC>(y + (int64_t)s * a.width, i0, width, f);
#pragma unroll
                for (int e = 0; e < 8; ++e) dot[j] = fmaf(g[e], f[e], dot[j]);
            }
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = w * g[e];
            store8<VEC>(dy + (int64_t)s * a.width, i0, width, o);
        }
    }
    if (!a.dweights) return;
#pragma unroll
    for (int j = 0; j < KM; ++j) dot[j] = warp_sum(dot[j]);
    if (lane == 0) {
#pragma unroll
        for (int j = 0; j < KM; ++j) dots[warp][j] = dot[j];
    }
    __syncthreads();
    if (live && warp % wpr == 0 && lane < a.choices) {
        float s = 0.f;
        for (int q = 0; q < wpr; ++q) s += dots[warp + q][lane];
        a.dweights[t * a.choices + lane] = s;          // 0 where the pair has no place
    }
}

template <typename T, bool VEC>
cudaError_t run_combine_bwd(const CombineArgs &a, unsigned grid, int wpr, cudaStream_t st)
{
    if (a.choices <= 1) expert_combine_bwd_kernel<T, VEC, 1><<<grid, 32 * kRowWarps, 0, st>>>(a, wpr);
    else if (a.choices <= 2) expert_combine_bwd_kernel<T, VEC, 2><<<grid, 32 * kRowWarps, 0, st>>>(a, wpr);
    else if (a.choices <= 4) expert_combine_bwd_kernel<T, VEC, 4><<<grid, 32 * kRowWarps, 0, st>>>(a, wpr);
    else if (a.choices <= 8) expert_combine_bwd_kernel<T, VEC, 8><<<grid, 32 * kRowWarps, 0, st>>>(a, wpr);
    else expert_combine_bwd_kernel<T, VEC, 16><<<grid, 32 * kRowWarps, 0, st>>>(a, wpr);
    return cudaGetLastError();
}

template <typename T, bool BWD>
cudaError_t run_combine(const CombineArgs &a, cudaStream_t st)
{
    if (a.tokens <= 0) return cudaSuccess;
    const int wpr = warps_per_row((a.width + 15) / 16);      // 512 elements per warp and turn
    const int per = kRowWarps / wpr;
    const unsigned grid = (unsigned)((a.tokens + per - 1) / per);
    const bool vec = a.width % 8 == 0;
    if constexpr (BWD) {
        return vec ? run_combine_bwd<T, true>(a, grid, wpr, st)
                   : run_combine_bwd<T, false>(a, grid, wpr, st);
    } else {
        if (vec) expert_combine_kernel<T, true><<<grid, 32 * kRowWarps, 0, st>>>(a, wpr);
        else expert_combine_kernel<T, false><<<grid, 32 * kRowWarps, 0, st>>>(a, wpr);
        return cudaGetLastError();
    }
}

}  // namespace

int sort_blocks(int64_t n)
{
    if (n <= kSortOneBlock) return 1;
    const int64_t b = (n + 2047) / 2048;
    return (int)(b < kSortMaxBlocks ? b : kSortMaxBlocks);
}

cudaError_t launch_expert_sort(const SortArgs &a, bool ids64, cudaStream_t st)
{
    return ids64 ? run_sort<int64_t>(a, st) : run_sort<int32_t>(a, st);
}

cudaError_t launch_expert_dispatch(const DispatchArgs &a, cudaStream_t st)
{
    if (a.tokens <= 0) return cudaSuccess;
    const int64_t rb = a.row_bytes;
    const int unit = rb % 16 == 0 ? 16 : rb % 8 == 0 ? 8 : rb % 4 == 0 ? 4 : rb % 2 == 0 ? 2 : 1;
    const int wpr = warps_per_row((rb + unit - 1) / unit);
    const int per = kRowWarps / wpr;
    const unsigned grid = (unsigned)((a.tokens + per - 1) / per);
    switch (unit) {
    case 16: expert_dispatch_kernel<uint4><<<grid, 32 * kRowWarps, 0, st>>>(a, wpr); break;
    case 8: expert_dispatch_kernel<uint2><<<grid, 32 * kRowWarps, 0, st>>>(a, wpr); break;
    case 4: expert_dispatch_kernel<uint32_t><<<grid, 32 * kRowWarps, 0, st>>>(a, wpr); break;
    case 2: expert_dispatch_kernel<uint16_t><<<grid, 32 * kRowWarps, 0, st>>>(a, wpr); break;
    default: expert_dispatch_kernel<uint8_t><<<grid, 32 * kRowWarps, 0, st>>>(a, wpr); break;
    }
    return cudaGetLastError();
}

cudaError_t launch_expert_combine(const CombineArgs &a, bool f32, cudaStream_t st)
{
    return f32 ? run_combine<float, false>(a, st) : run_combine<__nv_bfloat16, false>(a, st);
}

cudaError_t launch_expert_combine_bwd(const CombineArgs &a, bool f32, cudaStream_t st)
{
    return f32 ? run_combine<float, true>(a, st) : run_combine<__nv_bfloat16, true>(a, st);
}

}  // namespace hstu
