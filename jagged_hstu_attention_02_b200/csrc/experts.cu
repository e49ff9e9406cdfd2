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
// Pairs that one block sorts by itself: 2048 take 6.8 us (7.0 with two launches over several
// blocks), 4096 10.7 (7.0), 1024 5.2 (4.9), 512 3.9 (3.9).
constexpr int kSortOneBlock = 2048;
constexpr int kSortMaxBlocks = 148;
constexpr int kBatch = 4;               // ids per lane fetched at a time

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

// Calls f(pair, expert or -1) for the pairs [b, e) of this warp, 32 at a time and in order, all
// lanes together; the ids of kBatch steps are fetched at once.
template <typename I, typename F>
__device__ __forceinline__ void walk_run(const SortArgs &a, int64_t b, int64_t e, bool report, F f)
{
    const int lane = threadIdx.x & 31;
    for (int64_t p0 = b; p0 < e; p0 += 32 * kBatch) {
        int x[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int64_t p = p0 + 32 * u + lane;
            x[u] = p < e ? expert_of<I>(a, p, report) : -1;
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (p0 + 32 * u < e) f(p0 + 32 * u + lane, x[u]);       // (warp-uniform)
    }
}

// Counts this warp's pairs per expert into its own row of shared memory.
template <typename I>
__device__ __forceinline__ void count_run(const SortArgs &a, int64_t b, int64_t e, int32_t *mine,
                                          bool report)
{
    const int lane = threadIdx.x & 31;
    walk_run<I>(a, b, e, report, [&](int64_t, int x) {
        const unsigned same = __match_any_sync(kFullMask, x);
        if (x >= 0 && lane == __ffs(same) - 1) mine[x] += __popc(same);
        __syncwarp();
    });
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
    walk_run<I>(a, b, e, false, [&](int64_t p, int x) {
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
    });
}

// ONE: the whole sort in one block.  Otherwise the second launch of two: expert_count_kernel
// has left every block's counts in a.hist, and each block adds those of the blocks before it.
template <typename I, bool ONE>
__global__ void __launch_bounds__(kSortThreads) expert_place_kernel(const __grid_constant__ SortArgs a)
{
    extern __shared__ int32_t sh[];                  // [kSortWarps][experts]
    __shared__ int wsum[kSortWarps];
    __shared__ int32_t sums[2][ONE ? 1 : kMaxExperts];   // pairs of all blocks, of earlier blocks
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t chunk = (a.n + gridDim.x - 1) / gridDim.x;
    const int64_t lo = min(a.n, (int64_t)blockIdx.x * chunk), hi = min(a.n, lo + chunk);
    int64_t b, e;
    warp_run(lo, hi, warp, b, e);
    for (int x = tid; x < kSortWarps * a.experts; x += kSortThreads) sh[x] = 0;
    if constexpr (ONE) {
        grid_dep_wait();
        grid_dep_release();
    }
    __syncthreads();
    count_run<I>(a, b, e, sh + warp * a.experts, ONE);
    if constexpr (!ONE) {
        // the blocks' counts: 32 experts and a share of the blocks per warp
        for (int x = tid; x < a.experts; x += kSortThreads) sums[0][x] = sums[1][x] = 0;
        grid_dep_wait();
        grid_dep_release();
        __syncthreads();
        const int chunks = (a.experts + 31) / 32;
        const int shares = chunks >= kSortWarps ? 1 : kSortWarps / chunks;
        const int per = ((int)gridDim.x + shares - 1) / shares;
        for (int task = warp; task < chunks * shares; task += kSortWarps) {
            const int x = task % chunks * 32 + lane, q0 = task / chunks * per;
            const int q1 = min(q0 + per, (int)gridDim.x);
            int all = 0, before = 0;
            if (x < a.experts) {
#pragma unroll 16
                for (int q = q0; q < q1; ++q) {
                    const int v = a.hist[(int64_t)q * a.experts + x];
                    all += v;
                    if (q < (int)blockIdx.x) before += v;
                }
                atomicAdd(&sums[0][x], all);
                atomicAdd(&sums[1][x], before);
            }
        }
    }
    __syncthreads();
    int base = 0;
    for (int x0 = 0; x0 < a.experts; x0 += kSortThreads) {
        const int x = x0 + tid;
        int all = 0, before = 0;
        if (x < a.experts) {
            if constexpr (ONE) {
                for (int w = 0; w < kSortWarps; ++w) all += sh[w * a.experts + x];
            } else {
                all = sums[0][x];
                before = sums[1][x];
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
    grid_dep_wait();
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
        e = allow_smem<expert_place_kernel<I, true>>(smem);
        if (e != cudaSuccess) return e;
        return launch_pdl(expert_place_kernel<I, true>, dim3(1), dim3(kSortThreads), smem, st, a);
    }
    e = allow_smem<expert_count_kernel<I>>(smem);
    if (e == cudaSuccess) e = allow_smem<expert_place_kernel<I, false>>(smem);
    if (e != cudaSuccess) return e;                       // (before the first launch)
    e = launch_pdl(expert_count_kernel<I>, dim3(blocks), dim3(kSortThreads), smem, st, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(expert_place_kernel<I, false>, dim3(blocks), dim3(kSortThreads), smem, st, a);
}

// ------------------------------------------------------------------ rows of tokens

constexpr int kRowWarps = 8;            // per block

// Warps that share a token's row of `pieces` pieces, `per_lane` of them per lane.
int warps_per_row(int64_t pieces, int per_lane)
{
    int w = 1;
    while (w < kRowWarps && w * 32 * per_lane < pieces) w *= 2;
    return w;
}

constexpr int kLaneElems = 4;

// An element as it lies in memory, if `yes`, else 0.  (Inline for the reason at load16_if.)
__device__ __forceinline__ void load_elem(const void *p, bool yes, uint8_t &v)
{
    uint16_t w;
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\tmov.b16 %0, 0;\n\t@q ld.global.b8 %0, [%1];\n\t}"
                 : "=&h"(w) : "l"(p), "r"((int)yes));
    v = (uint8_t)w;
}
__device__ __forceinline__ void load_elem(const void *p, bool yes, uint16_t &v)
{
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\tmov.b16 %0, 0;\n\t@q ld.global.b16 %0, [%1];\n\t}"
                 : "=&h"(v) : "l"(p), "r"((int)yes));
}
__device__ __forceinline__ void load_elem(const void *p, bool yes, uint32_t &v)
{
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\tmov.b32 %0, 0;\n\t@q ld.global.b32 %0, [%1];\n\t}"
                 : "=&r"(v) : "l"(p), "r"((int)yes));
}
__device__ __forceinline__ void load_elem(const void *p, bool yes, uint64_t &v)
{
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\tmov.b64 %0, 0;\n\t@q ld.global.b64 %0, [%1];\n\t}"
                 : "=&l"(v) : "l"(p), "r"((int)yes));
}
__device__ __forceinline__ float elem(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ float elem(uint32_t v) { return __uint_as_float(v); }
__device__ __forceinline__ void store_elem(__nv_bfloat16 *p, float f) { *p = __float2bfloat16_rn(f); }
__device__ __forceinline__ void store_elem(float *p, float f) { *p = f; }
template <typename T> struct ElemBits { using type = uint32_t; };
template <> struct ElemBits<__nv_bfloat16> { using type = uint16_t; };

// The elements p[0], p[32], ..., `n` of them.
template <typename T, typename B>
__device__ __forceinline__ void load_apart(const T *p, int n, B (&v)[kLaneElems])
{
#pragma unroll
    for (int i = 0; i < kLaneElems; ++i) load_elem(p + 32 * i, i < n, v[i]);
}

// Rows wider than 16 pieces: wpr warps per token read its row once, 4 pieces per lane in
// flight, and write it to each of the token's places.
__global__ void __launch_bounds__(32 * kRowWarps)
    expert_dispatch_kernel(const __grid_constant__ DispatchArgs a, int wpr)
{
    grid_dep_wait();
    grid_dep_release();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * (kRowWarps / wpr) + warp / wpr;
    if (t >= a.tokens) return;
    const int part = warp % wpr;
    int mine = lane < a.choices ? a.slots[t * a.choices + lane] : -1;
    if (mine >= a.max_rows) mine = -1;
    const int64_t per = a.row_bytes / 16;
    const uint4 *src = reinterpret_cast<const uint4 *>(a.x + t * a.row_bytes);
    for (int64_t c0 = part * 32 + lane; c0 - lane < per; c0 += 4 * 32 * wpr) {
        uint4 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t c = c0 + u * 32 * wpr;
            if (c < per) v[u] = src[c];
        }
        for (int j = 0; j < a.choices; ++j) {
            const int s = __shfl_sync(kFullMask, mine, j);
            if (s < 0) continue;
            uint4 *dst = reinterpret_cast<uint4 *>(a.out + (int64_t)s * a.row_bytes);
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

// Rows that start anywhere, of whole elements E (1 to 8 bytes): 128 elements per warp and turn, a
// lane's 4 lying 32 apart.  One element per access is what all alignments have in common, and a
// warp's access is still a run of neighbours.  (By aligned pieces of 16 bytes, shifted into place,
// 16384 x 4 places: 1001 bf16 46.4 us against 36.9, 1003 fp32 82 against 57, 1001 bytes 42 against 34.)
template <typename E>
__global__ void __launch_bounds__(32 * kRowWarps)
    expert_dispatch_apart_kernel(const __grid_constant__ DispatchArgs a, int wpr)
{
    grid_dep_wait();
    grid_dep_release();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * (kRowWarps / wpr) + warp / wpr;
    if (t >= a.tokens) return;
    const int part = warp % wpr;
    int mine = lane < a.choices ? a.slots[t * a.choices + lane] : -1;
    if (mine >= a.max_rows) mine = -1;
    const int64_t width = a.row_bytes / (int64_t)sizeof(E);
    const E *src = reinterpret_cast<const E *>(a.x) + t * width;
    E *out = reinterpret_cast<E *>(a.out);
    for (int64_t c0 = part * 128; c0 < width; c0 += 128 * wpr) {
        const int64_t c = c0 + lane;
        const int n = (int)min((width - c + 31) >> 5, (int64_t)kLaneElems);
        E v[kLaneElems];
        load_apart(src + c, n, v);
        for (int j = 0; j < a.choices; ++j) {
            const int s = __shfl_sync(kFullMask, mine, j);
            if (s < 0) continue;
            E *to = out + s * width + c;
#pragma unroll
            for (int i = 0; i < kLaneElems; ++i)
                if (i < n) to[32 * i] = v[i];
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

// Narrow rows (up to 16 pieces): 2^shift lanes per (token, choice) pair, one piece each, 4 pairs
// per lane.  262144 pairs, against a warp per token: 64-byte rows 35 us there, 256-byte rows 37
// against 31, 512-byte rows (which the other kernel takes) 41 against 59.
template <typename V>
__global__ void __launch_bounds__(256)
    expert_dispatch_narrow_kernel(const __grid_constant__ DispatchArgs a, int shift)
{
    grid_dep_wait();
    grid_dep_release();
    const int lanes = 1 << shift, c = threadIdx.x & (lanes - 1);
    const int64_t n = a.tokens * a.choices, step = 256 >> shift;
    const int64_t first = (int64_t)blockIdx.x * 4 * step + (threadIdx.x >> shift);
    const int per = (int)(a.row_bytes / (int64_t)sizeof(V));
    int s[4];
    uint32_t t[4];
    V v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int64_t pair = first + u * step;
        s[u] = pair < n ? a.slots[pair] : -1;
        if (s[u] >= a.max_rows) s[u] = -1;
        t[u] = (uint32_t)pair / (uint32_t)a.choices;           // tokens * choices < 2^31
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
        if (s[u] >= 0 && c < per) v[u] = reinterpret_cast<const V *>(a.x + (int64_t)t[u] * a.row_bytes)[c];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        if (s[u] < 0) continue;
        if (c < per) reinterpret_cast<V *>(a.out + (int64_t)s[u] * a.row_bytes)[c] = v[u];
        if (a.scales)
            for (int g = c; g < a.n_scales; g += lanes)
                a.scales_out[(int64_t)s[u] * a.n_scales + g] = a.scales[(int64_t)t[u] * a.n_scales + g];
    }
}

template <typename V>
cudaError_t run_dispatch(const DispatchArgs &a, cudaStream_t st)
{
    const int64_t per = a.row_bytes / (int64_t)sizeof(V);
    if (per <= 16) {
        int shift = 0;
        while ((1 << shift) < per) ++shift;
        const int64_t per_block = 4 * (256 >> shift);
        return launch_pdl(expert_dispatch_narrow_kernel<V>,
                          dim3((unsigned)((a.tokens * a.choices + per_block - 1) / per_block)), dim3(256),
                          0, st, a, shift);
    }
    const int wpr = warps_per_row((a.row_bytes + 15) / 16, sizeof(V) == 16 ? 4 : 1);
    const int tokens = kRowWarps / wpr;
    auto k = sizeof(V) == 16  ? expert_dispatch_kernel
             : sizeof(V) == 8 ? expert_dispatch_apart_kernel<uint64_t>
             : sizeof(V) == 4 ? expert_dispatch_apart_kernel<uint32_t>
             : sizeof(V) == 2 ? expert_dispatch_apart_kernel<uint16_t>
                              : expert_dispatch_apart_kernel<uint8_t>;
    return launch_pdl(k, dim3((unsigned)((a.tokens + tokens - 1) / tokens)), dim3(32 * kRowWarps), 0,
                      st, a, wpr);
}

// How a token's lanes lie, for the combine kernels.  Wide rows: wpr warps per token, 256
// elements per warp and turn.  Narrow rows (VEC, at most 128 elements): lanes = 2^k >= width / 8
// neighbours per token and 32 / lanes tokens per warp.
struct RowLanes {
    int wpr, lanes;
};

// A lane's part in a block's `tile` of tokens.
struct TokenPart {
    int64_t t;
    int c0, step;              // first element of the warp's turns (wide), their distance
    int lane;                  // among the token's lanes of this warp
};

__device__ __forceinline__ int tokens_per_tile(const RowLanes &r)
{
    return kRowWarps / r.wpr * (32 / r.lanes);
}

__device__ __forceinline__ TokenPart token_part(const RowLanes &r, int64_t tile)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    TokenPart p;
    p.t = tile * tokens_per_tile(r) + (r.lanes == 32 ? warp / r.wpr : (warp * 32 + lane) / r.lanes);
    p.c0 = r.lanes == 32 ? warp % r.wpr * 256 : 0;
    p.step = 256 * r.wpr;
    p.lane = lane & (r.lanes - 1);
    return p;
}

// A token's places (-1: none) and weights.
template <int KM>
struct Places {
    int s[KM];
    float w[KM];
    __device__ __forceinline__ void load(const CombineArgs &a, int64_t t)
    {
#pragma unroll
        for (int j = 0; j < KM; ++j) {
            const bool has = t < a.tokens && j < a.choices;
            s[j] = has ? a.slots[t * a.choices + j] : -1;
            w[j] = a.weights && has ? a.weights[t * a.choices + j] : 1.f;
        }
    }
    // Pairs without a row weigh 0, so that their (zero) rows may be added like the others': a
    // branch around each pair's use pulled its fetch in too, one latency after another.
    __device__ __forceinline__ void clip(int64_t max_rows)
    {
#pragma unroll
        for (int j = 0; j < KM; ++j)
            if (s[j] < 0 || s[j] >= max_rows) {
                s[j] = -1;
                w[j] = 0.f;
            }
    }
    // Row of pair j, and how much of it there is to read.
    __device__ __forceinline__ int64_t row(int j) const { return s[j] < 0 ? 0 : s[j]; }
    __device__ __forceinline__ int width(int j, int width) const { return s[j] < 0 ? 0 : width; }
};

// A narrow row's lanes may start anywhere in the warp: the c0 that makes elem8 count from them.
__device__ __forceinline__ int lane_c0(int c0, int lane) { return c0 + 8 * (lane - (int)(threadIdx.x & 31)); }

// Blocks per SM, so that the pieces of 4 choices fit the registers (fp32 takes twice as many).
template <typename T, int KM, bool BWD>
constexpr int combine_blocks()
{
    return sizeof(T) == 2 ? (KM <= 4 && !BWD ? 4 : KM <= 8 ? 3 : 2) : KM <= 4 ? 3 : 2;
}

// KM: the choices, rounded up to a power of two.  Blocks stay and walk the tokens; the places
// and weights of the next token are fetched while this one's rows move, and the rows of 4
// choices before the first of them is used.
template <typename T, int KM>
__global__ void __launch_bounds__(32 * kRowWarps, combine_blocks<T, KM, false>())
    expert_combine_kernel(const __grid_constant__ CombineArgs a, const RowLanes r)
{
    constexpr int KB = KM < 4 ? KM : 4;
    grid_dep_wait();
    grid_dep_release();
    const T *y = reinterpret_cast<const T *>(a.y), *y_end = y + a.max_rows * a.width;   // rows
    const T *resid = reinterpret_cast<const T *>(a.resid), *r_end = resid + a.tokens * a.width;
    const int per = tokens_per_tile(r);
    Places<KM> now, next;
    next.load(a, token_part(r, blockIdx.x).t);
    for (int64_t tile = blockIdx.x; tile * per < a.tokens; tile += gridDim.x) {
        const TokenPart p = token_part(r, tile);
        now = next;
        now.clip(a.max_rows);
        next.load(a, token_part(r, tile + gridDim.x).t);
        if (p.t >= a.tokens) continue;
        T *out = reinterpret_cast<T *>(a.out) + p.t * a.width;
        for (int turn = p.c0; turn < a.width; turn += p.step) {
            const int c0 = lane_c0(turn, p.lane);
            float acc[8];
            Piece<T, true> first, f[KB];
            if (resid) first.load(resid + p.t * a.width, c0, a.width, resid, r_end);
#pragma unroll
            for (int j0 = 0; j0 < KM; j0 += KB) {
#pragma unroll
                for (int u = 0; u < KB; ++u)
                    f[u].load(y + now.row(j0 + u) * a.width, c0, now.width(j0 + u, a.width), y, y_end);
                if (j0 == 0) {
                    if (resid) {
                        first.get(acc);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
                    }
                }
#pragma unroll
                for (int u = 0; u < KB; ++u) {
                    float v[8];
                    f[u].get(v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[e] = fmaf(now.w[j0 + u], v[e], acc[e]);
                }
            }
            store8<true>(out, c0, a.width, acc);
        }
    }
}

template <typename T, int KM>
__global__ void __launch_bounds__(32 * kRowWarps, combine_blocks<T, KM, true>())
    expert_combine_bwd_kernel(const __grid_constant__ CombineArgs a, const RowLanes r)
{
    constexpr int KB = KM < 4 ? KM : 4;
    __shared__ float dots[2][kRowWarps][KM];
    grid_dep_wait();
    grid_dep_release();
    const T *y = reinterpret_cast<const T *>(a.y), *y_end = y + a.max_rows * a.width;
    const T *g_end = reinterpret_cast<const T *>(a.dout) + a.tokens * a.width;
    T *dy = reinterpret_cast<T *>(a.dy);
    const int warp = threadIdx.x >> 5, per = tokens_per_tile(r);
    int flip = 0;
    Places<KM> now, next;
    next.load(a, token_part(r, blockIdx.x).t);
    for (int64_t tile = blockIdx.x; tile * per < a.tokens; tile += gridDim.x, flip ^= 1) {
        const TokenPart p = token_part(r, tile);
        now = next;
        now.clip(a.max_rows);
        next.load(a, token_part(r, tile + gridDim.x).t);
        const bool live = p.t < a.tokens;
        const int width = live ? a.width : 0;
        const T *dout = reinterpret_cast<const T *>(a.dout) + (live ? p.t * a.width : 0);
        float dot[KM];
#pragma unroll
        for (int j = 0; j < KM; ++j) dot[j] = 0.f;
        for (int turn = p.c0; turn < width; turn += p.step) {
            const int c0 = lane_c0(turn, p.lane);
            Piece<T, true> first, f[KB];
            float g[8];
            first.load(dout, c0, width, dout, g_end);
#pragma unroll
            for (int j0 = 0; j0 < KM; j0 += KB) {
                if (a.dweights) {
#pragma unroll
                    for (int u = 0; u < KB; ++u)
                        f[u].load(y + now.row(j0 + u) * a.width, c0, now.width(j0 + u, width), y, y_end);
                }
                if (j0 == 0) first.get(g);
#pragma unroll
                for (int u = 0; u < KB; ++u) {
                    const int j = j0 + u;
                    if (a.dweights && now.s[j] >= 0) {     // (0 times dout may be NaN)
                        float v[8];
                        f[u].get(v);
#pragma unroll
                        for (int e = 0; e < 8; ++e) dot[j] = fmaf(g[e], v[e], dot[j]);
                    }
                    if (now.s[j] < 0) continue;
                    float o[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] = now.w[j] * g[e];
                    store8<true>(dy + (int64_t)now.s[j] * a.width, c0, width, o);
                }
            }
        }
        if (!a.dweights) continue;
#pragma unroll
        for (int j = 0; j < KM; ++j)
            for (int o = r.lanes / 2; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(kFullMask, dot[j], o);
        // (0 where a pair has no place)
        if (r.wpr == 1) {
            if (live && p.lane == 0) {
#pragma unroll
                for (int j = 0; j < KM; ++j)
                    if (j < a.choices) a.dweights[p.t * a.choices + j] = dot[j];
            }
        } else {
            if (p.lane == 0) {
#pragma unroll
                for (int j = 0; j < KM; ++j) dots[flip][warp][j] = dot[j];
            }
            __syncthreads();
            if (live && warp % r.wpr == 0 && p.lane < a.choices) {
                float sum = 0.f;
                for (int q = 0; q < r.wpr; ++q) sum += dots[flip][warp + q][p.lane];
                a.dweights[p.t * a.choices + p.lane] = sum;
            }
        }
    }
}

// The same for rows that start anywhere: wpr warps per token, 128 elements per warp and turn, a
// lane's 4 lying 32 apart as in the dispatch, those of 4 choices fetched before the first is used.
// (Aligned pieces of 16 bytes, shifted into place, 1001 wide: bf16 65.8 us against 53.4, backward 100.7
// against 74.8; fp32 77.4 against 71.4, 142 against 109.  100 wide: 187 against 90, 358 against 134.)
template <typename T>
__global__ void __launch_bounds__(32 * kRowWarps, 5)
    expert_combine_apart_kernel(const __grid_constant__ CombineArgs a, int wpr)
{
    grid_dep_wait();
    grid_dep_release();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * (kRowWarps / wpr) + warp / wpr;
    if (t >= a.tokens) return;
    int place = lane < a.choices ? a.slots[t * a.choices + lane] : -1;
    if (place >= a.max_rows) place = -1;
    const float weight = a.weights && place >= 0 ? a.weights[t * a.choices + lane] : 1.f;
    const T *y = reinterpret_cast<const T *>(a.y);
    const T *resid = a.resid ? reinterpret_cast<const T *>(a.resid) + t * a.width : nullptr;
    T *out = reinterpret_cast<T *>(a.out) + t * a.width;
    int s[4];
    float w[4];
    auto places = [&](int j0) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            s[u] = __shfl_sync(kFullMask, place, j0 + u);
            w[u] = s[u] < 0 ? 0.f : __shfl_sync(kFullMask, weight, j0 + u);    // (warp-uniform)
        }
    };
    places(0);
    for (int c0 = warp % wpr * 128; c0 < a.width; c0 += 128 * wpr) {
        const int c = c0 + lane, n = (a.width - c + 31) >> 5;  // elements from c on, 32 apart
        typename ElemBits<T>::type r[kLaneElems], v[4][kLaneElems];
        load_apart(resid + c, resid ? n : 0, r);
        float acc[kLaneElems];
        for (int j0 = 0;;) {
#pragma unroll
            for (int u = 0; u < 4; ++u) load_apart(y + (int64_t)s[u] * a.width + c, s[u] >= 0 ? n : 0, v[u]);
#pragma unroll
            for (int i = 0; i < kLaneElems; ++i) {
                if (j0 == 0) acc[i] = elem(r[i]);
#pragma unroll
                for (int u = 0; u < 4; ++u) acc[i] = fmaf(w[u], elem(v[u][i]), acc[i]);
            }
            j0 += 4;
            if (j0 < a.choices) places(j0);
            else break;
        }
        if (a.choices > 4) places(0);
#pragma unroll
        for (int i = 0; i < kLaneElems; ++i)
            if (i < n) store_elem(out + c + 32 * i, acc[i]);
    }
}

template <typename T>
__global__ void __launch_bounds__(32 * kRowWarps, 4)
    expert_combine_bwd_apart_kernel(const __grid_constant__ CombineArgs a, int wpr)
{
    __shared__ float dots[kRowWarps][kMaxChoices];
    grid_dep_wait();
    grid_dep_release();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * (kRowWarps / wpr) + warp / wpr;
    const bool live = t < a.tokens;
    int place = live && lane < a.choices ? a.slots[t * a.choices + lane] : -1;
    if (place >= a.max_rows) place = -1;
    const float weight = a.weights && place >= 0 ? a.weights[t * a.choices + lane] : 1.f;
    const T *y = reinterpret_cast<const T *>(a.y);
    const T *dout = reinterpret_cast<const T *>(a.dout) + (live ? t * a.width : 0);
    T *dy = reinterpret_cast<T *>(a.dy);
    float mine = 0.f;                                      // lane j: the dot product of pair j
    for (int j0 = 0; live && j0 < a.choices; j0 += 4) {
        int s[4];
        float w[4], d[4] = {};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            s[u] = __shfl_sync(kFullMask, place, j0 + u);
            w[u] = __shfl_sync(kFullMask, weight, j0 + u);
        }
        for (int c = warp % wpr * 128 + lane; c < a.width; c += 128 * wpr) {
            const int n = (a.width - c + 31) >> 5;
            typename ElemBits<T>::type g[kLaneElems], v[4][kLaneElems];
            load_apart(dout + c, n, g);
            if (a.dweights) {
#pragma unroll
                for (int u = 0; u < 4; ++u) load_apart(y + (int64_t)s[u] * a.width + c, s[u] >= 0 ? n : 0, v[u]);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (s[u] < 0) continue;                    // (warp-uniform)
                T *to = dy + (int64_t)s[u] * a.width + c;
#pragma unroll
                for (int i = 0; i < kLaneElems; ++i) {
                    const float x = elem(g[i]);
                    if (a.dweights) d[u] = fmaf(x, elem(v[u][i]), d[u]);
                    if (i < n) store_elem(to + 32 * i, w[u] * x);
                }
            }
        }
        if (!a.dweights) continue;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float sum = warp_sum(d[u]);
            if (lane == j0 + u) mine = sum;
        }
    }
    if (!a.dweights) return;
    if (lane < a.choices) dots[warp][lane] = mine;
    __syncthreads();
    if (live && warp % wpr == 0 && lane < a.choices) {
        float sum = 0.f;
        for (int q = 0; q < wpr; ++q) sum += dots[warp + q][lane];
        a.dweights[t * a.choices + lane] = sum;            // (0 where the pair has no place)
    }
}

template <typename T, int KM, bool BWD>
cudaError_t run_combine_km(const CombineArgs &a, int64_t tiles, const RowLanes &r, cudaStream_t st)
{
    const int64_t most = (int64_t)num_sms() * combine_blocks<T, KM, BWD>();
    const unsigned grid = (unsigned)(tiles < most ? tiles : most);
    if constexpr (BWD)
        return launch_pdl(expert_combine_bwd_kernel<T, KM>, dim3(grid), dim3(32 * kRowWarps), 0, st, a, r);
    else
        return launch_pdl(expert_combine_kernel<T, KM>, dim3(grid), dim3(32 * kRowWarps), 0, st, a, r);
}

template <typename T, bool BWD>
cudaError_t run_combine(const CombineArgs &a, cudaStream_t st)
{
    if (a.tokens <= 0) return cudaSuccess;
    if (a.width % 8 != 0) {
        const int wpr = warps_per_row((a.width + 7) / 8, 4);
        const int64_t per = kRowWarps / wpr;
        return launch_pdl(BWD ? expert_combine_bwd_apart_kernel<T> : expert_combine_apart_kernel<T>,
                          dim3((unsigned)((a.tokens + per - 1) / per)), dim3(32 * kRowWarps), 0, st, a,
                          wpr);
    }
    RowLanes r;
    r.lanes = 32;
    r.wpr = 1;
    if (a.width <= 128) {
        r.lanes = 1;
        while (r.lanes * 8 < a.width) r.lanes *= 2;
    } else {
        // a warp takes 4 turns of 512 bytes (2 of 1024), or one where that leaves SMs without a
        // token (64 tokens of 1024 bf16: 4.4 us against 3.1)
        r.wpr = warps_per_row((a.width + 7) / 8, sizeof(T) == 2 ? 4 : 2);
        if (a.tokens * r.wpr <= (int64_t)num_sms() * kRowWarps) r.wpr = warps_per_row((a.width + 7) / 8, 1);
    }
    const int64_t per = (int64_t)kRowWarps / r.wpr * (32 / r.lanes);
    const int64_t tiles = (a.tokens + per - 1) / per;
    if (a.choices <= 1) return run_combine_km<T, 1, BWD>(a, tiles, r, st);
    if (a.choices <= 2) return run_combine_km<T, 2, BWD>(a, tiles, r, st);
    if (a.choices <= 4) return run_combine_km<T, 4, BWD>(a, tiles, r, st);
    if (a.choices <= 8) return run_combine_km<T, 8, BWD>(a, tiles, r, st);
    return run_combine_km<T, 16, BWD>(a, tiles, r, st);
}

}  // namespace

int sort_blocks(int64_t n)
{
    if (n <= kSortOneBlock) return 1;
    const int64_t b = (n + 1023) / 1024;
    return (int)(b < kSortMaxBlocks ? b : kSortMaxBlocks);
}

cudaError_t launch_expert_sort(const SortArgs &a, bool ids64, cudaStream_t st)
{
    return ids64 ? run_sort<int64_t>(a, st) : run_sort<int32_t>(a, st);
}

cudaError_t launch_expert_dispatch(const DispatchArgs &a, cudaStream_t st)
{
    if (a.tokens <= 0) return cudaSuccess;
    switch (a.row_bytes & 15) {
    case 0: return run_dispatch<uint4>(a, st);
    case 8: return run_dispatch<uint2>(a, st);
    case 4: case 12: return run_dispatch<uint32_t>(a, st);
    default: return a.row_bytes % 2 == 0 ? run_dispatch<uint16_t>(a, st) : run_dispatch<uint8_t>(a, st);
    }
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
