// experts.h -- launchers of the kernels of the mixture-of-experts layer: the RMS norm of
// rows (rmsnorm.cu), sorting rows by expert and bringing them back (experts.cu) and the
// experts' products (expert_gemm.cu).  Internal; the C ABI is include/hstu_attn.h.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "hstu_attn.h"

namespace hstu {

// Lets Kern use `bytes` of dynamic shared memory.  Without the attribute a block may have 48 KB,
// what the kernel declares itself included.  Its own part is asked for once per kernel, and the
// attribute raised once per kernel and device (asking the runtime at every call took a fifth of a
// small call's time on the host).
template <auto Kern>
cudaError_t allow_smem(size_t bytes)
{
    constexpr int kMaxDev = 64;
    static std::atomic<int64_t> own{-1};
    static std::atomic<size_t> allowed[kMaxDev];
    int64_t fixed = own.load(std::memory_order_relaxed);
    if (fixed < 0) {
        cudaFuncAttributes fa;
        const cudaError_t e = cudaFuncGetAttributes(&fa, Kern);
        if (e != cudaSuccess) return e;
        fixed = (int64_t)fa.sharedSizeBytes;
        own.store(fixed, std::memory_order_relaxed);
    }
    if (bytes + (size_t)fixed <= 48 * 1024) return cudaSuccess;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDev && allowed[dev].load(std::memory_order_acquire) >= bytes) return cudaSuccess;
    int most = 0;
    e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    if (e != cudaSuccess) return e;
    const size_t room = (size_t)(most - fixed);
    if (bytes > room) return cudaErrorInvalidValue;
    e = cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)room);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDev) allowed[dev].store(room, std::memory_order_release);
    return cudaSuccess;
}

// ------------------------------------------------------------------ rmsnorm.cu
constexpr int kMaxNormWidth = 16384;

struct RmsArgs {
    const void *x, *resid;      // [rows, width]; resid may be null
    const float *weight;        // [width] or null
    int64_t rows;
    int width;
    float eps;
    int group;                  // e4m3: columns per scale (0: the row)
    void *y, *sum;              // y [rows, width]; sum (x + resid) or null
    float *scales, *rstd;       // scales with e4m3 output; rstd or null
};

struct RmsBwdArgs {
    const void *dy, *h;         // [rows, width]
    const void *dsum;           // [rows, width] or null
    const float *rstd, *weight; // [rows]; [width] or null
    int64_t rows;
    int width;
    void *dx;                   // [rows, width]
    float *dweight;             // [width] or null
    float *part;                // rms_bwd_blocks(...) x width floats, when dweight is wanted
};

cudaError_t launch_rms_norm(const RmsArgs &a, bool f32, bool e4m3, cudaStream_t st);
// Blocks (rows of partial weight gradients) of the backward for this shape.
int rms_bwd_blocks(int64_t rows, int width);
cudaError_t launch_rms_norm_bwd(const RmsBwdArgs &a, bool f32, cudaStream_t st);

// ------------------------------------------------------------------ experts.cu
constexpr int kMaxExperts = 1024;
constexpr int kMaxChoices = 16;
constexpr int kMaxCombineWidth = 1 << 30;   // (element counters of a row step past its end in 32 bits)

struct SortArgs {
    const void *ids;            // [n] int32 or int64
    int64_t n;                  // tokens * choices
    int choices, experts;
    int32_t *slots;             // [n]
    int64_t *offsets;           // [experts + 1]
    int64_t *rows;              // [n] or null
    int32_t *status;            // or null
    int32_t *hist;              // sort_blocks(n) x experts counters, when sort_blocks(n) > 1
};

int sort_blocks(int64_t n);
cudaError_t launch_expert_sort(const SortArgs &a, bool ids64, cudaStream_t st);

struct DispatchArgs {
    const uint8_t *x;           // [tokens] rows of row_bytes
    const float *scales;        // [tokens, n_scales] or null
    const int32_t *slots;       // [tokens, choices]
    int64_t tokens, row_bytes, max_rows;
    int choices, n_scales;
    uint8_t *out;
    float *scales_out;
};
cudaError_t launch_expert_dispatch(const DispatchArgs &a, cudaStream_t st);

struct CombineArgs {
    const void *y;              // [max_rows, width]
    const int32_t *slots;       // [tokens, choices]
    const float *weights;       // [tokens, choices] or null (all one)
    const void *resid;          // [tokens, width] or null
    const void *dout;           // backward: [tokens, width]
    int64_t tokens, max_rows;
    int choices, width;
    void *out;                  // forward: [tokens, width]
    void *dy;                   // backward: [max_rows, width]
    float *dweights;            // backward: [tokens, choices] or null
};
cudaError_t launch_expert_combine(const CombineArgs &a, bool f32, cudaStream_t st);
cudaError_t launch_expert_combine_bwd(const CombineArgs &a, bool f32, cudaStream_t st);

// ------------------------------------------------------------------ expert_gemm.cu
struct ProjArgs {
    const void *x, *w;          // x [rows, k]; w [experts, k, n] (e4m3: [experts, n, k])
    const float *x_scales, *w_scales;   // e4m3: [rows], [experts, n]
    const int64_t *offsets;     // [experts + 1]
    int64_t rows;
    int experts, k, n;
    int silu;
    void *out, *pre;            // [rows, n]; pre (x w before the SiLU) or null
    const void *dout;           // backward: [rows, n]
    const void *silu_pre;       // backward: [rows, k] or null
    void *dx, *dw;              // backward: [rows, k], [experts, k, n]
    float *partial;             // dw: expert_dw_plan(...).slices x experts x k x n floats when > 1
    int32_t *status;
    long long wait_limit;
    int stall_test;
};
cudaError_t launch_expert_proj(const ProjArgs &a, bool e4m3, cudaStream_t st);
cudaError_t launch_expert_proj_dx(const ProjArgs &a, cudaStream_t st);
// How the weights' gradient runs: by pairs of CTAs or single ones, and the parts that the
// experts' rows are cut into.
struct DwPlan {
    bool pair;
    int slices;
};
DwPlan expert_dw_plan(int64_t rows, int experts, int k, int n);
cudaError_t launch_expert_proj_dw(const ProjArgs &a, cudaStream_t st);

}  // namespace hstu
