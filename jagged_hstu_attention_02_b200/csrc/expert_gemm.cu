// expert_gemm.cu -- the experts' products on rows sorted by expert (a jagged tensor whose
// sequences are the experts; offsets in device memory), on the tcgen05 tensor cores:
//
//   P_FWD   out_s = x_s W_e            bf16, W [E, K, N]; optional SiLU in the epilogue
//   P_E4M3  out_s = xs_s ws_e (x_s W_e)  e4m3 values, W [E, N, K], fp32 scales per row and column
//   P_DX    dx_s = (dout_s W_e^T) (.) SiLU'(pre_s)
//   P_DW    dW_e = X_e^T dOut_e        contraction over the expert's rows
//
// Persistent CTAs take 128 x BN output tiles; a tile lies in one expert.  The host never reads
// the offsets: every CTA sums up the experts' row tiles in shared memory at its start and finds
// a tile's expert by bisection.  Warp 0 streams 128-byte-wide slices of both operands through a
// TMA ring (128-byte swizzle), warp 1 issues tcgen05.mma into one of two TMEM accumulators,
// eight warps read the other accumulator back and store it.  Rows of a tile past the
// expert's end hold another expert's rows (or nothing): they are computed, not stored.  In P_DW
// they would enter the sums, so the MMA warp zeroes them in shared memory first.
// Every wait is bounded.
#include <cudaTypedefs.h>

#include <cstring>

#include "experts.h"
#include "kernels.h"
#include "sm100.cuh"
#include "units.cuh"

namespace hstu {

using namespace sm100;

namespace {

enum Product { P_FWD = 0, P_E4M3 = 1, P_DX = 2, P_DW = 3 };

constexpr int EBM = 128;             // rows of an output tile (TMEM lanes)
constexpr int kSlice = 128;          // bytes of the contraction per stage and row
constexpr int kSmallBox = 16;        // rows of the small A box, for tiles with few rows
constexpr int kEpiWarps = 8;
constexpr int kEThreads = 32 * (2 + kEpiWarps);

struct EGemmArgs {
    CUtensorMap ta, ta_small, tb;
    const int64_t *offsets;
    int64_t rows;                    // rows of the sorted tensors
    int experts;
    int kc;                          // contraction length (P_DW: the expert's rows instead)
    int m, n;                        // P_DW: rows of an output tile's matrix; output columns
    int silu;
    const float *x_scales, *w_scales;
    const __nv_bfloat16 *silu_pre;   // P_DX
    __nv_bfloat16 *out, *pre;
    int32_t *status;
    long long wait_limit;
    int stall_test;                  // test only: the MMA warp first waits for nothing
};

template <int BN>
struct ELayout {
    static constexpr int STAGES = BN == 256 ? 4 : 6;
    static constexpr int AB = EBM * kSlice;           // 16 KB
    static constexpr int BB = BN * kSlice;
    static constexpr int A_OFF = 0;
    static constexpr int B_OFF = STAGES * AB;
    static constexpr int BAR_OFF = B_OFF + STAGES * BB;
    static constexpr int TAB_OFF = BAR_OFF + 256;     // tile prefix and row starts
};

__device__ __forceinline__ void load_2d(void *dst, const CUtensorMap *map, uint64_t *bar, int c0,
                                        int c1)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
        : "memory");
}

// D (TMEM) += A (smem) B (smem), e4m3 values, fp32 accumulator: 32 of the contraction per MMA.
__device__ __forceinline__ void umma_f8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Instruction descriptor of kind::f8f6f4 with e4m3 A and B (format 0), K-major, fp32 D.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N)
{
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void egemm_flag(const EGemmArgs &a, int bits)
{
    if (a.status) atomicOr(a.status, bits);
}

// The experts' rows and row tiles, in shared memory: expert e's rows are [row0[e], row0[e] +
// cnt[e]) and its row tiles [tile0[e], tile0[e + 1]).
struct ExpertTable {
    int32_t *tile0, *row0, *cnt;
};

// Fills the table (all threads of the block).  An expert whose offsets are invalid has no rows.
__device__ __forceinline__ void fill_table(const EGemmArgs &a, const ExpertTable &t, int32_t *wsum)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kWarps = kEThreads / 32;
    int base = 0;
    for (int e0 = 0; e0 < a.experts; e0 += kEThreads) {
        const int e = e0 + tid;
        int tiles = 0;
        if (e < a.experts) {
            int64_t lo = a.offsets[e], hi = a.offsets[e + 1];
            if (lo < 0 || hi < lo || hi > a.rows) {
                if (blockIdx.x == 0) egemm_flag(a, HSTU_DEV_BAD_OFFSETS);
                lo = hi = 0;
            }
            t.row0[e] = (int)lo;
            t.cnt[e] = (int)(hi - lo);
            tiles = (int)((hi - lo + EBM - 1) / EBM);
        }
        int s = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += u;
        }
        if (lane == 31) wsum[warp] = s;
        __syncthreads();
        int before = base, all = 0;
        for (int w = 0; w < kWarps; ++w) {
            const int u = wsum[w];
            if (w < warp) before += u;
            all += u;
        }
        if (e < a.experts) t.tile0[e] = before + s - tiles;
        base += all;
        __syncthreads();
    }
    if (tid == 0) t.tile0[a.experts] = base;
}

struct ETile {
    int e;         // expert
    int m0, rows;  // first row (of the sorted rows; P_DW: of the matrix) and rows to store
    int n0;        // first output column
    int kbeg, kcnt;   // contraction: first index and length
};

template <int P, int BN>
__device__ __forceinline__ int tile_count(const EGemmArgs &a, const ExpertTable &t)
{
    const int nt = (a.n + BN - 1) / BN;
    return P == P_DW ? a.experts * ((a.m + EBM - 1) / EBM) * nt : t.tile0[a.experts] * nt;
}

template <int P, int BN>
__device__ __forceinline__ ETile tile_of(const EGemmArgs &a, const ExpertTable &t, int tile)
{
    const int nt = (a.n + BN - 1) / BN;
    ETile r;
    r.n0 = (tile % nt) * BN;
    const int q = tile / nt;
    if constexpr (P == P_DW) {
        const int mt = (a.m + EBM - 1) / EBM;
        r.e = q / mt;
        r.m0 = (q % mt) * EBM;
        r.rows = min(EBM, a.m - r.m0);
        r.kbeg = t.row0[r.e];
        r.kcnt = t.cnt[r.e];
    } else {
        int lo = 0, hi = a.experts;          // the last expert whose first tile is <= q
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (t.tile0[mid] <= q) lo = mid; else hi = mid;
        }
        r.e = lo;
        const int off = (q - t.tile0[lo]) * EBM;
        r.m0 = t.row0[lo] + off;
        r.rows = min(EBM, t.cnt[lo] - off);
        r.kbeg = 0;
        r.kcnt = a.kc;
    }
    return r;
}

enum EBar { E_FULL = 0, E_EMPTY = 8, EACC_FULL = 16, EACC_EMPTY = 18, E_DONE = 20, E_STALL = 21,
            E_NBARS = 22 };

template <int P, int BN>
__global__ void __launch_bounds__(kEThreads, 1) expert_gemm_kernel(const __grid_constant__ EGemmArgs a)
{
    using L = ELayout<BN>;
    constexpr int ST = L::STAGES;
    constexpr int KB = P == P_E4M3 ? 128 : 64;          // contraction per stage
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::BAR_OFF);
    uint32_t *slot = reinterpret_cast<uint32_t *>(sm + L::BAR_OFF + 8 * 24);
    int32_t *wsum = reinterpret_cast<int32_t *>(sm + L::BAR_OFF + 8 * 25);
    ExpertTable tab;
    tab.tile0 = reinterpret_cast<int32_t *>(sm + L::TAB_OFF);
    tab.row0 = tab.tile0 + a.experts + 1;
    tab.cnt = tab.row0 + a.experts;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        for (int x = 0; x < E_NBARS; ++x)
            mbar_init(&bars[x], x == EACC_EMPTY || x == EACC_EMPTY + 1 ? kEpiWarps : 1);
        fence_mbar_init();
    }
    if (warp == 2) tmem_alloc(slot, 2 * BN);
    fill_table(a, tab, wsum);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *slot;
    const uint32_t sm_base = smem_u32(sm);
    const int ntiles = tile_count<P, BN>(a, tab);

    if (warp == 0) {
        if (lane == 0) {
            // ---------------------------------------------------------------- TMA producer
            prefetch_tmap(&a.ta);
            prefetch_tmap(&a.tb);
            int g = 0;
            bool ok = true;
            for (int tile = blockIdx.x; ok && tile < ntiles; tile += gridDim.x) {
                const ETile r = tile_of<P, BN>(a, tab, tile);
                const int kch = (r.kcnt + KB - 1) / KB;
                const bool small = P != P_DW && r.rows <= 64;
                const int boxes = small ? (r.rows + kSmallBox - 1) / kSmallBox : 1;
                const uint32_t abytes = small ? boxes * kSmallBox * kSlice : L::AB;
                for (int kc = 0; kc < kch; ++kc, ++g) {
                    const int s = g % ST;
                    if (g >= ST && !mbar_wait(&bars[E_EMPTY + s], ((g / ST) - 1) & 1, a.wait_limit)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&bars[E_FULL + s], abytes + L::BB);
                    uint8_t *as = sm + L::A_OFF + s * L::AB, *bs = sm + L::B_OFF + s * L::BB;
                    uint64_t *full = &bars[E_FULL + s];
                    if constexpr (P == P_DW) {
                        // both operands lie along their rows: blocks of 64 columns x 64 rows
                        for (int b = 0; b < EBM / 64; ++b)
                            load_2d(as + b * 8192, &a.ta, full, r.m0 + 64 * b, r.kbeg + kc * KB);
                        for (int b = 0; b < BN / 64; ++b)
                            load_2d(bs + b * 8192, &a.tb, full, r.n0 + 64 * b, r.kbeg + kc * KB);
                    } else {
                        if (small) {
                            for (int b = 0; b < boxes; ++b)
                                load_2d(as + b * kSmallBox * kSlice, &a.ta_small, full, kc * KB,
                                        r.m0 + b * kSmallBox);
                        } else {
                            load_2d(as, &a.ta, full, kc * KB, r.m0);
                        }
                        if constexpr (P == P_FWD) {
                            for (int b = 0; b < BN / 64; ++b)
                                tma_load_3d(bs + b * 8192, &a.tb, full, r.n0 + 64 * b, kc * KB, r.e);
                        } else {
                            tma_load_3d(bs, &a.tb, full, kc * KB, r.n0, r.e);
                        }
                    }
                }
            }
            if (!ok) egemm_flag(a, HSTU_DEV_WAIT_TIMEOUT);
            // every copy issued has landed before the block may exit
            bool drained = true;
            for (int x = g - 1; x >= 0 && x >= g - ST; --x)
                drained &= mbar_wait(&bars[E_FULL + x % ST], (x / ST) & 1, kWaitLimitCycles);
            if (!drained) egemm_flag(a, HSTU_DEV_WAIT_TIMEOUT);
        }
    } else if (warp == 1) {
        // -------------------------------------------------------------------- MMA issuer
        // the whole warp walks the tiles (it zeroes rows together); lane 0 issues
        constexpr uint32_t idesc = P == P_E4M3 ? idesc_e4m3(EBM, BN)
                                               : idesc_bf16(EBM, BN, P == P_DW, P != P_DX);
        int g = 0, t = 0;
        bool ok = !a.stall_test || warp_wait(&bars[E_STALL], 0, a.wait_limit);
        for (int tile = blockIdx.x; ok && tile < ntiles; tile += gridDim.x) {
            const ETile r = tile_of<P, BN>(a, tab, tile);
            const int kch = (r.kcnt + KB - 1) / KB;
            if (kch == 0) continue;                     // (P_DW: an expert without rows)
            const int acc = t & 1;
            if (t >= 2 && !warp_wait(&bars[EACC_EMPTY + acc], ((t >> 1) - 1) & 1, a.wait_limit)) {
                ok = false;
                break;
            }
            ++t;
            tc_fence_after();
            const uint32_t d = tmem + acc * BN;
            for (int kc = 0; kc < kch; ++kc, ++g) {
                const int s = g % ST;
                if (!warp_wait(&bars[E_FULL + s], (g / ST) & 1, a.wait_limit)) {
                    ok = false;
                    break;
                }
                if constexpr (P == P_DW) {
                    // rows of this slice past the expert's end: zeros in both operands
                    const int valid = r.kcnt - kc * KB;
                    if (valid < KB) {
                        const int per = (KB - valid) * 8;            // 16-byte pieces per block
                        for (int b = 0; b < (EBM + BN) / 64; ++b) {
                            uint8_t *blk = b < EBM / 64 ? sm + L::A_OFF + s * L::AB + b * 8192
                                                        : sm + L::B_OFF + s * L::BB + (b - EBM / 64) * 8192;
                            uint4 *z = reinterpret_cast<uint4 *>(blk + valid * 128);
                            for (int x = lane; x < per; x += 32) z[x] = make_uint4(0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                }
                tc_fence_after();
                if (lane == 0) {
                    const uint32_t aa = sm_base + L::A_OFF + s * L::AB;
                    const uint32_t bb = sm_base + L::B_OFF + s * L::BB;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        // K-major: 32 bytes per step within the 128-byte rows, 8-row groups at
                        // 1 KB.  Otherwise 64-column blocks at 8 KB, 8-row groups of the
                        // contraction at 1 KB, 16 rows per step.
                        const uint64_t ad = P == P_DW ? sw128_desc(aa + kk * 2048, 8192, 1024)
                                                      : sw128_desc(aa + kk * 32, 16, 1024);
                        const uint64_t bd = P == P_FWD || P == P_DW
                                                ? sw128_desc(bb + kk * 2048, 8192, 1024)
                                                : sw128_desc(bb + kk * 32, 16, 1024);
                        if constexpr (P == P_E4M3)
                            umma_f8_ss(d, ad, bd, idesc, (kc | kk) ? 1u : 0u);
                        else
                            umma_bf16_ss(d, ad, bd, idesc, (kc | kk) ? 1u : 0u);
                    }
                    umma_commit(&bars[E_EMPTY + s]);
                }
                __syncwarp();
            }
            if (!ok) break;
            if (lane == 0) umma_commit(&bars[EACC_FULL + acc]);
            __syncwarp();
        }
        if (lane == 0) {
            if (!ok) egemm_flag(a, HSTU_DEV_WAIT_TIMEOUT);
            umma_commit(&bars[E_DONE]);
            if (!mbar_wait(&bars[E_DONE], 0, kWaitLimitCycles)) egemm_flag(a, HSTU_DEV_WAIT_TIMEOUT);
        }
        __syncwarp();
    } else {
        // -------------------------------------------------------------------- epilogue
        // 64 columns per step: a lane converts its row's values into 8 chunks of 8 bf16, a
        // transpose over groups of 8 lanes then lets 8 lanes store one row's 128 bytes
        const int q = warp & 3;                          // TMEM lane quarter: rows 32q ..
        const int half = (warp - 2) >> 2;                // columns [half BN/2, (half+1) BN/2)
        const int rr = q * 32 + lane;                    // row of the tile == TMEM lane
        const uint32_t lane_base = (uint32_t)(q * 32) << 16;
        const int j = lane & 7;                          // chunk this lane stores
        int t = 0;
        bool ok = true;
        for (int tile = blockIdx.x; tile < ntiles; tile += gridDim.x) {
            const ETile r = tile_of<P, BN>(a, tab, tile);
            const bool none = P == P_DW && r.kcnt == 0;  // a gradient of zeros, without an MMA
            const int acc = t & 1;
            if (!none) {
                if (!warp_wait(&bars[EACC_FULL + acc], (t >> 1) & 1, a.wait_limit)) {
                    ok = false;
                    break;
                }
                ++t;
                tc_fence_after();
            }
            const int64_t out0 = P == P_DW ? ((int64_t)r.e * a.m + r.m0) * a.n
                                           : (int64_t)r.m0 * a.n;
            const bool mine = rr < r.rows;
            float xs = 1.f;
            if (P == P_E4M3 && mine) xs = __ldg(a.x_scales + r.m0 + rr);
#pragma unroll 1
            for (int c0 = half * (BN / 2); c0 < (half + 1) * (BN / 2); c0 += 64) {
                const int nb = r.n0 + c0;
                if (nb >= a.n) break;                    // (warp-uniform)
                if (q * 32 >= r.rows) break;             // no row of this warp is stored
                __syncwarp();                            // the warp-wide TMEM loads below
                uint32_t v[32], w[32];
                if (!none) {
                    tmem_ld32(tmem + lane_base + acc * BN + c0, v);
                    tmem_ld32(tmem + lane_base + acc * BN + c0 + 32, w);
                    tmem_wait_ld();
                    reg_fence(v);
                    reg_fence(w);
                }
                float4 o[8], po[8];                      // 8 chunks of 8 bf16 (as 16 bytes)
#pragma unroll
                for (int hh = 0; hh < 8; ++hh) {
                    float f[8];
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        f[x] = none ? 0.f : __uint_as_float(hh < 4 ? v[8 * hh + x] : w[8 * hh - 32 + x]);
                    const int nc = nb + 8 * hh;          // n is a multiple of 8
                    if constexpr (P == P_E4M3) {
                        if (nc < a.n) {
                            const float4 *sp = reinterpret_cast<const float4 *>(
                                a.w_scales + (int64_t)r.e * a.n + nc);
                            const float4 s0 = __ldg(sp), s1 = __ldg(sp + 1);
                            f[0] *= xs * s0.x; f[1] *= xs * s0.y; f[2] *= xs * s0.z; f[3] *= xs * s0.w;
                            f[4] *= xs * s1.x; f[5] *= xs * s1.y; f[6] *= xs * s1.z; f[7] *= xs * s1.w;
                        }
                    }
                    if constexpr (P == P_DX) {
                        if (a.silu_pre && mine && nc < a.n) {
                            const uint4 pv = *reinterpret_cast<const uint4 *>(
                                a.silu_pre + (int64_t)(r.m0 + rr) * a.n + nc);
                            const uint32_t u4[4] = {pv.x, pv.y, pv.z, pv.w};
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                const float p0 = __uint_as_float(u4[y] << 16);
                                const float p1 = __uint_as_float(u4[y] & 0xFFFF0000u);
                                const float s0 = __fdividef(1.f, 1.f + __expf(-p0));
                                const float s1 = __fdividef(1.f, 1.f + __expf(-p1));
                                f[2 * y] *= s0 * (1.f + p0 * (1.f - s0));
                                f[2 * y + 1] *= s1 * (1.f + p1 * (1.f - s1));
                            }
                        }
                    }
                    if constexpr (P == P_FWD) {
                        if (a.pre)
                            po[hh] = make_float4(__uint_as_float(pack_bf16x2(f[0], f[1])),
                                                 __uint_as_float(pack_bf16x2(f[2], f[3])),
                                                 __uint_as_float(pack_bf16x2(f[4], f[5])),
                                                 __uint_as_float(pack_bf16x2(f[6], f[7])));
                    }
                    if constexpr (P == P_FWD || P == P_E4M3) {
                        if (a.silu) {
#pragma unroll
                            for (int x = 0; x < 8; ++x)
                                f[x] = f[x] * __fdividef(1.0f, 1.0f + __expf(-f[x]));
                        }
                    }
                    o[hh] = make_float4(__uint_as_float(pack_bf16x2(f[0], f[1])),
                                        __uint_as_float(pack_bf16x2(f[2], f[3])),
                                        __uint_as_float(pack_bf16x2(f[4], f[5])),
                                        __uint_as_float(pack_bf16x2(f[6], f[7])));
                }
                // lane l now stores chunk j = l % 8 of rows l - j .. l - j + 7 of this warp
                transpose_chunks<8>(o);
                const int row = q * 32 + lane - j, col = nb + 8 * j;
                const int64_t at = out0 + (int64_t)row * a.n + col;
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    if (row + c < r.rows && col < a.n)
                        *reinterpret_cast<float4 *>(a.out + at + (int64_t)c * a.n) = o[c];
                if constexpr (P == P_FWD) {
                    if (a.pre) {
                        transpose_chunks<8>(po);
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            if (row + c < r.rows && col < a.n)
                                *reinterpret_cast<float4 *>(a.pre + at + (int64_t)c * a.n) = po[c];
                    }
                }
            }
            if (!none) {
                __syncwarp();
                tc_fence_before();
                warp_arrive(&bars[EACC_EMPTY + acc]);
            }
        }
        if (!ok && lane == 0) egemm_flag(a, HSTU_DEV_WAIT_TIMEOUT);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, 2 * BN);
    }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
        return nullptr;
    }();
    return fn;
}

// A row-major [d2, d1, d0] tensor (d2 = 1: a matrix) of bf16 or 8-bit values as a TMA tensor
// whose box is 128 bytes of d0 by box1 rows, 128-byte swizzle.
bool encode(CUtensorMap *m, const void *base, bool bytes, int64_t d0, int64_t d1, int64_t d2,
            int box1)
{
    auto fn = encode_fn();
    if (!fn) return false;
    const int es = bytes ? 1 : 2;
    cuuint64_t dims[3] = {(cuuint64_t)d0, (cuuint64_t)d1, (cuuint64_t)d2};
    cuuint64_t strides[2] = {(cuuint64_t)(d0 * es), (cuuint64_t)(d0 * d1 * es)};
    cuuint32_t box[3] = {(cuuint32_t)(kSlice / es), (cuuint32_t)box1, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
              d2 > 0 ? 3 : 2, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

template <int P, int BN>
cudaError_t run_egemm(EGemmArgs &a, int64_t most_tiles, cudaStream_t st)
{
    using L = ELayout<BN>;
    const int smem = L::TAB_OFF + (3 * a.experts + 1) * 4 + 1024;
    static_assert(L::TAB_OFF + (3 * kMaxExperts + 1) * 4 + 1024 <= 232448, "shared memory");
    auto k = expert_gemm_kernel<P, BN>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    int64_t grid = num_sms();
    if (most_tiles < grid) grid = most_tiles;
    if (grid <= 0) return cudaSuccess;
    k<<<(unsigned)grid, kEThreads, smem, st>>>(a);
    return cudaGetLastError();
}

// The most row tiles that `rows` rows of `experts` experts can have.
int64_t most_row_tiles(int64_t rows, int experts)
{
    return rows / EBM + (rows < experts ? rows : experts);
}

// 256-wide tiles feed the tensor cores from shared memory at their full rate; 128-wide ones
// are taken where the wider ones would leave the last wave of the persistent grid emptier.
bool wide_tiles(int64_t row_tiles, int n)
{
    const int64_t sms = num_sms();
    const int64_t wide = row_tiles * ((n + 255) / 256), narrow = row_tiles * ((n + 127) / 128);
    const int64_t wide_time = 2 * ((wide + sms - 1) / sms), narrow_time = (narrow + sms - 1) / sms;
    return wide_time <= narrow_time;
}

template <int P>
cudaError_t run_by_width(EGemmArgs &a, const void *b, int64_t row_tiles, cudaStream_t st)
{
    const bool wide = wide_tiles(row_tiles, a.n);
    const int bn = wide ? 256 : 128;
    bool ok = true;
    if constexpr (P == P_FWD) ok = encode(&a.tb, b, false, a.n, a.kc, a.experts, 64);
    if constexpr (P == P_E4M3) ok = encode(&a.tb, b, true, a.kc, a.n, a.experts, bn);
    if constexpr (P == P_DX) ok = encode(&a.tb, b, false, a.kc, a.n, a.experts, bn);
    if (!ok) return cudaErrorInvalidValue;
    const int64_t tiles = row_tiles * ((a.n + bn - 1) / bn);
    return wide ? run_egemm<P, 256>(a, tiles, st) : run_egemm<P, 128>(a, tiles, st);
}

EGemmArgs common(const ProjArgs &p)
{
    EGemmArgs a;
    std::memset(&a, 0, sizeof(a));
    a.offsets = p.offsets;
    a.rows = p.rows;
    a.experts = p.experts;
    a.status = p.status;
    a.wait_limit = p.wait_limit;
    a.stall_test = p.stall_test;
    return a;
}

}  // namespace

cudaError_t launch_expert_proj(const ProjArgs &p, bool e4m3, cudaStream_t st)
{
    if (p.rows <= 0) return cudaSuccess;
    EGemmArgs a = common(p);
    if (!encode(&a.ta, p.x, e4m3, p.k, p.rows, 0, EBM) ||
        !encode(&a.ta_small, p.x, e4m3, p.k, p.rows, 0, kSmallBox))
        return cudaErrorInvalidValue;
    a.kc = p.k;
    a.n = p.n;
    a.silu = p.silu;
    a.x_scales = p.x_scales;
    a.w_scales = p.w_scales;
    a.out = reinterpret_cast<__nv_bfloat16 *>(p.out);
    a.pre = reinterpret_cast<__nv_bfloat16 *>(p.pre);
    const int64_t rt = most_row_tiles(p.rows, p.experts);
    return e4m3 ? run_by_width<P_E4M3>(a, p.w, rt, st) : run_by_width<P_FWD>(a, p.w, rt, st);
}

cudaError_t launch_expert_proj_dx(const ProjArgs &p, cudaStream_t st)
{
    if (p.rows <= 0) return cudaSuccess;
    EGemmArgs a = common(p);
    if (!encode(&a.ta, p.dout, false, p.n, p.rows, 0, EBM) ||
        !encode(&a.ta_small, p.dout, false, p.n, p.rows, 0, kSmallBox))
        return cudaErrorInvalidValue;
    a.kc = p.n;
    a.n = p.k;
    a.silu_pre = reinterpret_cast<const __nv_bfloat16 *>(p.silu_pre);
    a.out = reinterpret_cast<__nv_bfloat16 *>(p.dx);
    return run_by_width<P_DX>(a, p.w, most_row_tiles(p.rows, p.experts), st);
}

cudaError_t launch_expert_proj_dw(const ProjArgs &p, cudaStream_t st)
{
    if (p.rows <= 0)
        return cudaMemsetAsync(p.dw, 0, (size_t)p.experts * p.k * p.n * 2, st);
    EGemmArgs a = common(p);
    if (!encode(&a.ta, p.x, false, p.k, p.rows, 0, 64) ||
        !encode(&a.tb, p.dout, false, p.n, p.rows, 0, 64))
        return cudaErrorInvalidValue;
    a.m = p.k;
    a.n = p.n;
    a.out = reinterpret_cast<__nv_bfloat16 *>(p.dw);
    const int64_t rt = (int64_t)p.experts * ((p.k + EBM - 1) / EBM);
    const bool wide = wide_tiles(rt, p.n);
    const int64_t tiles = rt * ((p.n + (wide ? 255 : 127)) / (wide ? 256 : 128));
    return wide ? run_egemm<P_DW, 256>(a, tiles, st) : run_egemm<P_DW, 128>(a, tiles, st);
}

}  // namespace hstu
