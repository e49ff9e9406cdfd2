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

#include <atomic>
#include <cstring>

#include "experts.h"
#include "kernels.h"
#include "sm100.cuh"
#include "units.cuh"

namespace hstu {

using namespace sm100;

namespace {

enum Product { P_FWD = 0, P_E4M3 = 1, P_DX = 2, P_DW = 3 };

constexpr int EBM = 128;             // rows of a CTA's output tile (TMEM lanes)
constexpr int EBN = 128;             // columns of the second operand that a CTA stages
constexpr int kSlice = 128;          // bytes of the contraction per stage and row
constexpr int kStages = 5;
constexpr int kSmallBox = 16;        // rows of the small A box, for tiles with few rows
constexpr int kEpiWarps = 16;
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

// Shared memory of a CTA.  CG CTAs work on one tile of CG * 128 rows x CG * 128 columns: each
// stages 128 rows of A and 128 columns of B, 32 KB per stage.
struct ELayout {
    static constexpr int AB = EBM * kSlice;           // 16 KB
    static constexpr int BB = EBN * kSlice;           // 16 KB
    static constexpr int A_OFF = 0;
    static constexpr int B_OFF = kStages * AB;
    static constexpr int C_OFF = B_OFF + kStages * BB;      // 2 KB per epilogue warp
    static constexpr int BAR_OFF = C_OFF + kEpiWarps * 2048;
    static constexpr int TAB_OFF = BAR_OFF + 512;     // tile prefix and row starts
};

// TMA loads into this CTA's shared memory.  CG = 2: `bar` is an address in the pair's shared
// memory, of this CTA's barrier or of the leader's.
template <int CG>
__device__ __forceinline__ void load_2d(void *dst, const CUtensorMap *map, uint32_t bar, int c0,
                                        int c1)
{
    if constexpr (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
            ".cta_group::2 [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
            : "memory");
}

template <int CG>
__device__ __forceinline__ void load_3d(void *dst, const CUtensorMap *map, uint32_t bar, int c0,
                                        int c1, int c2)
{
    if constexpr (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
            ".cta_group::2 [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
            : "memory");
}

// Address of the leader's (rank 0) copy of `bar` in the pair's shared memory.
__device__ __forceinline__ uint32_t leader_addr(uint64_t *bar)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(bar)));
    return r;
}

// D (TMEM) += A (smem) B (smem), fp32 accumulator: 16 bf16 or 32 e4m3 of the contraction per
// MMA.  CG = 2: both CTAs of the pair hold half of A's rows, B's columns and D's rows, at the
// same shared-memory and TMEM addresses; one thread of the pair issues.
#define HSTU_MMA(GROUP, KIND)                                              \
    asm volatile(                                                          \
        "{\n\t.reg .pred p;\n\t"                                           \
        "setp.ne.b32 p, %4, 0;\n\t"                                        \
        "tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem), \
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)              \
        : "memory")

template <int CG, bool E4M3>
__device__ __forceinline__ void umma(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                     uint32_t idesc, uint32_t accumulate)
{
    if constexpr (CG == 1 && !E4M3) HSTU_MMA("1", "f16");
    if constexpr (CG == 1 && E4M3) HSTU_MMA("1", "f8f6f4");
    if constexpr (CG == 2 && !E4M3) HSTU_MMA("2", "f16");
    if constexpr (CG == 2 && E4M3) HSTU_MMA("2", "f8f6f4");
}
#undef HSTU_MMA

// Arrives on `bar` (CG = 2: of both CTAs) when the MMAs issued so far by this thread complete.
template <int CG>
__device__ __forceinline__ void commit(uint64_t *bar)
{
    if constexpr (CG == 1) {
        umma_commit(bar);
    } else {
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster"
            ".b64 [%0], %1;" ::"r"(smem_u32(bar)),
            "h"((uint16_t)3)
            : "memory");
    }
}

// The same, on this CTA's barrier alone.
template <int CG>
__device__ __forceinline__ void commit_here(uint64_t *bar)
{
    if constexpr (CG == 1)
        umma_commit(bar);
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                smem_u32(bar))
            : "memory");
}

template <int CG>
__device__ __forceinline__ void tmem_take(uint32_t *slot, uint32_t ncols)
{
    if constexpr (CG == 1) {
        tmem_alloc(slot, ncols);
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(slot)),
                     "r"(ncols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}

template <int CG>
__device__ __forceinline__ void tmem_give(uint32_t taddr, uint32_t ncols)
{
    if constexpr (CG == 1)
        tmem_dealloc(taddr, ncols);
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr),
                     "r"(ncols)
                     : "memory");
}

// All threads of both CTAs of a pair.
__device__ __forceinline__ void pair_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// One arrival on the leader's copy of `bar`, after what this thread did before.
__device__ __forceinline__ void arrive_leader(uint64_t *bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                     leader_addr(bar))
                 : "memory");
}

// The same without ordering this thread's memory: for what it has read from TMEM into registers
// (a release would also wait for its stores to global memory, which cost more than the MMAs).
__device__ __forceinline__ void arrive_leader_relaxed(uint64_t *bar)
{
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                     leader_addr(bar))
                 : "memory");
}

// mbar_wait for barriers on which the pair's other CTA arrives.
__device__ __forceinline__ bool pair_wait(uint64_t *bar, uint32_t parity, long long limit)
{
    const long long t0 = clock64();
    while (true) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity), "r"(kSuspendHintNs)
            : "memory");
        if (ok) return true;
        if (clock64() - t0 > limit) return false;
    }
}

template <int CG>
__device__ __forceinline__ bool warp_wait_cg(uint64_t *bar, uint32_t parity, long long limit)
{
    if constexpr (CG == 1) return warp_wait(bar, parity, limit);
    return __all_sync(0xffffffffu, pair_wait(bar, parity, limit));
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
template <int CG>
__device__ __forceinline__ void fill_table(const EGemmArgs &a, const ExpertTable &t, int32_t *wsum)
{
    constexpr int kRows = CG * EBM;
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
            tiles = (int)((hi - lo + kRows - 1) / kRows);
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

// Bytes that a CTA with `rows` rows of A loads per stage.
template <int P>
__device__ __forceinline__ uint32_t stage_bytes(int rows)
{
    const bool small = P != P_DW && rows <= 64;
    return ELayout::BB + (small ? (rows + kSmallBox - 1) / kSmallBox * kSmallBox * kSlice
                                : (uint32_t)ELayout::AB);
}

struct ETile {
    int e;            // expert
    int m0, rows;     // first row (of the sorted rows; P_DW: of the matrix) and rows to store
    int n0;           // first output column
    int kbeg, kcnt;   // contraction: first index and length
};

template <int P, int CG>
__device__ __forceinline__ int tile_count(const EGemmArgs &a, const ExpertTable &t)
{
    const int nt = (a.n + CG * EBN - 1) / (CG * EBN);
    return P == P_DW ? a.experts * ((a.m + CG * EBM - 1) / (CG * EBM)) * nt
                     : t.tile0[a.experts] * nt;
}

template <int P, int CG>
__device__ __forceinline__ ETile tile_of(const EGemmArgs &a, const ExpertTable &t, int tile)
{
    constexpr int kRows = CG * EBM;
    const int nt = (a.n + CG * EBN - 1) / (CG * EBN);
    ETile r;
    r.n0 = (tile % nt) * (CG * EBN);
    const int q = tile / nt;
    if constexpr (P == P_DW) {
        const int mt = (a.m + kRows - 1) / kRows;
        r.e = q / mt;
        r.m0 = (q % mt) * kRows;
        r.rows = min(kRows, a.m - r.m0);
        r.kbeg = t.row0[r.e];
        r.kcnt = t.cnt[r.e];
    } else {
        int lo = 0, hi = a.experts;          // the last expert whose first tile is <= q
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (t.tile0[mid] <= q) lo = mid; else hi = mid;
        }
        r.e = lo;
        const int off = (q - t.tile0[lo]) * kRows;
        r.m0 = t.row0[lo] + off;
        r.rows = min(kRows, t.cnt[lo] - off);
        r.kbeg = 0;
        r.kcnt = a.kc;
    }
    return r;
}

// x * sigmoid(x) and its slope, on the hardware's exponential and reciprocal (2 ulp each).
__device__ __forceinline__ float sigmoid_fast(float x)
{
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8])
{
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

// 16-byte piece c of row `row` of a warp's 32 x 64 bytes, swizzled so that 8 rows' pieces c, and
// the pieces of 2 rows, lie in different banks.
__device__ __forceinline__ uint4 *staged(uint8_t *stage, int row, int c)
{
    return reinterpret_cast<uint4 *>(stage + row * 64 + ((c ^ ((row >> 1) & 3)) * 16));
}

// This lane's row (32 bf16) of the warp's 32 to shared memory, and from there 4 lanes a row to
// out[(out0 + row) * n + nb ...], rows and columns that exist.
__device__ __forceinline__ void store_rows(uint8_t *stage, const uint4 (&o)[4], __nv_bfloat16 *out,
                                           int64_t out0, int rows, int nb, int n)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 4; ++i) *staged(stage, lane, i) = o[i];
    __syncwarp();
    const int r0 = lane / 4, col = nb + 8 * (lane & 3);
    __nv_bfloat16 *at = out + (out0 + r0) * n + col;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint4 x = *staged(stage, 8 * i + r0, lane & 3);
        if (8 * i + r0 < rows && col < n) *reinterpret_cast<uint4 *>(at) = x;
        at += (int64_t)8 * n;
    }
    __syncwarp();
}

// 32 accumulator columns to bf16: scales, SiLU or the SiLU's slope applied in fp32 before the
// one rounding.  xs, ws: the row's scale and the columns' (P_E4M3); pv: this row's silu_pre
// (P_DX); po: the product itself (P_FWD with pre).
template <int P>
__device__ __forceinline__ void convert32(const EGemmArgs &a, bool none, float xs, const float4 *ws,
                                          const uint32_t (&v)[32], const uint4 (&pv)[4],
                                          uint4 (&o)[4], uint4 (&po)[4])
{
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        float f[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) f[x] = none ? 0.f : __uint_as_float(v[8 * h + x]);
        if constexpr (P == P_E4M3) {
            const float4 s0 = ws[2 * h], s1 = ws[2 * h + 1];
            f[0] *= xs * s0.x; f[1] *= xs * s0.y; f[2] *= xs * s0.z; f[3] *= xs * s0.w;
            f[4] *= xs * s1.x; f[5] *= xs * s1.y; f[6] *= xs * s1.z; f[7] *= xs * s1.w;
        }
        if constexpr (P == P_DX) {
            if (a.silu_pre) {
                const uint32_t u4[4] = {pv[h].x, pv[h].y, pv[h].z, pv[h].w};
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const float p0 = __uint_as_float(u4[y] << 16);
                    const float p1 = __uint_as_float(u4[y] & 0xFFFF0000u);
                    const float s0 = sigmoid_fast(p0), s1 = sigmoid_fast(p1);
                    f[2 * y] *= s0 * fmaf(p0, 1.f - s0, 1.f);
                    f[2 * y + 1] *= s1 * fmaf(p1, 1.f - s1, 1.f);
                }
            }
        }
        if constexpr (P == P_FWD) {
            if (a.pre) po[h] = pack8(f);
        }
        if constexpr (P == P_FWD || P == P_E4M3) {
            if (a.silu) {
#pragma unroll
                for (int x = 0; x < 8; ++x) f[x] *= sigmoid_fast(f[x]);
            }
        }
        o[h] = pack8(f);
    }
}

// FULL (the leader's): both CTAs' copies of a stage have landed.  EMPTY (each CTA's): the MMAs
// that read a stage are done.  P_DW with pairs, for a stage that needs zeroed rows: TAIL, the
// other CTA's copies have landed (on its own barrier), READY, it has zeroed its rows.
// (Both per stage: several tiles' last slices can be under way at once.)
enum EBar { E_FULL = 0, E_EMPTY = 8, E_TAIL = 16, E_READY = 24, EACC_FULL = 32, EACC_EMPTY = 34,
            E_DONE = 36, E_STALL = 37, E_NBARS = 38 };

template <int P, int CG>
__global__ void __launch_bounds__(kEThreads, 1) expert_gemm_kernel(const __grid_constant__ EGemmArgs a)
{
    using L = ELayout;
    constexpr int ST = kStages;
    constexpr int BN = CG * EBN;                        // columns of the pair's tile
    constexpr int KB = P == P_E4M3 ? 128 : 64;          // contraction per stage
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::BAR_OFF);
    uint32_t *slot = reinterpret_cast<uint32_t *>(sm + L::BAR_OFF + 8 * 40);
    int32_t *wsum = reinterpret_cast<int32_t *>(sm + L::BAR_OFF + 8 * 41);
    ExpertTable tab;
    tab.tile0 = reinterpret_cast<int32_t *>(sm + L::TAB_OFF);
    tab.row0 = tab.tile0 + a.experts + 1;
    tab.cnt = tab.row0 + a.experts;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = CG == 2 ? (int)(blockIdx.x & 1) : 0;
    const int first = blockIdx.x / CG, stride = gridDim.x / CG;
    if (threadIdx.x == 0) {
        for (int x = 0; x < E_NBARS; ++x)
            mbar_init(&bars[x], x == EACC_EMPTY || x == EACC_EMPTY + 1 ? CG * kEpiWarps : 1);
        fence_mbar_init();
    }
    if (warp == 2) tmem_take<CG>(slot, 2 * BN);
    fill_table<CG>(a, tab, wsum);
    tc_fence_before();
    __syncthreads();
    if constexpr (CG == 2) pair_sync();
    tc_fence_after();
    const uint32_t tmem = *slot;
    const uint32_t sm_base = smem_u32(sm);
    const int ntiles = tile_count<P, CG>(a, tab);

    if (warp == 0) {
        if (lane == 0) {
            // ---------------------------------------------------------------- TMA producer
            prefetch_tmap(&a.ta);
            prefetch_tmap(&a.tb);
            int g = 0;
            bool ok = true;
            for (int tile = first; ok && tile < ntiles; tile += stride) {
                const ETile r = tile_of<P, CG>(a, tab, tile);
                const int kch = (r.kcnt + KB - 1) / KB;
                const int m0 = r.m0 + rank * EBM, n0 = r.n0 + rank * EBN;
                const int rows = max(0, min(EBM, r.rows - rank * EBM));   // of this CTA
                const bool small = P != P_DW && rows <= 64;
                const int boxes = (rows + kSmallBox - 1) / kSmallBox;
                const uint32_t bytes = stage_bytes<P>(rows);
                const uint32_t both = CG == 1 ? bytes : bytes + stage_bytes<P>(
                    max(0, min(EBM, r.rows - EBM)));
                for (int kc = 0; kc < kch; ++kc, ++g) {
                    const int s = g % ST;
                    if (g >= ST && !mbar_wait(&bars[E_EMPTY + s], ((g / ST) - 1) & 1, a.wait_limit)) {
                        ok = false;
                        break;
                    }
                    uint8_t *as = sm + L::A_OFF + s * L::AB, *bs = sm + L::B_OFF + s * L::BB;
                    const bool tail = CG == 2 && P == P_DW && r.kcnt - kc * KB < KB;
                    if (rank == 0) mbar_arrive_expect_tx(&bars[E_FULL + s], tail ? bytes : both);
                    else if (tail) mbar_arrive_expect_tx(&bars[E_TAIL + s], bytes);
                    uint32_t full = smem_u32(&bars[E_FULL + s]);
                    if (rank != 0) full = tail ? smem_u32(&bars[E_TAIL + s]) : leader_addr(&bars[E_FULL + s]);
                    if constexpr (P == P_DW) {
                        // both operands lie along their rows: blocks of 64 columns x 64 rows
                        for (int b = 0; b < EBM / 64; ++b)
                            load_2d<CG>(as + b * 8192, &a.ta, full, m0 + 64 * b, r.kbeg + kc * KB);
                        for (int b = 0; b < EBN / 64; ++b)
                            load_2d<CG>(bs + b * 8192, &a.tb, full, n0 + 64 * b, r.kbeg + kc * KB);
                    } else {
                        if (small) {
                            for (int b = 0; b < boxes; ++b)
                                load_2d<CG>(as + b * kSmallBox * kSlice, &a.ta_small, full, kc * KB,
                                            m0 + b * kSmallBox);
                        } else {
                            load_2d<CG>(as, &a.ta, full, kc * KB, m0);
                        }
                        if constexpr (P == P_FWD) {
                            for (int b = 0; b < EBN / 64; ++b)
                                load_3d<CG>(bs + b * 8192, &a.tb, full, n0 + 64 * b, kc * KB, r.e);
                        } else {
                            load_3d<CG>(bs, &a.tb, full, kc * KB, n0, r.e);
                        }
                    }
                }
            }
            if (!ok) egemm_flag(a, HSTU_DEV_WAIT_TIMEOUT);
            // Every copy issued has landed before the block may exit: seen on the barriers that
            // it arrived on, or, by the other CTA of a pair, from the MMAs that have read it.
            // (A producer that gave up has waited the limit since its last copy.)
            bool drained = true;
            if (rank == 0) {
                for (int x = g - 1; x >= 0 && x >= g - ST; --x)
                    drained &= mbar_wait(&bars[E_FULL + x % ST], (x / ST) & 1, kWaitLimitCycles);
            } else {
                for (int x = g > ST ? g - ST : 0; ok && drained && x < g; ++x)
                    drained = mbar_wait(&bars[E_EMPTY + x % ST], (x / ST) & 1, kWaitLimitCycles);
            }
            if (!drained) egemm_flag(a, HSTU_DEV_WAIT_TIMEOUT);
        }
    } else if (warp == 1) {
        // -------------------------------------------------------------------- MMA issuer
        // the whole warp walks the tiles (it zeroes rows together); the leader's lane 0 issues,
        // the other CTA's warp only zeroes its rows
        constexpr uint32_t idesc = P == P_E4M3 ? idesc_e4m3(CG * EBM, BN)
                                               : idesc_bf16(CG * EBM, BN, P == P_DW, P != P_DX);
        int g = 0, t = 0;
        int tails = 0;                                  // bit s: parity of TAIL and READY[s]
        bool ok = !a.stall_test || warp_wait(&bars[E_STALL], 0, a.wait_limit);
        for (int tile = first; ok && tile < ntiles; tile += stride) {
            const ETile r = tile_of<P, CG>(a, tab, tile);
            const int kch = (r.kcnt + KB - 1) / KB;
            if (kch == 0) continue;                     // (P_DW: an expert without rows)
            const int acc = t & 1;
            if (rank == 0 && t >= 2 &&
                !warp_wait_cg<CG>(&bars[EACC_EMPTY + acc], ((t >> 1) - 1) & 1, a.wait_limit)) {
                ok = false;
                break;
            }
            ++t;
            tc_fence_after();
            const uint32_t d = tmem + acc * BN;
            for (int kc = 0; kc < kch; ++kc, ++g) {
                const int s = g % ST;
                const int valid = r.kcnt - kc * KB;     // P_DW: rows of this slice
                const bool tail = P == P_DW && valid < KB;
                if (rank != 0 && !tail) continue;
                if (!warp_wait(&bars[(rank == 0 ? E_FULL : E_TAIL) + s],
                               (rank == 0 ? g / ST : tails >> s) & 1, a.wait_limit)) {
                    ok = false;
                    break;
                }
                if (tail) {
                    // rows of this slice past the expert's end: zeros in both operands
                    const int per = (KB - valid) * 8;                // 16-byte pieces per block
                    for (int b = 0; b < (EBM + EBN) / 64; ++b) {
                        uint8_t *blk = b < EBM / 64 ? sm + L::A_OFF + s * L::AB + b * 8192
                                                    : sm + L::B_OFF + s * L::BB + (b - EBM / 64) * 8192;
                        uint4 *z = reinterpret_cast<uint4 *>(blk + valid * 128);
                        for (int x = lane; x < per; x += 32) z[x] = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if constexpr (CG == 2) {
                        if (rank != 0) {
                            if (lane == 0) arrive_leader(&bars[E_READY + s]);
                        } else if (!warp_wait_cg<2>(&bars[E_READY + s], (tails >> s) & 1, a.wait_limit)) {
                            ok = false;
                            break;
                        }
                    }
                    tails ^= 1 << s;
                    if (rank != 0) continue;
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
                        umma<CG, P == P_E4M3>(d, ad, bd, idesc, (kc | kk) ? 1u : 0u);
                    }
                    commit<CG>(&bars[E_EMPTY + s]);
                }
                __syncwarp();
            }
            if (!ok) break;
            if (rank == 0 && lane == 0) commit<CG>(&bars[EACC_FULL + acc]);
            __syncwarp();
        }
        if (lane == 0) {
            if (!ok) egemm_flag(a, HSTU_DEV_WAIT_TIMEOUT);
            if (rank == 0) {
                commit_here<CG>(&bars[E_DONE]);
                if (!mbar_wait(&bars[E_DONE], 0, kWaitLimitCycles))
                    egemm_flag(a, HSTU_DEV_WAIT_TIMEOUT);
            }
        }
        __syncwarp();
    } else {
        // -------------------------------------------------------------------- epilogue
        // 32 columns per step: a lane converts its row's values to bf16 and puts them, 16 bytes
        // at a time and swizzled, into the warp's 2 KB of shared memory, from where 4 lanes
        // store one row's 64 bytes side by side.  A step is a chain of latencies (TMEM, shared
        // memory, stores), so four warps per lane quarter work side by side.
        const int q = warp & 3;                          // TMEM lane quarter: rows 32q ..
        const int quarter = (warp - 2) >> 2;             // a quarter of the columns
        const int rr = q * 32 + lane;                    // row of the tile == TMEM lane
        const uint32_t lane_base = (uint32_t)(q * 32) << 16;
        uint8_t *stage = sm + L::C_OFF + (warp - 2) * 2048;
        int t = 0;
        bool ok = true;
        for (int tile = first; tile < ntiles; tile += stride) {
            const ETile r = tile_of<P, CG>(a, tab, tile);
            const int m0 = r.m0 + rank * EBM;
            // rows and columns of the tile that this warp stores (none: <= 0)
            const int rows = min(EBM, r.rows - rank * EBM) - q * 32;
            const int cbeg = quarter * (BN / 4);
            const int cend = rows > 0 ? min((quarter + 1) * (BN / 4), a.n - r.n0) : cbeg;
            const bool none = P == P_DW && r.kcnt == 0;  // a gradient of zeros, without an MMA
            const int acc = t & 1;
            const int64_t out0 = (P == P_DW ? (int64_t)r.e * a.m + m0 : (int64_t)m0) + q * 32;
            // scales: this lane's row's, and per step this lane's column's, fetched while the
            // accumulator is not there yet (loading them column by column in the step, through
            // L1, took as long as the MMAs of 512 of the contraction)
            float xs = 1.f, ws[BN / 128];
            if constexpr (P == P_E4M3) {
                if (lane < rows) xs = __ldg(a.x_scales + m0 + rr);
#pragma unroll
                for (int i = 0; i < BN / 128; ++i) {
                    const int col = r.n0 + cbeg + 32 * i + lane;
                    ws[i] = col < a.n ? __ldg(a.w_scales + (int64_t)r.e * a.n + col) : 0.f;
                }
            }
            if (!none) {
                if (!warp_wait(&bars[EACC_FULL + acc], (t >> 1) & 1, a.wait_limit)) {
                    ok = false;
                    break;
                }
                ++t;
                tc_fence_after();
            }
            const uint32_t src = tmem + lane_base + acc * BN;
#pragma unroll
            for (int i = 0; i < BN / 128; ++i) {
                const int c0 = cbeg + 32 * i, nb = r.n0 + c0;
                if (c0 >= cend) break;
                uint32_t v[32];
                if (!none) {
                    __syncwarp();                        // the warp-wide TMEM load
                    tmem_ld32(src + c0, v);
                }
                uint4 pv[4];
                if constexpr (P == P_E4M3) reinterpret_cast<float *>(stage)[lane] = ws[i];
                if constexpr (P == P_DX) {
                    if (a.silu_pre) {                    // 4 lanes a row in, each lane its own out
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const int row = 8 * u + lane / 4, col = nb + 8 * (lane & 3);
                            pv[u] = make_uint4(0u, 0u, 0u, 0u);
                            if (row < rows && col < a.n)
                                pv[u] = *reinterpret_cast<const uint4 *>(a.silu_pre + (out0 + row) * a.n + col);
                        }
#pragma unroll
                        for (int u = 0; u < 4; ++u) *staged(stage, 8 * u + lane / 4, lane & 3) = pv[u];
                        __syncwarp();
#pragma unroll
                        for (int u = 0; u < 4; ++u) pv[u] = *staged(stage, lane, u);
                        __syncwarp();
                    }
                }
                if (!none) {
                    tmem_wait_ld();
                    reg_fence(v);
                }
                uint4 o[4], po[4];
                __syncwarp();
                convert32<P>(a, none, xs, reinterpret_cast<const float4 *>(stage), v, pv, o, po);
                __syncwarp();
                store_rows(stage, o, a.out, out0, rows, nb, a.n);
                if constexpr (P == P_FWD) {
                    if (a.pre) store_rows(stage, po, a.pre, out0, rows, nb, a.n);
                }
            }
            if (!none) {
                __syncwarp();
                tc_fence_before();
                if constexpr (CG == 1) warp_arrive(&bars[EACC_EMPTY + acc]);
                else if (lane == 0) arrive_leader_relaxed(&bars[EACC_EMPTY + acc]);
            }
        }
        if (!ok && lane == 0) egemm_flag(a, HSTU_DEV_WAIT_TIMEOUT);
    }
    tc_fence_before();
    __syncthreads();
    // the leader's MMAs read both CTAs' shared memory and arrive on both CTAs' barriers
    if constexpr (CG == 2) pair_sync();
    if (warp == 2) {
        tc_fence_after();
        tmem_give<CG>(tmem, 2 * BN);
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

// CTA pairs that the device runs at a time (cached per device ordinal).
template <typename K>
int most_pairs(K kern, int smem)
{
    constexpr int kMaxDev = 64;
    static std::atomic<int> cache[kMaxDev];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return num_sms() / 2;
    int v = cache[dev].load(std::memory_order_relaxed);
    if (v > 0) return v;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(num_sms() / 2 * 2));
    cfg.blockDim = dim3(kEThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&v, kern, &cfg) != cudaSuccess || v <= 0) {
        cudaGetLastError();
        v = num_sms() / 2;
    }
    cache[dev].store(v, std::memory_order_relaxed);
    return v;
}

template <int P, int CG>
cudaError_t run_egemm(const EGemmArgs &a, int64_t most_tiles, cudaStream_t st)
{
    const int smem = ELayout::TAB_OFF + (3 * a.experts + 1) * 4 + 1024;
    static_assert(ELayout::TAB_OFF + (3 * kMaxExperts + 1) * 4 + 1024 <= 232448, "shared memory");
    auto k = expert_gemm_kernel<P, CG>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    int64_t tiles = CG == 2 ? most_pairs(k, smem) : num_sms();
    if (most_tiles < tiles) tiles = most_tiles;
    if (tiles <= 0) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(CG * tiles));
    cfg.blockDim = dim3(kEThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = CG;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = CG == 2 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k, a);
}

// The most row tiles that `rows` rows of `experts` experts can have.
int64_t most_row_tiles(int64_t rows, int experts, int tile)
{
    return rows / tile + (rows < experts ? rows : experts);
}

// Pairs of CTAs (256 x 256 tiles) read each operand half as often and reach the higher rate;
// single CTAs (128 x 128) waste less on short experts and fill the device with fewer tiles.
template <int P>
cudaError_t run_by_size(const EGemmArgs &a, int64_t rows, cudaStream_t st)
{
    auto tiles = [&](int cg) {
        const int64_t bm = cg * EBM, bn = cg * EBN, nt = (a.n + bn - 1) / bn;
        return (P == P_DW ? a.experts * ((a.m + bm - 1) / bm)
                          : most_row_tiles(rows, a.experts, (int)bm)) * nt;
    };
    const bool pair = P == P_DW ? tiles(2) >= num_sms() / 2
                                : rows >= (int64_t)a.experts * 192 && tiles(2) >= num_sms() / 2;
    return pair ? run_egemm<P, 2>(a, tiles(2), st) : run_egemm<P, 1>(a, tiles(1), st);
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
        !encode(&a.ta_small, p.x, e4m3, p.k, p.rows, 0, kSmallBox) ||
        !(e4m3 ? encode(&a.tb, p.w, true, p.k, p.n, p.experts, EBN)
               : encode(&a.tb, p.w, false, p.n, p.k, p.experts, 64)))
        return cudaErrorInvalidValue;
    a.kc = p.k;
    a.n = p.n;
    a.silu = p.silu;
    a.x_scales = p.x_scales;
    a.w_scales = p.w_scales;
    a.out = reinterpret_cast<__nv_bfloat16 *>(p.out);
    a.pre = reinterpret_cast<__nv_bfloat16 *>(p.pre);
    return e4m3 ? run_by_size<P_E4M3>(a, p.rows, st) : run_by_size<P_FWD>(a, p.rows, st);
}

cudaError_t launch_expert_proj_dx(const ProjArgs &p, cudaStream_t st)
{
    if (p.rows <= 0) return cudaSuccess;
    EGemmArgs a = common(p);
    if (!encode(&a.ta, p.dout, false, p.n, p.rows, 0, EBM) ||
        !encode(&a.ta_small, p.dout, false, p.n, p.rows, 0, kSmallBox) ||
        !encode(&a.tb, p.w, false, p.n, p.k, p.experts, EBN))
        return cudaErrorInvalidValue;
    a.kc = p.n;
    a.n = p.k;
    a.silu_pre = reinterpret_cast<const __nv_bfloat16 *>(p.silu_pre);
    a.out = reinterpret_cast<__nv_bfloat16 *>(p.dx);
    return run_by_size<P_DX>(a, p.rows, st);
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
    return run_by_size<P_DW>(a, p.rows, st);
}

}  // namespace hstu
