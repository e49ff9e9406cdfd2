// expert_gemm.cu -- the experts' products on rows sorted by expert (a jagged tensor whose
// sequences are the experts; offsets in device memory), on the tcgen05 tensor cores:
//
//   P_FWD   out_s = x_s W_e            bf16, W [E, K, N]; optional SiLU in the epilogue
//   P_E4M3  out_s = xs_s ws_e (x_s W_e)  e4m3 values, W [E, N, K], fp32 scales per row and column
//   P_DX    dx_s = (dout_s W_e^T) (.) SiLU'(pre_s)
//   P_DW    dW_e = X_e^T dOut_e        contraction over the expert's rows
//
// Persistent: a CTA takes 128 x 128 output tiles (CG = 1), or a pair of CTAs 256 x 256 ones with
// cta_group::2 (CG = 2); a tile lies in one expert.  The host never reads the offsets: every CTA
// sums up the experts' row tiles in shared memory at its start and finds a tile's expert by
// bisection.  Warp 0 streams 128-byte-wide slices of both operands through a TMA ring (128-byte
// swizzle), warp 1 issues tcgen05.mma into one of two TMEM accumulators, two groups of eight warps
// read them back and store them in turn.  Rows of a tile past the expert's end hold another expert's
// rows (or nothing): they are computed, not stored.  In P_DW they would enter the sums, so the MMA
// warp zeroes them in shared memory first.  Every wait is bounded.
//
// Products of few tiles share a tile's contraction among the CTAs of a cluster
// (expert_gemm_parts_kernel), weight gradients of few tiles cut the rows (expert_dw_plan).
//
// What bounds it: with 256 x 256 tiles each slice brings 32 KB per CTA from L2 for 512 cycles of
// MMAs, and that traffic (with the results going the other way) paces the loop: 740 to 800 cycles
// per slice.  8192^3 bf16 takes 0.71 ms in a burst (1.55 PFLOP/s, 0.96 of the measured peak) and
// 0.87 ms at the power limit; e4m3 0.37 ms (2.96 PFLOP/s).  Few rows per expert: the weights' bytes
// (256 rows of 64 experts, 1024 x 2048: 46 us, 5.7 TB/s).  Measured and dropped: 128 x 256 tiles of
// one CTA (0.94 PFLOP/s: shared memory's bandwidth), A kept in shared memory for all column tiles of
// a short contraction (too few stages left for B: 46 -> 64 us), the second CTA's warp reporting every
// slice to the leader (a cluster-scope release per slice: 0.57 PFLOP/s).
#include <cudaTypedefs.h>

#include <algorithm>
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
constexpr int kMaxStages = 6;
constexpr int kSmallBox = 16;        // rows of the small A box, for tiles with few rows
constexpr int kPartStages = 4;       // where the contraction is shared
constexpr int kEpiWarps = 16;
constexpr int kBand = 8;             // column tiles that the tiles in flight share
constexpr int kMaxSorted = 256;      // experts that P_DW puts in order of their rows
constexpr int kEThreads = 32 * (2 + kEpiWarps);
constexpr int kMaxSmem = 232448;     // of a block (227 KB)

struct EGemmArgs {
    CUtensorMap ta, ta_small, tb;
    const int64_t *offsets;
    int64_t rows;                    // rows of the sorted tensors
    int experts;
    int kc;                          // contraction length (P_DW: the expert's rows instead)
    int m, n;                        // P_DW: rows of an output tile's matrix; output columns
    int silu;
    int stages;                      // of the ring
    int slices;                      // P_DW: parts that an expert's rows are cut into
    float *partial;                  // P_DW with slices > 1: their sums [slices, experts, m, n]
    const float *x_scales, *w_scales;
    const __nv_bfloat16 *silu_pre;   // P_DX
    __nv_bfloat16 *out, *pre;
    int32_t *status;
    long long wait_limit;
    int stall_test;                  // test only: the MMA warp first waits for nothing
};

// Shared memory of a CTA.  CG CTAs work on one tile of CG * 128 rows x CG * 128 columns: each
// stages 128 rows of A and 128 columns of B, 16 KB each per slice of the contraction, in as many
// stages as there is room for (4 to 6, by the size of the experts' table).
constexpr int AB = EBM * kSlice, BB = EBN * kSlice;

template <int CG>
struct ELayout {
    static constexpr int kWarpStage = CG * 2048;      // of an epilogue warp: 32 rows x 32 CG columns
    static constexpr int kBarBytes = 512;
    // [A stages][B stages][epilogue][barriers][table]
    static __host__ __device__ int c_off(int stages) { return stages * (AB + BB); }
    static __host__ __device__ int bar_off(int stages) { return c_off(stages) + kEpiWarps * kWarpStage; }
    static __host__ int bytes(int stages, int experts)
    {
        return bar_off(stages) + kBarBytes + (3 * experts + 1) * 4 + 1024 /* alignment */;
    }
    static __host__ int stages(int experts)
    {
        int n = kMaxStages;
        while (bytes(n, experts) > kMaxSmem) --n;
        return n;
    }
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

// All threads of all CTAs of a cluster.
__device__ __forceinline__ void cluster_sync()
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
// cnt[e]) and its row tiles [tile0[e], tile0[e + 1]).  P_DW, whose tiles cost what their expert
// has rows: tile0 lists the experts, those with the most rows first.
struct ExpertTable {
    int32_t *tile0, *row0, *cnt;
};

// Fills the table (all threads of the block).  An expert whose offsets are invalid has no rows.
template <int P, int CG>
__device__ __forceinline__ void fill_table(const EGemmArgs &a, const ExpertTable &t, int32_t *wsum)
{
    constexpr int kRows = CG * EBM;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kWarps = kEThreads / 32;
    if constexpr (P == P_DW) {
        for (int e = tid; e < a.experts; e += kEThreads) {
            int64_t lo = a.offsets[e], hi = a.offsets[e + 1];
            if (lo < 0 || hi < lo || hi > a.rows) {
                if (blockIdx.x == 0) egemm_flag(a, HSTU_DEV_BAD_OFFSETS);
                lo = hi = 0;
            }
            t.row0[e] = (int)lo;
            t.cnt[e] = (int)(hi - lo);
        }
        __syncthreads();
        for (int e = tid; e < a.experts; e += kEThreads) {
            int rank = e;
            if (a.experts <= kMaxSorted) {
                const int mine = t.cnt[e];
                rank = 0;
                for (int o = 0; o < a.experts; ++o) rank += t.cnt[o] > mine || (t.cnt[o] == mine && o < e);
            }
            t.tile0[rank] = e;
        }
        return;
    }
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
    return BB + (small ? (rows + kSmallBox - 1) / kSmallBox * kSmallBox * kSlice
                                : (uint32_t)AB);
}

struct ETile {
    int e;            // expert
    int m0, rows;     // first row (of the sorted rows; P_DW: of the matrix) and rows to store
    int n0;           // first output column
    int kbeg, kcnt;   // contraction: first index and length
    int slice;        // P_DW: of the expert's rows
};

template <int P, int CG>
__device__ __forceinline__ int tile_count(const EGemmArgs &a, const ExpertTable &t)
{
    const int nt = (a.n + CG * EBN - 1) / (CG * EBN);
    return P == P_DW ? a.slices * a.experts * ((a.m + CG * EBM - 1) / (CG * EBM)) * nt
                     : t.tile0[a.experts] * nt;
}

// The tile that CTA (pair) `first` of `stride` takes in its turn w, or -1 after its last.
// P_DW deals back and forth, so that whoever takes the longest tile of one turn takes the
// shortest of the next.
template <int P>
__device__ __forceinline__ int deal(int w, int first, int stride, int ntiles)
{
    const int tile = w * stride + (P == P_DW && (w & 1) ? stride - 1 - first : first);
    return tile < ntiles ? tile : -1;
}

// An expert's tiles are numbered along bands of kBand column tiles, rows first: the tiles that
// run at the same time then cover about as many rows as columns of the product, and share their
// operands in L2 (8192 x 8192 x 8192 bf16 with whole rows of tiles: 765 us).
template <int P, int CG>
__device__ __forceinline__ ETile tile_of(const EGemmArgs &a, const ExpertTable &t, int tile)
{
    constexpr int kRows = CG * EBM;
    const int nt = (a.n + CG * EBN - 1) / (CG * EBN);
    ETile r;
    int mt, i;                               // the expert's row tiles, the tile's number in it
    r.slice = 0;
    if constexpr (P == P_DW) {
        if (a.slices > 1) {
            r.slice = tile % a.slices;
            tile /= a.slices;
        }
        mt = (a.m + kRows - 1) / kRows;
        const int q = tile / (mt * nt);
        r.e = t.tile0[q];
        i = tile - q * (mt * nt);
    } else {
        const int q = tile / nt;
        int lo = 0, hi = a.experts;          // the last expert whose first tile is <= q
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (t.tile0[mid] <= q) lo = mid; else hi = mid;
        }
        r.e = lo;
        mt = t.tile0[lo + 1] - t.tile0[lo];
        i = tile - t.tile0[lo] * nt;
    }
    const int band = i / (mt * kBand), j = i - band * (mt * kBand);
    const int cols = min(kBand, nt - band * kBand);
    const int row = j / cols;
    r.n0 = (band * kBand + j - row * cols) * (CG * EBN);
    if constexpr (P == P_DW) {
        r.m0 = row * kRows;
        r.rows = min(kRows, a.m - r.m0);
        r.kbeg = t.row0[r.e];
        r.kcnt = t.cnt[r.e];
        if (a.slices > 1) {                  // whole steps of 64 rows, as evenly as they go
            const int steps = (r.kcnt + 63) / 64;
            const int beg = (int)((int64_t)steps * r.slice / a.slices) * 64;
            const int end = min(r.kcnt, (int)((int64_t)steps * (r.slice + 1) / a.slices) * 64);
            r.kbeg += beg;
            r.kcnt = max(0, end - beg);
        }
    } else {
        r.m0 = t.row0[r.e] + row * kRows;
        r.rows = min(kRows, t.cnt[r.e] - row * kRows);
        r.kbeg = 0;
        r.kcnt = a.kc;
    }
    return r;
}

// a b, results below the normal numbers 0.
__device__ __forceinline__ float mul_ftz(float a, float b)
{
    float r;
    asm("mul.ftz.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// sigmoid(x) and sigmoid(y) on the hardware's exponential and reciprocal (2 ulp each), one
// reciprocal for both: 1 / a = b / (a b).  The special-function unit takes 8 cycles per warp and
// call, so 4 calls for two values of a 256-wide tile would outlast its MMAs below 512 of the
// contraction.  a and b = 1 + exp(-.) are kept times 2^-63, so that a b stays in fp32's range up to
// where exponents stop, at 2^126.5 (x = -87.7).  There 1 / a is 2^-126.5, which the last product
// flushes to 0: x sigmoid(x) is 0 for any x from there down, and the other value does not notice.
// With both far down (a b above 2^189) both are 0, an error of x sigmoid(x) below 1e-17.  (21846 rows
// of 8 experts, 512 x 2048: 48.0 us in a burst; 47.5 without the product by 2^-63 and wrong far down,
// 48.2 with the values clamped at -43.)
// rx, ry: 1 - sigmoid, as exp(-x) sigmoid(x), which goes to 0 with exp(-x) (and is 0 where sigmoid
// is: its users multiply by that).  1.f - sx would keep the reciprocal's rounding, which depends on
// the other value, and times x = 1e6 or more that rounding is what the slope of SiLU would be.
__device__ __forceinline__ void sigmoid2(float x, float y, float &sx, float &sy, float &rx, float &ry)
{
    constexpr float kDown = 0x1p-63f;
    float ex, ey, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(ex) : "f"(fminf(x * -1.4426950408889634f, 126.5f)));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(ey) : "f"(fminf(y * -1.4426950408889634f, 126.5f)));
    const float a = fmaf(ex, kDown, kDown), b = fmaf(ey, kDown, kDown);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a * b));
    r = mul_ftz(r, kDown);
    sx = mul_ftz(r, b);
    sy = mul_ftz(r, a);
    rx = ex * sx;
    ry = ey * sy;
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8])
{
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

// Piece c (16 bytes) of row `row` of a warp's 32 rows x NP pieces in shared memory, swizzled so
// that 8 rows' pieces c, and neighbouring pieces of a row, lie in different banks.
template <int NP>
__device__ __forceinline__ uint4 *staged(uint8_t *stage, int row, int c)
{
    return reinterpret_cast<uint4 *>(
        stage + row * (16 * NP) + ((c ^ (NP == 8 ? row & 7 : (row >> 1) & 3)) * 16));
}

// The staged rows to out[(out0 + row) * n + nb ...], NP lanes a row, rows and columns that exist.
template <int NP>
__device__ __forceinline__ void store_rows(uint8_t *stage, __nv_bfloat16 *out, int64_t out0, int rows,
                                           int nb, int n)
{
    const int lane = threadIdx.x & 31;
    const int r0 = lane / NP, col = nb + 8 * (lane % NP);
    __nv_bfloat16 *at = out + (out0 + r0) * n + col;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int row = i * (32 / NP) + r0;
        const uint4 x = *staged<NP>(stage, row, lane % NP);
        if (row < rows && col < n) *reinterpret_cast<uint4 *>(at) = x;
        at += (int64_t)(32 / NP) * n;
    }
}

// 8 accumulator columns to bf16: scales, SiLU or the SiLU's slope applied in fp32 before the
// one rounding.  xs, s0, s1: the row's scale and the columns' (P_E4M3); pv: this row's silu_pre
// (P_DX).  product: without the SiLU.
template <int P>
__device__ __forceinline__ uint4 convert8(const EGemmArgs &a, float xs, const float4 &s0, const float4 &s1,
                                          const uint4 &pv, bool product, float (&f)[8])
{
    if constexpr (P == P_E4M3) {
        f[0] *= xs * s0.x; f[1] *= xs * s0.y; f[2] *= xs * s0.z; f[3] *= xs * s0.w;
        f[4] *= xs * s1.x; f[5] *= xs * s1.y; f[6] *= xs * s1.z; f[7] *= xs * s1.w;
    }
    if constexpr (P == P_DX) {
        if (a.silu_pre) {
            const uint32_t u4[4] = {pv.x, pv.y, pv.z, pv.w};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const float p0 = __uint_as_float(u4[y] << 16);
                const float p1 = __uint_as_float(u4[y] & 0xFFFF0000u);
                float g0, g1, r0, r1;
                sigmoid2(p0, p1, g0, g1, r0, r1);
                f[2 * y] *= g0 * fmaf(p0, r0, 1.f);
                f[2 * y + 1] *= g1 * fmaf(p1, r1, 1.f);
            }
        }
    }
    if constexpr (P == P_FWD || P == P_E4M3) {
        if (a.silu && !product) {
#pragma unroll
            for (int x = 0; x < 8; x += 2) {
                float g0, g1, r0, r1;
                sigmoid2(f[x], f[x + 1], g0, g1, r0, r1);
                f[x] *= g0;
                f[x + 1] *= g1;
            }
        }
    }
    return pack8(f);
}

// The same for 32 columns of a lane's row.
template <int P>
__device__ __forceinline__ void convert32(const EGemmArgs &a, bool none, float xs, const float4 *ws,
                                          const uint32_t (&v)[32], const uint4 (&pv)[4], bool product,
                                          uint4 (&o)[4])
{
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        float f[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) f[x] = none ? 0.f : __uint_as_float(v[8 * h + x]);
        o[h] = convert8<P>(a, xs, ws[2 * h], ws[2 * h + 1], pv[h], product, f);
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
    using L = ELayout<CG>;
    const int ST = a.stages;
    constexpr int BN = CG * EBN;                        // columns of the pair's tile
    constexpr int KB = P == P_E4M3 ? 128 : 64;          // contraction per stage
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::bar_off(ST));
    uint32_t *slot = reinterpret_cast<uint32_t *>(bars + 40);
    int32_t *wsum = reinterpret_cast<int32_t *>(bars + 41);
    ExpertTable tab;
    tab.tile0 = reinterpret_cast<int32_t *>(sm + L::bar_off(ST) + L::kBarBytes);
    tab.row0 = tab.tile0 + a.experts + 1;
    tab.cnt = tab.row0 + a.experts;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = CG == 2 ? (int)(blockIdx.x & 1) : 0;
    const int first = blockIdx.x / CG, stride = gridDim.x / CG;
    if (threadIdx.x == 0) {
        prefetch_tmap(&a.ta);
        prefetch_tmap(&a.ta_small);
        prefetch_tmap(&a.tb);
        for (int x = 0; x < E_NBARS; ++x)
            mbar_init(&bars[x], x == EACC_EMPTY || x == EACC_EMPTY + 1 ? CG * kEpiWarps / 2 : 1);
        fence_mbar_init();
    }
    if (warp == 2) tmem_take<CG>(slot, 2 * BN);
    grid_dep_wait();
    grid_dep_release();
    fill_table<P, CG>(a, tab, wsum);
    tc_fence_before();
    __syncthreads();
    if constexpr (CG == 2) cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *slot;
    const uint32_t sm_base = smem_u32(sm);
    const int ntiles = tile_count<P, CG>(a, tab);

    if (warp == 0) {
        if (lane == 0) {
            // ---------------------------------------------------------------- TMA producer
            int s = 0, issued = 0;                       // stage, copies of stages so far
            uint32_t phase = 0;                          // of the stage's next use
            bool ok = true;
            for (int turn = 0; ok; ++turn) {
                const int tile = deal<P>(turn, first, stride, ntiles);
                if (tile < 0) break;
                const ETile r = tile_of<P, CG>(a, tab, tile);
                const int kch = (r.kcnt + KB - 1) / KB;
                const int m0 = r.m0 + rank * EBM, n0 = r.n0 + rank * EBN;
                const int rows = max(0, min(EBM, r.rows - rank * EBM));   // of this CTA
                const bool small = P != P_DW && rows <= 64;
                const int boxes = (rows + kSmallBox - 1) / kSmallBox;
                const uint32_t bytes = stage_bytes<P>(rows);
                const uint32_t both = CG == 1 ? bytes : bytes + stage_bytes<P>(
                    max(0, min(EBM, r.rows - EBM)));
                for (int kc = 0; kc < kch; ++kc) {
                    // (the phase before the first counts as over)
                    if (!mbar_wait(&bars[E_EMPTY + s], phase ^ 1, a.wait_limit)) {
                        ok = false;
                        break;
                    }
                    uint8_t *as = sm + s * AB, *bs = sm + ST * AB + s * BB;
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
                    ++issued;
                    if (++s == ST) {
                        s = 0;
                        phase ^= 1;
                    }
                }
            }
            if (!ok) egemm_flag(a, HSTU_DEV_WAIT_TIMEOUT);
            // Every copy issued has landed before the block may exit: seen on the barriers that
            // it arrived on, or, by the other CTA of a pair, from the MMAs that have read it.
            // (The other CTA sees no barrier of copies that no MMA has read; where it gave up it has
            // waited the limit since its last copy, and the leader, which it meets before it exits,
            // drains the barriers that both CTAs' copies arrive on.)
            bool drained = true;
            for (int x = min(issued, ST); x > 0 && (rank == 0 || (ok && drained)); --x) {
                if (--s < 0) {
                    s = ST - 1;
                    phase ^= 1;
                }
                drained &= mbar_wait(&bars[(rank == 0 ? E_FULL : E_EMPTY) + s], phase, kWaitLimitCycles);
            }
            if (!drained) egemm_flag(a, HSTU_DEV_WAIT_TIMEOUT);
        }
    } else if (warp == 1) {
        // -------------------------------------------------------------------- MMA issuer
        // the whole warp walks the tiles (it zeroes rows together); the leader's lane 0 issues,
        // the other CTA's warp only zeroes its rows
        constexpr uint32_t idesc = P == P_E4M3 ? idesc_e4m3(CG * EBM, BN)
                                               : idesc_bf16(CG * EBM, BN, P == P_DW, P != P_DX);
        int s = 0, t = 0;
        uint32_t phase = 0;
        int tails = 0;                                  // bit s: parity of TAIL and READY[s]
        bool ok = !a.stall_test || warp_wait(&bars[E_STALL], 0, a.wait_limit);
        for (int turn = 0; ok; ++turn) {
            const int tile = deal<P>(turn, first, stride, ntiles);
            if (tile < 0) break;
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
            for (int kc = 0; kc < kch; ++kc, phase ^= s + 1 == ST, s = s + 1 == ST ? 0 : s + 1) {
                const int valid = r.kcnt - kc * KB;     // P_DW: rows of this slice
                const bool tail = P == P_DW && valid < KB;
                if (rank != 0 && !tail) continue;
                if (!warp_wait(&bars[(rank == 0 ? E_FULL : E_TAIL) + s],
                               rank == 0 ? phase : (tails >> s) & 1, a.wait_limit)) {
                    ok = false;
                    break;
                }
                if (tail) {
                    // rows of this slice past the expert's end: zeros in both operands
                    const int per = (KB - valid) * 8;                // 16-byte pieces per block
                    for (int b = 0; b < (EBM + EBN) / 64; ++b) {
                        uint8_t *blk = b < EBM / 64 ? sm + s * AB + b * 8192
                                                    : sm + ST * AB + s * BB + (b - EBM / 64) * 8192;
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
                    const uint32_t aa = sm_base + s * AB;
                    const uint32_t bb = sm_base + ST * AB + s * BB;
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
        // A lane converts its row's values, 32 columns at a time, to bf16 and puts them, 16 bytes
        // at a time and swizzled, into the warp's shared memory, from where NP lanes store one
        // row's pieces side by side.  That is a chain of latencies (TMEM, shared memory,
        // stores), so two warps per lane quarter work side by side, each on half of the columns,
        // and two such groups of eight warps take the accumulators in turn: one computes SiLUs while
        // the other stores.  (All sixteen on one tile: 21846 rows of 8 experts, 512 x 2048 with SiLU
        // 56.3 -> 54.3 us, of 64 x 2048 35.9 -> 33.4; without SiLU 49.6 -> 49.4 and 22.1 -> 23.1.)
        const int q = warp & 3;                          // TMEM lane quarter: rows 32q ..
        const int group = (warp - 2) >> 3, half = (warp - 2) >> 2 & 1;
        const int rr = q * 32 + lane;                    // row of the tile == TMEM lane
        const uint32_t lane_base = (uint32_t)(q * 32) << 16;
        uint8_t *stage = sm + L::c_off(ST) + (warp - 2) * L::kWarpStage;
        int t = 0;
        bool ok = true;
        for (int turn = 0;; ++turn) {
            const int tile = deal<P>(turn, first, stride, ntiles);
            if (tile < 0) break;
            const ETile r = tile_of<P, CG>(a, tab, tile);
            const int m0 = r.m0 + rank * EBM;
            // rows and columns of the tile that this warp stores (none: <= 0)
            const int rows = min(EBM, r.rows - rank * EBM) - q * 32;
            const int cbeg = half * (BN / 2);
            const int cend = rows > 0 ? min((half + 1) * (BN / 2), a.n - r.n0) : cbeg;
            const bool none = P == P_DW && r.kcnt == 0;  // a gradient of zeros, without an MMA
            const int acc = t & 1;
            if (((none ? turn : t) & 1) != group) {      // the other group's
                if (!none) ++t;
                continue;
            }
            const int64_t out0 = (P == P_DW ? (int64_t)r.e * a.m + m0 : (int64_t)m0) + q * 32;
            // scales: this lane's row's, and per step this lane's column's, fetched while the
            // accumulator is not there yet (loading them column by column in the step, through
            // L1, took as long as the MMAs of 512 of the contraction)
            float xs = 1.f, ws[BN / 64];
            if constexpr (P == P_E4M3) {
                if (lane < rows) xs = __ldg(a.x_scales + m0 + rr);
#pragma unroll
                for (int i = 0; i < BN / 64; ++i) {
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
            constexpr int STEPS = BN / 128, NP = 4 * STEPS;   // pieces of 16 bytes of a lane's row
            if (P == P_DW && a.partial) {
                // a slice's sums stay in fp32: as below, 16 CG columns at a time
                float *to = a.partial + (((int64_t)r.slice * a.experts + r.e) * a.m + m0 + q * 32) * a.n;
                constexpr int FP = 4 * CG;               // pieces of 16 bytes of a lane's row
                for (int c0 = cbeg; c0 < cend; c0 += 32) {
                    uint32_t v[32];
                    __syncwarp();
                    if (!none) {
                        tmem_ld32(src + c0, v);
                        tmem_wait_ld();
                        reg_fence(v);
                    }
#pragma unroll
                    for (int h = 0; h < 32; h += 4 * FP) {
#pragma unroll
                        for (int u = 0; u < FP; ++u)
                            *staged<FP>(stage, lane, u) =
                                none ? make_uint4(0u, 0u, 0u, 0u)
                                     : make_uint4(v[h + 4 * u], v[h + 4 * u + 1], v[h + 4 * u + 2], v[h + 4 * u + 3]);
                        __syncwarp();
                        const int col = r.n0 + c0 + h + 4 * (lane % FP);
#pragma unroll
                        for (int u = 0; u < FP; ++u) {
                            const int row = u * (32 / FP) + lane / FP;
                            const uint4 x = *staged<FP>(stage, row, lane % FP);
                            if (row < rows && col < a.n)
                                *reinterpret_cast<uint4 *>(to + (int64_t)row * a.n + col) = x;
                        }
                        __syncwarp();
                    }
                }
            }
            bool given = false;
            auto give = [&] {
                __syncwarp();
                tc_fence_before();
                if constexpr (CG == 1) warp_arrive(&bars[EACC_EMPTY + acc]);
                else if (lane == 0) arrive_leader_relaxed(&bars[EACC_EMPTY + acc]);
                given = true;
            };
            // the product itself first, where it is wanted, then what becomes of it
            for (int pass = P == P_FWD && a.pre ? 0 : 1; pass < 2 && cbeg < cend && !(P == P_DW && a.partial);
                 ++pass) {
#pragma unroll
                for (int i = 0; i < 2 * STEPS; ++i) {
                    const int c0 = cbeg + 32 * i, nb = r.n0 + c0, at = 4 * (i % STEPS);
                    uint32_t v[32];
                    if (!none) {
                        __syncwarp();                    // the warp-wide TMEM load
                        tmem_ld32(src + c0, v);
                    }
                    // what a lane needs of other rows' or columns' lines passes through the place
                    // that its results take afterwards
                    uint4 pv[4];
                    if constexpr (P == P_E4M3) {
                        reinterpret_cast<float *>(staged<NP>(stage, lane / 4, at))[lane & 3] = ws[i];
                    }
                    if constexpr (P == P_DX) {
                        if (a.silu_pre) {                // 4 lanes a row in, each lane its own out
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                const int row = 8 * u + lane / 4, col = nb + 8 * (lane & 3);
                                pv[u] = make_uint4(0u, 0u, 0u, 0u);
                                if (row < rows && col < a.n)
                                    pv[u] = *reinterpret_cast<const uint4 *>(a.silu_pre + (out0 + row) * a.n + col);
                            }
#pragma unroll
                            for (int u = 0; u < 4; ++u)
                                *staged<NP>(stage, 8 * u + lane / 4, at + (lane & 3)) = pv[u];
                            __syncwarp();
#pragma unroll
                            for (int u = 0; u < 4; ++u) pv[u] = *staged<NP>(stage, lane, at + u);
                        }
                    }
                    if (!none) {
                        tmem_wait_ld();
                        reg_fence(v);
                        if (pass == 1 && i == 2 * STEPS - 1) give();   // the accumulator's last read
                    }
                    uint4 o[4];
                    float4 w4[8];
                    if constexpr (P == P_E4M3) {
                        __syncwarp();
#pragma unroll
                        for (int u = 0; u < 8; ++u)
                            w4[u] = *reinterpret_cast<const float4 *>(staged<NP>(stage, u, at));
                        __syncwarp();
                    }
                    convert32<P>(a, none, xs, w4, v, pv, pass == 0, o);
#pragma unroll
                    for (int u = 0; u < 4; ++u) *staged<NP>(stage, lane, at + u) = o[u];
                    if (i % STEPS == STEPS - 1) {
                        __syncwarp();
                        store_rows<NP>(stage, pass == 0 ? a.pre : a.out, out0, rows,
                                       nb - 32 * (STEPS - 1), a.n);
                        __syncwarp();
                    }
                }
            }
            if (!none && !given) give();
        }
        if (!ok && lane == 0) egemm_flag(a, HSTU_DEV_WAIT_TIMEOUT);
    }
    tc_fence_before();
    __syncthreads();
    // the leader's MMAs read both CTAs' shared memory and arrive on both CTAs' barriers
    if constexpr (CG == 2) cluster_sync();
    if (warp == 2) {
        tc_fence_after();
        tmem_give<CG>(tmem, 2 * BN);
    }
}

// Few tiles (few rows, or narrow matrices): the CTAs of a cluster share one 128 x 128 tile and cut
// its contraction into contiguous parts.  Each hands its fp32 sums to the shared memory of those that
// own their columns, and each adds up, converts and stores its columns, the parts in the order of
// their ranks.
enum SBar { S_FULL = 0, S_EMPTY = 8, S_ACC = 16, S_STALL = 17, S_NBARS = 18 };

// The sums that a CTA receives: [rank they come from][row][columns it owns].  PIECES of 16 bytes a
// row, swizzled so that neighbouring rows' pieces lie in different banks.
template <int PARTS>
struct Joined {
    static constexpr int kCols = EBN / PARTS, kPieces = kCols / 4;
    static constexpr int kBytes = PARTS * EBM * kCols * 4;
    static __device__ __forceinline__ uint32_t at(int rank, int row, int piece)
    {
        const int swizzled = piece ^ (kPieces == 4 ? row >> 1 & 3 : row & 7);
        return (uint32_t)(((rank * EBM + row) * kPieces + swizzled) * 16);
    }
};

// 16 bytes to the same place of CTA `rank`'s shared memory.
__device__ __forceinline__ void store_to(uint32_t at, int rank, const uint32_t *v)
{
    asm volatile(
        "{\n\t.reg .b32 a;\n\t"
        "mapa.shared::cluster.u32 a, %0, %1;\n\t"
        "st.shared::cluster.v4.b32 [a], {%2, %3, %4, %5};\n\t}" ::"r"(at),
        "r"(rank), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
        : "memory");
}

template <int P, int PARTS>
__global__ void __launch_bounds__(kEThreads, 1) expert_gemm_parts_kernel(const __grid_constant__ EGemmArgs a)
{
    using L = ELayout<1>;
    using J = Joined<PARTS>;
    constexpr int ST = kPartStages;
    constexpr int KB = P == P_E4M3 ? 128 : 64;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    // [A stages][B stages][sums of the parts][barriers][table]
    uint8_t *joined = sm + L::c_off(ST);
    uint64_t *bars = reinterpret_cast<uint64_t *>(joined + J::kBytes);
    uint32_t *slot = reinterpret_cast<uint32_t *>(bars + 40);
    int32_t *wsum = reinterpret_cast<int32_t *>(bars + 41);
    ExpertTable tab;
    tab.tile0 = reinterpret_cast<int32_t *>(reinterpret_cast<uint8_t *>(bars) + L::kBarBytes);
    tab.row0 = tab.tile0 + a.experts + 1;
    tab.cnt = tab.row0 + a.experts;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = blockIdx.x % PARTS;
    if (threadIdx.x == 0) {
        prefetch_tmap(&a.ta);
        prefetch_tmap(&a.ta_small);
        prefetch_tmap(&a.tb);
        for (int x = 0; x < S_NBARS; ++x) mbar_init(&bars[x], 1);
        fence_mbar_init();
    }
    if (warp == 2) tmem_take<1>(slot, EBN);
    grid_dep_wait();
    grid_dep_release();
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    fill_table<P, 1>(a, tab, wsum);
    tc_fence_before();
    __syncthreads();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");   // all CTAs have begun
    tc_fence_after();
    const uint32_t tmem = *slot;
    const int ntiles = tile_count<P, 1>(a, tab);
    const int kch = (a.kc + KB - 1) / KB;
    const int beg = kch * rank / PARTS, end = kch * (rank + 1) / PARTS;    // beg < end (the host)
    int issued = 0;                                     // slices so far (warps 0 and 1)
    // (a turn each, unless offsets that overlap make more tiles than the rows have)
    for (int turn = 0, tile = blockIdx.x / PARTS; tile < ntiles; ++turn, tile += gridDim.x / PARTS) {
        const ETile r = tile_of<P, 1>(a, tab, tile);
        if (warp == 0) {
            if (lane == 0) {
                const int rows = r.rows;
                const bool small = rows <= 64;
                bool ok = true;
                const int before = issued;
                for (int kc = beg; kc < end; ++kc) {
                    const int s = issued % ST;
                    if (!mbar_wait(&bars[S_EMPTY + s], (issued / ST + 1) & 1, a.wait_limit)) {
                        ok = false;
                        break;
                    }
                    uint8_t *as = sm + s * AB, *bs = sm + ST * AB + s * BB;
                    mbar_arrive_expect_tx(&bars[S_FULL + s], stage_bytes<P>(rows));
                    const uint32_t full = smem_u32(&bars[S_FULL + s]);
                    if (small) {
                        for (int b = 0; b * kSmallBox < rows; ++b)
                            load_2d<1>(as + b * kSmallBox * kSlice, &a.ta_small, full, kc * KB,
                                       r.m0 + b * kSmallBox);
                    } else {
                        load_2d<1>(as, &a.ta, full, kc * KB, r.m0);
                    }
                    if constexpr (P == P_FWD) {
                        for (int b = 0; b < EBN / 64; ++b)
                            load_3d<1>(bs + b * 8192, &a.tb, full, r.n0 + 64 * b, kc * KB, r.e);
                    } else {
                        load_3d<1>(bs, &a.tb, full, kc * KB, r.n0, r.e);
                    }
                    ++issued;
                }
                // every copy issued has landed before the memory is used again or the block exits
                for (int x = max(before, issued - ST); x < issued; ++x)
                    ok &= mbar_wait(&bars[S_FULL + x % ST], (x / ST) & 1, kWaitLimitCycles);
                if (!ok) egemm_flag(a, HSTU_DEV_WAIT_TIMEOUT);
            }
        } else if (warp == 1) {
            constexpr uint32_t idesc = P == P_E4M3 ? idesc_e4m3(EBM, EBN) : idesc_bf16(EBM, EBN, false, P != P_DX);
            bool ok = !a.stall_test || warp_wait(&bars[S_STALL], 0, a.wait_limit);
            for (int kc = beg; ok && kc < end; ++kc, ++issued) {
                const int s = issued % ST;
                if (!warp_wait(&bars[S_FULL + s], (issued / ST) & 1, a.wait_limit)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (lane == 0) {
                    const uint32_t aa = smem_u32(sm) + s * AB, bb = smem_u32(sm) + ST * AB + s * BB;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const uint64_t ad = sw128_desc(aa + kk * 32, 16, 1024);
                        const uint64_t bd = P == P_FWD ? sw128_desc(bb + kk * 2048, 8192, 1024)
                                                       : sw128_desc(bb + kk * 32, 16, 1024);
                        umma<1, P == P_E4M3>(tmem, ad, bd, idesc, (kc - beg) | kk ? 1u : 0u);
                    }
                    commit<1>(&bars[S_EMPTY + s]);
                }
                __syncwarp();
            }
            // (after a wait that ran out too: what was issued completes before the block goes on)
            if (lane == 0) {
                if (!ok) egemm_flag(a, HSTU_DEV_WAIT_TIMEOUT);
                commit_here<1>(&bars[S_ACC]);
            }
            __syncwarp();
        } else {
            const int q = warp & 3, c0 = (warp - 2) / 4 * 32;
            const bool ok = warp_wait(&bars[S_ACC], turn & 1, kWaitLimitCycles);
            if (!ok && lane == 0) egemm_flag(a, HSTU_DEV_WAIT_TIMEOUT);
            tc_fence_after();
            if (ok && q * 32 < r.rows) {
                uint32_t v[32];
                tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + c0, v);
                tmem_wait_ld();
                reg_fence(v);
                const int row = q * 32 + lane;
                if (row < r.rows) {
#pragma unroll
                    for (int x = 0; x < 32; x += 4)
                        store_to(smem_u32(joined) + J::at(rank, row, (c0 + x) % J::kCols / 4),
                                 (c0 + x) / J::kCols, v + x);
                }
            }
        }
        tc_fence_before();
        __syncthreads();
        cluster_sync();                                  // the sums have arrived
        constexpr int PIECES = J::kCols / 8;             // of 8 columns, of a row's owned ones
        for (int it = threadIdx.x; it < r.rows * PIECES; it += kEThreads) {
            const int row = it / PIECES, col = r.n0 + rank * J::kCols + it % PIECES * 8;
            if (col >= a.n) continue;
            const int64_t at = (int64_t)(r.m0 + row) * a.n + col;
            float xs = 1.f;
            float4 s0 = {}, s1 = {}, lo[PARTS], hi[PARTS];
            uint4 pv = {};
            if constexpr (P == P_E4M3) {
                xs = __ldg(a.x_scales + r.m0 + row);
                const float4 *ws = reinterpret_cast<const float4 *>(a.w_scales + (int64_t)r.e * a.n + col);
                s0 = __ldg(ws);
                s1 = __ldg(ws + 1);
            }
            if constexpr (P == P_DX)
                if (a.silu_pre) pv = *reinterpret_cast<const uint4 *>(a.silu_pre + at);
#pragma unroll
            for (int u = 0; u < PARTS; ++u) {
                lo[u] = *reinterpret_cast<const float4 *>(joined + J::at(u, row, it % PIECES * 2));
                hi[u] = *reinterpret_cast<const float4 *>(joined + J::at(u, row, it % PIECES * 2 + 1));
            }
            float f[8] = {};
#pragma unroll
            for (int u = 0; u < PARTS; ++u) {
                f[0] += lo[u].x; f[1] += lo[u].y; f[2] += lo[u].z; f[3] += lo[u].w;
                f[4] += hi[u].x; f[5] += hi[u].y; f[6] += hi[u].z; f[7] += hi[u].w;
            }
            if (P == P_FWD && a.pre)
                *reinterpret_cast<uint4 *>(a.pre + at) = convert8<P>(a, xs, s0, s1, pv, true, f);
            *reinterpret_cast<uint4 *>(a.out + at) = convert8<P>(a, xs, s0, s1, pv, false, f);
        }
        // before the next turn's sums arrive
        if (tile + (int)gridDim.x / PARTS < ntiles) {
            __syncthreads();
            cluster_sync();
        }
        tc_fence_after();
    }
    if (warp == 2) {
        tc_fence_after();
        tmem_give<1>(tmem, EBN);
    }
}

// out = the slices' sums added up in order, 4 elements per thread.
__global__ void __launch_bounds__(128) sum_slices_kernel(const float *__restrict__ partial, int slices,
                                                         int64_t n, __nv_bfloat16 *__restrict__ out)
{
    grid_dep_wait();
    grid_dep_release();
    const int64_t i = ((int64_t)blockIdx.x * 128 + threadIdx.x) * 4;
    if (i >= n) return;
    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 16
    for (int s = 0; s < slices; ++s) {
        const float4 a = *reinterpret_cast<const float4 *>(partial + s * n + i);
        f.x += a.x; f.y += a.y; f.z += a.z; f.w += a.w;
    }
    *reinterpret_cast<uint2 *>(out + i) = make_uint2(pack_bf16x2(f.x, f.y), pack_bf16x2(f.z, f.w));
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

// Clusters of SIZE CTAs of Kern that the device runs at a time, with the `smem` bytes that Kern asks
// for at most (cached per kernel and device).
template <auto Kern, int SIZE>
int most_clusters(int smem)
{
    constexpr int kMaxDev = 64;
    static std::atomic<int> cache[kMaxDev];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return num_sms() / SIZE;
    int v = cache[dev].load(std::memory_order_relaxed);
    if (v > 0) return v;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(num_sms() / SIZE * SIZE));
    cfg.blockDim = dim3(kEThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = SIZE;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&v, Kern, &cfg) != cudaSuccess || v <= 0) {
        cudaGetLastError();
        v = num_sms() / SIZE;
    }
    cache[dev].store(v, std::memory_order_relaxed);
    return v;
}

template <typename K>
cudaError_t launch_clusters(K k, const EGemmArgs &a, int size, int64_t clusters, int smem, cudaStream_t st)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(size * clusters));
    cfg.blockDim = dim3(kEThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = size;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = size > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k, a);
}

template <int P, int CG>
cudaError_t run_egemm(const EGemmArgs &args, int64_t most_tiles, cudaStream_t st)
{
    EGemmArgs a = args;
    a.stages = ELayout<CG>::stages(a.experts);
    const int smem = ELayout<CG>::bytes(a.stages, a.experts);
    constexpr auto k = expert_gemm_kernel<P, CG>;
    cudaError_t e = allow_smem<k>(smem);
    if (e != cudaSuccess) return e;
    int64_t tiles = CG == 2 ? most_clusters<k, 2>(kMaxSmem) : num_sms();
    if (most_tiles < tiles) tiles = most_tiles;
    if (tiles <= 0) return cudaSuccess;
    return launch_clusters(k, a, CG, tiles, smem, st);
}

// One cluster of PARTS CTAs for each tile, if all clusters run at a time, each CTA has two slices of
// the contraction at least, and the slices saved (0.3 us each) outweigh handing over the tile's rows
// (2 us for 128).  *done says whether.  Whole against shared, bf16 with SiLU: 8 rows of 8 experts,
// 1024 x 1024 10.5 and 7.7 us; 64 rows of one, 4096 x 1024 27.5 and 10.1; 2048 rows of 8, 2048 x 128
// 17.0 and 10.9; with too few slices saved, 2048 rows of 2, 512 x 512 8.1 and 8.5 (e4m3 7.4 and 8.3).
template <int P, int PARTS>
cudaError_t run_parts(const EGemmArgs &args, int64_t most_tiles, cudaStream_t st, bool *done)
{
    constexpr int KB = P == P_E4M3 ? 128 : 64;
    *done = false;
    const int slices = (args.kc + KB - 1) / KB;
    const int64_t tile_rows = std::min<int64_t>(EBM, args.rows / args.experts);
    if (slices < 2 * PARTS || (slices - slices / PARTS) * 16 <= tile_rows || most_tiles * PARTS > num_sms())
        return cudaSuccess;
    auto bytes = [](int experts) {
        return ELayout<1>::c_off(kPartStages) + Joined<PARTS>::kBytes + ELayout<1>::kBarBytes +
               (3 * experts + 1) * 4 + 1024 /* alignment */;
    };
    const int smem = bytes(args.experts);
    constexpr auto k = expert_gemm_parts_kernel<P, PARTS>;
    cudaError_t e = allow_smem<k>(smem);
    if (e != cudaSuccess || most_tiles > most_clusters<k, PARTS>(bytes(kMaxExperts))) return e;
    *done = true;
    return launch_clusters(k, args, PARTS, most_tiles, smem, st);
}

// The most row tiles that `rows` rows of `experts` experts can have.
int64_t most_row_tiles(int64_t rows, int experts, int tile)
{
    return rows / tile + (rows < experts ? rows : experts);
}

// Pairs of CTAs (256 x 256 tiles) read each operand half as often and reach the higher rate; single
// CTAs (128 x 128) waste less on experts of few rows, and fill the device with fewer tiles.  32
// experts, 1024 x 1024 bf16, single against pair: 64 rows each 18.7 against 22.8 us, 128 rows 24.6
// against 24.9, 192 rows 30.7 against 29.7, 768 rows 84 against 64.  The host knows the experts'
// average alone: where one of 64 experts takes nearly all of 10000 rows, 1024 x 1024, single CTAs
// run although pairs would be faster (52 against 47 us).
template <int P>
cudaError_t run_by_size(const EGemmArgs &a, int64_t rows, cudaStream_t st)
{
    auto tiles = [&](int cg) {
        return most_row_tiles(rows, a.experts, cg * EBM) * ((a.n + cg * EBN - 1) / (cg * EBN));
    };
    bool done = false;
    cudaError_t e = run_parts<P, 8>(a, tiles(1), st, &done);
    if (e == cudaSuccess && !done) e = run_parts<P, 4>(a, tiles(1), st, &done);
    if (e == cudaSuccess && !done) e = run_parts<P, 2>(a, tiles(1), st, &done);
    if (e != cudaSuccess || done) return e;
    const bool pair = rows >= (int64_t)a.experts * 160 && tiles(2) >= num_sms() / 2;
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

// Tiles of the weights' gradient for CTAs (cg = 1) or pairs (cg = 2).
static int64_t dw_tiles(int cg, int experts, int k, int n)
{
    return (int64_t)experts * ((k + cg * EBM - 1) / (cg * EBM)) * ((n + cg * EBN - 1) / (cg * EBN));
}

// Few tiles and many rows: the experts' rows are cut so that the device has work for its SMs, but
// to no less than 256 rows on average.  The slices' fp32 sums are at most 148 tiles of 64 KB, or 74 of
// 256 KB by pairs (one expert of 512 x 512: 18.9 MB).  16384 rows over experts of 512 x 512, whole
// against parts by single CTAs against parts by pairs: two experts 72, 26 and 23 us; four 51, 31 and
// 25; one of 32768 rows 189, 33 and 31.
DwPlan expert_dw_plan(int64_t rows, int experts, int k, int n)
{
    constexpr int64_t kSms = 148;            // (the workspace's size must not depend on the device)
    const int64_t t1 = dw_tiles(1, experts, k, n), t2 = dw_tiles(2, experts, k, n);
    const int64_t most = rows / experts / 256;
    DwPlan p;
    // pairs where they fill the device, or where parts of the rows do; matrices below 192 leave
    // most of a pair's tile empty
    p.pair = t2 >= kSms / 2 || (k >= 192 && n >= 192 && kSms / 2 / t2 >= 2 && most >= 2);
    int64_t s = p.pair ? kSms / 2 / t2 : kSms / t1;
    if (s > 32) s = 32;                      // (the sum of the parts is a chain)
    if (s > most) s = most;
    p.slices = (int)(s < 1 ? 1 : s);
    return p;
}

cudaError_t launch_expert_proj_dw(const ProjArgs &p, cudaStream_t st)
{
    const int64_t all = (int64_t)p.experts * p.k * p.n;
    if (p.rows <= 0) return cudaMemsetAsync(p.dw, 0, (size_t)all * 2, st);
    EGemmArgs a = common(p);
    if (!encode(&a.ta, p.x, false, p.k, p.rows, 0, 64) ||
        !encode(&a.tb, p.dout, false, p.n, p.rows, 0, 64))
        return cudaErrorInvalidValue;
    a.m = p.k;
    a.n = p.n;
    a.out = reinterpret_cast<__nv_bfloat16 *>(p.dw);
    const DwPlan plan = expert_dw_plan(p.rows, p.experts, p.k, p.n);
    a.slices = plan.slices;
    if (a.slices > 1) a.partial = p.partial;
    const int64_t tiles = a.slices * dw_tiles(plan.pair ? 2 : 1, p.experts, p.k, p.n);
    cudaError_t e = plan.pair ? run_egemm<P_DW, 2>(a, tiles, st) : run_egemm<P_DW, 1>(a, tiles, st);
    if (e != cudaSuccess || a.slices == 1) return e;
    return launch_pdl(sum_slices_kernel, dim3((unsigned)((all / 4 + 127) / 128)), dim3(128), 0, st,
                      (const float *)p.partial, a.slices, all, a.out);
}

}  // namespace hstu
