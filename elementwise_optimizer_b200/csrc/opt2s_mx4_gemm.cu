// opt2s_mx4_gemm.cu -- products of microscaled 4-bit matrices on the tensor
// cores (tcgen05, kind::mxf4 with one E8M0 scale per 32 elements).
//
// D = P Q^T, both operands in blocks along the contraction axis.  A CTA owns
// a tile of 128 rows of P by BN rows of Q:
//   warp 0      moves tiles of codes (128-byte swizzled rows of 256 elements)
//               and of scales into a ring of shared-memory stages with TMA;
//   warps 4-7   copy a stage's scale words from shared memory into TMEM, in
//               the layout the block-scaled MMA reads (row r of 32 in lane r
//               of every quadrant, 4 blocks to a 32-bit column);
//   warp 1      issues the MMAs, 64 elements of the contraction each, into an
//               fp32 accumulator in TMEM;
//   warps 8-11  read finished accumulators and store them.
// Scales are stored by 128-column group, [group][row][4 bytes], so a tile's
// scales are contiguous whatever row it starts at: groups of rows that begin
// anywhere (experts) need no copy and no padding.
//
// Every wait is bounded: a wait that runs out raises the CTA's abort flag and
// the library's error flag (opt2s_mx4_errors), and the CTA drains its copies,
// frees its TMEM and returns.
#include <cuda.h>

#include "opt2s_mx4.cuh"

namespace opt2s {
namespace {

constexpr int kThreads = 384;
constexpr int kPRows = 128;
constexpr uint32_t kWaitLimit = 1u << 22;   // try_wait attempts, each suspending for up to microseconds

__device__ unsigned int g_mx4_errors;

// ---------------------------------------------------------------------------
// PTX
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t smem_u32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" :: "r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" :: "r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(bar) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(done) : "r"(bar), "r"(parity) : "memory");
    return done != 0;
}

// Bounded wait; false when it ran out or the CTA is aborting.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag)
{
    if (bar_try(bar, parity)) return true;
    for (uint32_t i = 0; i < kWaitLimit; ++i) {
        if (bar_try(bar, parity)) return true;
        if ((i & 255u) == 255u && *abort_flag) return false;
    }
    *abort_flag = 1;
    atomicAdd(&g_mx4_errors, 1u);
    return false;
}

// The same by a whole warp, which then goes on or stops as one.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag)
{
    return __all_sync(0xFFFFFFFFu, bar_wait(bar, parity, abort_flag));
}

__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3}], [%4];"
                 :: "r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}

__device__ __forceinline__ void mma_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" :: "r"(bar) : "memory");
}

__device__ __forceinline__ void mma_mx4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.b32 p, %6, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
                 :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate) : "memory");
}

__device__ __forceinline__ void tmem_st4(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};"
                 :: "r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// TMEM loads of consecutive columns of the thread's lane.  They wait inside
// the same statement, so that nothing can use the registers before they are
// filled.
__device__ __forceinline__ void tmem_ld(uint32_t at, float (&x)[4])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];\n\ttcgen05.wait::ld.sync.aligned;"
                 : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void tmem_ld(uint32_t at, float (&x)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7]),
                   "=f"(x[8]), "=f"(x[9]), "=f"(x[10]), "=f"(x[11]), "=f"(x[12]), "=f"(x[13]), "=f"(x[14]), "=f"(x[15])
                 : "r"(at) : "memory");
}
__device__ __forceinline__ void tmem_ld(uint32_t at, float (&x)[32])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7]),
                   "=f"(x[8]), "=f"(x[9]), "=f"(x[10]), "=f"(x[11]), "=f"(x[12]), "=f"(x[13]), "=f"(x[14]), "=f"(x[15]),
                   "=f"(x[16]), "=f"(x[17]), "=f"(x[18]), "=f"(x[19]), "=f"(x[20]), "=f"(x[21]), "=f"(x[22]), "=f"(x[23]),
                   "=f"(x[24]), "=f"(x[25]), "=f"(x[26]), "=f"(x[27]), "=f"(x[28]), "=f"(x[29]), "=f"(x[30]), "=f"(x[31])
                 : "r"(at) : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Shared-memory descriptor of a K-major tile with 128-byte swizzled rows:
// 8-row groups 1,024 bytes apart.
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr)
{
    return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | 1ull << 16 | static_cast<uint64_t>(1024 >> 4) << 32 |
           1ull << 46 | 2ull << 61;
}

// ---------------------------------------------------------------------------
// Geometry
// ---------------------------------------------------------------------------
constexpr int round_up(int x, int k) { return (x + k - 1) / k * k; }

template <int BN>
struct Geo {
    static constexpr int kStages = BN == 256 ? 4 : 5;
    // Two accumulators.  At BN = 256 they overlap by 96 of TMEM's columns
    // (the scales need the rest): the epilogue takes those columns into
    // registers first and hands them back at once, so the next tile's MMAs
    // wait for 96 columns to be read, not for the tile to be stored.
    static constexpr int kAccStep = BN == 256 ? 160 : BN;
    static constexpr int kOverlap = BN - kAccStep;
    static constexpr int kAccLag = kOverlap ? 1 : 2;            // a tile's MMAs wait for the epilogue of the tile this many before
    static constexpr int kSfP = 132;                            // words a scale box has per 128-column group
    static constexpr int kSfQ = BN == 256 ? 256 : BN + 4;
    static constexpr int kCodesP = kPRows * 128, kCodesQ = BN * 128;
    static constexpr int kScalesP = kSfP * 8, kScalesQ = kSfQ * 8;
    static constexpr int kTx = kCodesP + kCodesQ + kScalesP + kScalesQ;
    static constexpr int kStageCodes = kCodesP + round_up(kCodesQ, 1024);
    static constexpr int kStageScales = round_up(kScalesP, 128) + round_up(kScalesQ, 128);
    static constexpr int kScalesQAt = round_up(kScalesP, 128);  // where a stage's Q scales start
    static constexpr int kSmem = kStages * (kStageCodes + kStageScales) + 1024;
    static constexpr int kQCols = BN < 128 ? 4 : BN / 32;       // TMEM columns of one group's Q scales
    static constexpr int kSfCols = 8 + 2 * kQCols;
    static constexpr int kSfBase = kAccStep + BN;
    static constexpr int kUsedCols = kSfBase + kStages * kSfCols;
    static constexpr int kTmemCols = kUsedCols <= 128 ? 128 : (kUsedCols <= 256 ? 256 : 512);
    static_assert(kUsedCols <= 512, "TMEM columns");
};

struct Mx4GemmMaps {
    CUtensorMap p_codes, q_codes, p_scales, q_scales;
};

// Elements of the contraction per stage: 256, one 128-byte row of codes (two
// 128-column groups of scales, four 64-element MMAs).

// One output tile.
struct Tile {
    int p_row, q_row;      // first row in the operands' code maps
    int p_sf, q_sf;        // and in their scale maps
    int kg0;               // first 128-column group of the contraction
    int k64;               // 64-element steps of the contraction
    int64_t d_row;         // first row of D the tile's token (or output-row) side writes
    int d_rows;            // rows left from there (may exceed the tile)
    int d_col;             // first column of D
};

template <int BN, bool SWAP>
__device__ __forceinline__ Tile tile_at(const Mx4GemmArgs& a, const int32_t* start, const int32_t* first, int t)
{
    Tile o;
    if (a.ragged_k) {
        const int per = a.p_tiles * a.q_tiles, e = t / per, u = t - e * per;
        const int pi = u % a.p_tiles, qi = u / a.p_tiles;
        o.p_row = o.p_sf = pi * kPRows;
        o.q_row = o.q_sf = qi * BN;
        o.kg0 = first[e];
        o.k64 = (start[e + 1] - start[e] + 63) / 64;
        o.d_row = e * a.p_rows + pi * kPRows;
        o.d_rows = static_cast<int>(a.p_rows) - pi * kPRows;
        o.d_col = qi * BN;
        return o;
    }
    int e = 0, u = t, x0 = 0, x1 = static_cast<int>(a.x_rows);
    if (a.offsets) {
        e = group_of(first, a.groups, t);
        u = t - first[e];
        x0 = start[e];
        x1 = start[e + 1];
    }
    constexpr int kX = SWAP ? BN : kPRows, kW = SWAP ? kPRows : BN;
    // weight tiles inside bands of kBand token tiles, so that neighbouring CTAs share both operands in L2
    constexpr int kBand = 8;
    const int xt = (x1 - x0 + kX - 1) / kX, wt = a.w_tiles;
    const int band = u / (kBand * wt), in = u - band * kBand * wt;
    const int height = min(kBand, xt - band * kBand);
    const int xi = band * kBand + in % height, wi = in / height;
    const int xr = x0 + xi * kX, wr = wi * kW;
    const int w_row = e * static_cast<int>(a.w_rows) + wr, w_sf = e * static_cast<int>(a.w_sf_rows) + wr;
    o.p_row = SWAP ? w_row : xr;
    o.q_row = SWAP ? xr : w_row;
    o.p_sf = SWAP ? w_sf : xr;
    o.q_sf = SWAP ? xr : w_sf;
    o.kg0 = 0;
    o.k64 = a.k64;
    o.d_row = xr;
    o.d_rows = x1 - xr;
    o.d_col = wr;
    return o;
}

// ---------------------------------------------------------------------------
// Epilogue
// ---------------------------------------------------------------------------
template <int DT> __device__ __forceinline__ float load_out(const void* d, int64_t i)
{
    if (DT == kF32) return static_cast<const float*>(d)[i];
    if (DT == kF16) return __half2float(static_cast<const __half*>(d)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16*>(d)[i]);
}
template <int DT> __device__ __forceinline__ void store_out(void* d, int64_t i, float x)
{
    if (DT == kF32) static_cast<float*>(d)[i] = x;
    else if (DT == kF16) static_cast<__half*>(d)[i] = __float2half_rn(x);
    else static_cast<__nv_bfloat16*>(d)[i] = __float2bfloat16_rn(x);
}
template <int DT> __device__ __forceinline__ uint32_t pack_out(float lo, float hi)
{
    if (DT == kF16) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// A 32-byte store to a 32-byte aligned address.
__device__ __forceinline__ void store32(void* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t e, uint32_t f,
                                        uint32_t g, uint32_t h)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 :: "l"(p), "r"(a), "r"(b), "r"(c), "r"(d), "r"(e), "r"(f), "r"(g), "r"(h) : "memory");
}

// Accumulator columns c0 .. c0+N-1 of this thread's lane (row of P).
template <int N, int DT, bool SWAP>
__device__ __forceinline__ void store_cols(const Mx4GemmArgs& a, const Tile& t, int lane_row, int c0, const float (&x)[N])
{
    const int cols = static_cast<int>(a.d_cols);
    if (SWAP) {
        // the lane is a column of D, the accumulator's columns are its rows:
        // a warp stores 32 neighbouring elements of one row
        const int col = t.d_col + lane_row;
        if (col >= cols) return;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if (c0 + j >= t.d_rows) break;
            const int64_t i = (t.d_row + c0 + j) * a.ldd + col;
            store_out<DT>(a.d, i, a.accumulate ? __fadd_rn(load_out<DT>(a.d, i), x[j]) : x[j]);
        }
        return;
    }
    if (lane_row >= t.d_rows) return;
    const int col = t.d_col + c0;
    const int64_t i = (t.d_row + lane_row) * a.ldd + col;
    if (N >= 16 && a.vec && !a.accumulate && col + N <= cols) {
        // whole 32-byte sectors a lane
        if (DT == kF32) {
            uint32_t* d = static_cast<uint32_t*>(a.d) + i;
#pragma unroll
            for (int k = 0; k < N; k += 8)
                store32(d + k, __float_as_uint(x[k]), __float_as_uint(x[k + 1]), __float_as_uint(x[k + 2]),
                        __float_as_uint(x[k + 3]), __float_as_uint(x[k + 4]), __float_as_uint(x[k + 5]),
                        __float_as_uint(x[k + 6]), __float_as_uint(x[k + 7]));
        } else {
            uint16_t* d = static_cast<uint16_t*>(a.d) + i;
#pragma unroll
            for (int k = 0; k < N; k += 16)
                store32(d + k, pack_out<DT>(x[k], x[k + 1]), pack_out<DT>(x[k + 2], x[k + 3]),
                        pack_out<DT>(x[k + 4], x[k + 5]), pack_out<DT>(x[k + 6], x[k + 7]),
                        pack_out<DT>(x[k + 8], x[k + 9]), pack_out<DT>(x[k + 10], x[k + 11]),
                        pack_out<DT>(x[k + 12], x[k + 13]), pack_out<DT>(x[k + 14], x[k + 15]));
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < N; ++j)
        if (col + j < cols) store_out<DT>(a.d, i + j, a.accumulate ? __fadd_rn(load_out<DT>(a.d, i + j), x[j]) : x[j]);
}

template <int N, bool SWAP>
__device__ __forceinline__ void store_any(const Mx4GemmArgs& a, const Tile& t, int lane_row, int c0, const float (&x)[N])
{
    if (a.dtype == kF32) store_cols<N, kF32, SWAP>(a, t, lane_row, c0, x);
    else if (a.dtype == kF16) store_cols<N, kF16, SWAP>(a, t, lane_row, c0, x);
    else store_cols<N, kBF16, SWAP>(a, t, lane_row, c0, x);
}

// ---------------------------------------------------------------------------
// The kernel.  Cluster of a.split CTAs along the contraction (1: none, and
// each CTA walks tiles blockIdx.x, + gridDim.x, ...; else each cluster has
// one tile).
// ---------------------------------------------------------------------------
template <int BN, bool SWAP>
__global__ void __launch_bounds__(kThreads, 1)
mx4_gemm_kernel(const __grid_constant__ Mx4GemmMaps maps, const Mx4GemmArgs a)
{
    using G = Geo<BN>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int32_t start[kMaxGroups + 1], first[kMaxGroups + 1];
    __shared__ __align__(8) uint64_t bars[3 * G::kStages + 5];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t{1023});
    uint8_t* sf_smem = smem + G::kStages * G::kStageCodes;
    const uint32_t codes_at = smem_u32(smem), sf_at = smem_u32(sf_smem), bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (G::kStages + s); };
    auto sf_full = [&](int s) { return bar0 + 8u * (2 * G::kStages + s); };
    auto acc_full = [&](int b) { return bar0 + 8u * (3 * G::kStages + b); };
    auto acc_empty = [&](int b) { return bar0 + 8u * (3 * G::kStages + 2 + b); };
    const uint32_t drain = bar0 + 8u * (3 * G::kStages + 4);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int s = 0; s < G::kStages; ++s) {
            bar_init(full(s), 1);
            bar_init(empty(s), 1);
            bar_init(sf_full(s), 4);
        }
        for (int b = 0; b < 2; ++b) {
            bar_init(acc_full(b), 1);
            bar_init(acc_empty(b), 4);
        }
        bar_init(drain, 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(smem_u32(&tmem_slot)), "r"(G::kTmemCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (a.offsets) {
        if (a.ragged_k) ragged_table(a.offsets, a.groups, a.x_rows, 128, 1, start, first, tid, kThreads);
        else ragged_table(a.offsets, a.groups, a.x_rows, SWAP ? BN : kPRows, a.w_tiles, start, first, tid, kThreads);
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_slot;

    const int split = a.split;
    int rank = 0;
    if (split > 1) asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    const int tiles = (a.offsets && !a.ragged_k) ? first[a.groups] : a.tiles;
    const int t0 = blockIdx.x / split, dt = gridDim.x / split;

    // the 64-element steps [k_lo, k_hi) of a tile that this CTA sums: whole stages, evenly over the ranks
    auto k_range = [&](const Tile& t, int* lo, int* hi) {
        const int stages = (t.k64 + 3) / 4;
        *lo = min(t.k64, stages * rank / split * 4);
        *hi = min(t.k64, stages * (rank + 1) / split * 4);
    };

    if (warp == 0) {
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int t = t0; t < tiles && ok; t += dt) {
                const Tile o = tile_at<BN, SWAP>(a, start, first, t);
                int lo, hi;
                k_range(o, &lo, &hi);
                const int px = o.p_sf & ~3, qx = o.q_sf & ~3;
                for (int k = lo; k < hi; k += 4, ++it) {
                    const int s = it % G::kStages;
                    if (it >= G::kStages && !(ok = bar_wait(empty(s), (it / G::kStages - 1) & 1, &abort_flag))) break;
                    const uint32_t c = codes_at + s * G::kStageCodes, f = sf_at + s * G::kStageScales;
                    const int kg = o.kg0 + k / 2;
                    bar_expect(full(s), G::kTx);
                    tma_2d(c, &maps.p_codes, kg * 64, o.p_row, full(s));
                    tma_2d(c + G::kCodesP, &maps.q_codes, kg * 64, o.q_row, full(s));
                    tma_2d(f, &maps.p_scales, px, kg, full(s));
                    tma_2d(f + G::kScalesQAt, &maps.q_scales, qx, kg, full(s));
                }
            }
            if (abort_flag)      // let the copies in flight land before the CTA's memory goes away
                for (int s = 0; s < G::kStages; ++s) {
                    const uint32_t uses = it > static_cast<uint32_t>(s) ? (it - s - 1) / G::kStages + 1 : 0;
                    for (uint32_t i = 0; uses > 0 && i < kWaitLimit && !bar_try(full(s), (uses - 1) & 1); ++i) {}
                }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // kind::mxf4: E2M1 operands (1), E8M0 scales, M = 128, N = BN
            constexpr uint32_t kIdesc = 1u << 7 | 1u << 10 | static_cast<uint32_t>(BN >> 3) << 17 | 1u << 23 | 1u << 27;
            uint32_t it = 0, n = 0;
            bool ok = true;
            for (int t = t0; t < tiles && ok; t += dt) {
                const Tile o = tile_at<BN, SWAP>(a, start, first, t);
                int lo, hi;
                k_range(o, &lo, &hi);
                if (lo >= hi) continue;                  // nothing to sum: the epilogue takes zeros
                const int b = n & 1;
                if (n >= G::kAccLag) {
                    const uint32_t m = n - G::kAccLag;
                    if (!(ok = bar_wait(acc_empty(m & 1), (m >> 1) & 1, &abort_flag))) break;
                }
                fence_after();
                const uint32_t d = tmem + b * G::kAccStep;
                for (int k = lo; k < hi; k += 4, ++it) {
                    const int s = it % G::kStages;
                    const uint32_t ph = (it / G::kStages) & 1;
                    if (!(ok = bar_wait(full(s), ph, &abort_flag))) break;
                    if (!(ok = bar_wait(sf_full(s), ph, &abort_flag))) break;
                    fence_after();
                    const uint32_t c = codes_at + s * G::kStageCodes;
                    const uint64_t pd = tile_desc(c), qd = tile_desc(c + G::kCodesP);
                    const uint32_t sf = tmem + G::kSfBase + s * G::kSfCols;
                    const int steps = min(4, hi - k);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (j >= steps) break;
                        const uint32_t id = 2u * (j & 1);
                        mma_mx4(d, pd + 2 * j, qd + 2 * j, kIdesc | id << 4 | id << 29, sf + 4 * (j >> 1),
                                sf + 8 + G::kQCols * (j >> 1), k > lo || j > 0);
                    }
                    mma_commit(empty(s));
                }
                if (!ok) break;
                mma_commit(acc_full(b));
                ++n;
            }
            if (abort_flag) {
                mma_commit(drain);
                for (uint32_t i = 0; i < kWaitLimit && !bar_try(drain, 0); ++i) {}
            }
        }
    } else if (warp == 3) {
        if (a.fill_rest && a.offsets) {          // zeros for the rows in no group
            const int64_t before = start[0], behind = a.x_rows - start[a.groups];
            for (int64_t i = blockIdx.x; i < before + behind; i += gridDim.x) {
                const int64_t at = (i < before ? i : start[a.groups] + (i - before)) * a.ldd;
                for (int64_t c = lane; c < a.d_cols; c += 32) {
                    if (a.dtype == kF32) static_cast<float*>(a.d)[at + c] = 0.0f;
                    else static_cast<uint16_t*>(a.d)[at + c] = 0;
                }
            }
        }
    } else if (warp >= 4 && warp < 8) {
        const uint32_t quad = static_cast<uint32_t>(warp & 3) << 21;     // lane field: 32 * quadrant << 16
        uint32_t it = 0;
        bool ok = true;
        for (int t = t0; t < tiles && ok; t += dt) {
            const Tile o = tile_at<BN, SWAP>(a, start, first, t);
            int lo, hi;
            k_range(o, &lo, &hi);
            const int pr = o.p_sf & 3, qr = o.q_sf & 3;
            for (int k = lo; k < hi; k += 4, ++it) {
                const int s = it % G::kStages;
                if (!(ok = warp_wait(full(s), (it / G::kStages) & 1, &abort_flag))) break;
                const uint32_t* ps = reinterpret_cast<const uint32_t*>(sf_smem + s * G::kStageScales) + pr;
                const uint32_t* qs = reinterpret_cast<const uint32_t*>(sf_smem + s * G::kStageScales + G::kScalesQAt) + qr;
                const uint32_t at = tmem + quad + G::kSfBase + s * G::kSfCols;
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const uint32_t* p = ps + g * G::kSfP;
                    tmem_st4(at + 4 * g, p[lane], p[32 + lane], p[64 + lane], p[96 + lane]);
                    const uint32_t* q = qs + g * G::kSfQ;
#pragma unroll
                    for (int c = 0; c < G::kQCols; c += 4) {
                        uint32_t w[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int r = (c + j) * 32 + lane;
                            w[j] = r < BN ? q[r] : 0u;
                        }
                        tmem_st4(at + 8 + g * G::kQCols + c, w[0], w[1], w[2], w[3]);
                    }
                }
                tmem_st_wait();
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(sf_full(s));
            }
        }
    } else if (warp >= 8) {
        const int lane_row = (warp & 3) * 32 + lane;
        const uint32_t quad = static_cast<uint32_t>(warp & 3) << 21;
        uint32_t n = 0;
        for (int t = t0; t < tiles; t += dt) {
            const Tile o = tile_at<BN, SWAP>(a, start, first, t);
            int lo, hi;
            k_range(o, &lo, &hi);
            if (lo < hi) {
                const int b = n & 1;
                if (!warp_wait(acc_full(b), (n >> 1) & 1, &abort_flag)) break;
                fence_after();
                if (split == 1) {
                    const uint32_t acc = tmem + quad + b * G::kAccStep;
                    constexpr int kChunk = BN < 32 ? 16 : 32, kFirst = G::kOverlap / 32;
                    // the shared columns first: the last ones of accumulator 0, the first ones of 1
                    const int c0 = b == 0 ? BN - G::kOverlap : 0;
                    if constexpr (kFirst > 0) {
                        float x[kFirst][32];
#pragma unroll
                        for (int i = 0; i < kFirst; ++i) tmem_ld(acc + c0 + 32 * i, x[i]);
                        fence_before();
                        __syncwarp();
                        if (lane == 0) bar_arrive(acc_empty(b));
#pragma unroll
                        for (int i = 0; i < kFirst; ++i) store_any<32, SWAP>(a, o, lane_row, c0 + 32 * i, x[i]);
                    }
#pragma unroll 1
                    for (int i = kFirst; i < BN / kChunk; ++i) {
                        const int c = (c0 + kChunk * i) % BN;
                        float x[kChunk];
                        tmem_ld(acc + c, x);
                        store_any<kChunk, SWAP>(a, o, lane_row, c, x);
                    }
                    if constexpr (kFirst == 0) {
                        fence_before();
                        __syncwarp();
                        if (lane == 0) bar_arrive(acc_empty(b));
                    }
                }
                ++n;
            } else if (split == 1 && !a.accumulate) {
                const float zero[16] = {};
#pragma unroll 1
                for (int c = 0; c < BN; c += 16) store_any<16, SWAP>(a, o, lane_row, c, zero);
            }
        }
    }

    if (split > 1) {
        // Partial sums meet by reduce-scatter in distributed shared memory:
        // the tile's token columns go round the ranks four at a time, each
        // rank gets the others' partial sums of its columns, adds them in rank
        // order and stores them.  Columns without a token are not exchanged.
        // All MMAs of the cluster are done here (every CTA's epilogue warps
        // have waited for them), so the stages' memory is free.
        __syncthreads();
        cluster_sync();
        const bool mine = t0 < tiles && !abort_flag;
        Tile o{};
        int lo = 0, hi = 0, quads = 0;
        if (mine) {
            o = tile_at<BN, SWAP>(a, start, first, t0);
            k_range(o, &lo, &hi);
            quads = (min(BN, o.d_rows) + 3) / 4;
        }
        const int lane_row = (warp & 3) * 32 + lane;
        const uint32_t acc = tmem + (static_cast<uint32_t>(warp & 3) << 21);
        constexpr int kQuadBytes = kPRows * 16;
        const int slots = (BN / 4 + split - 1) / split;
        fence_after();
        if (warp >= 8) {
            for (int g = 0; g < quads; ++g) {
                const int owner = g % split;
                if (owner == rank) continue;
                float r[4] = {};
                if (lo < hi) tmem_ld(acc + 4 * g, r);
                const uint32_t local = codes_at + (rank * slots + g / split) * kQuadBytes + lane_row * 16;
                uint32_t remote;
                asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(owner));
                asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};"
                             :: "r"(remote), "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]) : "memory");
            }
        }
        cluster_sync();
        if (warp >= 8 && (o.k64 > 0 || !a.accumulate)) {
            for (int g = rank; g < quads; g += split) {
                float r[4] = {}, x[4] = {};
                if (lo < hi) tmem_ld(acc + 4 * g, r);
                for (int q = 0; q < split; ++q) {
                    float4 v;
                    if (q == rank)
                        v = make_float4(r[0], r[1], r[2], r[3]);
                    else
                        v = *reinterpret_cast<const float4*>(smem + (q * slots + g / split) * kQuadBytes + lane_row * 16);
                    x[0] = __fadd_rn(x[0], v.x);
                    x[1] = __fadd_rn(x[1], v.y);
                    x[2] = __fadd_rn(x[2], v.z);
                    x[3] = __fadd_rn(x[3], v.w);
                }
                store_any<4, SWAP>(a, o, lane_row, 4 * g, x);
            }
        }
    }
    fence_before();
    __syncthreads();
    if (warp == 2)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(G::kTmemCols));
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

cudaError_t encoder(EncodeTiled* out)
{
    static EncodeTiled found = nullptr;         // the driver's entry point: the same for every device and thread
    if (!found) {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
        if (e != cudaSuccess) return e;
        if (!fn || q != cudaDriverEntryPointSuccess) return cudaErrorNotSupported;
        found = reinterpret_cast<EncodeTiled>(fn);
    }
    *out = found;
    return cudaSuccess;
}

// A map of `rows` code rows of `pitch` bytes, boxes of 128 bytes x box_rows.
cudaError_t codes_map(EncodeTiled enc, CUtensorMap* m, const uint8_t* base, int64_t rows, int64_t pitch, int box_rows)
{
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(pitch), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch)};
    const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(box_rows)}, ones[2] = {1, 1};
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(base), dims, strides, box, ones,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// A map of the scale words: `words` rows by `groups` 128-column groups.
cudaError_t scales_map(EncodeTiled enc, CUtensorMap* m, const uint8_t* base, int64_t words, int64_t groups, int box_words)
{
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(words), static_cast<cuuint64_t>(groups)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(words) * 4};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_words), 2}, ones[2] = {1, 1};
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<uint8_t*>(base), dims, strides, box, ones,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int BN, bool SWAP>
cudaError_t launch_as(Mx4GemmArgs a, const Mx4GemmOperands& op, int sms, cudaStream_t stream)
{
    using G = Geo<BN>;
    EncodeTiled enc = nullptr;
    cudaError_t e = encoder(&enc);
    if (e != cudaSuccess) return e;
    const Mx4Operand& p = SWAP ? op.w : op.x;
    const Mx4Operand& q = SWAP ? op.x : op.w;
    Mx4GemmMaps maps;
    if ((e = codes_map(enc, &maps.p_codes, p.codes, p.code_rows, p.pitch, kPRows)) != cudaSuccess) return e;
    if ((e = codes_map(enc, &maps.q_codes, q.codes, q.code_rows, q.pitch, BN)) != cudaSuccess) return e;
    if ((e = scales_map(enc, &maps.p_scales, p.scales, p.scale_rows, p.pitch / 64, G::kSfP)) != cudaSuccess) return e;
    if ((e = scales_map(enc, &maps.q_scales, q.scales, q.scale_rows, q.pitch / 64, G::kSfQ)) != cudaSuccess) return e;
    constexpr int kX = SWAP ? BN : kPRows, kW = SWAP ? kPRows : BN;
    a.w_tiles = static_cast<int>((a.w_rows + kW - 1) / kW);
    a.p_tiles = static_cast<int>((a.p_rows + kPRows - 1) / kPRows);
    a.q_tiles = a.w_tiles;
    int64_t tiles;                      // exact, or (groups of rows) at most
    if (a.ragged_k) tiles = static_cast<int64_t>(a.groups) * a.p_tiles * a.q_tiles;
    else tiles = ((a.x_rows + kX - 1) / kX + (a.offsets ? a.groups : 0)) * a.w_tiles;
    if (tiles > INT32_MAX / 8) return cudaErrorInvalidConfiguration;
    a.tiles = static_cast<int>(tiles);
    if (tiles == 0) return cudaSuccess;
    const int64_t ctas = a.split > 1 ? tiles * a.split : std::min<int64_t>(tiles, sms * (512 / G::kTmemCols > 1 && G::kSmem < 110000 ? 2 : 1));
    auto* k = mx4_gemm_kernel<BN, SWAP>;
    if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, G::kSmem)) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = G::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(a.split);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k, maps, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_mx4_gemm(Mx4GemmArgs a, const Mx4GemmOperands& op, cudaStream_t stream)
{
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    a.split = 1;
    if (a.ragged_k) return launch_as<128, false>(a, op, sms, stream);
    // Few token rows a group: the weights take the 128-row side of the tile,
    // the tokens its narrow side, and the contraction is cut over a cluster
    // so that the weights' tiles reach every SM.
    const int64_t mean = a.offsets ? (a.x_rows + a.groups - 1) / a.groups : a.x_rows;
    if (mean <= 64) {
        const int bn = mean <= 16 ? 16 : (mean <= 32 ? 32 : 64);
        const int64_t wt = (a.w_rows + kPRows - 1) / kPRows;
        const int64_t xt = (a.x_rows + bn - 1) / bn + (a.offsets ? std::min<int64_t>(a.groups, a.x_rows) : 0);
        const int stages = (a.k64 + 3) / 4, most = bn == 16 ? 8 : 4;
        while (a.split < most && a.split * 2 <= stages && wt * xt * a.split * 2 <= sms) a.split *= 2;
        if (bn == 16) return launch_as<16, true>(a, op, sms, stream);
        if (bn == 32) return launch_as<32, true>(a, op, sms, stream);
        return launch_as<64, true>(a, op, sms, stream);
    }
    if (a.w_rows > 128) return launch_as<256, false>(a, op, sms, stream);
    return launch_as<128, false>(a, op, sms, stream);
}

cudaError_t mx4_error_count(unsigned int* out) { return cudaMemcpyFromSymbol(out, g_mx4_errors, sizeof(*out)); }

}  // namespace opt2s
