// opt2s_mx4_gemm.cu -- products of microscaled 4-bit matrices on the tensor
// cores (tcgen05, kind::mxf4 with one E8M0 scale per 32 elements).
//
// D = P Q^T, both operands in blocks along the contraction axis.  A CTA owns
// a tile of 128 rows of P by BN rows of Q:
//   warp 0      moves tiles of codes (128-byte swizzled rows of 256 elements)
//               and of scales into a ring of shared-memory stages with TMA;
//   warps 4-7   bring a stage's scale words, in shared memory, into the order
//               in which they are copied to TMEM, a warp every fourth stage;
//   warp 1      issues the copies of the scales to TMEM and the MMAs, 64
//               elements of the contraction each, into an fp32 accumulator in
//               TMEM;
//   warps 8-11  read finished accumulators and store them.
// Scales are stored by 128-column group, [group][row][4 bytes], so a tile's
// scales are contiguous whatever row it starts at: groups of rows that begin
// anywhere (experts) need no copy and no padding.
//
// What bounds it, at 8,192 x 8,192 x 2,048 (65 us: 4.2 PFLOP/s, 2.5 times the
// library's measured bf16 rate): a pair's stage takes 730 cycles where its
// MMAs take 512, the copies of its scales to TMEM about 40 each (six, in the
// same pipe), and between two tiles the pipe stands still for about 900 cycles
// (the accumulators' hand-over).  8,192^3 takes 190 us (5.8 PFLOP/s) from a
// cool chip and 236 us (4.7) for seconds on end, where the power limit lowers
// the clock.  The contraction's loads arrive about 1,000 cycles before they are
// needed.
//
// Every wait on a shared-memory barrier is bounded: one that runs out raises
// the CTA's abort flag and adds to the library's count (opt2s_mx4_errors), and
// the CTA drains its copies, frees its TMEM and returns.  The other waits have
// no limit and need none: every thread of a cluster reaches its barriers,
// since all loops before them end, and TMEM is free at once, since shared
// memory lets no more of these CTAs share an SM than two of 128 columns.
#include <type_traits>

#include <cuda.h>

#include "opt2s_mx4.cuh"
#include "opt2s_mx4_wait.cuh"

namespace opt2s {
namespace {

constexpr int kThreads = 384;
constexpr int kPRows = 128;
constexpr uint32_t kWaitLimit = 1u << 25;   // attempts; a wait that nothing ends gives up after about a second

__device__ unsigned int g_mx4_errors;

// ---------------------------------------------------------------------------
// PTX
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t smem_u32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" :: "r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(bar) : "memory");
}

__device__ __forceinline__ uint32_t in_rank(uint32_t addr, int rank)      // addr in another CTA of the cluster
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void bar_arrive_cluster(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" :: "r"(bar) : "memory");
}

__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag)
{
    return bar_wait(bar, parity, kWaitLimit, abort_flag, &g_mx4_errors);
}

// The same by a whole warp, which then goes on or stops as one.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag)
{
    return __all_sync(0xFFFFFFFFu, bar_wait(bar, parity, abort_flag));
}

// A tile into this CTA's shared memory; PAIR: `bar` may be the other CTA's.
template <bool PAIR = false>
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar)
{
    if (PAIR)
        asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                     " [%0], [%1, {%2, %3}], [%4];"
                     :: "r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
    else
        asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                     " [%0], [%1, {%2, %3}], [%4];"
                     :: "r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, int x, int y, uint32_t src)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];\n\t"
                 "cp.async.bulk.commit_group;" :: "l"(map), "r"(x), "r"(y), "r"(src) : "memory");
}

// Arrives at `bar` (PAIR: in both CTAs) when the MMAs issued so far are done.
template <bool PAIR>
__device__ __forceinline__ void mma_commit(uint32_t bar)
{
    if (PAIR)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                     :: "r"(bar), "h"(static_cast<uint16_t>(3)) : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" :: "r"(bar) : "memory");
}

template <bool PAIR>
__device__ __forceinline__ void mma_mx4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        uint32_t accumulate)
{
    if (PAIR)
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "setp.ne.b32 p, %6, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
                     :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate) : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "setp.ne.b32 p, %6, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
                     :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate) : "memory");
}

// 512 bytes of scales, [32][4] words, to four TMEM columns: word [r][j] to lane
// r (and 32 + r, 64 + r, 96 + r) of column j.  PAIR: in both CTAs.  In order
// with the MMAs that the thread issues after it.
template <bool PAIR>
__device__ __forceinline__ void copy_scales(uint32_t tmem_col, uint32_t addr)
{
    const uint64_t desc = static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | static_cast<uint64_t>(128 >> 4) << 32 | 1ull << 46;
    if (PAIR) asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" :: "r"(tmem_col), "l"(desc) : "memory");
    else asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" :: "r"(tmem_col), "l"(desc) : "memory");
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
// 64 columns at `at` and 32 at `more`, one wait.
__device__ __forceinline__ void tmem_ld(uint32_t at, uint32_t more, float (&x)[3][32])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
                 "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
                 "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
                 "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%96];\n\t"
                 "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
                 "%64, %65, %66, %67, %68, %69, %70, %71, %72, %73, %74, %75, %76, %77, %78, %79, "
                 "%80, %81, %82, %83, %84, %85, %86, %87, %88, %89, %90, %91, %92, %93, %94, %95}, [%97];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=f"(x[0][0]), "=f"(x[0][1]), "=f"(x[0][2]), "=f"(x[0][3]), "=f"(x[0][4]), "=f"(x[0][5]),
                   "=f"(x[0][6]), "=f"(x[0][7]), "=f"(x[0][8]), "=f"(x[0][9]), "=f"(x[0][10]), "=f"(x[0][11]),
                   "=f"(x[0][12]), "=f"(x[0][13]), "=f"(x[0][14]), "=f"(x[0][15]), "=f"(x[0][16]), "=f"(x[0][17]),
                   "=f"(x[0][18]), "=f"(x[0][19]), "=f"(x[0][20]), "=f"(x[0][21]), "=f"(x[0][22]), "=f"(x[0][23]),
                   "=f"(x[0][24]), "=f"(x[0][25]), "=f"(x[0][26]), "=f"(x[0][27]), "=f"(x[0][28]), "=f"(x[0][29]),
                   "=f"(x[0][30]), "=f"(x[0][31]), "=f"(x[1][0]), "=f"(x[1][1]), "=f"(x[1][2]), "=f"(x[1][3]),
                   "=f"(x[1][4]), "=f"(x[1][5]), "=f"(x[1][6]), "=f"(x[1][7]), "=f"(x[1][8]), "=f"(x[1][9]),
                   "=f"(x[1][10]), "=f"(x[1][11]), "=f"(x[1][12]), "=f"(x[1][13]), "=f"(x[1][14]), "=f"(x[1][15]),
                   "=f"(x[1][16]), "=f"(x[1][17]), "=f"(x[1][18]), "=f"(x[1][19]), "=f"(x[1][20]), "=f"(x[1][21]),
                   "=f"(x[1][22]), "=f"(x[1][23]), "=f"(x[1][24]), "=f"(x[1][25]), "=f"(x[1][26]), "=f"(x[1][27]),
                   "=f"(x[1][28]), "=f"(x[1][29]), "=f"(x[1][30]), "=f"(x[1][31]), "=f"(x[2][0]), "=f"(x[2][1]),
                   "=f"(x[2][2]), "=f"(x[2][3]), "=f"(x[2][4]), "=f"(x[2][5]), "=f"(x[2][6]), "=f"(x[2][7]),
                   "=f"(x[2][8]), "=f"(x[2][9]), "=f"(x[2][10]), "=f"(x[2][11]), "=f"(x[2][12]), "=f"(x[2][13]),
                   "=f"(x[2][14]), "=f"(x[2][15]), "=f"(x[2][16]), "=f"(x[2][17]), "=f"(x[2][18]), "=f"(x[2][19]),
                   "=f"(x[2][20]), "=f"(x[2][21]), "=f"(x[2][22]), "=f"(x[2][23]), "=f"(x[2][24]), "=f"(x[2][25]),
                   "=f"(x[2][26]), "=f"(x[2][27]), "=f"(x[2][28]), "=f"(x[2][29]), "=f"(x[2][30]), "=f"(x[2][31])
                 : "r"(at), "r"(more) : "memory");
}
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

template <int BN, bool SWAP, bool PAIR>
struct Geo {
    // pairs give one stage's room to the epilogue, whose stores would otherwise bound short contractions
    static constexpr int kStages = PAIR ? 4 : 5;
    static constexpr int kOutBuffers = SWAP ? 0 : (PAIR ? 4 : 2);       // 32-row x 128-byte store buffers an epilogue warp
    // Two accumulators.  At BN = 256 they overlap by 96 of TMEM's columns
    // (the scales need the rest): the epilogue takes those columns into
    // registers first and hands them back at once, so the next tile's MMAs
    // wait for 96 columns to be read, not for the tile to be stored.
    static constexpr int kAccStep = BN == 256 ? 160 : BN;
    static constexpr int kOverlap = BN - kAccStep;
    static constexpr int kAccLag = kOverlap ? 1 : 2;            // a tile's MMAs wait for the epilogue of the tile this many before
    static constexpr int kQRows = PAIR ? BN / 2 : BN;           // rows of Q's codes a CTA holds
    static constexpr int kSfP = 132;                            // words a scale box has per 128-column group
    static constexpr int kSfQ = BN == 256 ? 256 : BN + 4;
    static constexpr int kCodesP = kPRows * 128, kCodesQ = kQRows * 128;
    static constexpr int kScalesP = kSfP * 8, kScalesQ = kSfQ * 8;
    static constexpr int kTxCodes = kCodesP + kCodesQ, kTxScales = kScalesP + kScalesQ;
    static constexpr int kStageCodes = kCodesP + round_up(kCodesQ, 1024);
    static constexpr int kQAtoms = BN <= 128 ? 1 : BN / 128;    // 128-row pieces of Q's scales
    static constexpr int kStageScales = round_up(kScalesP, 128) + (kScalesQ > 1024 ? round_up(kScalesQ, 128) : 1024);
    static constexpr int kScalesQAt = round_up(kScalesP, 128);  // where a stage's Q scales start
    static constexpr int kOutBytes = 4 * kOutBuffers * 4096;
    static constexpr int kSmem = kStages * (kStageCodes + kStageScales) + kOutBytes + 1024;
    static constexpr int kQCols = 4 * kQAtoms;                  // TMEM columns of one group's Q scales
    static constexpr int kSfCols = 8 + 2 * kQCols;
    // A stage's scales have TMEM columns of their own, free again when the stage is.
    static constexpr int kSfBase = kAccStep + BN;
    static constexpr int kUsedCols = kSfBase + kStages * kSfCols;
    static constexpr int kTmemCols = kUsedCols <= 128 ? 128 : (kUsedCols <= 256 ? 256 : 512);
    static_assert(kUsedCols <= 512, "TMEM columns");
    static_assert(kSmem + 2 * 4 * (kMaxGroups + 1) + 512 <= 232448, "shared memory");
};

struct Mx4GemmMaps {
    CUtensorMap p_codes, q_codes, p_scales, q_scales, d;
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

// Tile t as CTA `half` of a pair sees it (0 without pairs): its 128 rows of P.
template <int BN, bool SWAP, bool PAIR>
__device__ __forceinline__ Tile tile_at(const Mx4GemmArgs& a, const int32_t* start, const int32_t* first, int t, int half)
{
    constexpr int kP = PAIR ? 2 * kPRows : kPRows;
    Tile o;
    if (a.ragged_k) {
        const int per = a.p_tiles * a.q_tiles, e = t / per, u = t - e * per;
        const int pi = u % a.p_tiles, qi = u / a.p_tiles;
        o.p_row = o.p_sf = pi * kP + half * kPRows;
        o.q_sf = qi * BN;
        o.q_row = o.q_sf + half * (BN / 2);
        o.kg0 = first[e];
        o.k64 = (start[e + 1] - start[e] + 63) / 64;
        o.d_row = e * a.p_rows + o.p_row;
        o.d_rows = static_cast<int>(a.p_rows) - o.p_row;
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
    constexpr int kX = SWAP ? BN : kP, kW = SWAP ? kPRows : BN;
    // weight tiles inside bands of kBand token tiles, so that neighbouring CTAs share both operands in L2
    constexpr int kBand = 8;
    const int xt = (x1 - x0 + kX - 1) / kX, wt = a.w_tiles;
    const int band = u / (kBand * wt), in = u - band * kBand * wt;
    const int height = min(kBand, xt - band * kBand);
    const int xi = band * kBand + in % height, wi = in / height;
    const int xr = x0 + xi * kX + half * kPRows, wr = wi * kW;
    const int w_row = e * static_cast<int>(a.w_rows) + wr, w_sf = e * static_cast<int>(a.w_sf_rows) + wr;
    o.p_row = SWAP ? w_row : xr;
    o.q_row = SWAP ? xr : w_row + half * (BN / 2);
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

// Swapped operands: the lane is a column of D, the accumulator's columns c0 ..
// c0+N-1 are rows of it, so a warp stores 32 neighbouring elements of a row.
template <int N, int DT>
__device__ __forceinline__ void store_swapped(const Mx4GemmArgs& a, const Tile& t, int lane_row, int c0, const float (&x)[N])
{
    const int col = t.d_col + lane_row;
    if (col >= a.d_cols) return;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        if (c0 + j >= t.d_rows) break;
        const int64_t i = (t.d_row + c0 + j) * a.ldd + col;
        store_out<DT>(a.d, i, a.accumulate ? __fadd_rn(load_out<DT>(a.d, i), x[j]) : x[j]);
    }
}
template <int N>
__device__ __forceinline__ void store_swapped(const Mx4GemmArgs& a, const Tile& t, int lane_row, int c0, const float (&x)[N])
{
    if (a.dtype == kF32) store_swapped<N, kF32>(a, t, lane_row, c0, x);
    else if (a.dtype == kF16) store_swapped<N, kF16>(a, t, lane_row, c0, x);
    else store_swapped<N, kBF16>(a, t, lane_row, c0, x);
}

__device__ __forceinline__ void store_shared16(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" :: "r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// The warp's bulk stores, whichever lanes issued them, have read their buffers.
__device__ __forceinline__ void stores_read()
{
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
}

// `bytes` (a multiple of 16) from shared to global memory, both 16-byte aligned.
__device__ __forceinline__ void bulk_store(void* to, uint32_t from, uint32_t bytes)
{
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n\t"
                 "cp.async.bulk.commit_group;" :: "l"(to), "r"(from), "r"(bytes) : "memory");
}

// An epilogue warp's 32 rows of a tile from its accumulator (columns acc ..) to
// D, whose rows start on 32 bytes: through NB buffers of 32 rows x 128 bytes.
// With PART false all 32 rows exist and a buffer is stored by TMA in whole
// lines (swizzled as the output's tensor map expects, whose bounds cut columns
// behind D's last, which end on 16 bytes).  With PART true `rows` of them
// exist, and each of these is a bulk copy of its lane's (the buffer's rows are
// 144 bytes apart against bank conflicts).  chunk(i) is the first of
// the 32 columns that come i-th; release() is called once the first FIRST of
// them (three, in registers together) or all (FIRST = 0) are read.  ZERO:
// zeros instead.
// Direct stores, 32 bytes a lane in 32 different rows, bounded a product of
// 2,048 columns (80 us against 65 us for 8,192 x 8,192 x 2,048); rows of a
// partial tile stored 64 bytes an instruction made eight uneven experts of
// 2,048 x 2,048 take 38 us where now 28.
template <int DT, int BN, int FIRST, int NB, bool PART, bool ZERO, typename Chunk, typename Release>
__device__ __forceinline__ void store_tile(const CUtensorMap& map, const Mx4GemmArgs& a, const Tile& t, uint32_t acc, int warp,
                                           int lane, int rows, uint32_t buf0, Chunk chunk, Release release)
{
    constexpr bool kWide = DT == kF32;                   // a buffer holds 32 columns, else 64: two chunks that come together
    constexpr int kBuffers = PART ? NB * 4096 / (32 * 144) : NB, kBytes = PART ? 32 * 144 : 4096;
    const uint32_t row = buf0 + lane * (PART ? 144 : 128);
    const uint32_t sw = PART ? 0u : static_cast<uint32_t>(lane & 7) << 4;
    const int d_cols = static_cast<int>(a.d_cols);
    const int64_t y = t.d_row + (warp & 3) * 32;
    auto put = [&](int i, const float (&x)[32]) {
        constexpr int kRound = kWide ? kBuffers : 2 * kBuffers;
        if (i % kRound == 0) stores_read();
        const int c = chunk(i), k = kWide ? i % kBuffers : i / 2 % kBuffers;
        const uint32_t at = row + k * kBytes;
        if constexpr (kWide) {
#pragma unroll
            for (uint32_t j = 0; j < 8; ++j)
                store_shared16(at + ((j << 4) ^ sw), __float_as_uint(x[4 * j]), __float_as_uint(x[4 * j + 1]),
                               __float_as_uint(x[4 * j + 2]), __float_as_uint(x[4 * j + 3]));
        } else {
            const uint32_t half = static_cast<uint32_t>(c & 32) << 1;           // the row's second 64 bytes
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j)
                store_shared16(at + ((half + (j << 4)) ^ sw), pack_out<DT>(x[8 * j], x[8 * j + 1]),
                               pack_out<DT>(x[8 * j + 2], x[8 * j + 3]), pack_out<DT>(x[8 * j + 4], x[8 * j + 5]),
                               pack_out<DT>(x[8 * j + 6], x[8 * j + 7]));
        }
        if (kWide || i % 2 == 1) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            const int col = t.d_col + (kWide ? c : c & ~32);
            if constexpr (PART) {
                constexpr int es = kWide ? 4 : 2;
                const int bytes = min(128, (d_cols - col) * es);
                if (lane < rows && bytes > 0)
                    bulk_store(static_cast<uint8_t*>(a.d) + ((y + lane) * a.ldd + col) * es, row + k * kBytes, static_cast<uint32_t>(bytes));
            } else if (lane == 0 && col < d_cols) {
                tma_store_2d(&map, col, static_cast<int>(y), buf0 + k * kBytes);
            }
        }
    };
    if constexpr (FIRST == 3 && !ZERO) {
        float x[3][32];
        tmem_ld(acc + chunk(0), acc + chunk(2), x);
        release();
#pragma unroll
        for (int i = 0; i < 3; ++i) put(i, x[i]);
    }
#pragma unroll 1
    for (int i = ZERO ? 0 : FIRST; i < BN / 32; ++i) {
        float x[32] = {};
        if (!ZERO) tmem_ld(acc + chunk(i), x);
        put(i, x);
    }
    if constexpr (FIRST == 0 && !ZERO) release();
}

// The same (1 to 32 rows exist) where D's rows do not start on 32 bytes or do
// not end on 16, or D is added to: each row as 32 neighbouring elements of the warp
// (stored by the lanes that hold the rows, 32 rows an instruction, 999 x 531 x
// 1,000 into fp32 took 28 us; so, 8 us).  From zeros when ZERO.
template <int DT, int BN, int FIRST, bool ZERO, typename Chunk, typename Release>
__device__ __forceinline__ void store_rows(const Mx4GemmArgs& a, const Tile& t, uint32_t acc, int warp, int lane, float* buf,
                                           Chunk chunk, Release release)
{
    const int rows = min(32, t.d_rows - (warp & 3) * 32);
    stores_read();                                       // of earlier tiles
    auto put = [&](int i, const float (&x)[32]) {
        const int col = t.d_col + chunk(i) + lane;
        if (col - lane >= a.d_cols) return;
#pragma unroll
        for (int k = 0; k < 32; ++k) buf[lane * 32 + (k ^ lane)] = x[k];
        __syncwarp();
        if (col < a.d_cols) {
            const int64_t at = (t.d_row + (warp & 3) * 32) * a.ldd + col;
            // eight rows' loads before their stores, which the compiler may not move them across
            for (int r0 = 0; r0 < rows; r0 += 8) {
                float v[8];
#pragma unroll
                for (int r = 0; r < 8; ++r) v[r] = buf[(r0 + r) * 32 + (lane ^ (r0 + r))];
                if (a.accumulate) {
                    float old[8];
#pragma unroll
                    for (int r = 0; r < 8; ++r) old[r] = r0 + r < rows ? load_out<DT>(a.d, at + (r0 + r) * a.ldd) : 0.0f;
#pragma unroll
                    for (int r = 0; r < 8; ++r) v[r] = __fadd_rn(old[r], v[r]);
                }
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (r0 + r < rows) store_out<DT>(a.d, at + (r0 + r) * a.ldd, v[r]);
            }
        }
        __syncwarp();
    };
    if constexpr (FIRST == 3 && !ZERO) {
        float x[3][32];
        tmem_ld(acc + chunk(0), acc + chunk(2), x);
        release();
#pragma unroll
        for (int i = 0; i < 3; ++i) put(i, x[i]);
    }
#pragma unroll 1
    for (int i = ZERO ? 0 : FIRST; i < BN / 32; ++i) {
        float x[32] = {};
        if (!ZERO) tmem_ld(acc + chunk(i), x);
        put(i, x);
    }
    if constexpr (FIRST == 0 && !ZERO) release();
}

// f with the output's type as a constant.
template <typename F> __device__ __forceinline__ void with_dtype(int dtype, F f)
{
    if (dtype == kF32) f(std::integral_constant<int, kF32>());
    else if (dtype == kF16) f(std::integral_constant<int, kF16>());
    else f(std::integral_constant<int, kBF16>());
}

// ---------------------------------------------------------------------------
// The kernel.  Cluster of a.split CTAs along the contraction (1: none, and
// each CTA walks tiles blockIdx.x, + gridDim.x, ...; else each cluster has
// one tile).  PAIR: two CTAs work on one tile of 256 x BN with the MMA that
// spans both (cta_group::2).  Each holds its 128 rows of P and half of Q's
// rows, so a tile's operands are read once by the pair: a third less traffic
// from L2 per product, which bounds the main loop.  The first CTA issues the
// MMAs; loads, scales and the epilogue run in both.
// ---------------------------------------------------------------------------
template <int BN, bool SWAP, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
mx4_gemm_kernel(const __grid_constant__ Mx4GemmMaps maps, const Mx4GemmArgs a)
{
    using G = Geo<BN, SWAP, PAIR>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int32_t start[kMaxGroups + 1], first[kMaxGroups + 1];
    __shared__ __align__(8) uint64_t bars[4 * G::kStages + 5];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t{1023});
    uint8_t* out_smem = smem + G::kStages * G::kStageCodes;          // 1,024-byte aligned store buffers
    uint8_t* sf_smem = out_smem + G::kOutBytes;
    const uint32_t codes_at = smem_u32(smem), sf_at = smem_u32(sf_smem), bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (G::kStages + s); };
    // a stage's scales are in order, and its codes have landed
    auto ready = [&](int s) { return bar0 + 8u * (2 * G::kStages + s); };
    // where a stage's scales land: on their own in a pair, whose codes all land on the first CTA's `full`
    auto sf_land = [&](int s) { return bar0 + 8u * (PAIR ? 3 * G::kStages + s : s); };
    auto acc_full = [&](int b) { return bar0 + 8u * (4 * G::kStages + b); };
    auto acc_empty = [&](int b) { return bar0 + 8u * (4 * G::kStages + 2 + b); };
    const uint32_t drain = bar0 + 8u * (4 * G::kStages + 4);
    const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
    const int split = a.split;
    int rank = 0;
    if (PAIR || split > 1) asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    const int half = PAIR ? rank : 0, ctas = PAIR ? 2 : split;
    // arrives at the first CTA's barrier
    auto arrive_first = [&](uint32_t bar) {
        if (PAIR) bar_arrive_cluster(in_rank(bar, 0));
        else bar_arrive(bar);
    };

    if (tid == 0) {
        for (int s = 0; s < G::kStages; ++s) {
            bar_init(full(s), 1);
            bar_init(empty(s), 1);
            bar_init(ready(s), PAIR ? 2 : 1);
            if (PAIR) bar_init(sf_land(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            bar_init(acc_full(b), 1);
            bar_init(acc_empty(b), PAIR ? 8 : 4);
        }
        bar_init(drain, 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 2) {
        if (PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                         :: "r"(smem_u32(&tmem_slot)), "r"(G::kTmemCols) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                         :: "r"(smem_u32(&tmem_slot)), "r"(G::kTmemCols) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        }
    }
    if (a.offsets) {
        constexpr int kX = SWAP ? BN : (PAIR ? 2 * kPRows : kPRows);
        if (a.ragged_k) ragged_table(a.offsets, a.groups, a.x_rows, 128, 1, start, first, tid, kThreads);
        else ragged_table(a.offsets, a.groups, a.x_rows, kX, a.w_tiles, start, first, tid, kThreads);
    }
    fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();            // the barriers exist before the other CTA's loads and arrivals reach them
    fence_after();
    const uint32_t tmem = tmem_slot;

    const int tiles = (a.offsets && !a.ragged_k) ? first[a.groups] : a.tiles;
    const int t0 = blockIdx.x / ctas, dt = gridDim.x / ctas;

    // the 64-element steps [k_lo, k_hi) of a tile that this CTA sums: whole stages, evenly over the ranks
    auto k_range = [&](const Tile& t, int* lo, int* hi) {
        const int stages = (t.k64 + 3) / 4, part = PAIR ? 0 : rank;
        *lo = min(t.k64, stages * part / split * 4);
        *hi = min(t.k64, stages * (part + 1) / split * 4);
    };

    if (warp == 0) {
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int t = t0; t < tiles && ok; t += dt) {
                const Tile o = tile_at<BN, SWAP, PAIR>(a, start, first, t, half);
                int lo, hi;
                k_range(o, &lo, &hi);
                const int px = o.p_sf & ~3, qx = o.q_sf & ~3;
                for (int k = lo; k < hi; k += 4, ++it) {
                    const int s = it % G::kStages;
                    if (it >= G::kStages && !(ok = bar_wait(empty(s), (it / G::kStages - 1) & 1, &abort_flag))) break;
                    const uint32_t c = codes_at + s * G::kStageCodes, f = sf_at + s * G::kStageScales;
                    const int kg = o.kg0 + k / 2;
                    uint32_t land = full(s);
                    if (PAIR) {
                        bar_expect(sf_land(s), G::kTxScales);
                        if (rank == 0) bar_expect(full(s), 2 * G::kTxCodes);
                        land = in_rank(full(s), 0);
                    } else {
                        bar_expect(full(s), G::kTxCodes + G::kTxScales);
                    }
                    tma_2d<PAIR>(c, &maps.p_codes, kg * 64, o.p_row, land);
                    tma_2d<PAIR>(c + G::kCodesP, &maps.q_codes, kg * 64, o.q_row, land);
                    tma_2d(f, &maps.p_scales, px, kg, sf_land(s));
                    tma_2d(f + G::kScalesQAt, &maps.q_scales, qx, kg, sf_land(s));
                }
            }
            // every stage's last use is over before the CTA's memory goes
            // away: its copies have landed and its commits have arrived (the
            // wait stays bounded; after an abort it looks at the copies only)
            for (int s = 0; s < G::kStages; ++s) {
                const uint32_t uses = it > static_cast<uint32_t>(s) ? (it - s - 1) / G::kStages + 1 : 0;
                if (uses == 0) continue;
                if (ok && !abort_flag) {
                    bar_wait(empty(s), (uses - 1) & 1, &abort_flag);
                } else {
                    for (uint32_t i = 0; i < kWaitLimit && !bar_try(sf_land(s), (uses - 1) & 1); ++i) {}
                    if (PAIR && rank == 0) for (uint32_t i = 0; i < kWaitLimit && !bar_try(full(s), (uses - 1) & 1); ++i) {}
                }
            }
        }
    } else if (warp == 1) {
        if (half == 0) {
            // The whole warp runs the loop and one elected lane issues, so
            // that the compiler sees uniform control flow and keeps the
            // descriptors in uniform registers: issued by a single lane's own
            // branch, a stage took 1,300 cycles to issue and 512 to compute.
            // kind::mxf4: E2M1 operands (1), E8M0 scales, M = 128 (pair: 256), N = BN
            constexpr uint32_t kIdesc = 1u << 7 | 1u << 10 | static_cast<uint32_t>(BN >> 3) << 17 | 1u << 23 | (PAIR ? 2u : 1u) << 27;
            uint32_t n = 0, s = 0, ph = 0;
            bool ok = true;
            for (int t = t0; t < tiles && ok; t += dt) {
                const Tile o = tile_at<BN, SWAP, PAIR>(a, start, first, t, half);
                int lo, hi;
                k_range(o, &lo, &hi);
                const int steps = __shfl_sync(0xFFFFFFFFu, hi - lo, 0);
                if (steps <= 0) continue;                // nothing to sum: the epilogue takes zeros
                const uint32_t b = n & 1;
                if (n >= G::kAccLag) {
                    const uint32_t m = n - G::kAccLag;
                    if (!(ok = warp_wait(acc_empty(m & 1), (m >> 1) & 1, &abort_flag))) break;
                }
                const uint32_t d = tmem + b * G::kAccStep;
                for (int k = 0; k < steps; k += 4) {
                    if (!(ok = warp_wait(ready(s), ph, &abort_flag))) break;
                    fence_after();
                    const uint32_t c = codes_at + s * G::kStageCodes, sf_from = sf_at + s * G::kStageScales;
                    const uint32_t sf = tmem + G::kSfBase + s * G::kSfCols;
                    const uint64_t pd = tile_desc(c), qd = tile_desc(c + G::kCodesP);
                    if (elect_one()) {
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            copy_scales<PAIR>(sf + 4 * g, sf_from + 512 * g);
#pragma unroll
                            for (int q = 0; q < G::kQAtoms; ++q)
                                copy_scales<PAIR>(sf + 8 + G::kQCols * g + 4 * q, sf_from + G::kScalesQAt + 512 * (G::kQAtoms * g + q));
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if (k + j >= steps) break;
                            const uint32_t id = 2u * (j & 1);
                            mma_mx4<PAIR>(d, pd + 2 * j, qd + 2 * j, kIdesc | id << 4 | id << 29, sf + 4 * (j >> 1),
                                          sf + 8 + G::kQCols * (j >> 1), k + j > 0);
                        }
                        mma_commit<PAIR>(empty(s));
                        if (k + 4 >= steps) mma_commit<PAIR>(acc_full(b));
                    }
                    __syncwarp();
                    if (++s == G::kStages) { s = 0; ph ^= 1; }
                }
                ++n;
            }
            if (abort_flag) {
                if (elect_one()) {
                    mma_commit<PAIR>(drain);
                    for (uint32_t i = 0; i < kWaitLimit && !bar_try(drain, 0); ++i) {}
                }
                __syncwarp();
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
        // Scales of every fourth stage: from rows in order to the order that
        // copy_scales takes (row 32 j + r at word [r][j]), in place.
        uint32_t it = 0;
        bool ok = true;
        for (int t = t0; t < tiles && ok; t += dt) {
            const Tile o = tile_at<BN, SWAP, PAIR>(a, start, first, t, half);
            int lo, hi;
            k_range(o, &lo, &hi);
            const int pr = o.p_sf & 3, qr = o.q_sf & 3;
            for (int k = lo; k < hi; k += 4, ++it) {
                if ((it & 3) != (warp & 3u)) continue;
                const int s = it % G::kStages;
                // This warp has not seen the stage's use before, whose landing
                // another warp waited for, and a parity only tells two
                // neighbouring uses apart: first wait until that use is over.
                // (The use before that one is over: the loads of it - 4, which
                // this warp saw land, were issued after those of it - 5, which
                // waited for it.)
                if (it >= G::kStages && !(ok = warp_wait(empty(s), (it / G::kStages - 1) & 1, &abort_flag))) break;
                if (!(ok = warp_wait(sf_land(s), (it / G::kStages) & 1, &abort_flag))) break;
                uint32_t* ps = reinterpret_cast<uint32_t*>(sf_smem + s * G::kStageScales);
                uint32_t* qs = ps + G::kScalesQAt / 4;
                uint32_t p[2][4], q[2][G::kQAtoms][4];
#pragma unroll
                for (int g = 0; g < 2; ++g)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        p[g][j] = ps[g * G::kSfP + pr + 32 * j + lane];
#pragma unroll
                        for (int n = 0; n < G::kQAtoms; ++n) {
                            const int r = 128 * n + 32 * j + lane;
                            q[g][n][j] = BN >= 128 || r < BN ? qs[g * G::kSfQ + qr + r] : 0u;
                        }
                    }
                __syncwarp();
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    reinterpret_cast<uint4*>(ps)[32 * g + lane] = make_uint4(p[g][0], p[g][1], p[g][2], p[g][3]);
#pragma unroll
                    for (int n = 0; n < G::kQAtoms; ++n)
                        reinterpret_cast<uint4*>(qs)[32 * (G::kQAtoms * g + n) + lane] =
                            make_uint4(q[g][n][0], q[g][n][1], q[g][n][2], q[g][n][3]);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                // the pair's codes land on the first CTA's barrier: its arrival says that they are there too
                if (PAIR && half == 0 && !(ok = warp_wait(full(s), (it / G::kStages) & 1, &abort_flag))) break;
                if (lane == 0) arrive_first(ready(s));
            }
        }
    } else if (warp >= 8) {
        const int lane_row = (warp & 3) * 32 + lane;
        const uint32_t quad = static_cast<uint32_t>(warp & 3) << 21;
        uint8_t* buf = out_smem + (warp & 3) * G::kOutBuffers * 4096;
        constexpr int kFirst = G::kOverlap / 32;
        uint32_t n = 0;
        for (int t = t0; t < tiles; t += dt) {
            const Tile o = tile_at<BN, SWAP, PAIR>(a, start, first, t, half);
            int lo, hi;
            k_range(o, &lo, &hi);
            const int rows = o.d_rows - (warp & 3) * 32;         // of this warp (tokens on the lanes' side)
            if (lo < hi) {
                const int b = n & 1;
                if (!warp_wait(acc_full(b), (n >> 1) & 1, &abort_flag)) break;
                fence_after();
                if (split == 1) {
                    const uint32_t acc = tmem + quad + b * G::kAccStep;
                    auto release = [&] {
                        fence_before();
                        __syncwarp();
                        if (lane == 0) arrive_first(acc_empty(b));
                    };
                    if constexpr (SWAP) {
                        constexpr int kChunk = BN < 32 ? 16 : 32;
#pragma unroll 1
                        for (int c = 0; c < BN; c += kChunk) {
                            float x[kChunk];
                            tmem_ld(acc + c, x);
                            store_swapped<kChunk>(a, o, lane_row, c, x);
                        }
                        release();
                    } else if (rows <= 0) {
                        release();
                    } else {
                        // The shared columns first: the last ones of accumulator 0, the first ones of 1.
                        // Chunks that share a 64-column store buffer stay neighbours.
                        static_assert(kFirst == 0 || kFirst == 3, "the order here");
                        auto chunk = [&](int i) {
                            if constexpr (kFirst == 0) return 32 * i;
                            else return 32 * (b ? i : (i < 2 ? 6 + i : (i < 4 ? 7 - i : i - 4)));
                        };
                        with_dtype(a.dtype, [&](auto dt_) {
                            constexpr int DT = decltype(dt_)::value;
                            if (a.tma_store && rows >= 32)
                                store_tile<DT, BN, kFirst, G::kOutBuffers, false, false>(maps.d, a, o, acc, warp, lane, 32, smem_u32(buf),
                                                                                  chunk, release);
                            else if (a.tma_store)
                                store_tile<DT, BN, kFirst, G::kOutBuffers, true, false>(maps.d, a, o, acc, warp, lane, rows, smem_u32(buf),
                                                                                 chunk, release);
                            else
                                store_rows<DT, BN, kFirst, false>(a, o, acc, warp, lane, reinterpret_cast<float*>(buf), chunk, release);
                        });
                    }
                }
                ++n;
            } else if (!SWAP && !a.accumulate && rows > 0) {     // an empty group's product
                if constexpr (!SWAP)
                    with_dtype(a.dtype, [&](auto dt_) {
                        constexpr int DT = decltype(dt_)::value;
                        auto chunk = [](int i) { return 32 * i; };
                        if (a.tma_store && rows >= 32)
                            store_tile<DT, BN, kFirst, G::kOutBuffers, false, true>(maps.d, a, o, 0u, warp, lane, 32, smem_u32(buf),
                                                                                    chunk, [] {});
                        else
                            store_rows<DT, BN, kFirst, true>(a, o, 0u, warp, lane, reinterpret_cast<float*>(buf), chunk, [] {});
                    });
            }
        }
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
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
            o = tile_at<BN, SWAP, PAIR>(a, start, first, t0, half);
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
                store_swapped<4>(a, o, lane_row, 4 * g, x);
            }
        }
    }
    fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();            // nothing of the other CTA reaches for this one's memory any more
    if (warp == 2) {
        if (PAIR) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(G::kTmemCols));
        else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(G::kTmemCols));
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

cudaError_t encoder(EncodeTiled* out)
{
    // the driver's entry point: the same for every device and thread
    static std::atomic<EncodeTiled> found{nullptr};
    EncodeTiled fn = found.load(std::memory_order_relaxed);
    if (!fn) {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q);
        if (e != cudaSuccess) return e;
        if (!p || q != cudaDriverEntryPointSuccess) return cudaErrorNotSupported;
        fn = reinterpret_cast<EncodeTiled>(p);
        found.store(fn, std::memory_order_relaxed);
    }
    *out = fn;
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

// D, for stores of 32 rows x 128 bytes.
cudaError_t out_map(EncodeTiled enc, CUtensorMap* m, const Mx4GemmArgs& a)
{
    const int es = elem_bytes(a.dtype);
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(a.d_cols), static_cast<cuuint64_t>(a.d_rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(a.ldd) * es};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / es), 32}, ones[2] = {1, 1};
    const CUtensorMapDataType type = a.dtype == kF32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : a.dtype == kF16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const CUresult r = enc(m, type, 2, a.d, dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int BN, bool SWAP, bool PAIR>
cudaError_t launch_as(Mx4GemmArgs a, const Mx4GemmOperands& op, int sms, cudaStream_t stream)
{
    using G = Geo<BN, SWAP, PAIR>;
    EncodeTiled enc = nullptr;
    cudaError_t e = encoder(&enc);
    if (e != cudaSuccess) return e;
    const Mx4Operand& p = SWAP ? op.w : op.x;
    const Mx4Operand& q = SWAP ? op.x : op.w;
    Mx4GemmMaps maps{};
    if ((e = codes_map(enc, &maps.p_codes, p.codes, p.code_rows, p.pitch, kPRows)) != cudaSuccess) return e;
    if ((e = codes_map(enc, &maps.q_codes, q.codes, q.code_rows, q.pitch, G::kQRows)) != cudaSuccess) return e;
    if ((e = scales_map(enc, &maps.p_scales, p.scales, p.scale_rows, p.pitch / 64, G::kSfP)) != cudaSuccess) return e;
    if ((e = scales_map(enc, &maps.q_scales, q.scales, q.scale_rows, q.pitch / 64, G::kSfQ)) != cudaSuccess) return e;
    // A bulk store writes whole 16-byte pieces: where D's columns end inside
    // one it would write into what stands behind them.
    a.tma_store = !SWAP && a.vec && !a.accumulate && a.d_cols * elem_bytes(a.dtype) % 16 == 0;
    if (a.tma_store && (e = out_map(enc, &maps.d, a)) != cudaSuccess) return e;
    constexpr int kP = PAIR ? 2 * kPRows : kPRows, kX = SWAP ? BN : kP, kW = SWAP ? kPRows : BN;
    a.w_tiles = static_cast<int>((a.w_rows + kW - 1) / kW);
    a.p_tiles = static_cast<int>((a.p_rows + kP - 1) / kP);
    a.q_tiles = a.w_tiles;
    int64_t tiles;                      // exact, or (groups of rows) at most
    if (a.ragged_k) tiles = static_cast<int64_t>(a.groups) * a.p_tiles * a.q_tiles;
    else tiles = ((a.x_rows + kX - 1) / kX + (a.offsets ? a.groups : 0)) * a.w_tiles;
    if (tiles > INT32_MAX / 8) return cudaErrorInvalidConfiguration;
    a.tiles = static_cast<int>(tiles);
    if (tiles == 0) return cudaSuccess;
    const int cluster = PAIR ? 2 : a.split;
    const int64_t ctas = a.split > 1 ? tiles * cluster : std::min<int64_t>(tiles, sms / cluster) * cluster;
    auto* k = mx4_gemm_kernel<BN, SWAP, PAIR>;
    static std::atomic<uint64_t> allowed{0};
    if ((e = allow_shared(k, G::kSmem, allowed)) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = G::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
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
    // 256 x 256 tiles by pairs of CTAs, or 128 x 128 tiles by single ones: the
    // fewer rounds of tiles, weighted by what a 256-element stage of each takes
    // (0.42 us for a pair's, 0.30 us for a single's), decide.  Measured, pairs
    // and singles: 256 x 8,192 x 2,048 8.4 and 7.1 us, 512 x 8,192 x 2,048 9.6
    // and 11.0, 4,096 x 2,048 x 8,192 32.6 and 46.2, 8,192 x 8,192 x 2,048 65
    // and 92, 999 x 531 x 1,000 14.9 and 9.3.
    auto pairs_win = [&](int64_t groups, int64_t rows, int64_t cols) {
        auto rounds = [&](int64_t tile, int64_t at_once) {
            const int64_t tiles = groups * ((rows + tile - 1) / tile) * ((cols + tile - 1) / tile);
            return (tiles + at_once - 1) / at_once;
        };
        return rounds(256, sms / 2) * 42 <= rounds(128, sms) * 30;
    };
    if (a.ragged_k)
        return pairs_win(a.groups, a.p_rows, a.w_rows) ? launch_as<256, false, true>(a, op, sms, stream)
                                                       : launch_as<128, false, false>(a, op, sms, stream);
    // Few token rows a group: the weights take the 128-row side of the tile,
    // the tokens its narrow side, and the contraction is cut over a cluster
    // so that the weights' tiles reach every SM.
    const int64_t mean = a.offsets ? (a.x_rows + a.groups - 1) / a.groups : a.x_rows;
    if (mean <= 64) {
        const int bn = mean <= 16 ? 16 : (mean <= 32 ? 32 : 64);
        const int64_t wt = (a.w_rows + kPRows - 1) / kPRows;
        const int64_t xt = (a.x_rows + bn - 1) / bn + (a.offsets ? std::min<int64_t>(a.groups, a.x_rows) : 0);
        // A cluster pays about 1 us to meet at 16 tokens and 3 us at 64, a stage
        // 0.29 us: 1 x 2,048 x 8,192 takes 12.8 us whole and 8.4 us in four,
        // 1 x 8,192 x 2,048 6.1 us whole and 7.3 us in two, 64 x 8,192 x 2,048
        // 6.9 us whole and 11.3 us in two.  So a part keeps 8 stages.
        const int stages = (a.k64 + 3) / 4;
        while (a.split < 4 && stages >= a.split * 2 * 8 && wt * xt * a.split * 2 <= sms) a.split *= 2;
        if (bn == 16) return launch_as<16, true, false>(a, op, sms, stream);
        if (bn == 32) return launch_as<32, true, false>(a, op, sms, stream);
        return launch_as<64, true, false>(a, op, sms, stream);
    }
    return pairs_win(a.offsets ? a.groups : 1, mean, a.w_rows) ? launch_as<256, false, true>(a, op, sms, stream)
                                                               : launch_as<128, false, false>(a, op, sms, stream);
}

cudaError_t mx4_error_count(unsigned int* out)
{
    // the copy's own stream does not wait for streams made non-blocking
    const cudaError_t e = cudaDeviceSynchronize();
    return e != cudaSuccess ? e : cudaMemcpyFromSymbol(out, g_mx4_errors, sizeof(*out));
}

}  // namespace opt2s
