// opt2s_mx4_step.cu -- the two-state step that also writes the 4-bit copies of
// the params it updates.
//
// A model that multiplies with 4-bit weights needs them again after every
// step, along their rows and, transposed, down their columns.  Written by the
// step itself they cost 17/16 byte an element and no second read of the
// param.  A CTA steps a tile of 128 rows x 64 columns (the element arithmetic
// of opt2s_device.cuh, so the same bits as opt2s_step), keeps the new params
// in shared memory as they are stored, and encodes both forms from there.
// Tensors without copies are stepped in the same launch, 8,192 elements a
// CTA, a warp on each of eight chunks.  Bound by memory traffic, as the plain
// step is: four tensors of 2,048 x 8,192 take 338 us with AdEMAMix over bf16
// (6.2 TB/s of 30 + 17/16 bytes an element; 315 us without copies) and 311 us
// with Adam over fp32 (6.3 TB/s); Adam over bf16, 283 us (5.5 TB/s; 231 us
// without), has the least traffic to hide the encoding behind.
//
// The records travel as kernel arguments (up to 256 a launch): no table in
// device memory, nothing kept between calls, and a captured launch holds all
// it needs.
#include "opt2s_device.cuh"
#include "opt2s_mx4.cuh"

namespace opt2s {
namespace {

constexpr int kStepThreads = 256;
constexpr int kStepCols = 64;
constexpr uint32_t kFlatElems = 8192, kWarpElems = kFlatElems / (kStepThreads / 32);

template <int CAP>
struct StepMx4Table {
    int32_t count;
    int32_t first[CAP + 1];         // tiles of the records before each; [count] is the total
    StepMx4Rec rec[CAP];
};

template <int DT, int ALGO, bool SKIP>
__device__ __forceinline__ void step_tile(const StepMx4Rec& t, int32_t u, uint8_t* tile, const StepScalars& s, int tid)
{
    using P = Param<DT>;
    constexpr int V = P::kVec, kChunks = kStepCols / V, kIters = kTileRows * kChunks / kStepThreads;
    const int64_t cols = t.cols, rows = t.rows;
    const int ct = static_cast<int>((cols + 127) / 128 * 2), rt = static_cast<int>((rows + 127) / 128);
    const int c_at = u % ct, rest = u / ct, r_at = rest % rt;
    const int64_t slab = rest / rt, row0 = static_cast<int64_t>(r_at) * kTileRows, col0 = static_cast<int64_t>(c_at) * kStepCols;
    const int n_rows = static_cast<int>(min(static_cast<int64_t>(kTileRows), rows - row0));
    const int n_cols = static_cast<int>(min(static_cast<int64_t>(kStepCols), cols - col0));      // <= 0: padding only
    const int64_t base = (slab * rows + row0) * cols + col0;

    if (t.vec) {
        constexpr int U = 8 / V;            // 8 elements a thread and iteration, as the plain step's vector body
        for (int it = 0; it < kIters; it += U) {
            typename P::Raw graw[U], praw[U];
            float m[U][V], v[U][V], m2[U][V];
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int x = (it + k) * kStepThreads + tid, r = x / kChunks, c = x % kChunks;
                if (r < n_rows && c * V < n_cols) {
                    const int64_t i = base + r * cols + c * V;
                    graw[k] = P::load(static_cast<const uint8_t*>(t.g) + i * P::kBytes, 0);
                    praw[k] = P::load(static_cast<const uint8_t*>(t.p) + i * P::kBytes, 0);
                    load_state<V>(t.m + i, 0, m[k]);
                    load_state<V>(t.v + i, 0, v[k]);
                    if (ALGO == kAdEMAMix) load_state<V>(t.m2 + i, 0, m2[k]);
                }
            }
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int x = (it + k) * kStepThreads + tid, r = x / kChunks, c = x % kChunks;
                typename P::Raw out{};
                if (r < n_rows && c * V < n_cols) {
                    const int64_t i = base + r * cols + c * V;
                    float g[V], p[V];
                    P::widen(graw[k], g);
                    P::widen(praw[k], p);
                    // the range test of four elements at a time (337 us where eight took 352, with AdEMAMix over bf16)
                    update_group<ALGO, SKIP, kPlain, 0, 4, V>(g, p, m[k], v[k], m2[k], s);
                    if constexpr (V == 8) update_group<ALGO, SKIP, kPlain, V - 4, 4, V>(g, p, m[k], v[k], m2[k], s);
                    out = P::narrow(p, praw[k], g, SKIP);
                    P::store(static_cast<uint8_t*>(t.p) + i * P::kBytes, 0, out);
                    store_state<V>(t.m + i, 0, m[k]);
                    store_state<V>(t.v + i, 0, v[k]);
                    if (ALGO == kAdEMAMix) store_state<V>(t.m2 + i, 0, m2[k]);
                }
                *reinterpret_cast<typename P::Raw*>(tile + tile_chunk<DT, kStepCols>(r, c)) = out;
            }
        }
    } else {
        // element by element, four a thread in flight
        constexpr int U = 4;
        for (int x0 = tid; x0 < kTileRows * kStepCols; x0 += U * kStepThreads) {
            float g[U] = {}, p[U] = {}, m[U] = {}, v[U] = {}, m2[U] = {};
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int x = x0 + k * kStepThreads, r = x / kStepCols, c = x % kStepCols;
                if (r < n_rows && c < n_cols) {
                    const int64_t i = base + r * cols + c;
                    g[k] = P::load1(static_cast<const uint8_t*>(t.g) + i * P::kBytes, 0);
                    p[k] = P::load1(static_cast<const uint8_t*>(t.p) + i * P::kBytes, 0);
                    m[k] = t.m[i];
                    v[k] = t.v[i];
                    if (ALGO == kAdEMAMix) m2[k] = t.m2[i];
                }
            }
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int x = x0 + k * kStepThreads, r = x / kStepCols, c = x % kStepCols;
                if (r < n_rows && c < n_cols && !(SKIP && g[k] == 0.0f)) {
                    const int64_t i = base + r * cols + c;
                    update<ALGO, false>(g[k], p[k], m[k], v[k], m2[k], s);
                    P::store1(static_cast<uint8_t*>(t.p) + i * P::kBytes, 0, p[k]);
                    t.m[i] = m[k];
                    t.v[i] = v[k];
                    if (ALGO == kAdEMAMix) t.m2[i] = m2[k];
                }
                P::store1(tile + tile_chunk<DT, kStepCols>(r, c / V) + c % V * P::kBytes, 0, p[k]);
            }
        }
    }
    __syncthreads();
    TileOut o{};
    if (t.codes) {
        const int64_t rp = (rows + 3) / 4 * 4;
        o.pitch = (cols + 127) / 128 * 64;
        o.codes = t.codes + (slab * rows + row0) * o.pitch + c_at * 32;
        o.scales = t.scales + ((static_cast<int64_t>(c_at / 2) * t.slabs + slab) * rp + row0) * 4 + c_at % 2 * 2;
        o.rows = n_rows;
        o.scale_rows = static_cast<int>(min(static_cast<int64_t>(kTileRows), rp - row0));
        tile_rows_out<DT, kStepCols, false, kStepThreads>(tile, nullptr, o, tid);
    }
    if (t.codes_t) {
        const int64_t cp = (cols + 3) / 4 * 4;
        o.pitch_t = static_cast<int64_t>(rt) * 64;
        o.codes_t = t.codes_t + (slab * cols + col0) * o.pitch_t + r_at * 64;
        o.scales_t = t.scales_t + ((static_cast<int64_t>(r_at) * t.slabs + slab) * cp + col0) * 4;
        o.cols = n_cols;
        o.scale_cols = static_cast<int>(min(static_cast<int64_t>(kStepCols), cp - col0));
        tile_cols_out<DT, kStepCols, false, kStepThreads>(tile, nullptr, o, tid);
    }
}

template <int DT, int ALGO, bool SKIP>
__device__ __forceinline__ void step_flat(const StepMx4Rec& t, int32_t u, const StepScalars& s, int tid)
{
    const int64_t at = static_cast<int64_t>(u) * kFlatElems + (tid >> 5) * kWarpElems;
    if (at >= t.numel) return;
    ChunkRec c;
    c.p = static_cast<uint8_t*>(t.p) + at * Param<DT>::kBytes;
    c.g = static_cast<const uint8_t*>(t.g) + at * Param<DT>::kBytes;
    c.m = t.m + at;
    c.v = t.v + at;
    c.m2 = t.m2 + at;
    c.len = static_cast<uint32_t>(min(static_cast<int64_t>(kWarpElems), t.numel - at));
    c.dtype = DT;
    run_chunk<DT, ALGO, SKIP>(c, s, tid & 31);
}

template <int DT, int ALGO, bool SKIP>
__device__ __forceinline__ void step_unit(const StepMx4Rec& t, int32_t u, uint8_t* tile, const StepScalars& s, int tid)
{
    if (t.codes || t.codes_t) step_tile<DT, ALGO, SKIP>(t, u, tile, s, tid);
    else step_flat<DT, ALGO, SKIP>(t, u, s, tid);
}

template <int CAP, int ALGO, bool SKIP>
// Three resident CTAs an SM (80 registers) overlap one's encoding with the
// others' memory traffic: AdEMAMix over bf16, 4 x 2048 x 8192, takes 397 us
// with the two that 96 registers allow and 352 us with three.
__global__ void __launch_bounds__(kStepThreads, 3)
step_mx4_kernel(const __grid_constant__ StepMx4Table<CAP> tab, const StepScalars s)
{
    __shared__ __align__(128) uint8_t tile[kTileRows * kStepCols * 4];
    const int32_t b = static_cast<int32_t>(blockIdx.x);
    const int e = group_of(tab.first, tab.count, b);
    const StepMx4Rec& t = tab.rec[e];
    const int32_t u = b - tab.first[e];
    if (t.dtype == kF32) step_unit<kF32, ALGO, SKIP>(t, u, tile, s, threadIdx.x);
    else if (t.dtype == kF16) step_unit<kF16, ALGO, SKIP>(t, u, tile, s, threadIdx.x);
    else step_unit<kBF16, ALGO, SKIP>(t, u, tile, s, threadIdx.x);
}

template <int CAP>
cudaError_t launch_cap(const StepMx4Rec* recs, int n, int algo, int skip, const StepScalars& s, cudaStream_t stream)
{
    StepMx4Table<CAP> tab;
    tab.count = n;
    int64_t total = 0;
    for (int i = 0; i < n; ++i) {
        tab.rec[i] = recs[i];
        tab.first[i] = static_cast<int32_t>(total);
        total += step_mx4_tiles(recs[i]);
        if (total > INT32_MAX) return cudaErrorInvalidConfiguration;
    }
    tab.first[n] = static_cast<int32_t>(total);
    const unsigned grid = static_cast<unsigned>(total);
    if (algo == kAdam) {
        if (skip) step_mx4_kernel<CAP, kAdam, true><<<grid, kStepThreads, 0, stream>>>(tab, s);
        else step_mx4_kernel<CAP, kAdam, false><<<grid, kStepThreads, 0, stream>>>(tab, s);
    } else {
        if (skip) step_mx4_kernel<CAP, kAdEMAMix, true><<<grid, kStepThreads, 0, stream>>>(tab, s);
        else step_mx4_kernel<CAP, kAdEMAMix, false><<<grid, kStepThreads, 0, stream>>>(tab, s);
    }
    return cudaGetLastError();
}

}  // namespace

int64_t step_mx4_tiles(const StepMx4Rec& t)
{
    if (t.codes || t.codes_t) return t.slabs * ((t.rows + 127) / 128) * ((t.cols + 127) / 128 * 2);
    return (t.numel + kFlatElems - 1) / kFlatElems;
}

cudaError_t launch_step_mx4(const StepMx4Rec* recs, int n, int algo, int skip_zeros, StepScalars s,
                            cudaStream_t stream)
{
    fill_reciprocals(&s);
    // small collections send small argument blocks
    return n <= 16 ? launch_cap<16>(recs, n, algo, skip_zeros, s, stream)
                   : launch_cap<kStepMx4MaxRecs>(recs, n, algo, skip_zeros, s, stream);
}

}  // namespace opt2s
