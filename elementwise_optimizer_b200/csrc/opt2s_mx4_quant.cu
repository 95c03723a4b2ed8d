// opt2s_mx4_quant.cu -- quantisation to microscaled 4-bit matrices and back.
//
// A quantised training step needs a matrix twice: in blocks along its rows
// (the contraction of the forward product) and in blocks down its columns,
// transposed (the contraction of the backward products).  One CTA reads a
// 128 x 128 tile once into shared memory and writes both forms from there.
// The kernel is bound by memory traffic: 16-bit sources read 2 bytes an
// element (3 with noise) and write 17/32 byte per form.
#include "opt2s_mx4.cuh"

namespace opt2s {
namespace {

constexpr int kQuantThreads = 256;
constexpr int kTileCols = 128;

// A 16-byte copy from global to shared memory that does not wait; zeros when
// !in (the address must then still be valid).
__device__ __forceinline__ void copy16(uint8_t* dst, const void* src, bool in)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 :: "r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))), "l"(src), "r"(in ? 16 : 0) : "memory");
}

// Starts the load of one tile of the source (zeros outside it) into shared
// memory; copies_done() waits for it.
template <int DT, bool NOISE>
__device__ __forceinline__ void load_tile(const Mx4QuantArgs& a, int64_t row0, int rows, int64_t slab, int64_t col0,
                                          uint8_t* tile, uint8_t* noise, int tid)
{
    using S = Src<DT>;
    constexpr int P = S::kPer, kChunks = kTileCols / P, kStep = kQuantThreads / kChunks;
    const int cols = static_cast<int>(min(static_cast<int64_t>(kTileCols), a.cols - col0));
    {
        const int c = tid % kChunks, at = c * P;
        const uint8_t* x = static_cast<const uint8_t*>(a.x) + (slab * a.slab_stride + row0 * a.row_stride + col0) * S::kBytes;
        if (a.vec && cols % P == 0) {
            const int64_t pitch = a.row_stride * S::kBytes;
            const uint8_t* p = x + c * 16;
#pragma unroll
            for (int r = tid / kChunks; r < kTileRows; r += kStep) {
                const bool in = r < rows && at < cols;
                copy16(tile + tile_chunk<DT, kTileCols>(r, c), in ? p + r * pitch : static_cast<const uint8_t*>(a.x), in);
            }
        } else {
            for (int r = tid / kChunks; r < kTileRows; r += kStep) {
                uint32_t w[4] = {0, 0, 0, 0};
                if (r < rows) {
#pragma unroll
                    for (int k = 0; k < P; ++k)
                        if (at + k < cols)
                            w[k * S::kBytes / 4] |= S::bits(x, r * a.row_stride + at + k) << (S::kBytes == 2 ? 16 * (k & 1) : 0);
                }
                *reinterpret_cast<uint4*>(tile + tile_chunk<DT, kTileCols>(r, c)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
    if (NOISE) {
        const int c = tid % 8, at = c * 16;
        const uint8_t* n = a.noise + (slab * a.rows + row0) * a.cols + col0;
        if (a.noise_vec && cols % 16 == 0) {
#pragma unroll
            for (int r = tid / 8; r < kTileRows; r += kQuantThreads / 8) {
                const bool in = r < rows && at < cols;
                copy16(noise + noise_chunk<kTileCols>(r, c), in ? n + r * a.cols + at : a.noise, in);
            }
        } else {
            for (int r = tid / 8; r < kTileRows; r += kQuantThreads / 8) {
                uint32_t w[4] = {0, 0, 0, 0};
                if (r < rows) {
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        if (at + k < cols) w[k / 4] |= static_cast<uint32_t>(n[r * a.cols + at + k]) << (8 * (k & 3));
                }
                *reinterpret_cast<uint4*>(noise + noise_chunk<kTileCols>(r, c)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
}

__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// grid: x = column tiles, y = row tiles (of all groups), z = slabs.
template <int DT, bool NOISE>
__global__ void __launch_bounds__(kQuantThreads) mx4_quantize_kernel(const Mx4QuantArgs a)
{
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* tile = smem;
    uint8_t* noise = smem + kTileRows * kTileCols * Src<DT>::kBytes;
    const int tid = threadIdx.x;
    const int64_t slab = blockIdx.z, col0 = static_cast<int64_t>(blockIdx.x) * kTileCols;
    const int64_t rt = blockIdx.y;
    int64_t row0 = rt * kTileRows, row_end = a.rows;
    if (a.offsets) {
        int32_t* start = reinterpret_cast<int32_t*>(smem);          // the tile's room, until it is loaded
        int32_t* first = start + kMaxGroups + 1;
        ragged_table(a.offsets, a.groups, a.rows, kTileRows, 1, start, first, tid, kQuantThreads);
        if (rt >= first[a.groups]) {                // behind the last group: only padding of the column form
            row0 = row_end = 0;
        } else {
            const int e = group_of(first, a.groups, static_cast<int32_t>(rt));
            row0 = start[e] + (rt - first[e]) * kTileRows;
            row_end = start[e + 1];
        }
        __syncthreads();
    }
    const int rows = static_cast<int>(min(static_cast<int64_t>(kTileRows), row_end - row0));
    load_tile<DT, NOISE>(a, row0, rows, slab, col0, tile, noise, tid);
    copies_done();
    __syncthreads();
    TileOut o{};
    const int64_t cg = col0 / 128;                  // 128-column group of the row form
    if (a.codes && rows > 0) {
        // the last tile of an ungrouped matrix also writes the scale bytes of its padding rows
        const int64_t rp = (a.rows + 3) / 4 * 4;
        o.pitch = (a.cols + 127) / 128 * 64;
        o.codes = a.codes + (slab * a.rows + row0) * o.pitch + cg * 64;
        o.scales = a.scales + ((cg * a.slabs + slab) * rp + row0) * 4;
        o.rows = rows;
        o.scale_rows = row_end == a.rows ? static_cast<int>(min(static_cast<int64_t>(kTileRows), rp - row0)) : rows;
        tile_rows_out<DT, kTileCols, NOISE, kQuantThreads>(tile, noise, o, tid);
    }
    if (a.codes_t) {
        const int64_t cp = (a.cols + 3) / 4 * 4;
        o.pitch_t = static_cast<int64_t>(gridDim.y) * 64;
        o.codes_t = a.codes_t + (slab * a.cols + col0) * o.pitch_t + rt * 64;
        o.scales_t = a.scales_t + ((rt * a.slabs + slab) * cp + col0) * 4;
        o.cols = static_cast<int>(min(static_cast<int64_t>(kTileCols), a.cols - col0));
        o.scale_cols = static_cast<int>(min(static_cast<int64_t>(kTileCols), cp - col0));
        tile_cols_out<DT, kTileCols, NOISE, kQuantThreads>(tile, noise, o, tid);
    }
}

// 2^(s - 127): s = 0 is the subnormal 2^-127, s = 255 NaN.
__device__ __forceinline__ float scale_value(uint32_t s)
{
    return s == 255u ? __uint_as_float(0x7FC00000u) : (s == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(s << 23));
}

// grid: x = groups of 4 rows, y = 4,096-column parts, z = slabs.  A thread
// takes 8 elements (4 bytes of codes) a step.
template <int DT>
__global__ void __launch_bounds__(256) mx4_dequantize_kernel(const Mx4DequantArgs a)
{
    constexpr int kRows = 4, kPart = 512 * 8;         // 4 rows of 512 x 8 columns a CTA: 8 steps of 256 threads
    const int64_t cp = (a.cols + 127) / 128 * 128, rp = (a.rows + 3) / 4 * 4;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kRows, slab = blockIdx.z, col0 = static_cast<int64_t>(blockIdx.y) * kPart;
#pragma unroll
    for (int it = 0; it < kRows * 2; ++it) {
        const int64_t r = row0 + it / 2, c0 = col0 + ((it & 1) * 256 + threadIdx.x) * 8;
        if (r >= a.rows || c0 >= a.cols) continue;
        const int64_t row = slab * a.rows + r;
        const uint32_t w = *reinterpret_cast<const uint32_t*>(a.codes + row * (cp / 2) + c0 / 2);
        const float scale = scale_value(a.scales[(((c0 >> 7) * a.slabs + slab) * rp + r) * 4 + ((c0 >> 5) & 3)]);
        float x[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 f = decode2(w >> (8 * k) & 255u);
            x[2 * k] = __fmul_rn(f.x, scale);
            x[2 * k + 1] = __fmul_rn(f.y, scale);
        }
        const int64_t at = row * a.cols + c0;
        const bool vec = a.vec && c0 + 8 <= a.cols;
        if (DT == kF32) {
            float* d = static_cast<float*>(a.out) + at;
            if (vec) {
                reinterpret_cast<float4*>(d)[0] = make_float4(x[0], x[1], x[2], x[3]);
                reinterpret_cast<float4*>(d)[1] = make_float4(x[4], x[5], x[6], x[7]);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) if (c0 + k < a.cols) d[k] = x[k];
            }
        } else {
            uint32_t h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (DT == kBF16) {
                    const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
                    h[k] = *reinterpret_cast<const uint32_t*>(&v);
                } else {
                    const __half2 v = __floats2half2_rn(x[2 * k], x[2 * k + 1]);
                    h[k] = *reinterpret_cast<const uint32_t*>(&v);
                }
            }
            uint16_t* d = static_cast<uint16_t*>(a.out) + at;
            if (vec) {
                *reinterpret_cast<uint4*>(d) = make_uint4(h[0], h[1], h[2], h[3]);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (c0 + k < a.cols) d[k] = static_cast<uint16_t>(h[k / 2] >> (16 * (k & 1)));
            }
        }
    }
}

template <int DT, bool NOISE>
cudaError_t launch_quantize_as(const Mx4QuantArgs& a, dim3 grid, cudaStream_t stream)
{
    constexpr int kBytes = kTileRows * kTileCols * (Src<DT>::kBytes + (NOISE ? 1 : 0));
    auto* k = mx4_quantize_kernel<DT, NOISE>;
    // an attribute of the function on the current device: set at every launch, it costs no synchronisation
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (e != cudaSuccess) return e;
    k<<<grid, kQuantThreads, kBytes, stream>>>(a);
    return cudaGetLastError();
}

template <int DT>
cudaError_t launch_quantize_dt(const Mx4QuantArgs& a, dim3 grid, cudaStream_t stream)
{
    return a.noise ? launch_quantize_as<DT, true>(a, grid, stream) : launch_quantize_as<DT, false>(a, grid, stream);
}

}  // namespace

cudaError_t launch_mx4_quantize(const Mx4QuantArgs& a, int dtype, int64_t row_tiles, cudaStream_t stream)
{
    const dim3 grid(static_cast<unsigned>((a.cols + kTileCols - 1) / kTileCols), static_cast<unsigned>(row_tiles),
                    static_cast<unsigned>(a.slabs));
    if (dtype == kF32) return launch_quantize_dt<kF32>(a, grid, stream);
    if (dtype == kF16) return launch_quantize_dt<kF16>(a, grid, stream);
    return launch_quantize_dt<kBF16>(a, grid, stream);
}

cudaError_t launch_mx4_dequantize(const Mx4DequantArgs& a, int dtype, cudaStream_t stream)
{
    const dim3 grid(static_cast<unsigned>((a.rows + 3) / 4), static_cast<unsigned>((a.cols + 4095) / 4096),
                    static_cast<unsigned>(a.slabs));
    if (dtype == kF32) mx4_dequantize_kernel<kF32><<<grid, 256, 0, stream>>>(a);
    else if (dtype == kF16) mx4_dequantize_kernel<kF16><<<grid, 256, 0, stream>>>(a);
    else mx4_dequantize_kernel<kBF16><<<grid, 256, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace opt2s
