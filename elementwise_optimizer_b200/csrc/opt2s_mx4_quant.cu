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

// Loads one tile of the source (zeros outside it) into shared memory.
template <int DT, bool NOISE>
__device__ __forceinline__ void load_tile(const Mx4QuantArgs& a, int64_t row0, int rows, int64_t slab, int64_t col0,
                                          uint8_t* tile, uint8_t* noise, int tid)
{
    using S = Src<DT>;
    constexpr int P = S::kPer, kChunks = kTileCols / P;
    const int64_t base = slab * a.slab_stride + row0 * a.row_stride + col0;
    const int cols = static_cast<int>(min(static_cast<int64_t>(kTileCols), a.cols - col0));
    for (int t = tid; t < kTileRows * kChunks; t += kQuantThreads) {
        const int r = t / kChunks, c = t % kChunks, at = c * P;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r < rows && at < cols) {
            const int64_t i = base + r * a.row_stride + at;
            if (a.vec && at + P <= cols) {
                v = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.x) + i * S::kBytes);
            } else {
                uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
                for (int k = 0; k < P; ++k)
                    if (at + k < cols) w[k * S::kBytes / 4] |= S::bits(a.x, i + k) << (S::kBytes == 2 ? 16 * (k & 1) : 0);
                v = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        *reinterpret_cast<uint4*>(tile + tile_chunk<DT, kTileCols>(r, c)) = v;
    }
    if (NOISE) {
        const int64_t nbase = (slab * a.rows + row0) * a.cols + col0;
        for (int t = tid; t < kTileRows * 8; t += kQuantThreads) {
            const int r = t / 8, c = t % 8, at = c * 16;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (r < rows && at < cols) {
                const int64_t i = nbase + r * a.cols + at;
                if (a.noise_vec && at + 16 <= cols) {
                    v = *reinterpret_cast<const uint4*>(a.noise + i);
                } else {
                    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        if (at + k < cols) w[k / 4] |= static_cast<uint32_t>(a.noise[i + k]) << (8 * (k & 3));
                    v = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            *reinterpret_cast<uint4*>(noise + noise_chunk<kTileCols>(r, c)) = v;
        }
    }
}

// grid: x = column tiles, y = row tiles (of all groups), z = slabs.
template <int DT, bool NOISE>
__global__ void __launch_bounds__(kQuantThreads) mx4_quantize_kernel(const Mx4QuantArgs a)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int32_t start[kMaxGroups + 1], first[kMaxGroups + 1];
    uint8_t* tile = smem;
    uint8_t* noise = smem + kTileRows * kTileCols * Src<DT>::kBytes;
    const int tid = threadIdx.x;
    const int64_t slab = blockIdx.z, col0 = static_cast<int64_t>(blockIdx.x) * kTileCols;
    const int64_t rt = blockIdx.y;
    int64_t row0 = rt * kTileRows, row_end = a.rows;
    if (a.offsets) {
        ragged_table(a.offsets, a.groups, a.rows, kTileRows, 1, start, first, tid, kQuantThreads);
        if (rt >= first[a.groups]) {                // behind the last group: only padding of the column form
            row0 = row_end = 0;
        } else {
            const int e = group_of(first, a.groups, static_cast<int32_t>(rt));
            row0 = start[e] + (rt - first[e]) * kTileRows;
            row_end = start[e + 1];
        }
    }
    const int rows = static_cast<int>(min(static_cast<int64_t>(kTileRows), row_end - row0));
    load_tile<DT, NOISE>(a, row0, rows, slab, col0, tile, noise, tid);
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

// A thread's 8 elements (4 bytes of codes) of one row.
template <int DT>
__global__ void __launch_bounds__(256) mx4_dequantize_kernel(const Mx4DequantArgs a)
{
    const int64_t cp = (a.cols + 127) / 128 * 128, per_row = cp / 8;
    const int64_t total = a.slabs * a.rows * per_row, rp = (a.rows + 3) / 4 * 4;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; t < total;
         t += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t row = t / per_row, c0 = (t - row * per_row) * 8;
        if (c0 >= a.cols) continue;
        const int64_t slab = row / a.rows, r = row - slab * a.rows;
        const uint32_t w = *reinterpret_cast<const uint32_t*>(a.codes + row * (cp / 2) + c0 / 2);
        const uint32_t s = a.scales[(((c0 >> 7) * a.slabs + slab) * rp + r) * 4 + ((c0 >> 5) & 3)];
        // 2^(s - 127): s = 0 is the subnormal 2^-127, s = 255 NaN
        const float scale = s == 255u ? __uint_as_float(0x7FC00000u)
                                      : (s == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(s << 23));
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
    const int64_t total = a.slabs * a.rows * ((a.cols + 127) / 128 * 16);
    const int64_t blocks = std::min<int64_t>((total + 255) / 256, 1 << 20);
    if (dtype == kF32) mx4_dequantize_kernel<kF32><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(a);
    else if (dtype == kF16) mx4_dequantize_kernel<kF16><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(a);
    else mx4_dequantize_kernel<kBF16><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace opt2s
