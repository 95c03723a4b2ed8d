// opt2s_mx4_quant.cu -- quantisation to microscaled 4-bit matrices and back.
//
// A quantised training step needs a matrix twice: in blocks along its rows
// (the contraction of the forward product) and in blocks down its columns,
// transposed (the contraction of the backward products).  One CTA reads a
// 128 x 64 tile once into shared memory and writes both forms from there.
// A 4,096 x 8,192 bf16 source takes 22 us (4.7 TB/s of its 103 MB; 16 us at
// the measured copy rate) and 37 us with noise (3.7 TB/s of 136 MB; 21 us):
// instructions bound it, 13 an element and 27 with noise (the ALU pipe 76 %
// busy); fp32 reaches 6.1 TB/s.  Loads by cp.async, all of a tile's in
// flight at once.  Tiles of 128 x 128 by 256 threads were slower (23 and 41 us:
// fewer, larger steps between barriers and a coarser last wave), as was a
// persistent form that loaded the next tile meanwhile (27 and 55 us); scaling
// two bf16 elements at once changed nothing.
#include <type_traits>

#include "opt2s_mx4.cuh"

namespace opt2s {
namespace {

constexpr int kQuantThreads = 128;
constexpr int kTileCols = 64;

// A 16-byte copy from global to shared memory that does not wait; zeros when
// !in (the address must then still be valid).
__device__ __forceinline__ void copy16(uint8_t* dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                 :: "r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16(uint8_t* dst, const void* src, bool in)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 :: "r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))), "l"(src), "r"(in ? 16 : 0) : "memory");
}

// The 16-byte chunks of a tile, CHUNKS a row of 16 * CHUNKS bytes from `x` on,
// into shared memory (chunk c of row r at chunk c ^ (r & 7)); zeros from row
// `rows` and chunk `chunks` on (`valid` is an address that may be read).  A
// whole tile needs two instructions a chunk; with the bounds of a partial one
// they were an eighth of all instructions.
template <int CHUNKS>
__device__ __forceinline__ void load_chunks(const uint8_t* x, int64_t pitch, int rows, int chunks, const void* valid,
                                            uint8_t* dst, int tid)
{
    constexpr int kStep = kQuantThreads / CHUNKS;
    constexpr int kMask = CHUNKS < 8 ? CHUNKS - 1 : 7;
    static_assert(kStep % 8 == 0, "a thread's rows have one swizzle");
    const int r0 = tid / CHUNKS, c = tid % CHUNKS;
    const uint8_t* p = x + r0 * pitch + c * 16;
    const int64_t step = pitch * kStep;
    uint8_t* d = dst + r0 * CHUNKS * 16 + ((c ^ (r0 & kMask)) << 4);
    if (rows == kTileRows && chunks == CHUNKS) {
#pragma unroll
        for (int k = 0; k < kTileRows / kStep; ++k, p += step) copy16(d + k * kStep * CHUNKS * 16, p);
    } else {
#pragma unroll
        for (int k = 0; k < kTileRows / kStep; ++k, p += step) {
            const bool in = r0 + k * kStep < rows && c < chunks;
            copy16(d + k * kStep * CHUNKS * 16, in ? p : valid, in);
        }
    }
}

// A tile of elements of B bytes whose rows do not start on 16 bytes: a warp
// takes neighbouring elements of a row, eight rows in flight.  `place` says
// where an element goes.
template <int B, int COLS, typename Place>
__device__ __forceinline__ void load_elements(const uint8_t* x, int64_t pitch, int rows, int cols, int tid, Place place)
{
    using T = std::conditional_t<B == 4, uint32_t, std::conditional_t<B == 2, uint16_t, uint8_t>>;
    constexpr int kAcross = COLS / 32, kRows = 8;
    const T* p = reinterpret_cast<const T*>(x);
    const int lane = tid & 31;
    for (int r0 = (tid >> 5) * kRows; r0 < kTileRows; r0 += kQuantThreads / 32 * kRows) {
        T v[kRows][kAcross];
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int k = 0; k < kAcross; ++k) {
                const int e = k * 32 + lane;
                v[r][k] = r0 + r < rows && e < cols ? p[(r0 + r) * pitch + e] : T{0};
            }
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int k = 0; k < kAcross; ++k) *reinterpret_cast<T*>(place(r0 + r, k * 32 + lane)) = v[r][k];
    }
}

// Starts the load of one tile of the source (zeros outside it) into shared
// memory; copies_done() waits for it.
template <int DT, bool NOISE>
__device__ __forceinline__ void load_tile(const Mx4QuantArgs& a, int64_t row0, int rows, int64_t slab, int64_t col0,
                                          uint8_t* tile, uint8_t* noise, int tid)
{
    using S = Src<DT>;
    constexpr int P = S::kPer;
    const int cols = static_cast<int>(min(static_cast<int64_t>(kTileCols), a.cols - col0));
    const uint8_t* x = static_cast<const uint8_t*>(a.x) + (slab * a.slab_stride + row0 * a.row_stride + col0) * S::kBytes;
    if (a.vec && cols % P == 0) {
        load_chunks<kTileCols / P>(x, a.row_stride * S::kBytes, rows, cols / P, a.x, tile, tid);
    } else {
        load_elements<S::kBytes, kTileCols>(x, a.row_stride, rows, cols, tid, [&](int r, int e) {
            return tile + tile_chunk<DT, kTileCols>(r, e / P) + e % P * S::kBytes;
        });
    }
    if (NOISE) {
        const uint8_t* n = a.noise + (slab * a.rows + row0) * a.cols + col0;
        if (a.noise_vec && cols % 16 == 0) {
            load_chunks<kTileCols / 16>(n, a.cols, rows, cols / 16, a.noise, noise, tid);
        } else {
            load_elements<1, kTileCols>(n, a.cols, rows, cols, tid,
                                        [&](int r, int e) { return noise + noise_chunk<kTileCols>(r, e / 16) + e % 16; });
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
    if (a.codes && rows > 0) {
        // the last tile of an ungrouped matrix also writes the scale bytes of its padding rows
        const int64_t rp = (a.rows + 3) / 4 * 4;
        o.pitch = (a.cols + 127) / 128 * 64;
        o.codes = a.codes + (slab * a.rows + row0) * o.pitch + col0 / 2;
        o.scales = a.scales + ((col0 / 128 * a.slabs + slab) * rp + row0) * 4 + col0 % 128 / 32;
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

template <int DT> __device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    if (DT == kF16) {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// grid: x = groups of 4 rows, y = 4,096-column parts, z = slabs.  A thread
// takes 16 elements (8 bytes of codes, half a block) of each row; all loads
// come first, and 16-bit outputs are stored 32 bytes a thread: 4,096 x 8,192
// to bf16 takes 12 us (7.1 TB/s).  Outputs whose rows do not start on 32 bytes
// (VEC false) take two elements a thread and step and one row a CTA instead,
// so that a warp still stores neighbouring elements.
template <int DT, bool VEC>
__global__ void __launch_bounds__(256) mx4_dequantize_kernel(const Mx4DequantArgs a)
{
    constexpr int kRows = VEC ? 4 : 1, kPart = 4096;
    const int64_t cp = (a.cols + 127) / 128 * 128, rp = (a.rows + 3) / 4 * 4;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kRows, slab = blockIdx.z, col0 = static_cast<int64_t>(blockIdx.y) * kPart;
    const int rows = static_cast<int>(min(static_cast<int64_t>(kRows), a.rows - row0));
    const uint8_t* codes = a.codes + (slab * a.rows + row0) * (cp / 2);
    const uint8_t* scales = a.scales + (slab * rp + row0) * 4;
    const int64_t group = a.slabs * rp * 4;           // bytes of scales per 128-column group
    const int64_t out0 = (slab * a.rows + row0) * a.cols;
    if constexpr (VEC) {
        const int64_t c0 = col0 + threadIdx.x * 16;
        if (c0 >= a.cols) return;
        uint2 w[kRows];
        uint32_t s[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (r < rows) {
                w[r] = *reinterpret_cast<const uint2*>(codes + r * (cp / 2) + c0 / 2);
                s[r] = scales[(c0 >> 7) * group + r * 4 + ((c0 >> 5) & 3)];
            }
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (r >= rows) break;
            const float scale = scale_value(s[r]);
            float x[16];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float2 f = decode2((k < 4 ? w[r].x : w[r].y) >> (8 * (k & 3)) & 255u);
                x[2 * k] = __fmul_rn(f.x, scale);
                x[2 * k + 1] = __fmul_rn(f.y, scale);
            }
            const int64_t at = out0 + r * a.cols + c0;
            if (DT == kF32) {
                uint32_t* d = static_cast<uint32_t*>(a.out) + at;
#pragma unroll
                for (int k = 0; k < 16; k += 8)
                    store32(d + k, __float_as_uint(x[k]), __float_as_uint(x[k + 1]), __float_as_uint(x[k + 2]),
                            __float_as_uint(x[k + 3]), __float_as_uint(x[k + 4]), __float_as_uint(x[k + 5]),
                            __float_as_uint(x[k + 6]), __float_as_uint(x[k + 7]));
            } else {
                store32(static_cast<uint16_t*>(a.out) + at, pack2<DT>(x[0], x[1]), pack2<DT>(x[2], x[3]),
                        pack2<DT>(x[4], x[5]), pack2<DT>(x[6], x[7]), pack2<DT>(x[8], x[9]), pack2<DT>(x[10], x[11]),
                        pack2<DT>(x[12], x[13]), pack2<DT>(x[14], x[15]));
            }
        }
        return;
    }
#pragma unroll
    for (int it = 0; it < kPart / 512; ++it) {
        const int64_t c0 = col0 + (it * 256 + threadIdx.x) * 2;
        if (c0 >= a.cols) break;
        const float2 f = decode2(codes[c0 / 2]);
        const float scale = scale_value(scales[(c0 >> 7) * group + ((c0 >> 5) & 3)]);
        const float x0 = __fmul_rn(f.x, scale), x1 = __fmul_rn(f.y, scale);
        const int64_t at = out0 + c0;
        if (DT == kF32) {
            float* d = static_cast<float*>(a.out) + at;
            d[0] = x0;
            if (c0 + 1 < a.cols) d[1] = x1;
        } else {
            uint16_t* d = static_cast<uint16_t*>(a.out) + at;
            const uint32_t h = pack2<DT>(x0, x1);
            d[0] = static_cast<uint16_t>(h);
            if (c0 + 1 < a.cols) d[1] = static_cast<uint16_t>(h >> 16);
        }
    }
}

template <int DT, bool NOISE>
cudaError_t launch_quantize_as(const Mx4QuantArgs& a, dim3 grid, cudaStream_t stream)
{
    constexpr int kBytes = kTileRows * kTileCols * (Src<DT>::kBytes + (NOISE ? 1 : 0));
    auto* k = mx4_quantize_kernel<DT, NOISE>;
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_shared(k, kBytes, allowed);
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
    const dim3 grid(static_cast<unsigned>((a.cols + 127) / 128 * (128 / kTileCols)), static_cast<unsigned>(row_tiles),
                    static_cast<unsigned>(a.slabs));
    if (dtype == kF32) return launch_quantize_dt<kF32>(a, grid, stream);
    if (dtype == kF16) return launch_quantize_dt<kF16>(a, grid, stream);
    return launch_quantize_dt<kBF16>(a, grid, stream);
}

cudaError_t launch_mx4_dequantize(const Mx4DequantArgs& a, int dtype, cudaStream_t stream)
{
    const dim3 grid(static_cast<unsigned>(a.vec ? (a.rows + 3) / 4 : a.rows), static_cast<unsigned>((a.cols + 4095) / 4096),
                    static_cast<unsigned>(a.slabs));
    auto go = [&](auto* wide, auto* any) {
        if (a.vec) wide<<<grid, 256, 0, stream>>>(a);
        else any<<<grid, 256, 0, stream>>>(a);
    };
    if (dtype == kF32) go(mx4_dequantize_kernel<kF32, true>, mx4_dequantize_kernel<kF32, false>);
    else if (dtype == kF16) go(mx4_dequantize_kernel<kF16, true>, mx4_dequantize_kernel<kF16, false>);
    else go(mx4_dequantize_kernel<kBF16, true>, mx4_dequantize_kernel<kBF16, false>);
    return cudaGetLastError();
}

}  // namespace opt2s
