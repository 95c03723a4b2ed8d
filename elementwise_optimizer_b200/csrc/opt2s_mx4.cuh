// opt2s_mx4.cuh -- device code shared by the microscaled 4-bit kernels: the
// E2M1 / E8M0 encoding of a block, the quantisation of a tile held in shared
// memory, and the table of ragged groups.
//
// The format is MXFP4 of the OCP Microscaling Formats (MX) specification
// v1.0: blocks of 32 elements share the scale 2^e, e = floor(log2 amax) - 2
// clamped to >= -127 and stored as the byte e + 127 (255 is NaN), and an
// element is the E2M1 value nearest to x / 2^e, ties to the even code,
// magnitudes above 6 taken as 6.  Every step is exact in fp32 (2^-e is a
// normal number and the product by it loses no bit that decides the
// rounding), so codes and scales do not depend on how a kernel orders them.
// A block holding an infinity or a NaN gets scale byte 255 and codes 0.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "opt2s_internal.h"

namespace opt2s {
namespace {

// ---------------------------------------------------------------------------
// Elements
// ---------------------------------------------------------------------------

// |x| as an integer that orders like |x|; at least kInfBits for inf and NaN.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
constexpr uint32_t kInfBits = 0x7F800000u;

// The scale byte of a block whose largest magnitude has the bits `amax`.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax)
{
    if (amax >= kInfBits) return 255u;
    const uint32_t biased = amax >> 23;             // floor(log2 amax) + 127, 0 for zero and subnormals
    return biased > 2u ? biased - 2u : 0u;
}

// 2^-(byte - 127), exactly: a normal number for every byte but 255 (for which
// it is 0, so that every code of a NaN block is 0).
__device__ __forceinline__ float inverse_scale(uint32_t byte)
{
    return byte == 255u ? 0.0f : __uint_as_float((254u - byte) << 23);
}

// Two E2M1 codes in one byte, `lo` in the low nibble: nearest, ties to even,
// magnitudes above 6 saturated.
__device__ __forceinline__ uint32_t encode2(float lo, float hi)
{
    uint32_t r;
    asm("{\n\t"
        ".reg .b8 t;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n\t"
        "cvt.u32.u8 %0, t;\n\t"
        "}" : "=r"(r) : "f"(lo), "f"(hi));
    return r;
}

// One E2M1 code rounded stochastically with the byte r: with c + f the
// position of |x| among the codes' magnitudes (linear between neighbours),
// the code is c + (f > (r + 0.5)/256).
__device__ __forceinline__ uint32_t encode_noise(float x, uint32_t r)
{
    // each difference below is exact, so the comparison decides on x itself
    const float a = fminf(fabsf(x), 6.0f);
    const float base = a < 2.0f ? 0.0f : (a < 4.0f ? 4.0f : 6.0f);
    const float pos = a < 2.0f ? __fmul_rn(a, 2.0f) : (a < 4.0f ? __fsub_rn(a, 2.0f) : __fmul_rn(__fsub_rn(a, 4.0f), 0.5f));
    const float c = floorf(pos);
    const float u = __fmul_rn(__fadd_rn(static_cast<float>(r), 0.5f), 1.0f / 256.0f);
    const uint32_t code = static_cast<uint32_t>(base + c) + (__fsub_rn(pos, c) > u ? 1u : 0u);
    return code | (__float_as_uint(x) >> 31 << 3);
}

// The two values of a byte of codes.
__device__ __forceinline__ float2 decode2(uint32_t byte)
{
    uint32_t h;
    asm("{\n\t"
        ".reg .b8 t;\n\t"
        "cvt.u8.u32 t, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, t;\n\t"
        "}" : "=r"(h) : "r"(byte));
    return __half22float2(*reinterpret_cast<__half2*>(&h));
}

// Storage traits of a 4-bit kernel's source: kPer elements in a 16-byte
// chunk, unpacked to fp32.
template <int DT> struct Src;
template <> struct Src<kF32> {
    static constexpr int kPer = 4, kBytes = 4;
    __device__ static void unpack(const uint4& c, float* x) {
        x[0] = __uint_as_float(c.x); x[1] = __uint_as_float(c.y);
        x[2] = __uint_as_float(c.z); x[3] = __uint_as_float(c.w);
    }
    __device__ static float one(const void* p, int64_t i) { return static_cast<const float*>(p)[i]; }
    __device__ static uint32_t bits(const void* p, int64_t i) { return static_cast<const uint32_t*>(p)[i]; }
};
template <> struct Src<kBF16> {
    static constexpr int kPer = 8, kBytes = 2;
    __device__ static float2 pair(uint32_t w) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
    __device__ static void unpack(const uint4& c, float* x) {
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) { const float2 f = pair(w[k]); x[2 * k] = f.x; x[2 * k + 1] = f.y; }
    }
    __device__ static uint32_t bits(const void* p, int64_t i) { return static_cast<const uint16_t*>(p)[i]; }
};
template <> struct Src<kF16> {
    static constexpr int kPer = 8, kBytes = 2;
    __device__ static float2 pair(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
    __device__ static void unpack(const uint4& c, float* x) {
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) { const float2 f = pair(w[k]); x[2 * k] = f.x; x[2 * k + 1] = f.y; }
    }
    __device__ static uint32_t bits(const void* p, int64_t i) { return static_cast<const uint16_t*>(p)[i]; }
};

// The scale byte and the 16 bytes of codes of one block.
template <bool NOISE>
__device__ __forceinline__ uint4 encode_block(const float (&x)[32], const uint32_t (&noise)[8], uint32_t* scale)
{
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) amax = max(amax, abs_bits(x[i]));
    *scale = scale_byte(amax);
    const float inv = inverse_scale(*scale);
    const bool dead = *scale == 255u;               // inf * 0 and NaN must not reach the encoder
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t word = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = __fmul_rn(x[8 * k + 2 * i], inv), b = __fmul_rn(x[8 * k + 2 * i + 1], inv);
            uint32_t byte;
            if (NOISE) {
                const uint32_t n = noise[2 * k + i / 2] >> (16 * (i & 1));
                byte = encode_noise(a, n & 255u) | encode_noise(b, n >> 8 & 255u) << 4;
            } else {
                byte = encode2(a, b);
            }
            word |= byte << (8 * i);
        }
        w[k] = dead ? 0u : word;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// ---------------------------------------------------------------------------
// A tile of 128 rows x TC columns in shared memory, in the source's type:
// 16-byte chunk c of row r stands at chunk c ^ (r & 7) of its row, so that
// threads reading one chunk of 8 consecutive rows and threads reading
// consecutive columns of one row both spread over all banks.
// ---------------------------------------------------------------------------
constexpr int kTileRows = 128;

template <int DT, int TC>
__device__ __forceinline__ uint32_t tile_chunk(int r, int c)   // byte offset of chunk c of row r
{
    constexpr int kRowBytes = TC * Src<DT>::kBytes;
    return static_cast<uint32_t>(r * kRowBytes + ((c ^ (r & 7)) << 4));
}

template <int TC>
__device__ __forceinline__ uint32_t noise_chunk(int r, int c)
{
    constexpr int kMask = TC / 16 - 1;              // 8 chunks a row for TC = 128, 4 for 64
    return static_cast<uint32_t>(r * TC + ((c ^ (r & kMask)) << 4));
}

// Where a tile's codes and scales go.  `codes` / `scales` of the row blocks
// are offset to the tile's first row and first column; those of the column
// blocks to the tile's first column and first row block.
struct TileOut {
    uint8_t* codes;        // row r: + r * pitch, TC/2 bytes
    uint8_t* scales;       // row r: + 4 r, TC/32 bytes
    int64_t pitch;
    int rows;              // rows of the tile that exist; scale bytes are written for scale_rows of them
    int scale_rows;
    uint8_t* codes_t;      // column c: + c * pitch_t, 64 bytes
    uint8_t* scales_t;     // column c: + 4 c, 4 bytes
    int64_t pitch_t;
    int cols, scale_cols;
};

// Blocks along the rows: a thread takes one row's TC/32/H blocks.  THREADS
// threads cover 128 rows x H parts, H = THREADS / 128.
template <int DT, int TC, bool NOISE, int THREADS>
__device__ __forceinline__ void tile_rows_out(const uint8_t* tile, const uint8_t* noise, const TileOut& o, int tid)
{
    constexpr int H = THREADS / kTileRows, B = TC / 32 / H, P = Src<DT>::kPer, C = 32 / P;
    static_assert(H * B * 32 == TC, "row parts");
    const int r = tid & 127, part = tid >> 7;
    if (r >= o.scale_rows) return;
    uint32_t bytes = 0;
#pragma unroll
    for (int b = 0; b < B; ++b) {
        const int blk = part * B + b;
        float x[32];
        uint32_t nz[8] = {};
#pragma unroll
        for (int c = 0; c < C; ++c)
            Src<DT>::unpack(*reinterpret_cast<const uint4*>(tile + tile_chunk<DT, TC>(r, blk * C + c)), x + c * P);
        if (NOISE) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const uint4 v = *reinterpret_cast<const uint4*>(noise + noise_chunk<TC>(r, blk * 2 + c));
                nz[4 * c] = v.x; nz[4 * c + 1] = v.y; nz[4 * c + 2] = v.z; nz[4 * c + 3] = v.w;
            }
        }
        uint32_t s;
        const uint4 codes = encode_block<NOISE>(x, nz, &s);
        bytes |= s << (8 * b);
        if (r < o.rows) *reinterpret_cast<uint4*>(o.codes + r * o.pitch + blk * 16) = codes;
    }
    uint8_t* at = o.scales + 4 * r + part * B;
    if (B == 4) *reinterpret_cast<uint32_t*>(at) = bytes;
    else if (B == 2) *reinterpret_cast<uint16_t*>(at) = static_cast<uint16_t>(bytes);
    else *at = static_cast<uint8_t>(bytes);
}

// Blocks down the columns, written transposed: a task is one block of 32 rows
// of the W columns that share a 32-bit word (W = 2 for 16-bit storage).
template <int DT, int TC, bool NOISE, int THREADS>
__device__ __forceinline__ void tile_cols_out(const uint8_t* tile, const uint8_t* noise, const TileOut& o, int tid)
{
    constexpr int W = 4 / Src<DT>::kBytes, kAcross = TC / W, kTasks = kAcross * 4;
    for (int t = tid; t < kTasks; t += THREADS) {
        const int c0 = (t % kAcross) * W, rb = t / kAcross;
        if (c0 >= o.scale_cols) continue;
        float x[W][32];
        uint32_t nz[W][8] = {};
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const int r = rb * 32 + i;
            constexpr int P = Src<DT>::kPer;
            const uint32_t w = *reinterpret_cast<const uint32_t*>(
                tile + tile_chunk<DT, TC>(r, c0 / P) + (c0 % P) * Src<DT>::kBytes);
            if constexpr (W == 1) {
                x[0][i] = __uint_as_float(w);
            } else {
                const float2 f = Src<DT>::pair(w);
                x[0][i] = f.x;
                x[W - 1][i] = f.y;
            }
            if (NOISE) {
                const uint8_t* np = noise + noise_chunk<TC>(r, c0 / 16) + c0 % 16;
#pragma unroll
                for (int j = 0; j < W; ++j) nz[j][i / 4] |= static_cast<uint32_t>(np[j]) << (8 * (i & 3));
            }
        }
#pragma unroll
        for (int j = 0; j < W; ++j) {
            if (c0 + j >= o.scale_cols) break;
            uint32_t s;
            const uint4 codes = encode_block<NOISE>(x[j], nz[j], &s);
            if (c0 + j < o.cols) *reinterpret_cast<uint4*>(o.codes_t + (c0 + j) * o.pitch_t + rb * 16) = codes;
            o.scales_t[4 * (c0 + j) + rb] = static_cast<uint8_t>(s);
        }
    }
}

// ---------------------------------------------------------------------------
// Ragged groups
// ---------------------------------------------------------------------------
constexpr int kMaxGroups = 1024;

// From the device offsets of `groups` row ranges over `rows` rows: start[e] =
// the clamped, non-decreasing offsets (groups + 1 of them, so that no input
// sends an access out of range), and first[e] = the number of tiles of `unit`
// rows in the groups before e, times `across`.  Called by the whole block;
// ends with a barrier.
__device__ __forceinline__ void ragged_table(const int32_t* offsets, int groups, int64_t rows, int unit,
                                             int across, int32_t* start, int32_t* first, int tid, int threads)
{
    for (int i = tid; i <= groups; i += threads)
        start[i] = static_cast<int32_t>(min(static_cast<int64_t>(max(offsets[i], 0)), rows));
    __syncthreads();
    if (tid < 32) {
        int32_t top = 0;
        for (int base = 0; base <= groups; base += 32) {
            const int i = base + tid;
            int32_t v = i <= groups ? start[i] : 0;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int32_t o = __shfl_up_sync(0xFFFFFFFFu, v, d);
                if (tid >= d) v = max(v, o);
            }
            v = max(v, top);
            if (i <= groups) start[i] = v;
            top = __shfl_sync(0xFFFFFFFFu, v, 31);
        }
        __syncwarp();
        int32_t sum = 0;
        for (int base = 0; base <= groups; base += 32) {
            const int i = base + tid;
            const int32_t n = i < groups ? (start[i + 1] - start[i] + unit - 1) / unit * across : 0;
            int32_t v = n;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int32_t o = __shfl_up_sync(0xFFFFFFFFu, v, d);
                if (tid >= d) v += o;
            }
            if (i <= groups) first[i] = sum + v - n;
            sum += __shfl_sync(0xFFFFFFFFu, v, 31);
        }
    }
    __syncthreads();
}

// The group that holds tile t (first[e] <= t < first[e + 1]).
__device__ __forceinline__ int group_of(const int32_t* first, int groups, int32_t t)
{
    int lo = 0, hi = groups - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= t) lo = mid; else hi = mid - 1;
    }
    return lo;
}

}  // namespace
}  // namespace opt2s
