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

// A 32-byte store to a 32-byte aligned address.
__device__ __forceinline__ void store32(void* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t e, uint32_t f,
                                        uint32_t g, uint32_t h)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 :: "l"(p), "r"(a), "r"(b), "r"(c), "r"(d), "r"(e), "r"(f), "r"(g), "r"(h) : "memory");
}

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

// Eight E2M1 codes in a word, x[0] in the lowest nibble: nearest, ties to
// even, magnitudes above 6 saturated.
__device__ __forceinline__ uint32_t encode8(float x0, float x1, float x2, float x3, float x4, float x5, float x6,
                                            float x7)
{
    uint32_t r;
    asm("{\n\t"
        ".reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t"
        "}" : "=r"(r) : "f"(x0), "f"(x1), "f"(x2), "f"(x3), "f"(x4), "f"(x5), "f"(x6), "f"(x7));
    return r;
}

// Stochastic rounding of a scaled element (|x| < 8) with the byte r: code c or
// c + 1, the upper one when |x| lies more than (r + 0.5)/256 of the way from
// c's magnitude to the next.  The complement of the code is the top byte of the
// result (8 for what pack_noise saturates to 7); `noise` holds four random
// bytes, `j` says which one is this element's.
//
// With a = |x|, y = a + max(a, 1) is 1 + a below 1 and 2 a from there on: its
// exponent and first mantissa bit count the codes, and the other 22 bits are
// the way to the next.  Shifted left by two, the code (plus 254) fills the top
// byte and the way the 24 bits under it, and the comparison is the carry of
// adding 2^24 - 1 - 256^2 r - 2^15.  The complement of that sum is one multiply
// and add with the random byte as it is.  The sum 1 + a is rounded up, which
// cannot take the way past a threshold (a multiple of 2^13 units of the last
// bit) that it had not passed, so the comparison is exact for every x.
__device__ __forceinline__ uint32_t noise_code(float x, uint32_t noise, int j)
{
    const float a = fabsf(x);
    const float y = __fadd_ru(a, fmaxf(a, 1.0f));
    const uint32_t c = __byte_perm(noise, 0x00FD8000u, 0x6054u | static_cast<uint32_t>(j) << 8);
    return c - 4u * __float_as_uint(y);
}

// The top bytes of four words as one word.
__device__ __forceinline__ uint32_t top_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    return __byte_perm(__byte_perm(a, b, 0x0073), __byte_perm(c, d, 0x0073), 0x5410);
}

// The signs of eight elements: the top bits of `even`'s bytes are those of
// elements 0, 2, 4 and 6, of `odd`'s those of 1, 3, 5 and 7.
struct Signs { uint32_t even, odd; };

// Eight codes in a word from noise_code's results and the signs.
__device__ __forceinline__ uint32_t pack_noise(const uint32_t (&t)[8], Signs s)
{
    const uint32_t even = top_bytes(t[0], t[2], t[4], t[6]), odd = top_bytes(t[1], t[3], t[5], t[7]) << 4;
    uint32_t w = ~((even & 0x0F0F0F0Fu) | (odd & 0xF0F0F0F0u));
    w -= w >> 3 & 0x11111111u;                      // 8 to 7
    const uint32_t sign = (s.even >> 4 & 0x0F0F0F0Fu) | (s.odd & 0xF0F0F0F0u);
    return (w & 0x77777777u) | (sign & 0x88888888u);
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
// chunk; element i of a run of words; for the 16-bit types one half of a
// word; the fp32 bits of a magnitude; the signs of eight elements.
template <int DT> struct Src;
template <> struct Src<kF32> {
    static constexpr int kPer = 4, kBytes = 4;
    __device__ static float element(const uint32_t* w, int i) { return __uint_as_float(w[i]); }
    __device__ static float half(uint32_t w, int) { return __uint_as_float(w); }
    __device__ static uint32_t magnitude(uint32_t bits) { return bits; }
    __device__ static Signs signs(const uint32_t* w)
    {
        return {top_bytes(w[0], w[2], w[4], w[6]), top_bytes(w[1], w[3], w[5], w[7])};
    }
    __device__ static Signs signs_down(const uint32_t* w, int) { return signs(w); }
};
struct Halves {
    // eight elements in four words
    __device__ static Signs signs(const uint32_t* w)
    {
        const uint32_t a = __byte_perm(w[0], w[1], 0x7531), b = __byte_perm(w[2], w[3], 0x7531);
        return {__byte_perm(a, b, 0x6420), __byte_perm(a, b, 0x7531)};
    }
    // half j of eight words (both halves share the first permutes)
    __device__ static Signs signs_down(const uint32_t* w, int j)
    {
        const uint32_t pick = j ? 0x7531 : 0x6420;
        return {__byte_perm(__byte_perm(w[0], w[2], 0x7531), __byte_perm(w[4], w[6], 0x7531), pick),
                __byte_perm(__byte_perm(w[1], w[3], 0x7531), __byte_perm(w[5], w[7], 0x7531), pick)};
    }
};
template <> struct Src<kBF16> : Halves {
    static constexpr int kPer = 8, kBytes = 2;
    __device__ static float half(uint32_t w, int j) { return __uint_as_float(j ? w & 0xFFFF0000u : w << 16); }
    __device__ static float element(const uint32_t* w, int i) { return half(w[i / 2], i & 1); }
    __device__ static uint32_t magnitude(uint32_t bits) { return bits << 16; }
};
template <> struct Src<kF16> : Halves {
    static constexpr int kPer = 8, kBytes = 2;
    __device__ static float half(uint32_t w, int j)
    {
        const __half2 h = *reinterpret_cast<const __half2*>(&w);
        return j ? __high2float(h) : __low2float(h);
    }
    __device__ static float element(const uint32_t* w, int i) { return half(w[i / 2], i & 1); }
    __device__ static uint32_t magnitude(uint32_t bits) { return abs_bits(half(bits, 0)); }
};

// The largest magnitudes of words of a 16-bit type, each half on its own: as
// signed numbers the positive ones win, as unsigned ones the negative.
struct Amax {
    uint32_t pos = 0, any = 0;
    __device__ void add(uint32_t v, uint32_t w)
    {
        pos = __vimax3_s16x2(pos, v, w);
        any = __vimax3_u16x2(any, v, w);
    }
    __device__ uint32_t halves() const { return __vmaxu2(pos, any & 0x7FFF7FFFu); }
};

// One word of a block's codes: eight elements x times 2^-e.  noise(i) and
// at(i) give element i's random byte as noise_code takes it, signs() theirs.
template <bool NOISE, typename Get, typename Noise, typename At, typename SignsOf>
__device__ __forceinline__ uint32_t encode_word(uint32_t scale, float inv, Get get, Noise noise, At at, SignsOf signs)
{
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __fmul_rn(get(i), inv);
    uint32_t w;
    if (NOISE) {
        uint32_t t[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = noise_code(x[i], noise(i), at(i));
        w = pack_noise(t, signs());
    } else {
        w = encode8(x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7]);
    }
    return scale == 255u ? 0u : w;               // a NaN block's codes are 0
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
    using S = Src<DT>;
    constexpr int H = THREADS / kTileRows, B = TC / 32 / H, C = 2 * S::kBytes;     // 16-byte chunks a block
    static_assert(H * B * 32 == TC, "row parts");
    const int r = tid & 127, part = tid >> 7;
    if (r >= o.scale_rows) return;
    uint32_t bytes = 0;
#pragma unroll
    for (int b = 0; b < B; ++b) {
        const int blk = part * B + b;
        uint32_t w[4 * C], nz[8] = {}, amax = 0;
        Amax most;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const uint4 v = *reinterpret_cast<const uint4*>(tile + tile_chunk<DT, TC>(r, blk * C + c));
            w[4 * c] = v.x; w[4 * c + 1] = v.y; w[4 * c + 2] = v.z; w[4 * c + 3] = v.w;
        }
        if (NOISE) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const uint4 v = *reinterpret_cast<const uint4*>(noise + noise_chunk<TC>(r, blk * 2 + c));
                nz[4 * c] = v.x; nz[4 * c + 1] = v.y; nz[4 * c + 2] = v.z; nz[4 * c + 3] = v.w;
            }
        }
#pragma unroll
        for (int i = 0; i < 4 * C; i += 2) {
            if (S::kBytes == 2) most.add(w[i], w[i + 1]);
            else amax = max(amax, max(w[i] & 0x7FFFFFFFu, w[i + 1] & 0x7FFFFFFFu));
        }
        if (S::kBytes == 2) amax = S::magnitude(max(most.halves() & 0xFFFFu, most.halves() >> 16));
        const uint32_t s = scale_byte(amax);
        const float inv = inverse_scale(s);
        uint32_t codes[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            codes[k] = encode_word<NOISE>(
                s, inv, [&](int i) { return S::element(w, 8 * k + i); }, [&](int i) { return nz[2 * k + i / 4]; },
                [](int i) { return i & 3; }, [&] { return S::signs(w + 8 * k / (4 / S::kBytes)); });
        bytes |= s << (8 * b);
        if (r < o.rows)
            *reinterpret_cast<uint4*>(o.codes + r * o.pitch + blk * 16) = make_uint4(codes[0], codes[1], codes[2], codes[3]);
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
    using S = Src<DT>;
    constexpr int W = 4 / S::kBytes, P = S::kPer, kAcross = TC / W, kTasks = kAcross * 4;
    for (int t = tid; t < kTasks; t += THREADS) {
        const int c0 = (t % kAcross) * W, rb = t / kAcross;
        if (c0 >= o.scale_cols) continue;
        uint32_t w[32], amax = 0;
        Amax most;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            w[i] = *reinterpret_cast<const uint32_t*>(tile + tile_chunk<DT, TC>(rb * 32 + i, c0 / P) + (c0 % P) * S::kBytes);
            if (W == 1) amax = max(amax, w[i] & 0x7FFFFFFFu);
            else if (i & 1) most.add(w[i - 1], w[i]);
        }
        if (W == 2) amax = most.halves();
        uint32_t s[W], codes[W][4];
        float inv[W];
#pragma unroll
        for (int j = 0; j < W; ++j) {
            s[j] = scale_byte(W == 2 ? S::magnitude(j ? amax >> 16 : amax & 0xFFFFu) : amax);
            inv[j] = inverse_scale(s[j]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t nz[8] = {};
            if (NOISE) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint8_t* np = noise + noise_chunk<TC>(rb * 32 + 8 * k + i, c0 / 16) + c0 % 16;
                    nz[i] = W == 2 ? static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(np)) : static_cast<uint32_t>(*np);
                }
            }
#pragma unroll
            for (int j = 0; j < W; ++j)
                codes[j][k] = encode_word<NOISE>(
                    s[j], inv[j], [&](int i) { return W == 2 ? S::half(w[8 * k + i], j) : __uint_as_float(w[8 * k + i]); },
                    [&](int i) { return nz[i]; }, [&](int) { return j; }, [&] { return S::signs_down(w + 8 * k, j); });
        }
#pragma unroll
        for (int j = 0; j < W; ++j) {
            if (c0 + j >= o.scale_cols) break;
            if (c0 + j < o.cols)
                *reinterpret_cast<uint4*>(o.codes_t + (c0 + j) * o.pitch_t + rb * 16) =
                    make_uint4(codes[j][0], codes[j][1], codes[j][2], codes[j][3]);
            o.scales_t[4 * (c0 + j) + rb] = static_cast<uint8_t>(s[j]);
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
