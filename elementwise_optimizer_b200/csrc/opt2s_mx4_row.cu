// opt2s_mx4_row.cu -- one row times a 4-bit weight, in one launch.
//
// A product with one token reads every weight once and computes next to
// nothing: it is bound by how soon the loads are under way.  Each warp takes
// two weight rows; a lane loads whole blocks (16 bytes of codes), so a warp's
// load is 512 contiguous bytes of a row, and the first of them are issued
// before the CTA quantises the token into shared memory itself, which saves
// the quantisation's launch and its round trip.  (Every CTA repeats that: 0.7
// us of instructions for one row against 8,192 rows of 2,048, but 2.9 us for
// four, more than the tensor-core path's second launch; so one row only.)
// Codes are multiplied as integers: twice an E2M1 magnitude is 0, 1, 2, 3, 4,
// 6, 8 or 12, which a byte permute looks up four at a time, and a block's sum
// of products is exact in 32-bit integers (at most 32 * 144).  Blocks are added
// in fp32, in a fixed order.
//
// 1 x 8,192 x 2,048 takes 5.6 us, against 8.4 us for the quantisation and the
// product on the tensor cores; 1 x 2,048 x 2,048 3.1 us against 8.2 us.
#include "opt2s_mx4.cuh"

namespace opt2s {
namespace {

constexpr int kRowThreads = 256, kWarps = kRowThreads / 32, R = 2;      // R: weight rows a warp

// Four codes of a word (the low or the high half) as signed bytes, doubled.
__device__ __forceinline__ uint32_t signed_bytes(uint32_t w, bool high)
{
    const uint32_t v = (w & 0x77777777u) >> (high ? 16 : 0);
    const uint32_t pos = __byte_perm(0x03020100u, 0x0C080604u, v);
    const uint32_t neg = __byte_perm(0xFDFEFF00u, 0xF4F8FAFCu, v);
    uint32_t sign;                       // 0xFF where the code's top bit is set
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(sign) : "r"(w << 4), "r"(w), "r"(high ? 0xFBEAu : 0xD9C8u));
    return (pos & ~sign) | (neg & sign);
}

// acc + x * 2^(ew - 127) * 2^(ex - 127) / 4 for an integer sum of doubled
// codes x.  The product is exact unless it leaves fp32's range, so the fused
// addition rounds once, as the separate one would.
__device__ __forceinline__ float add_scaled(float acc, int x, uint32_t ew, uint32_t ex)
{
    const int e = static_cast<int>(ew + ex) - 256;
    if (__builtin_expect(max(ew, ex) < 255u && static_cast<uint32_t>(e + 126) < 254u, 1))
        return __fmaf_rn(static_cast<float>(x), __uint_as_float(static_cast<uint32_t>(e + 127) << 23), acc);
    if (max(ew, ex) == 255u) return __uint_as_float(0x7FC00000u);
    // rare: in two factors, so that neither leaves fp32's range where the product does not
    auto power = [](int k) { return k >= -126 ? __uint_as_float(static_cast<uint32_t>(k + 127) << 23) : __uint_as_float(0x00800000u >> (-126 - k)); };
    const int e1 = e >> 1;
    return __fadd_rn(acc, __fmul_rn(__fmul_rn(static_cast<float>(x), power(e1)), power(e - e1)));
}

template <int DT> __device__ __forceinline__ float load_x(const void* p, int64_t i)
{
    if (DT == kF32) return static_cast<const float*>(p)[i];
    if (DT == kF16) return __half2float(static_cast<const __half*>(p)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
template <int DT> __device__ __forceinline__ void store_d(void* p, int64_t i, float x)
{
    if (DT == kF32) static_cast<float*>(p)[i] = x;
    else if (DT == kF16) static_cast<__half*>(p)[i] = __float2half_rn(x);
    else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(x);
}

// Quantises the row into shared memory: a block's 32 doubled codes as signed
// bytes, and its scale byte.  A thread takes four elements, eight neighbouring
// threads a block.
template <int DT>
__device__ __forceinline__ void quantize_row(const Mx4RowArgs& a, int blocks, uint32_t* xb, uint8_t* xs, int tid)
{
    constexpr int U = 4;                             // loads in flight a thread
    const int quads = blocks * 8;                    // a multiple of 32: whole warps stay together
    for (int q0 = tid; q0 < quads; q0 += U * kRowThreads) {
        float x[U][4] = {};
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = (q0 + u * kRowThreads) * 4;
            if (a.vec && c + 4 <= a.cols) {
                if constexpr (DT == kF32) {
                    const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(a.x) + c);
                    x[u][0] = v.x; x[u][1] = v.y; x[u][2] = v.z; x[u][3] = v.w;
                } else {
                    const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.x) + c);
                    x[u][0] = Src<DT>::half(v.x, 0); x[u][1] = Src<DT>::half(v.x, 1);
                    x[u][2] = Src<DT>::half(v.y, 0); x[u][3] = Src<DT>::half(v.y, 1);
                }
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (c + k < a.cols) x[u][k] = load_x<DT>(a.x, c + k);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int q = q0 + u * kRowThreads;
            if (q >= quads) break;
            uint32_t amax = max(max(abs_bits(x[u][0]), abs_bits(x[u][1])), max(abs_bits(x[u][2]), abs_bits(x[u][3])));
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, d));
            const uint32_t s = scale_byte(amax);
            const float inv = inverse_scale(s);
            const uint32_t w = encode8(__fmul_rn(x[u][0], inv), __fmul_rn(x[u][1], inv), __fmul_rn(x[u][2], inv),
                                       __fmul_rn(x[u][3], inv), 0.0f, 0.0f, 0.0f, 0.0f);
            xb[q] = signed_bytes(s == 255u ? 0u : w, false);
            if ((q & 7) == 0) xs[q >> 3] = static_cast<uint8_t>(s);
        }
    }
}

// grid: weight rows / 16.
template <int DT, int OUT>
__global__ void __launch_bounds__(kRowThreads, 4) mx4_row_kernel(const Mx4RowArgs a)
{
    extern __shared__ __align__(16) uint8_t smem[];
    const int blocks = static_cast<int>((a.cols + 127) / 128 * 4);
    uint4* xb = reinterpret_cast<uint4*>(smem);      // [blocks][2]
    uint8_t* xs = smem + blocks * 32;                // [blocks]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kWarps * R + warp * R;
    const int64_t pitch = static_cast<int64_t>(blocks) * 16, group = a.w_sf_rows * 4;
    const uint8_t* codes = a.codes + n0 * pitch;
    const uint8_t* scales = a.scales + n0 * 4;
    struct Loaded { uint4 w[R]; uint32_t s[R]; };
    auto load = [&](int b, Loaded& v) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool in = b < blocks && n0 + r < a.w_rows;
            v.w[r] = in ? *reinterpret_cast<const uint4*>(codes + r * pitch + b * 16) : make_uint4(0, 0, 0, 0);
            v.s[r] = in ? scales[(b >> 2) * group + r * 4 + (b & 3)] : 0u;
        }
    };
    Loaded one, two;
    load(lane, one);
    load(lane + 32, two);
    quantize_row<DT>(a, blocks, reinterpret_cast<uint32_t*>(xb), xs, tid);
    __syncthreads();
    float acc[R] = {};
    for (int b = lane; b < blocks; b += 32) {
        const Loaded v = one;
        one = two;
        load(b + 64, two);
        const uint4 x0 = xb[b * 2], x1 = xb[b * 2 + 1];
        const uint32_t ex = xs[b];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            int d = __dp4a(static_cast<int>(signed_bytes(v.w[r].x, false)), static_cast<int>(x0.x), 0);
            d = __dp4a(static_cast<int>(signed_bytes(v.w[r].x, true)), static_cast<int>(x0.y), d);
            d = __dp4a(static_cast<int>(signed_bytes(v.w[r].y, false)), static_cast<int>(x0.z), d);
            d = __dp4a(static_cast<int>(signed_bytes(v.w[r].y, true)), static_cast<int>(x0.w), d);
            d = __dp4a(static_cast<int>(signed_bytes(v.w[r].z, false)), static_cast<int>(x1.x), d);
            d = __dp4a(static_cast<int>(signed_bytes(v.w[r].z, true)), static_cast<int>(x1.y), d);
            d = __dp4a(static_cast<int>(signed_bytes(v.w[r].w, false)), static_cast<int>(x1.z), d);
            d = __dp4a(static_cast<int>(signed_bytes(v.w[r].w, true)), static_cast<int>(x1.w), d);
            acc[r] = add_scaled(acc[r], d, v.s[r], ex);
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float v = acc[r];
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
        if (lane == 0 && n0 + r < a.w_rows) store_d<OUT>(a.d, n0 + r, v);
    }
}

template <int DT, int OUT>
cudaError_t launch_row_as(const Mx4RowArgs& a, cudaStream_t stream)
{
    const int bytes = static_cast<int>((a.cols + 127) / 128 * 4 * 33);      // at most 33 KiB
    const unsigned grid = static_cast<unsigned>((a.w_rows + kWarps * R - 1) / (kWarps * R));
    mx4_row_kernel<DT, OUT><<<grid, kRowThreads, bytes, stream>>>(a);
    return cudaGetLastError();
}

template <int DT>
cudaError_t launch_row_out(const Mx4RowArgs& a, int out, cudaStream_t stream)
{
    if (out == kF32) return launch_row_as<DT, kF32>(a, stream);
    if (out == kF16) return launch_row_as<DT, kF16>(a, stream);
    return launch_row_as<DT, kBF16>(a, stream);
}

}  // namespace

cudaError_t launch_mx4_row(const Mx4RowArgs& a, int in, int out, cudaStream_t stream)
{
    if (in == kF32) return launch_row_out<kF32>(a, out, stream);
    if (in == kF16) return launch_row_out<kF16>(a, out, stream);
    return launch_row_out<kBF16>(a, out, stream);
}

}  // namespace opt2s
