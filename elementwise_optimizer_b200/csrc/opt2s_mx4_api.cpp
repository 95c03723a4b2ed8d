// opt2s_mx4_api.cpp -- the C ABI of the microscaled 4-bit operators
// (include/opt2s.h): argument validation and launches.  Nothing here keeps
// state: a call's tables travel as kernel arguments.
#include <cstdint>
#include <new>
#include <vector>

#include <cuda_runtime.h>

#include "opt2s.h"
#include "opt2s_internal.h"

#define OPT2S_API extern "C" __attribute__((visibility("default")))

using opt2s::Range;

namespace {

constexpr int64_t kMaxIndex = int64_t{1} << 30;     // rows and columns that tile indices may reach

int64_t up(int64_t x, int64_t k) { return (x + k - 1) / k * k; }

bool good_dtype(int32_t d) { return d == OPT2S_F32 || d == OPT2S_F16 || d == OPT2S_BF16; }

bool good_sizes(int64_t slabs, int64_t rows, int64_t cols)
{
    if (slabs < 1 || rows < 0 || cols < 1 || slabs > kMaxIndex || rows > kMaxIndex || cols > kMaxIndex) return false;
    return slabs * up(rows, 4) <= kMaxIndex;
}

Range span(const void* p, int64_t bytes, bool written)
{
    const auto lo = reinterpret_cast<uintptr_t>(p);
    return {lo, lo + static_cast<uintptr_t>(bytes), written};
}

// Whether n things `stride` elements apart span more than any address space.
bool too_far(int64_t n, int64_t stride) { return n > 1 && stride > (int64_t{1} << 54) / (n - 1); }

bool aligned(const void* p, uintptr_t k) { return reinterpret_cast<uintptr_t>(p) % k == 0; }

// Checks a matrix and appends its two ranges (none when it has no rows).
int matrix_ranges(const opt2s_mx4* m, bool written, Range* out, size_t* n)
{
    if (!m || !good_sizes(m->slabs, m->rows, m->cols)) return OPT2S_ERR_INVALID_ARG;
    if (m->rows == 0) return OPT2S_OK;
    if (!m->codes || !m->scales || !aligned(m->codes, 16) || !aligned(m->scales, 16)) return OPT2S_ERR_INVALID_ARG;
    out[(*n)++] = span(m->codes, opt2s_mx4_code_bytes(m->slabs, m->rows, m->cols), written);
    out[(*n)++] = span(m->scales, opt2s_mx4_scale_bytes(m->slabs, m->rows, m->cols), written);
    return OPT2S_OK;
}

int good_groups(const int32_t* offsets, int32_t groups)
{
    if (!offsets || groups < 1 || groups > OPT2S_MX4_MAX_GROUPS || !aligned(offsets, 4)) return OPT2S_ERR_INVALID_ARG;
    return OPT2S_OK;
}

opt2s::Mx4Operand operand(const opt2s_mx4* m)
{
    return {m->codes, m->scales, m->slabs * m->rows, up(m->cols, 128) / 2, m->slabs * up(m->rows, 4)};
}

// What the three products have in common.  d_rows rows of d_cols columns.
int product(const opt2s_mx4* a, const opt2s_mx4* b, const int32_t* offsets, int32_t groups, bool ragged, void* d,
            int64_t d_rows, int64_t ldd, int32_t dtype, int32_t accumulate, int32_t fill_rest, cudaStream_t stream)
{
    Range r[6];
    size_t n = 0;
    int st = matrix_ranges(a, false, r, &n);
    if (st == OPT2S_OK) st = matrix_ranges(b, false, r, &n);
    if (st != OPT2S_OK) return st;
    if (!good_dtype(dtype) || (accumulate != 0 && accumulate != 1) || (fill_rest != 0 && fill_rest != 1))
        return OPT2S_ERR_INVALID_ARG;
    if (a->cols != b->cols || a->slabs != 1 || (accumulate && fill_rest)) return OPT2S_ERR_INVALID_ARG;
    if (ldd < b->rows || ldd > (int64_t{1} << 40) || too_far(d_rows, ldd)) return OPT2S_ERR_INVALID_ARG;
    if (d_rows == 0 || b->rows == 0) return OPT2S_OK;
    const int es = opt2s::elem_bytes(dtype);
    if (!d || !aligned(d, es)) return OPT2S_ERR_INVALID_ARG;
    r[n++] = span(d, ((d_rows - 1) * ldd + b->rows) * es, true);
    if (offsets) r[n++] = span(offsets, (static_cast<int64_t>(groups) + 1) * 4, false);
    if ((st = opt2s::overlap_status(r, n)) != OPT2S_OK) return st;
    opt2s::Mx4GemmArgs g{};
    g.d = d;
    g.ldd = ldd;
    g.offsets = offsets;
    g.groups = groups;
    g.x_rows = ragged ? a->cols - 128 * static_cast<int64_t>(groups) : a->rows;
    g.w_rows = b->rows;
    g.w_sf_rows = up(b->rows, 4);
    g.p_rows = a->rows;
    g.d_rows = d_rows;
    g.d_cols = b->rows;
    g.k64 = static_cast<int32_t>((a->cols + 63) / 64);
    g.ragged_k = ragged;
    g.accumulate = accumulate;
    g.fill_rest = fill_rest;
    g.dtype = dtype;
    g.vec = aligned(d, 32) && ldd * es % 32 == 0;
    const cudaError_t e = opt2s::launch_mx4_gemm(g, {operand(a), operand(b)}, stream);
    if (e == cudaErrorInvalidConfiguration) return OPT2S_ERR_TOO_LARGE;
    if (e != cudaSuccess) return opt2s::record_cuda_error(e);
    opt2s::count_launches(1);
    return OPT2S_OK;
}

}  // namespace

OPT2S_API int64_t opt2s_mx4_code_bytes(int64_t slabs, int64_t rows, int64_t cols)
{
    return good_sizes(slabs, rows, cols) ? slabs * rows * (up(cols, 128) / 2) : -1;
}

OPT2S_API int64_t opt2s_mx4_scale_bytes(int64_t slabs, int64_t rows, int64_t cols)
{
    return good_sizes(slabs, rows, cols) ? up(cols, 128) / 128 * slabs * up(rows, 4) * 4 : -1;
}

OPT2S_API int opt2s_mx4_quantize(const opt2s_mx4_source* src, const opt2s_mx4* q, const opt2s_mx4* qt,
                                 const int32_t* offsets, int32_t groups, cudaStream_t stream)
{
    OPT2S_RANGE("opt2s_mx4_quantize");
    if (!src || src->reserved != 0 || !good_dtype(src->dtype)) return OPT2S_ERR_INVALID_ARG;
    if (!good_sizes(src->slabs, src->rows, src->cols) || src->row_stride < 0 || src->slab_stride < 0)
        return OPT2S_ERR_INVALID_ARG;
    if (src->row_stride > (int64_t{1} << 40) || src->slab_stride > (int64_t{1} << 40)) return OPT2S_ERR_INVALID_ARG;
    if (too_far(src->rows, src->row_stride) || too_far(src->slabs, src->slab_stride)) return OPT2S_ERR_INVALID_ARG;
    if (!offsets && groups != 0) return OPT2S_ERR_INVALID_ARG;
    if (offsets && (good_groups(offsets, groups) != OPT2S_OK || src->slabs != 1)) return OPT2S_ERR_INVALID_ARG;
    Range r[7];
    size_t n = 0;
    int st = OPT2S_OK;
    if (q) {
        if (q->slabs != src->slabs || q->rows != src->rows || q->cols != src->cols) return OPT2S_ERR_INVALID_ARG;
        if ((st = matrix_ranges(q, true, r, &n)) != OPT2S_OK) return st;
    }
    const int64_t t_cols = offsets ? up(src->rows, 128) + 128 * static_cast<int64_t>(groups) : src->rows;
    if (qt) {
        if (qt->slabs != src->slabs || qt->rows != src->cols || qt->cols != t_cols) return OPT2S_ERR_INVALID_ARG;
        if ((st = matrix_ranges(qt, true, r, &n)) != OPT2S_OK) return st;
    }
    const int64_t row_tiles = up(t_cols, 128) / 128;
    if (row_tiles > 65535 || src->slabs > 65535) return OPT2S_ERR_TOO_LARGE;
    if (row_tiles == 0 || (!q && !qt)) return OPT2S_OK;
    if (src->rows > 0) {
        const int es = opt2s::elem_bytes(src->dtype);
        if (!src->x || !aligned(src->x, es)) return OPT2S_ERR_INVALID_ARG;
        r[n++] = span(src->x, ((src->slabs - 1) * src->slab_stride + (src->rows - 1) * src->row_stride + src->cols) * es,
                      false);
        if (src->noise) r[n++] = span(src->noise, src->slabs * src->rows * src->cols, false);
    }
    if (offsets) r[n++] = span(offsets, (static_cast<int64_t>(groups) + 1) * 4, false);
    if ((st = opt2s::overlap_status(r, n)) != OPT2S_OK) return st;
    opt2s::Mx4QuantArgs a{};
    const int es = opt2s::elem_bytes(src->dtype);
    a.x = src->x;
    a.noise = src->noise;
    a.slabs = src->slabs;
    a.rows = src->rows;
    a.cols = src->cols;
    a.row_stride = src->row_stride;
    a.slab_stride = src->slab_stride;
    if (q) { a.codes = q->codes; a.scales = q->scales; }
    if (qt) { a.codes_t = qt->codes; a.scales_t = qt->scales; }
    a.offsets = offsets;
    a.groups = groups;
    a.vec = src->rows > 0 && aligned(src->x, 16) && src->row_stride * es % 16 == 0 && src->slab_stride * es % 16 == 0;
    a.noise_vec = src->rows > 0 && aligned(src->noise, 16) && src->cols % 16 == 0;
    const cudaError_t e = opt2s::launch_mx4_quantize(a, src->dtype, row_tiles, stream);
    if (e != cudaSuccess) return opt2s::record_cuda_error(e);
    opt2s::count_launches(1);
    return OPT2S_OK;
}

OPT2S_API int opt2s_mx4_dequantize(const opt2s_mx4* q, void* out, int32_t dtype, cudaStream_t stream)
{
    OPT2S_RANGE("opt2s_mx4_dequantize");
    Range r[3];
    size_t n = 0;
    int st = matrix_ranges(q, false, r, &n);
    if (st != OPT2S_OK) return st;
    if (!good_dtype(dtype)) return OPT2S_ERR_INVALID_ARG;
    if (q->rows == 0) return OPT2S_OK;
    if (q->slabs > 65535 || q->cols > 65535 * int64_t{4096}) return OPT2S_ERR_TOO_LARGE;
    const int es = opt2s::elem_bytes(dtype);
    if (!out || !aligned(out, es)) return OPT2S_ERR_INVALID_ARG;
    r[n++] = span(out, q->slabs * q->rows * q->cols * es, true);
    if ((st = opt2s::overlap_status(r, n)) != OPT2S_OK) return st;
    const opt2s::Mx4DequantArgs a{q->codes, q->scales, out, q->slabs, q->rows, q->cols,
                                  aligned(out, 32) && q->cols % 16 == 0};
    const cudaError_t e = opt2s::launch_mx4_dequantize(a, dtype, stream);
    if (e != cudaSuccess) return opt2s::record_cuda_error(e);
    opt2s::count_launches(1);
    return OPT2S_OK;
}

OPT2S_API int opt2s_mx4_matmul(const opt2s_mx4* a, const opt2s_mx4* b, void* d, int64_t ldd, int32_t dtype,
                               int32_t accumulate, cudaStream_t stream)
{
    OPT2S_RANGE("opt2s_mx4_matmul");
    if (!a || !b || b->slabs != 1) return OPT2S_ERR_INVALID_ARG;
    return product(a, b, nullptr, 0, false, d, a->rows, ldd, dtype, accumulate, 0, stream);
}

OPT2S_API int opt2s_mx4_matmul_grouped(const opt2s_mx4* a, const opt2s_mx4* b, const int32_t* offsets,
                                       int32_t groups, void* d, int64_t ldd, int32_t dtype, int32_t accumulate,
                                       int32_t fill_rest, cudaStream_t stream)
{
    OPT2S_RANGE("opt2s_mx4_matmul_grouped");
    if (!a || !b || good_groups(offsets, groups) != OPT2S_OK || b->slabs != groups) return OPT2S_ERR_INVALID_ARG;
    return product(a, b, offsets, groups, false, d, a->rows, ldd, dtype, accumulate, fill_rest, stream);
}

OPT2S_API int opt2s_mx4_matmul_ragged(const opt2s_mx4* a, const opt2s_mx4* b, const int32_t* offsets,
                                      int32_t groups, void* d, int64_t ldd, int32_t dtype, int32_t accumulate,
                                      cudaStream_t stream)
{
    OPT2S_RANGE("opt2s_mx4_matmul_ragged");
    if (!a || !b || good_groups(offsets, groups) != OPT2S_OK || b->slabs != 1) return OPT2S_ERR_INVALID_ARG;
    if (a->cols < 128 * static_cast<int64_t>(groups) || a->cols % 128 != 0) return OPT2S_ERR_INVALID_ARG;
    if (groups * a->rows > kMaxIndex) return OPT2S_ERR_TOO_LARGE;
    return product(a, b, offsets, groups, true, d, groups * a->rows, ldd, dtype, accumulate, 0, stream);
}

static_assert(OPT2S_MX4_PROJECT_COLS == opt2s::kRowMaxCols, "column limit");

OPT2S_API int opt2s_mx4_project_row(const void* x, int64_t cols, int32_t x_dtype, const opt2s_mx4* w, void* d,
                                    int32_t dtype, cudaStream_t stream)
{
    OPT2S_RANGE("opt2s_mx4_project_row");
    if (!good_dtype(x_dtype) || !good_dtype(dtype)) return OPT2S_ERR_INVALID_ARG;
    Range r[4];
    size_t n = 0;
    int st = matrix_ranges(w, false, r, &n);
    if (st != OPT2S_OK) return st;
    if (w->slabs != 1 || w->cols != cols) return OPT2S_ERR_INVALID_ARG;
    if (cols > OPT2S_MX4_PROJECT_COLS) return OPT2S_ERR_TOO_LARGE;
    if (w->rows == 0) return OPT2S_OK;
    const int xs = opt2s::elem_bytes(x_dtype), es = opt2s::elem_bytes(dtype);
    if (!x || !aligned(x, xs) || !d || !aligned(d, es)) return OPT2S_ERR_INVALID_ARG;
    r[n++] = span(x, cols * xs, false);
    r[n++] = span(d, w->rows * es, true);
    if ((st = opt2s::overlap_status(r, n)) != OPT2S_OK) return st;
    const opt2s::Mx4RowArgs a{x, cols, w->codes, w->scales, w->rows, up(w->rows, 4), d, aligned(x, 16)};
    const cudaError_t e = opt2s::launch_mx4_row(a, x_dtype, dtype, stream);
    if (e != cudaSuccess) return opt2s::record_cuda_error(e);
    opt2s::count_launches(1);
    return OPT2S_OK;
}

namespace {

// Checks one record of the step, appends its ranges and its kernel record.
int step_record(const opt2s_tensor_mx4& t, int32_t algo, std::vector<Range>* ranges,
                std::vector<opt2s::StepMx4Rec>* recs)
{
    const opt2s_tensor plain{t.param, t.grad, t.state1, t.state2, t.numel, t.dtype, t.reserved};
    Range r[8];
    int k = 0;
    int st = opt2s::record_ranges(plain, algo, r, &k);
    if (st != OPT2S_OK || k == 0) return st;
    size_t n = static_cast<size_t>(k);
    if (!t.codes != !t.scales || !t.codes_t != !t.scales_t) return OPT2S_ERR_INVALID_ARG;
    opt2s::StepMx4Rec rec{};
    rec.p = t.param;
    rec.g = t.grad;
    rec.m = t.state1;
    rec.v = t.state2;
    rec.m2 = t.state1 + t.numel;
    rec.numel = t.numel;
    rec.dtype = t.dtype;
    if (t.codes || t.codes_t) {
        if (!good_sizes(t.slabs, t.rows, t.cols) || !good_sizes(t.slabs, t.cols, t.rows)) return OPT2S_ERR_INVALID_ARG;
        if (t.numel % t.slabs || t.numel / t.slabs % t.rows || t.numel / t.slabs / t.rows != t.cols)
            return OPT2S_ERR_INVALID_ARG;
        const opt2s_mx4 q{t.codes, t.scales, t.slabs, t.rows, t.cols};
        const opt2s_mx4 qt{t.codes_t, t.scales_t, t.slabs, t.cols, t.rows};
        if (t.codes && (st = matrix_ranges(&q, true, r, &n)) != OPT2S_OK) return st;
        if (t.codes_t && (st = matrix_ranges(&qt, true, r, &n)) != OPT2S_OK) return st;
        rec.slabs = t.slabs;
        rec.rows = t.rows;
        rec.cols = t.cols;
        rec.codes = t.codes;
        rec.scales = t.scales;
        rec.codes_t = t.codes_t;
        rec.scales_t = t.scales_t;
        const int es = opt2s::elem_bytes(t.dtype);
        rec.vec = t.cols % (16 / es) == 0 && aligned(t.param, 16) && aligned(t.grad, 16) && aligned(t.state1, 16) &&
                  aligned(t.state2, 16) && (algo == OPT2S_ADAM || t.numel % 4 == 0);
    }
    ranges->insert(ranges->end(), r, r + n);
    recs->push_back(rec);
    return OPT2S_OK;
}

int step_mx4(const TensorListDescMx4* desc, const Hyper* hyper, int step, cudaStream_t stream)
{
    std::vector<Range> ranges;
    std::vector<opt2s::StepMx4Rec> recs;
    ranges.reserve(static_cast<size_t>(desc->count) * 8);
    recs.reserve(static_cast<size_t>(desc->count));
    int st;
    for (int32_t i = 0; i < desc->count; ++i)
        if ((st = step_record(desc->tensors[i], hyper->algo, &ranges, &recs)) != OPT2S_OK) return st;
    if ((st = opt2s::overlap_status(ranges.data(), ranges.size())) != OPT2S_OK) return st;
    const opt2s::StepScalars s = opt2s::make_scalars(hyper, step);
    constexpr size_t kMost = opt2s::kStepMx4MaxRecs;
    for (size_t at = 0; at < recs.size(); at += kMost) {        // nothing runs unless every launch can
        int64_t tiles = 0;
        for (size_t i = at; i < std::min(recs.size(), at + kMost); ++i) {
            tiles += opt2s::step_mx4_tiles(recs[i]);
            if (tiles > INT32_MAX) return OPT2S_ERR_TOO_LARGE;
        }
    }
    for (size_t at = 0; at < recs.size(); at += kMost) {
        const int n = static_cast<int>(std::min(kMost, recs.size() - at));
        const cudaError_t e = opt2s::launch_step_mx4(recs.data() + at, n, hyper->algo, hyper->skip_zeros, s, stream);
        if (e != cudaSuccess) return opt2s::record_cuda_error(e);
        opt2s::count_launches(1);
    }
    return OPT2S_OK;
}

}  // namespace

OPT2S_API int opt2s_step_mx4(const TensorListDescMx4* desc, const Hyper* hyper, int step, cudaStream_t stream)
{
    OPT2S_RANGE("opt2s_step_mx4");
    const int st = opt2s::validate_hyper(hyper, step);
    if (st != OPT2S_OK) return st;
    if (!desc || desc->count < 0 || (desc->count > 0 && !desc->tensors)) return OPT2S_ERR_INVALID_ARG;
    try {
        return step_mx4(desc, hyper, step, stream);
    } catch (const std::bad_alloc&) {
        return OPT2S_ERR_NO_MEMORY;
    }
}

OPT2S_API int opt2s_mx4_errors(uint32_t* count)
{
    if (!count) return OPT2S_ERR_INVALID_ARG;
    const cudaError_t e = opt2s::mx4_error_count(count);
    return e == cudaSuccess ? OPT2S_OK : opt2s::record_cuda_error(e);
}
