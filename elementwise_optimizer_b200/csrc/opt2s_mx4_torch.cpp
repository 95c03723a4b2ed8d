// opt2s_mx4_torch.cpp -- the torch side of the microscaled 4-bit operators
// (elementwise_optimizer_b200/mx4.py), part of the marshalling extension:
// checks of tensors, allocation of outputs, the calls of the C ABI on the
// tensors' device and current stream, and the layers' autograd function.  A
// layer's forward and backward make six library calls: 256 us of host time
// marshalled in Python, 102 us here, of which torch's engine takes 80 (a
// forward alone takes 20).  No arithmetic is here.  The library's entry points
// are handed over by address (mx4_set_library), so the extension does not link
// against it.
#include <torch/extension.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cstdint>
#include <optional>
#include <stdexcept>
#include <string>
#include <tuple>
#include <vector>

#include "opt2s.h"

namespace {

using at::Tensor;
using OptTensor = std::optional<Tensor>;

struct Library {
    decltype(&opt2s_mx4_quantize) quantize = nullptr;
    decltype(&opt2s_mx4_dequantize) dequantize = nullptr;
    decltype(&opt2s_mx4_matmul) matmul = nullptr;
    decltype(&opt2s_mx4_matmul_grouped) matmul_grouped = nullptr;
    decltype(&opt2s_mx4_matmul_ragged) matmul_ragged = nullptr;
    decltype(&opt2s_mx4_project_row) project_row = nullptr;
} lib;

// A failed library call; becomes binding.Opt2sError in Python.
struct CallFailed : std::runtime_error {
    CallFailed(const char* where, int status)
        : std::runtime_error(std::string(where) + " failed with status " + std::to_string(status)), where(where),
          status(status) {}
    const char* where;
    int status;
};

void check(int status, const char* where)
{
    if (status != OPT2S_OK) throw CallFailed(where, status);
}

// Message texts without streams: formatting numbers through an ostream of the
// compiler's libstdc++ crashes beside the older one that python has loaded.
std::string text(const char* s) { return s; }
std::string text(int64_t n) { return std::to_string(n); }
std::string text(const at::Device& d) { return d.str(); }
std::string text(at::IntArrayRef sizes)
{
    std::string out = "[";
    for (size_t i = 0; i < sizes.size(); ++i) out += (i ? ", " : "") + std::to_string(sizes[i]);
    return out + "]";
}
template <typename... A>
std::string message(const A&... parts) { return (text(parts) + ...); }

int64_t up(int64_t x, int64_t k) { return (x + k - 1) / k * k; }

int32_t dtype_code(c10::ScalarType t)
{
    switch (t) {
    case c10::ScalarType::Float: return OPT2S_F32;
    case c10::ScalarType::Half: return OPT2S_F16;
    case c10::ScalarType::BFloat16: return OPT2S_BF16;
    default: break;
    }
    TORCH_CHECK_TYPE(false, message("unsupported dtype ", c10::toString(t), " (float32, float16 or bfloat16 are supported)"));
}

// A 4-bit matrix: MX4Tensor's fields.
struct Matrix {
    Tensor codes, scales;
    int64_t slabs = 0, rows = 0, cols = 0;
    opt2s_mx4 c() const
    {
        auto ptr = [](const Tensor& t) { return t.numel() ? t.data_ptr<uint8_t>() : nullptr; };
        return {ptr(codes), ptr(scales), slabs, rows, cols};
    }
};

// A matrix of the extension's own: codes and scales in one allocation.
struct Packed {
    Tensor buffer;
    opt2s_mx4 c{};
};

int64_t code_bytes(int64_t slabs, int64_t rows, int64_t cols) { return slabs * rows * (up(cols, 128) / 2); }

opt2s_mx4 packed_view(const Tensor& buffer, int64_t slabs, int64_t rows, int64_t cols)
{
    uint8_t* at = buffer.data_ptr<uint8_t>();
    return {at, at + code_bytes(slabs, rows, cols), slabs, rows, cols};      // code rows are multiples of 64 bytes
}

Packed packed(int64_t slabs, int64_t rows, int64_t cols, const at::Device& device)
{
    const int64_t bytes = code_bytes(slabs, rows, cols) + up(cols, 128) / 128 * slabs * up(rows, 4) * 4;
    Packed p;
    p.buffer = at::empty({bytes}, at::TensorOptions().dtype(at::kByte).device(device));
    if (bytes) p.c = packed_view(p.buffer, slabs, rows, cols);
    else p.c = {nullptr, nullptr, slabs, rows, cols};
    return p;
}

Matrix empty_matrix(int64_t slabs, int64_t rows, int64_t cols, const at::Device& device)
{
    const auto o = at::TensorOptions().dtype(at::kByte).device(device);
    return {at::empty({slabs, rows, up(cols, 128) / 2}, o), at::empty({up(cols, 128) / 128, slabs, up(rows, 4), 4}, o),
            slabs, rows, cols};
}

int32_t check_offsets(const Tensor& offsets, const at::Device& device)
{
    TORCH_CHECK_VALUE(offsets.scalar_type() == at::kInt && offsets.dim() == 1 && offsets.is_contiguous() &&
                          offsets.device() == device,
                      "offsets must be a contiguous 1-D int32 tensor on the operands' device");
    const int64_t groups = offsets.numel() - 1;
    TORCH_CHECK_VALUE(groups >= 1 && groups <= OPT2S_MX4_MAX_GROUPS, message("offsets must hold 2 to ",
                      int64_t{OPT2S_MX4_MAX_GROUPS + 1}, " values"));
    return static_cast<int32_t>(groups);
}

cudaStream_t stream_of(const at::Device& d) { return c10::cuda::getCurrentCUDAStream(d.index()).stream(); }

// What a quantisation of x (2-D, or 3-D slabs) gets and gives.
struct Job {
    opt2s_mx4_source src;
    const int32_t* offsets = nullptr;
    int32_t groups = 0;
    int64_t t_cols;              // columns of the transposed form
};

Job job_of(const Tensor& x, const OptTensor& noise, const OptTensor& offsets)
{
    TORCH_CHECK_VALUE(x.is_cuda(), "a tensor to quantise must be on a CUDA device");
    TORCH_CHECK_VALUE(x.dim() == 2 || x.dim() == 3, "a tensor to quantise has 2 dimensions, or 3 with slabs");
    const bool three = x.dim() == 3;
    const int64_t slabs = three ? x.size(0) : 1, rows = x.size(-2), cols = x.size(-1);
    TORCH_CHECK_VALUE(cols >= 1 && slabs >= 1, "a tensor to quantise has at least one column and one slab");
    TORCH_CHECK_VALUE(cols == 1 || x.stride(-1) == 1,
                      "a tensor to quantise must have contiguous rows (stride 1 along the last axis)");
    if (noise) {
        TORCH_CHECK_VALUE(noise->scalar_type() == at::kByte && noise->sizes() == x.sizes() && noise->is_contiguous() &&
                              noise->device() == x.device(),
                          "noise must be a contiguous uint8 tensor of the source's shape and device");
    }
    Job j;
    if (offsets) {
        j.groups = check_offsets(*offsets, x.device());
        j.offsets = offsets->data_ptr<int32_t>();
        TORCH_CHECK_VALUE(slabs == 1, "only a single matrix is cut into groups of rows");
    }
    j.src = {x.data_ptr(), noise ? noise->data_ptr<uint8_t>() : nullptr, slabs, rows, cols,
             x.stride(-2), three ? x.stride(0) : 0, dtype_code(x.scalar_type()), 0};
    j.t_cols = j.groups ? up(rows, 128) + 128 * j.groups : rows;
    return j;
}

// On the current device, which is x's.
void run_job(const Job& j, const opt2s_mx4* q, const opt2s_mx4* qt, const at::Device& device)
{
    check(lib.quantize(&j.src, q, j.t_cols ? qt : nullptr, j.offsets, j.groups, stream_of(device)), "opt2s_mx4_quantize");
}

// The forms of x that are wanted, for the extension's own use.
void quantize(const Tensor& x, const OptTensor& noise, const OptTensor& offsets, Packed* q, Packed* qt)
{
    const Job j = job_of(x, noise, offsets);
    const c10::cuda::CUDAGuard guard(x.device());
    if (q) *q = packed(j.src.slabs, j.src.rows, j.src.cols, x.device());
    if (qt && j.t_cols) *qt = packed(j.src.slabs, j.src.cols, j.t_cols, x.device());
    run_job(j, q ? &q->c : nullptr, qt ? &qt->c : nullptr, x.device());
}

// The same for a caller: into q and/or qt, allocated where they are not given.
void quantize(const Tensor& x, const OptTensor& noise, const OptTensor& offsets, Matrix* q, Matrix* qt)
{
    const Job j = job_of(x, noise, offsets);
    const c10::cuda::CUDAGuard guard(x.device());
    auto fit = [&](Matrix* m, int64_t r, int64_t c) {
        if (!m) return;
        if (!m->codes.defined()) *m = empty_matrix(j.src.slabs, r, c, x.device());
        TORCH_CHECK_VALUE(m->slabs == j.src.slabs && m->rows == r && m->cols == c && m->codes.device() == x.device(),
                          "out does not fit the source on its device");
    };
    fit(q, j.src.rows, j.src.cols);
    if (j.t_cols == 0) qt = nullptr;             // no row, no transposed form
    fit(qt, j.src.cols, j.t_cols);
    const opt2s_mx4 cq = q ? q->c() : opt2s_mx4{}, ct = qt ? qt->c() : opt2s_mx4{};
    run_job(j, q ? &cq : nullptr, qt ? &ct : nullptr, x.device());
}

// The three products; d is [rows, cols] or [groups, rows, cols], or has the
// shape `as` of as many elements where it is made here.  (A view of a matrix
// could not be changed in place: autograd refuses that for a view made inside
// a function or without gradients.)
Tensor product(const opt2s_mx4& a, const opt2s_mx4& b, const at::Device& device, const OptTensor& offsets, bool ragged,
               c10::ScalarType dtype, const OptTensor& given, bool accumulate, at::IntArrayRef as = {})
{
    TORCH_CHECK_VALUE(a.cols == b.cols, message("the contractions differ: ", a.cols, " and ", b.cols));
    TORCH_CHECK_VALUE(a.slabs == 1, "the first operand of a product is a single matrix");
    int32_t groups = 0;
    if (offsets) groups = check_offsets(*offsets, device);
    const int64_t b_slabs = offsets && !ragged ? groups : 1;
    TORCH_CHECK_VALUE(b.slabs == b_slabs, message("the second operand has ", b.slabs, " slabs where this product takes ", b_slabs));
    if (ragged)
        TORCH_CHECK_VALUE(a.cols >= 128 * groups && a.cols % 128 == 0, "the operands were not quantised with these offsets");
    const std::vector<int64_t> shape =
        ragged ? std::vector<int64_t>{groups, a.rows, b.rows} : std::vector<int64_t>{a.rows, b.rows};
    const c10::cuda::CUDAGuard guard(device);
    Tensor d;
    int64_t ldd = b.rows;
    if (given) {
        d = *given;
        const int64_t n = d.dim();
        bool fits = d.sizes() == at::IntArrayRef(shape) && d.device() == device && (b.rows <= 1 || d.stride(-1) == 1);
        if (fits && a.rows > 1) ldd = d.stride(-2);
        else if (fits && ragged && groups > 1) ldd = d.stride(0);
        fits = fits && ldd >= b.rows && (n < 3 || groups <= 1 || a.rows == 0 || d.stride(0) == a.rows * ldd);
        TORCH_CHECK_VALUE(fits, message("out must be ", at::IntArrayRef(shape), " with contiguous, evenly spaced rows on ", device));
        if (!d.is_inference()) d.unsafeGetTensorImpl()->bump_version();       // autograd sees the write
    } else {
        TORCH_CHECK_VALUE(!accumulate, "accumulate needs the tensor to add to (out)");
        d = at::empty(as.empty() ? at::IntArrayRef(shape) : as, at::TensorOptions().dtype(dtype).device(device));
    }
    const int32_t code = dtype_code(d.scalar_type()), acc = accumulate ? 1 : 0;
    void* out = d.numel() ? d.data_ptr() : nullptr;
    const cudaStream_t s = stream_of(device);
    if (!offsets) check(lib.matmul(&a, &b, out, ldd, code, acc, s), "opt2s_mx4_matmul");
    else if (ragged)
        check(lib.matmul_ragged(&a, &b, offsets->data_ptr<int32_t>(), groups, out, ldd, code, acc, s), "opt2s_mx4_matmul_ragged");
    else
        check(lib.matmul_grouped(&a, &b, offsets->data_ptr<int32_t>(), groups, out, ldd, code, acc, given ? 0 : 1, s),
              "opt2s_mx4_matmul_grouped");
    return d;
}

// x as a matrix with contiguous rows.
Tensor rows_of(const Tensor& x)
{
    Tensor m = x.dim() == 2 ? x : x.reshape({-1, x.size(-1)});
    return m.size(-1) <= 1 || m.stride(-1) == 1 ? m : m.contiguous();
}

Tensor times(const opt2s_mx4& a, const opt2s_mx4& b, const at::Device& device, const OptTensor& offsets, c10::ScalarType dtype,
             at::IntArrayRef as)
{
    return product(a, b, device, offsets, false, dtype, std::nullopt, false, as);
}

// x's shape with n columns.
std::vector<int64_t> with_columns(const Tensor& x, int64_t n)
{
    std::vector<int64_t> shape = x.sizes().vec();
    shape.back() = n;
    return shape;
}

Tensor project(const Tensor& x, const Matrix& w, const OptTensor& offsets, std::optional<c10::ScalarType> dtype)
{
    TORCH_CHECK_VALUE(x.is_cuda(), "a tensor to quantise must be on a CUDA device");
    TORCH_CHECK_VALUE(x.dim() >= 1 && x.size(-1) == w.cols && (!offsets || x.dim() == 2), message("x ", x.sizes(),
                      " does not fit a weight of ", w.rows, " x ", w.cols));
    at::NoGradGuard no_grad;
    const at::Device device = x.device();
    TORCH_CHECK_VALUE(w.codes.device() == device, "a product's operands must be on one device");
    const int32_t groups = offsets ? check_offsets(*offsets, device) : 0, slabs = offsets ? groups : 1;
    TORCH_CHECK_VALUE(w.slabs == slabs, message("the weight has ", w.slabs, " slabs where this product takes ", slabs));
    const c10::ScalarType out = dtype.value_or(x.scalar_type());
    const Tensor rows = rows_of(x);
    const std::vector<int64_t> shape = with_columns(x, w.rows);
    if (rows.size(0) == 1 && !offsets && w.cols <= OPT2S_MX4_PROJECT_COLS) {
        // one row: 1 x 8,192 x 2,048 takes 5.6 us in one launch and 8.4 us in two
        const c10::cuda::CUDAGuard guard(device);
        Tensor y = at::empty(shape, at::TensorOptions().dtype(out).device(device));
        const opt2s_mx4 cw = w.c();
        check(lib.project_row(rows.data_ptr(), w.cols, dtype_code(x.scalar_type()), &cw, y.numel() ? y.data_ptr() : nullptr,
                              dtype_code(out), stream_of(device)),
              "opt2s_mx4_project_row");
        return y;
    }
    Packed q;
    quantize(rows, std::nullopt, std::nullopt, &q, nullptr);
    return times(q.c, w.c(), device, offsets, out, shape);
}

// y = Q(x) Q(w)^T with the straight-through gradients
// dx = Q(dy) Q(w^T)^T and dw = Q(dy^T) Q(x^T)^T.
struct Linear : torch::autograd::Function<Linear> {
    using Ctx = torch::autograd::AutogradContext;

    // Saved: the weight's and x's transposed forms, each as codes and scales (a
    // kept copy) or one buffer, and the shapes in one list.
    static Tensor forward(Ctx* ctx, const Tensor& x, const Tensor& weight, const OptTensor& offsets, const Matrix& wq,
                          const Matrix& wt, const OptTensor& noise, bool need_x, bool need_w)
    {
        const at::Device device = x.device();
        Packed own_q, own_t, xq, xt;
        opt2s_mx4 w;
        if (wq.codes.defined()) {
            w = wq.c();
        } else {
            quantize(weight, std::nullopt, std::nullopt, &own_q, need_x ? &own_t : nullptr);
            w = own_q.c;
        }
        const Tensor rows = rows_of(x);
        quantize(rows, std::nullopt, need_w ? offsets : std::nullopt, &xq, need_w ? &xt : nullptr);
        if (need_x || need_w) {
            const bool kept = wq.codes.defined();
            ctx->save_for_backward({need_x ? (kept ? wt.codes : own_t.buffer) : Tensor(), need_x && kept ? wt.scales : Tensor(),
                                    xt.buffer, offsets ? *offsets : Tensor(), noise ? *noise : Tensor()});
            std::vector<int64_t> facts{need_x, need_w, static_cast<int64_t>(weight.scalar_type()), xt.c.cols, weight.dim()};
            facts.insert(facts.end(), weight.sizes().begin(), weight.sizes().end());
            facts.insert(facts.end(), x.sizes().begin(), x.sizes().end());
            ctx->saved_data["facts"] = std::move(facts);
        }
        return times(xq.c, w, device, offsets, x.scalar_type(), with_columns(x, w.rows));
    }

    static torch::autograd::variable_list backward(Ctx* ctx, torch::autograd::variable_list grads)
    {
        const Tensor& dy = grads[0];
        TORCH_CHECK_NOT_IMPLEMENTED(!at::GradMode::is_enabled(),
                                    "a 4-bit layer's gradient has no gradient of its own (create_graph)");
        at::NoGradGuard no_grad;
        const auto saved = ctx->get_saved_variables();
        const auto facts = ctx->saved_data["facts"].toIntVector();
        const bool need_x = facts[0], need_w = facts[1];
        const auto w_dtype = static_cast<c10::ScalarType>(facts[2]);
        const auto w_at = facts.begin() + 5, x_at = w_at + facts[4];
        const at::IntArrayRef w_shape(&*w_at, static_cast<size_t>(facts[4]));
        const at::IntArrayRef x_shape(&*x_at, static_cast<size_t>(facts.end() - x_at));
        const OptTensor offsets = saved[3].defined() ? OptTensor(saved[3]) : std::nullopt;
        const OptTensor noise = saved[4].defined() ? OptTensor(saved[4]) : std::nullopt;
        const int64_t n = w_shape[w_shape.size() - 2], k = w_shape.back(), slabs = w_shape.size() == 3 ? w_shape[0] : 1;
        const at::Device device = dy.device();
        Tensor dx, dw;
        const Tensor rows = rows_of(dy);
        if (rows.size(0) == 0) {
            if (need_x) dx = at::zeros(x_shape, dy.options());
            if (need_w) dw = at::zeros(w_shape, dy.options().dtype(w_dtype));
        } else {
            Packed dq, dt;
            quantize(rows, noise, need_w ? offsets : std::nullopt, need_x ? &dq : nullptr, need_w ? &dt : nullptr);
            if (need_x) {
                const opt2s_mx4 wt = saved[1].defined() ? Matrix{saved[0], saved[1], slabs, k, n}.c() : packed_view(saved[0], slabs, k, n);
                dx = times(dq.c, wt, device, offsets, dy.scalar_type(), x_shape);
            }
            if (need_w)
                dw = product(dt.c, packed_view(saved[2], 1, k, facts[3]), device, offsets, offsets.has_value(), w_dtype, std::nullopt, false);
        }
        return {dx, dw, Tensor(), Tensor(), Tensor(), Tensor(), Tensor(), Tensor()};
    }
};

Tensor linear(const Tensor& x, const Tensor& weight, const OptTensor& offsets, const Matrix& wq, const Matrix& wt,
              const OptTensor& noise)
{
    TORCH_CHECK_VALUE(weight.dim() == (offsets ? 3 : 2) && x.dim() >= 1 && (!offsets || x.dim() == 2) &&
                          x.size(-1) == weight.size(-1),
                      message("x ", x.sizes(), " does not fit the weight ", weight.sizes()));
    TORCH_CHECK_VALUE(x.is_cuda() && x.device() == weight.device(), "x and weight must be on one CUDA device");
    const int64_t n = weight.size(-2);
    const bool grad = at::GradMode::is_enabled(), need_x = grad && x.requires_grad();
    TORCH_CHECK_VALUE(n >= 1, "a layer has at least one output");
    if (offsets)
        TORCH_CHECK_VALUE(check_offsets(*offsets, x.device()) == weight.size(0),
                          "offsets must hold one value more than there are experts");
    if (wq.codes.defined()) {
        const int64_t slabs = weight.dim() == 3 ? weight.size(0) : 1, k = weight.size(-1);
        const bool both = wt.codes.defined();
        TORCH_CHECK_VALUE(wq.slabs == slabs && wq.rows == n && wq.cols == k && wq.codes.device() == x.device() &&
                              (!both || (wt.slabs == slabs && wt.rows == k && wt.cols == n && wt.codes.device() == x.device())),
                          message("copies are not those of a weight ", weight.sizes()));
        TORCH_CHECK_VALUE(both || !need_x, "x needs a gradient, which takes the weight's transposed copy too");
    }
    OptTensor bytes;
    if (noise) {
        const std::vector<int64_t> want = with_columns(x, n);
        TORCH_CHECK_VALUE(noise->scalar_type() == at::kByte && noise->sizes() == at::IntArrayRef(want) &&
                              noise->device() == x.device(),
                          message("noise must be a uint8 tensor of the output's shape ", at::IntArrayRef(want), " on ", x.device()));
        bytes = noise->reshape({-1, n}).contiguous();
    }
    dtype_code(x.scalar_type());
    dtype_code(weight.scalar_type());
    return Linear::apply(x, weight, offsets, wq, wt, bytes, need_x, grad && weight.requires_grad());
}

using Fields = std::tuple<Tensor, Tensor, int64_t, int64_t, int64_t>;

Matrix matrix(const std::optional<Fields>& f)
{
    if (!f) return {};
    return {std::get<0>(*f), std::get<1>(*f), std::get<2>(*f), std::get<3>(*f), std::get<4>(*f)};
}

py::object fields(const Matrix& m)
{
    if (!m.codes.defined()) return py::none();
    return py::make_tuple(m.codes, m.scales, m.slabs, m.rows, m.cols);
}

}  // namespace

void bind_mx4(py::module& m)
{
    py::register_exception_translator([](std::exception_ptr p) {
        try {
            if (p) std::rethrow_exception(p);
        } catch (const CallFailed& e) {
            const py::module b = py::module::import("elementwise_optimizer_b200.binding");
            const py::object cls = b.attr("Opt2sError");
            const py::object err = cls(e.status, e.where, b.attr("lib")().attr("opt2s_last_cuda_error")());
            PyErr_SetObject(cls.ptr(), err.ptr());
        }
    });
    m.def("mx4_set_library", [](uintptr_t q, uintptr_t d, uintptr_t mm, uintptr_t mg, uintptr_t mr, uintptr_t pr) {
        lib.quantize = reinterpret_cast<decltype(lib.quantize)>(q);
        lib.dequantize = reinterpret_cast<decltype(lib.dequantize)>(d);
        lib.matmul = reinterpret_cast<decltype(lib.matmul)>(mm);
        lib.matmul_grouped = reinterpret_cast<decltype(lib.matmul_grouped)>(mg);
        lib.matmul_ragged = reinterpret_cast<decltype(lib.matmul_ragged)>(mr);
        lib.project_row = reinterpret_cast<decltype(lib.project_row)>(pr);
    });
    m.def("mx4_quantize", [](const Tensor& x, const OptTensor& noise, const OptTensor& offsets, bool want_q, bool want_t,
                             const std::optional<Fields>& out_q, const std::optional<Fields>& out_t) {
        Matrix q = matrix(out_q), t = matrix(out_t);
        at::NoGradGuard no_grad;
        quantize(x, noise, offsets, want_q ? &q : nullptr, want_t ? &t : nullptr);
        return py::make_tuple(fields(q), fields(t));
    });
    m.def("mx4_empty", [](int64_t slabs, int64_t rows, int64_t cols, const Tensor& like) {
        return fields(empty_matrix(slabs, rows, cols, like.device()));
    });
    m.def("mx4_dequantize", [](const Fields& f, const std::vector<int64_t>& shape, at::ScalarType st) {
        const Matrix q = matrix(f);
        const c10::cuda::CUDAGuard guard(q.codes.device());
        Tensor out = at::empty(shape, at::TensorOptions().dtype(st).device(q.codes.device()));
        const opt2s_mx4 c = q.c();
        check(lib.dequantize(&c, out.numel() ? out.data_ptr() : nullptr, dtype_code(st), stream_of(q.codes.device())),
              "opt2s_mx4_dequantize");
        return out;
    });
    m.def("mx4_product", [](const Fields& a, const Fields& b, const OptTensor& offsets, bool ragged,
                            std::optional<at::ScalarType> dtype, const OptTensor& out, bool accumulate) {
        TORCH_CHECK_VALUE(!out || !dtype || out->scalar_type() == *dtype, "out has another dtype than the one asked for");
        TORCH_CHECK_VALUE(!out || !at::GradMode::is_enabled() || !out->requires_grad(),
                          "out requires grad, and a product into a given tensor is not differentiated");
        at::NoGradGuard no_grad;
        const Matrix ma = matrix(a), mb = matrix(b);
        TORCH_CHECK_VALUE(ma.codes.device() == mb.codes.device(), "a product's operands must be on one device");
        return product(ma.c(), mb.c(), ma.codes.device(), offsets, ragged, dtype.value_or(at::kBFloat16), out, accumulate);
    });
    m.def("mx4_project", [](const Tensor& x, const Fields& w, const OptTensor& offsets,
                            std::optional<at::ScalarType> dtype) { return project(x, matrix(w), offsets, dtype);
    });
    m.def("mx4_linear", [](const Tensor& x, const Tensor& weight, const OptTensor& offsets, const std::optional<Fields>& wq,
                           const std::optional<Fields>& wt, const OptTensor& noise) {
        return linear(x, weight, offsets, matrix(wq), matrix(wt), noise);
    });
}
