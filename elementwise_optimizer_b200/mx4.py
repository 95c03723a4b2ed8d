"""Microscaled 4-bit matrices and their products, for torch tensors.

The weights that the optimizer steps are used by a model's products; here
those products read them in MXFP4 (blocks of 32 E2M1 elements with one E8M0
scale, OCP Microscaling Formats v1.0; the layout is described in
include/opt2s.h) and give the gradients that the next step reads:

    linear(x, w)              y = Q(x) Q(w)^T,  dx = Q(dy) Q(w^T)^T,
                              dw = Q(dy^T) Q(x^T)^T
    linear_grouped(x, w, offsets)   the same for experts: rows
                              [offsets[e], offsets[e+1]) of x with w[e]

Q cuts its operand into blocks along the contraction, so every matrix of a
training step is needed in two forms: ``quantize_pair`` makes both from one
read.  Rounding to 4 bits is to nearest (even), or stochastic from random
bytes that the caller gives; its gradient is taken as one (straight-through).
``copies`` skips the weight's quantisation: pass the pair that the optimizer
keeps up to date (``optim.AdamW32bit(..., mx4=True)``, ``mx4_copies(w)``: its
step writes them, see ``opt2s_step_mx4``), or one from ``quantize_pair``.

All work happens in the kernels of libopt2s.so, on the tensors' device and
torch's current stream of it; nothing is kept between calls, and every call
may be captured in a CUDA graph.  Errors raise ``Opt2sError`` (the library's
status) or ValueError/TypeError for arguments that do not fit together.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import binding as B
from .binding import TensorListMX4, opt2s_step_mx4  # noqa: F401  (the step that writes the copies)

BLOCK = B.MX4_BLOCK
MAX_GROUPS = B.MX4_MAX_GROUPS


def _on_device(index):
    """Makes CUDA device `index` current for a launch."""
    if index == torch._C._cuda_getDevice():
        return contextlib.nullcontext()
    return torch.cuda.device(index)


def _up(n: int, k: int) -> int:
    return (n + k - 1) // k * k


class MX4Tensor:
    """A 4-bit matrix, or slabs of them: ``codes`` uint8 [slabs, rows, cols_p/2]
    and ``scales`` uint8 [cols_p/128, slabs, rows_p, 4] (cols_p = cols rounded
    up to 128, rows_p = rows rounded up to 4), CUDA and contiguous; ``shape``
    is (rows, cols) or (slabs, rows, cols)."""

    __slots__ = ("codes", "scales", "shape", "slabs", "rows", "cols", "_c")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, shape):
        shape = tuple(int(n) for n in shape)
        if len(shape) not in (2, 3):
            raise ValueError("an MX4Tensor has shape (rows, cols) or (slabs, rows, cols)")
        rows, cols = shape[-2:]
        slabs = shape[0] if len(shape) == 3 else codes.shape[0] if codes.dim() == 3 else 1
        for t in (codes, scales):
            if t.dtype != torch.uint8 or not t.is_cuda or not t.is_contiguous():
                raise ValueError("codes and scales must be contiguous uint8 CUDA tensors")
        if codes.device != scales.device:
            raise ValueError("codes and scales must be on one device")
        if slabs < 1 or rows < 0 or cols < 1:
            raise ValueError("an MX4Tensor has slabs >= 1, rows >= 0 and cols >= 1")
        if (codes.numel() != slabs * rows * (_up(cols, 128) // 2)
                or scales.numel() != _up(cols, 128) // 128 * slabs * _up(rows, 4) * 4):
            raise ValueError(f"codes {tuple(codes.shape)} and scales {tuple(scales.shape)} do not fit {shape}")
        self.codes, self.scales = codes, scales
        self.slabs, self.rows, self.cols = slabs, rows, cols
        self.shape = shape if slabs == 1 or len(shape) == 3 else (slabs, rows, cols)
        self._c = B.opt2s_mx4(codes.data_ptr() or None, scales.data_ptr() or None, slabs, rows, cols)

    @property
    def device(self) -> torch.device:
        return self.codes.device

    def dequantize(self, dtype: torch.dtype = torch.float32) -> torch.Tensor:
        """The values it stands for (exact in fp32 and bf16)."""
        out = torch.empty(self.shape, dtype=dtype, device=self.device)
        with _on_device(self.device.index):
            B.check(B.lib().opt2s_mx4_dequantize(ctypes.byref(self._c), out.data_ptr() or None,
                                                 B._torch_dtype_code(out), B._stream_handle(None)),
                    "opt2s_mx4_dequantize")
        return out

    def __repr__(self):
        return f"MX4Tensor(shape={self.shape}, device={self.device})"


def _empty(shape, device) -> MX4Tensor:
    *slabs, rows, cols = shape
    n = slabs[0] if slabs else 1
    codes = torch.empty((n, rows, _up(cols, 128) // 2), dtype=torch.uint8, device=device)
    scales = torch.empty((_up(cols, 128) // 128, n, _up(rows, 4), 4), dtype=torch.uint8, device=device)
    return MX4Tensor(codes, scales, shape)


def empty_pair(x: torch.Tensor) -> tuple:
    """Uninitialised storage for the two forms of x (2-D, or 3-D slabs)."""
    if x.dim() not in (2, 3):
        raise ValueError("a 4-bit matrix has 2 dimensions, or 3 with slabs")
    *slabs, rows, cols = x.shape
    return _empty((*slabs, rows, cols), x.device), _empty((*slabs, cols, rows), x.device)


def _check_offsets(offsets: torch.Tensor, device) -> int:
    if offsets.dtype != torch.int32 or offsets.dim() != 1 or not offsets.is_contiguous() or offsets.device != device:
        raise ValueError("offsets must be a contiguous 1-D int32 tensor on the operands' device")
    groups = offsets.numel() - 1
    if not 1 <= groups <= MAX_GROUPS:
        raise ValueError(f"offsets must hold 2 to {MAX_GROUPS + 1} values")
    return groups


def _quantize(x, noise, offsets, want_q, want_t, out=None):
    if not x.is_cuda:
        raise ValueError("a tensor to quantise must be on a CUDA device")
    if x.dim() not in (2, 3):
        raise ValueError("a tensor to quantise has 2 dimensions, or 3 with slabs")
    if x.shape[-1] < 1 or x.dim() == 3 and x.shape[0] < 1:
        raise ValueError("a tensor to quantise has at least one column and one slab")
    if x.shape[-1] > 1 and x.stride(-1) != 1:
        raise ValueError("a tensor to quantise must have contiguous rows (stride 1 along the last axis)")
    if noise is not None and (noise.dtype != torch.uint8 or noise.shape != x.shape or not noise.is_contiguous()
                              or noise.device != x.device):
        raise ValueError("noise must be a contiguous uint8 tensor of the source's shape and device")
    dtype = B._torch_dtype_code(x)
    slabs = x.shape[0] if x.dim() == 3 else 1
    rows, cols = x.shape[-2:]
    groups = 0
    if offsets is not None:
        groups = _check_offsets(offsets, x.device)
        if slabs != 1:
            raise ValueError("only a single matrix is cut into groups of rows")
    src = B.opt2s_mx4_source(x.data_ptr() or None, None if noise is None else noise.data_ptr() or None, slabs, rows,
                             cols, x.stride(-2), x.stride(0) if x.dim() == 3 else 0, dtype, 0)
    lead = x.shape[:-2]
    t_cols = _up(rows, 128) + 128 * groups if groups else rows
    if out is not None:
        q, qt = out
        for m, want in zip(out, ((slabs, rows, cols), (slabs, cols, t_cols))):
            if (m.slabs, m.rows, m.cols) != want or m.device != x.device:
                raise ValueError(f"out {m.shape} does not fit a source {tuple(x.shape)} on its device")
    else:
        q = _empty((*lead, rows, cols), x.device) if want_q else None
        qt = _empty((*lead, cols, t_cols), x.device) if want_t and t_cols else None
    with _on_device(x.device.index):
        B.check(B.lib().opt2s_mx4_quantize(
            ctypes.byref(src), ctypes.byref(q._c) if q else None, ctypes.byref(qt._c) if qt else None,
            None if offsets is None else offsets.data_ptr(), groups, B._stream_handle(None)), "opt2s_mx4_quantize")
    return q, qt


def quantize(x: torch.Tensor, noise: torch.Tensor | None = None) -> MX4Tensor:
    """x ([rows, cols] or [slabs, rows, cols]; fp32, fp16 or bf16; rows of any
    stride) in blocks along its last axis.  noise: random bytes (uint8, x's
    shape) for stochastic rounding."""
    return _quantize(x.detach(), noise, None, True, False)[0]


def quantize_pair(x: torch.Tensor, noise: torch.Tensor | None = None, offsets: torch.Tensor | None = None,
                  out: tuple | None = None) -> tuple:
    """Both forms of x from one read: (blocks along the last axis, blocks down
    the columns of the transposed matrix).  offsets (int32 on the device,
    groups + 1 values): the rows' groups; the transposed form then starts each
    group at a multiple of 128 columns, as ``matmul_ragged`` reads it.  The
    second is None for a matrix without rows and offsets.  out: a pair to
    write to."""
    return _quantize(x.detach(), noise, offsets, True, True, out)


def _product(name, a, b, d_shape, offsets, dtype, out, accumulate, fill_rest=False):
    for m in (a, b):
        if not isinstance(m, MX4Tensor):
            raise TypeError("a product's operands are MX4Tensors")
    if a.device != b.device:
        raise ValueError("a product's operands must be on one device")
    if a.cols != b.cols:
        raise ValueError(f"the contractions differ: {a.shape} and {b.shape}")
    if a.slabs != 1:
        raise ValueError("the first operand of a product is a single matrix")
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs the tensor to add to (out)")
        out = torch.empty(d_shape, dtype=dtype or torch.bfloat16, device=a.device)
    else:
        if dtype is not None and dtype != out.dtype:
            raise ValueError("out has another dtype than the one asked for")
        fits = tuple(out.shape) == tuple(d_shape) and out.device == a.device and (out.shape[-1] <= 1 or out.stride(-1) == 1)
        if fits and out.dim() == 3:
            fits = out.stride(0) == out.shape[1] * out.stride(1) or out.shape[0] <= 1
        if not fits or out.shape[-2] > 1 and out.stride(-2) < out.shape[-1]:
            raise ValueError(f"out must be {tuple(d_shape)} with contiguous, evenly spaced rows on {a.device}")
    ldd = max(out.stride(-2), out.shape[-1]) if out.dim() > 1 else out.shape[-1]
    args = [ctypes.byref(a._c), ctypes.byref(b._c)]
    if offsets is not None:
        args += [offsets.data_ptr(), offsets.numel() - 1]
    args += [out.data_ptr() or None, ldd, B._torch_dtype_code(out), int(bool(accumulate))]
    if name == "opt2s_mx4_matmul_grouped":
        args.append(int(bool(fill_rest)))
    with _on_device(a.device.index):
        B.check(getattr(B.lib(), name)(*args, B._stream_handle(None)), name)
    return out


def matmul(a: MX4Tensor, b: MX4Tensor, dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
           accumulate: bool = False) -> torch.Tensor:
    """a [M, K] times b [N, K] transposed: [M, N] in `dtype` (bf16), sums in
    fp32.  out: where to write; accumulate: add to what it holds."""
    if isinstance(b, MX4Tensor) and b.slabs != 1:
        raise ValueError("matmul takes two single matrices; see matmul_grouped")
    return _product("opt2s_mx4_matmul", a, b, (a.rows, b.rows), None, dtype, out, accumulate)


def matmul_grouped(a: MX4Tensor, b: MX4Tensor, offsets: torch.Tensor, dtype: torch.dtype | None = None,
                   out: torch.Tensor | None = None, accumulate: bool = False) -> torch.Tensor:
    """Rows [offsets[e], offsets[e+1]) of a [T, K] times slab e of b [E, N, K]
    transposed: [T, N].  Rows in no group are zero, or with `out` left as they
    were."""
    if _check_offsets(offsets, a.device) != b.slabs:
        raise ValueError("offsets must hold one value more than the second operand has slabs")
    return _product("opt2s_mx4_matmul_grouped", a, b, (a.rows, b.rows), offsets, dtype, out, accumulate,
                    fill_rest=out is None)


def matmul_ragged(a: MX4Tensor, b: MX4Tensor, offsets: torch.Tensor, dtype: torch.dtype | None = None,
                  out: torch.Tensor | None = None, accumulate: bool = False) -> torch.Tensor:
    """For each group e of tokens, the product over its tokens: a [N, .] and
    b [K, .] are the transposed forms that ``quantize_pair`` made with these
    offsets; [E, N, K].  An empty group gives zeros."""
    groups = _check_offsets(offsets, a.device)
    if a.cols < 128 * groups or a.cols % 128:
        raise ValueError("the operands were not quantised with these offsets")
    if isinstance(b, MX4Tensor) and b.slabs != 1:
        raise ValueError("matmul_ragged takes two single matrices")
    return _product("opt2s_mx4_matmul_ragged", a, b, (groups, a.rows, b.rows), offsets, dtype, out, accumulate)


def project(x: torch.Tensor, wq: MX4Tensor, dtype: torch.dtype | None = None) -> torch.Tensor:
    """x [..., K] quantised (to nearest) and multiplied with a kept 4-bit
    weight [N, K]: [..., N] in x's dtype.  For serving: no autograd."""
    if x.shape[-1] != wq.cols or wq.slabs != 1:
        raise ValueError(f"x {tuple(x.shape)} does not fit the weight {wq.shape}")
    x2 = _rows(x.detach())
    return matmul(quantize(x2), wq, dtype or x.dtype).view(*x.shape[:-1], wq.rows)


def project_grouped(x: torch.Tensor, wq: MX4Tensor, offsets: torch.Tensor,
                    dtype: torch.dtype | None = None) -> torch.Tensor:
    """``project`` for experts: rows [offsets[e], offsets[e+1]) of x [T, K]
    with slab e of wq [E, N, K].  Rows in no group are zero."""
    if x.dim() != 2 or x.shape[-1] != wq.cols:
        raise ValueError(f"x {tuple(x.shape)} does not fit the weight {wq.shape}")
    return matmul_grouped(quantize(_rows(x.detach())), wq, offsets, dtype or x.dtype)


def _rows(x: torch.Tensor) -> torch.Tensor:
    """x as a matrix with contiguous rows."""
    x = x.reshape(-1, x.shape[-1])
    return x if x.shape[-1] <= 1 or x.stride(-1) == 1 else x.contiguous()


class _Linear(torch.autograd.Function):
    """y and its gradients; offsets None for one matrix."""

    @staticmethod
    def forward(ctx, x, weight, offsets, wq, wt, noise):
        need_x, need_w = ctx.needs_input_grad[:2]
        if wq is None:
            if need_x:
                wq, wt = quantize_pair(weight)
            else:
                wq = quantize(weight)
        rows = _rows(x)
        xq, xt = _quantize(rows, None, offsets if need_w else None, True, need_w)
        ctx.offsets, ctx.noise, ctx.shapes = offsets, noise, (x.shape, weight.shape, weight.dtype)
        ctx.wt, ctx.xt = (wt if need_x else None), xt
        if offsets is None:
            return matmul(xq, wq, x.dtype).view(*x.shape[:-1], wq.rows)
        return matmul_grouped(xq, wq, offsets, x.dtype)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        need_x, need_w = ctx.needs_input_grad[:2]
        x_shape, w_shape, w_dtype = ctx.shapes
        rows, offsets = _rows(dy), ctx.offsets
        dx = dw = None
        if rows.shape[0] == 0:
            return (dy.new_zeros(x_shape) if need_x else None,
                    torch.zeros(w_shape, dtype=w_dtype, device=dy.device) if need_w else None, None, None, None, None)
        if not (need_x or need_w):
            return None, None, None, None, None, None
        dq, dqt = _quantize(rows, ctx.noise, offsets if need_w else None, need_x, need_w)
        if need_x:
            dx = matmul(dq, ctx.wt, dy.dtype).view(x_shape) if offsets is None else \
                matmul_grouped(dq, ctx.wt, offsets, dy.dtype)
        if need_w:
            dw = matmul(dqt, ctx.xt, w_dtype) if offsets is None else matmul_ragged(dqt, ctx.xt, offsets, w_dtype)
        return dx, dw, None, None, None, None


def _copies(weight, copies):
    if copies is None:
        return None, None
    q, qt = copies
    want = tuple(weight.shape)
    if q.shape != want or qt.shape != (*want[:-2], want[-1], want[-2]):
        raise ValueError(f"copies {q.shape}, {qt.shape} are not those of a weight {want}")
    return q, qt


def _check_noise(noise, x, n_out):
    if noise is None:
        return None
    want = (*x.shape[:-1], n_out)
    if noise.dtype != torch.uint8 or tuple(noise.shape) != want or noise.device != x.device:
        raise ValueError(f"noise must be a uint8 tensor of the output's shape {want} on {x.device}")
    return noise.reshape(-1, n_out).contiguous()


def linear(x: torch.Tensor, weight: torch.Tensor, copies: tuple | None = None,
           noise: torch.Tensor | None = None) -> torch.Tensor:
    """x [..., K] through weight [N, K] in 4 bits: [..., N] in x's dtype, with
    gradients in x's and weight's dtypes.  copies: the weight's pair, kept by
    the caller; noise: random bytes (uint8, the output's shape) that round the
    output's gradient stochastically."""
    if weight.dim() != 2 or x.dim() < 1 or x.shape[-1] != weight.shape[1]:
        raise ValueError(f"x {tuple(x.shape)} does not fit the weight {tuple(weight.shape)}")
    if x.device != weight.device:
        raise ValueError("x and weight must be on one device")
    return _Linear.apply(x, weight, None, *_copies(weight, copies), _check_noise(noise, x, weight.shape[0]))


def linear_grouped(x: torch.Tensor, weight: torch.Tensor, offsets: torch.Tensor, copies: tuple | None = None,
                   noise: torch.Tensor | None = None) -> torch.Tensor:
    """``linear`` for experts: rows [offsets[e], offsets[e+1]) of x [T, K] with
    weight[e], weight [E, N, K].  offsets: int32 on the device, E + 1 values,
    non-decreasing.  Rows in no group, and their gradients, are zero."""
    if weight.dim() != 3 or x.dim() != 2 or x.shape[-1] != weight.shape[2]:
        raise ValueError(f"x {tuple(x.shape)} does not fit the weight {tuple(weight.shape)}")
    if x.device != weight.device:
        raise ValueError("x and weight must be on one device")
    if _check_offsets(offsets, x.device) != weight.shape[0]:
        raise ValueError("offsets must hold one value more than there are experts")
    return _Linear.apply(x, weight, offsets, *_copies(weight, copies), _check_noise(noise, x, weight.shape[1]))
