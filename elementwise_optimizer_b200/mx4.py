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
Stochastic rounding keeps the mean of all but a block's largest elements:
magnitudes between 6 and 8 times the block's scale 2^(floor(log2 amax) - 2)
are cut to 6 either way, up to a quarter of them.
``copies`` skips the weight's quantisation: pass the pair that the optimizer
keeps up to date (``optim.AdamW32bit(..., mx4=True)``, ``mx4_copies(w)``: its
step writes them, see ``opt2s_step_mx4``), or one from ``quantize_pair``.

All work happens in the kernels of libopt2s.so, on the tensors' device and
torch's current stream of it; nothing is kept between calls, and every call
may be captured in a CUDA graph (a backward pass as torch allows it: while it
is captured, no graph of the same leaves made outside may be alive).  Errors
raise ``Opt2sError`` (the library's status) or ValueError/TypeError for
arguments that do not fit together.  What only the device can know, a product
that gave up waiting for its own copies, ``check_errors`` reports: it waits
for the device, so the calls themselves do not ask.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding as B
from .binding import TensorListMX4, opt2s_step_mx4  # noqa: F401  (the step that writes the copies)

BLOCK = B.MX4_BLOCK
MAX_GROUPS = B.MX4_MAX_GROUPS

_ext = None
_ext_lib = None


def _extension():
    """The marshalling extension (csrc/opt2s_mx4_torch.cpp), with the entry
    points of the library in use; there is no fallback in Python."""
    global _ext, _ext_lib
    L = B.lib()
    if _ext_lib is not L:
        from .optim import _marshal_module
        m = _marshal_module()
        if m is None:
            raise RuntimeError("the marshalling extension is missing: build the package first "
                               "(python -m elementwise_optimizer_b200._build)")
        m.mx4_set_library(*(B.address_of(L, n) for n in (
            "opt2s_mx4_quantize", "opt2s_mx4_dequantize", "opt2s_mx4_matmul", "opt2s_mx4_matmul_grouped",
            "opt2s_mx4_matmul_ragged", "opt2s_mx4_project_row")))
        _ext, _ext_lib = m, L
    return _ext


def _up(n: int, k: int) -> int:
    return (n + k - 1) // k * k


class MX4Tensor:
    """A 4-bit matrix, or slabs of them: ``codes`` uint8 [slabs, rows, cols_p/2]
    and ``scales`` uint8 [cols_p/128, slabs, rows_p, 4] (cols_p = cols rounded
    up to 128, rows_p = rows rounded up to 4), CUDA and contiguous; ``shape``
    is (rows, cols) or (slabs, rows, cols)."""

    __slots__ = ("codes", "scales", "slabs", "rows", "cols", "shape")

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
        self.codes, self.scales, self.slabs, self.rows, self.cols = codes, scales, slabs, rows, cols
        self.shape = shape if slabs == 1 or len(shape) == 3 else (slabs, rows, cols)

    @classmethod
    def _made(cls, fields, slabbed):
        """From the extension's (codes, scales, slabs, rows, cols)."""
        if fields is None:
            return None
        t = object.__new__(cls)
        t.codes, t.scales, t.slabs, t.rows, t.cols = fields
        t.shape = fields[2:] if slabbed else fields[3:]
        return t

    @property
    def _fields(self):
        return self.codes, self.scales, self.slabs, self.rows, self.cols

    @property
    def device(self) -> torch.device:
        return self.codes.device

    def dequantize(self, dtype: torch.dtype = torch.float32) -> torch.Tensor:
        """The values it stands for (exact in fp32 and bf16)."""
        return _extension().mx4_dequantize(self._fields, self.shape, dtype)

    def __repr__(self):
        return f"MX4Tensor(shape={self.shape}, device={self.device})"


def _fields(m):
    if not isinstance(m, MX4Tensor):
        raise TypeError("a product's operands are MX4Tensors")
    return m._fields


def check_errors(device=None) -> None:
    """Raises if a product on `device` (the current one) gave up waiting for
    its own copies since the library was loaded: the hardware or the library
    is then at fault, and that product's outputs are undefined.  Waits for all
    streams of the device (not while one is captured)."""
    count = ctypes.c_uint32()
    with torch.cuda.device(device):
        B.check(B.lib().opt2s_mx4_errors(ctypes.byref(count)), "opt2s_mx4_errors")
    if count.value:
        raise RuntimeError(f"{count.value} CTAs of 4-bit products gave up waiting for their copies; "
                           "the outputs of those products are undefined")


def empty_pair(x: torch.Tensor) -> tuple:
    """Uninitialised storage for the two forms of x (2-D, or 3-D slabs)."""
    if x.dim() not in (2, 3):
        raise ValueError("a 4-bit matrix has 2 dimensions, or 3 with slabs")
    slabs = x.shape[0] if x.dim() == 3 else 1
    rows, cols = x.shape[-2:]
    if slabs < 1 or rows < 1 or cols < 1:
        raise ValueError("a pair of 4-bit forms needs at least one element")
    if not x.is_cuda:
        raise ValueError("4-bit matrices are on CUDA devices")
    e = _extension()
    return (MX4Tensor._made(e.mx4_empty(slabs, rows, cols, x), x.dim() == 3),
            MX4Tensor._made(e.mx4_empty(slabs, cols, rows, x), x.dim() == 3))


def quantize(x: torch.Tensor, noise: torch.Tensor | None = None) -> MX4Tensor:
    """x ([rows, cols] or [slabs, rows, cols]; fp32, fp16 or bf16; rows of any
    stride) in blocks along its last axis.  noise: random bytes (uint8, x's
    shape) for stochastic rounding."""
    return MX4Tensor._made(_extension().mx4_quantize(x, noise, None, True, False, None, None)[0], x.dim() == 3)


def quantize_pair(x: torch.Tensor, noise: torch.Tensor | None = None, offsets: torch.Tensor | None = None,
                  out: tuple | None = None) -> tuple:
    """Both forms of x from one read: (blocks along the last axis, blocks down
    the columns of the transposed matrix).  offsets (int32 on the device,
    groups + 1 values): the rows' groups; the transposed form then starts each
    group at a multiple of 128 columns, as ``matmul_ragged`` reads it.  The
    second is None for a matrix without rows and offsets.  out: a pair to
    write to."""
    oq, ot = (None, None) if out is None else (_fields(out[0]), _fields(out[1]))
    q, t = _extension().mx4_quantize(x, noise, offsets, True, True, oq, ot)
    if out is not None:
        B.bump_versions([m.codes for m in out])
        return tuple(out)
    return MX4Tensor._made(q, x.dim() == 3), MX4Tensor._made(t, x.dim() == 3)


def matmul(a: MX4Tensor, b: MX4Tensor, dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
           accumulate: bool = False) -> torch.Tensor:
    """a [M, K] times b [N, K] transposed: [M, N] in `dtype` (bf16), sums in
    fp32.  out: where to write (not differentiated); accumulate: add to what it
    holds."""
    return _extension().mx4_product(_fields(a), _fields(b), None, False, dtype, out, accumulate)


def matmul_grouped(a: MX4Tensor, b: MX4Tensor, offsets: torch.Tensor, dtype: torch.dtype | None = None,
                   out: torch.Tensor | None = None, accumulate: bool = False) -> torch.Tensor:
    """Rows [offsets[e], offsets[e+1]) of a [T, K] times slab e of b [E, N, K]
    transposed: [T, N].  Rows in no group are zero, or with `out` left as they
    were."""
    return _extension().mx4_product(_fields(a), _fields(b), offsets, False, dtype, out, accumulate)


def matmul_ragged(a: MX4Tensor, b: MX4Tensor, offsets: torch.Tensor, dtype: torch.dtype | None = None,
                  out: torch.Tensor | None = None, accumulate: bool = False) -> torch.Tensor:
    """For each group e of tokens, the product over its tokens: a [N, .] and
    b [K, .] are the transposed forms that ``quantize_pair`` made with these
    offsets; [E, N, K].  An empty group gives zeros."""
    return _extension().mx4_product(_fields(a), _fields(b), offsets, True, dtype, out, accumulate)


def project(x: torch.Tensor, wq: MX4Tensor, dtype: torch.dtype | None = None) -> torch.Tensor:
    """x [..., K] quantised (to nearest) and multiplied with a kept 4-bit
    weight [N, K]: [..., N] in x's dtype.  For serving: no autograd."""
    return _extension().mx4_project(x, _fields(wq), None, dtype)


def project_grouped(x: torch.Tensor, wq: MX4Tensor, offsets: torch.Tensor,
                    dtype: torch.dtype | None = None) -> torch.Tensor:
    """``project`` for experts: rows [offsets[e], offsets[e+1]) of x [T, K]
    with slab e of wq [E, N, K].  Rows in no group are zero."""
    return _extension().mx4_project(x, _fields(wq), offsets, dtype)


def _copies(copies):
    if copies is None:
        return None, None
    return _fields(copies[0]), None if copies[1] is None else _fields(copies[1])


def linear(x: torch.Tensor, weight: torch.Tensor, copies: tuple | None = None,
           noise: torch.Tensor | None = None) -> torch.Tensor:
    """x [..., K] through weight [N, K] in 4 bits: [..., N] in x's dtype, with
    gradients in x's and weight's dtypes.  x and the output's gradient may have
    any strides (where rows are not contiguous they are copied); the weight,
    which is read in place, has contiguous rows: a transposed view is refused.
    copies: the weight's pair, kept by the caller (its second form may be None
    where x needs no gradient); noise: random bytes (uint8, the output's shape)
    that round the output's gradient stochastically."""
    return _extension().mx4_linear(x, weight, None, *_copies(copies), noise)


def linear_grouped(x: torch.Tensor, weight: torch.Tensor, offsets: torch.Tensor, copies: tuple | None = None,
                   noise: torch.Tensor | None = None) -> torch.Tensor:
    """``linear`` for experts: rows [offsets[e], offsets[e+1]) of x [T, K] with
    weight[e], weight [E, N, K].  offsets: int32 on the device, E + 1 values,
    non-decreasing.  Rows in no group, and their gradients, are zero."""
    return _extension().mx4_linear(x, weight, offsets, *_copies(copies), noise)
