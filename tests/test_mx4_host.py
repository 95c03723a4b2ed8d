"""The microscaled 4-bit operators without a GPU: sizes, struct layout, and
every refusal of the C ABI and of the Python front end (all before any CUDA
call)."""
import ctypes
import os
import subprocess
import tempfile

import pytest
import torch

from elementwise_optimizer_b200 import binding as B
from elementwise_optimizer_b200 import mx4, optim

INVALID, ALIAS, TOO_LARGE, CUDA = -1, -2, -6, -4
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def L():
    return B.lib()


class Fake:
    """Disjoint made-up device addresses, 256-byte aligned."""

    def __init__(self):
        self.at = 1 << 40

    def __call__(self, n):
        p = self.at
        self.at += (n + 511) // 256 * 256
        return p


def matrix(L, fake, n_slabs, n_rows, n_cols, **change):
    m = B.opt2s_mx4(fake(max(1, L.opt2s_mx4_code_bytes(n_slabs, n_rows, n_cols))),
                    fake(max(1, L.opt2s_mx4_scale_bytes(n_slabs, n_rows, n_cols))), n_slabs, n_rows, n_cols)
    for k, v in change.items():
        setattr(m, k, v)
    return m


needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only where nothing can run")


def test_sizes(L):
    assert L.opt2s_mx4_code_bytes(1, 3, 1) == 3 * 64
    assert L.opt2s_mx4_code_bytes(2, 5, 130) == 2 * 5 * 128
    assert L.opt2s_mx4_scale_bytes(1, 3, 1) == 1 * 4 * 4
    assert L.opt2s_mx4_scale_bytes(2, 5, 130) == 2 * 2 * 8 * 4
    assert L.opt2s_mx4_code_bytes(1, 0, 5) == 0
    for bad in ((0, 1, 1), (1, -1, 1), (1, 1, 0), (1, 1 << 31, 1), (1 << 20, 1 << 20, 1)):
        assert L.opt2s_mx4_code_bytes(*bad) == -1 and L.opt2s_mx4_scale_bytes(*bad) == -1


def test_struct_layout(L):
    prog = r"""
    #include <stddef.h>
    #include <stdio.h>
    #include "opt2s.h"
    int main(void) {
      printf("%zu %zu %zu %zu\n", sizeof(opt2s_mx4), offsetof(opt2s_mx4, cols), sizeof(opt2s_mx4_source),
             offsetof(opt2s_mx4_source, dtype));
      printf("%zu %zu %zu %zu %zu\n", sizeof(opt2s_tensor_mx4), offsetof(opt2s_tensor_mx4, dtype),
             offsetof(opt2s_tensor_mx4, slabs), offsetof(opt2s_tensor_mx4, scales_t), sizeof(TensorListDescMx4));
      printf("%d %d %d\n", OPT2S_MX4_BLOCK, OPT2S_MX4_MAX_GROUPS, OPT2S_MX4_PROJECT_COLS);
      return 0;
    }"""
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "p.c"), os.path.join(d, "p")
        open(c, "w").write(prog)
        cuda_inc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
        subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), "-I", cuda_inc, "-o", exe, c], check=True)
        got = [list(map(int, line.split())) for line in subprocess.run([exe], check=True, capture_output=True,
                                                                        text=True).stdout.splitlines()]
    M, S, T = B.opt2s_mx4, B.opt2s_mx4_source, B.opt2s_tensor_mx4
    assert got[0] == [ctypes.sizeof(M), M.cols.offset, ctypes.sizeof(S), S.dtype.offset]
    assert got[1] == [ctypes.sizeof(T), T.dtype.offset, T.slabs.offset, T.scales_t.offset,
                      ctypes.sizeof(B.TensorListDescMx4)]
    assert got[2] == [B.MX4_BLOCK, B.MX4_MAX_GROUPS, 32768]


def source(fake, rows=8, cols=40, slabs=1, dtype=B.OPT2S_F32, noise=False, **change):
    s = B.opt2s_mx4_source(fake(slabs * rows * cols * 4), fake(slabs * rows * cols) if noise else None, slabs, rows, cols,
                           cols, rows * cols, dtype, 0)
    for k, v in change.items():
        setattr(s, k, v)
    return s


@pytest.mark.parametrize("change", [dict(dtype=3), dict(reserved=1), dict(rows=-1), dict(cols=0), dict(slabs=0),
                                    dict(row_stride=-1), dict(slab_stride=-4), dict(x=None), dict(x=(1 << 40) + 2),
                                    dict(row_stride=1 << 41)])
def test_quantize_refuses_a_bad_source(L, change):
    f = Fake()
    s, q = source(f, **change), matrix(L, f, 1, 8, 40)
    assert L.opt2s_mx4_quantize(ctypes.byref(s), ctypes.byref(q), None, None, 0, None) == INVALID


def test_quantize_refuses(L):
    f = Fake()
    s = source(f)
    q, qt = matrix(L, f, 1, 8, 40), matrix(L, f, 1, 40, 8)
    call = lambda s_, q_, t_, off=None, g=0: L.opt2s_mx4_quantize(  # noqa: E731
        s_ and ctypes.byref(s_), q_ and ctypes.byref(q_), t_ and ctypes.byref(t_), off, g, None)
    assert call(None, q, None) == INVALID
    for bad in (dict(rows=7), dict(cols=41), dict(slabs=2), dict(codes=None), dict(scales=None), dict(codes=(1 << 40) + 8)):
        assert call(s, matrix(L, f, 1, 8, 40, **bad), None) == INVALID
        assert call(s, None, matrix(L, f, 1, 40, 8, **{k: v for k, v in bad.items() if k != "cols"} | (
            {"cols": 9} if "cols" in bad else {}))) == INVALID
    # groups: their count, the transposed form's columns, one slab only
    off = f(64)
    grouped = matrix(L, f, 1, 40, 128 + 2 * 128)
    assert call(s, q, qt, off, 2) == INVALID                  # not the padded columns
    assert call(s, q, grouped, None, 2) == INVALID            # a count without offsets
    assert call(s, q, grouped, off, 0) == INVALID
    assert call(s, q, grouped, off, B.MX4_MAX_GROUPS + 1) == INVALID
    assert call(s, q, grouped, off + 1, 2) == INVALID         # unaligned
    s2, q2 = source(f, slabs=2), matrix(L, f, 2, 8, 40)
    assert call(s2, q2, None, off, 2) == INVALID
    # overlaps
    assert call(s, matrix(L, f, 1, 8, 40, codes=s.x), None) == ALIAS
    assert call(s, q, matrix(L, f, 1, 40, 8, codes=q.codes)) == ALIAS
    sn = source(f, noise=True)
    assert call(sn, matrix(L, f, 1, 8, 40, scales=sn.noise & ~15), None) == ALIAS
    # nothing to do
    assert call(s, None, None) == 0
    assert call(source(f, rows=0), B.opt2s_mx4(None, None, 1, 0, 40), None) == 0
    # more row tiles than a launch takes
    big = source(f, rows=65536 * 128, cols=1)
    assert call(big, matrix(L, f, 1, 65536 * 128, 1), None) == TOO_LARGE


def test_dequantize_refuses(L):
    f = Fake()
    q, out = matrix(L, f, 1, 8, 40), f(8 * 40 * 4)
    call = lambda q_, o, d: L.opt2s_mx4_dequantize(q_ and ctypes.byref(q_), o, d, None)  # noqa: E731
    assert call(None, out, 0) == INVALID and call(q, None, 0) == INVALID
    assert call(q, out, 7) == INVALID and call(q, out + 2, 0) == INVALID
    assert call(q, q.codes, 0) == ALIAS
    assert call(B.opt2s_mx4(None, None, 1, 0, 40), None, 0) == 0


def test_products_refuse(L):
    f = Fake()
    a, b = matrix(L, f, 1, 6, 256), matrix(L, f, 1, 10, 256)
    d, off = f(6 * 10 * 4), f(64)
    mm = lambda a_, b_, d_=d, ldd=10, dt=0, acc=0: L.opt2s_mx4_matmul(  # noqa: E731
        a_ and ctypes.byref(a_), b_ and ctypes.byref(b_), d_, ldd, dt, acc, None)
    assert mm(None, b) == INVALID and mm(a, None) == INVALID
    assert mm(a, matrix(L, f, 1, 10, 255)) == INVALID            # contractions
    assert mm(matrix(L, f, 2, 6, 256), b) == INVALID and mm(a, matrix(L, f, 2, 10, 256)) == INVALID
    assert mm(a, b, ldd=9) == INVALID and mm(a, b, dt=5) == INVALID and mm(a, b, acc=2) == INVALID
    assert mm(a, b, d_=None) == INVALID and mm(a, b, d_=d + 1) == INVALID
    assert mm(a, b, d_=b.codes) == ALIAS and mm(a, b, d_=a.scales) == ALIAS
    assert mm(B.opt2s_mx4(None, None, 1, 0, 256), b) == 0        # no rows: nothing to do
    gr = lambda a_, b_, o=off, g=2, fill=0, acc=0: L.opt2s_mx4_matmul_grouped(  # noqa: E731
        ctypes.byref(a_), ctypes.byref(b_), o, g, d, 10, 0, acc, fill, None)
    b2 = matrix(L, f, 2, 10, 256)
    assert gr(a, b2, o=None) == INVALID and gr(a, b2, g=0) == INVALID and gr(a, b2, g=3) == INVALID
    assert gr(a, b2, fill=1, acc=1) == INVALID and gr(a, b2, fill=2) == INVALID and gr(a, b2, o=off + 2) == INVALID
    assert gr(a, b) == INVALID
    assert gr(a, b2, o=d) == ALIAS
    rg = lambda a_, b_, g=2: L.opt2s_mx4_matmul_ragged(  # noqa: E731
        ctypes.byref(a_), ctypes.byref(b_), off, g, d, 10, 0, 0, None)
    assert rg(a, b, g=3) == INVALID                              # fewer columns than the groups' padding
    assert rg(matrix(L, f, 1, 6, 300), matrix(L, f, 1, 10, 300)) == INVALID       # not whole 128-column groups
    assert rg(a, b2) == INVALID


def test_project_row_refuses(L):
    f = Fake()
    w, x, d = matrix(L, f, 1, 10, 256), f(256 * 4), f(10 * 4)
    call = lambda w_, x_=x, cols=256, xd=0, d_=d, dt=0: L.opt2s_mx4_project_row(  # noqa: E731
        x_, cols, xd, w_ and ctypes.byref(w_), d_, dt, None)
    assert call(None) == INVALID and call(w, x_=None) == INVALID and call(w, d_=None) == INVALID
    assert call(w, cols=255) == INVALID and call(w, xd=9) == INVALID and call(w, dt=-1) == INVALID
    assert call(w, x_=x + 2) == INVALID and call(w, d_=d + 1) == INVALID
    assert call(matrix(L, f, 2, 10, 256)) == INVALID
    assert call(matrix(L, f, 1, 10, 32769), cols=32769) == TOO_LARGE
    assert call(w, d_=w.codes) == ALIAS and call(w, d_=x) == ALIAS


def record(L, fake, with_copies=True, **change):
    n = 8 * 40
    t = B.opt2s_tensor_mx4(fake(n * 4), fake(n * 4), fake(n * 8), fake(n * 4), n, 0, 0, 1, 8, 40)
    if with_copies:
        q, qt = matrix(L, fake, 1, 8, 40), matrix(L, fake, 1, 40, 8)
        t.codes, t.scales, t.codes_t, t.scales_t = q.codes, q.scales, qt.codes, qt.scales
    for k, v in change.items():
        setattr(t, k, v)
    return t


def step(L, *recs, hyper=None, t=1):
    arr = (B.opt2s_tensor_mx4 * max(1, len(recs)))(*recs)
    d = B.TensorListDescMx4(arr, len(recs))
    return L.opt2s_step_mx4(ctypes.byref(d), ctypes.byref(hyper or B.make_hyper("adam")), t, None)


@pytest.mark.parametrize("change", [dict(param=None), dict(grad=None), dict(state1=None), dict(state2=None), dict(numel=-1),
                                    dict(dtype=4), dict(reserved=1), dict(rows=7), dict(cols=41), dict(slabs=2),
                                    dict(slabs=0), dict(codes=None), dict(scales=None), dict(codes_t=None),
                                    dict(scales_t=None), dict(codes=(1 << 40) + 4), dict(rows=0)])
def test_step_refuses_a_bad_record(L, change):
    f = Fake()
    assert step(L, record(L, f), record(L, f, **change)) == INVALID


def test_step_refuses(L):
    f = Fake()
    good = record(L, f)
    assert step(L, good, t=0) == INVALID
    assert step(L, good, hyper=B.make_hyper("adam", beta1=1.0)) == INVALID
    assert L.opt2s_step_mx4(None, ctypes.byref(B.make_hyper("adam")), 1, None) == INVALID
    bad = B.TensorListDescMx4(None, 2)
    assert L.opt2s_step_mx4(ctypes.byref(bad), ctypes.byref(B.make_hyper("adam")), 1, None) == INVALID
    assert step(L, good, record(L, f, codes=good.codes_t)) == ALIAS
    assert step(L, record(L, f, codes=good.param), good) == ALIAS
    assert step(L, good, good) == ALIAS                          # one tensor twice
    assert step(L) == 0 and step(L, record(L, f, numel=0)) == 0
    assert L.opt2s_mx4_errors(None) == INVALID


@needs_no_gpu
def test_well_formed_calls_reach_the_device(L):
    """Without a GPU a call that passes validation ends in OPT2S_ERR_CUDA."""
    f = Fake()
    s, q, qt = source(f), matrix(L, f, 1, 8, 40), matrix(L, f, 1, 40, 8)
    assert L.opt2s_mx4_quantize(ctypes.byref(s), ctypes.byref(q), ctypes.byref(qt), None, 0, None) == CUDA
    assert L.opt2s_mx4_dequantize(ctypes.byref(q), f(4 * 8 * 40), 0, None) == CUDA
    assert L.opt2s_mx4_matmul(ctypes.byref(q), ctypes.byref(matrix(L, f, 1, 9, 40)), f(4 * 72), 9, 0, 0, None) == CUDA
    assert step(L, record(L, f), record(L, f, with_copies=False)) == CUDA


# ---------------------------------------------------------------------------
# The Python front end
# ---------------------------------------------------------------------------

def test_python_refusals():
    x, w = torch.zeros(3, 64), torch.zeros(5, 64)
    for call in (lambda: mx4.quantize(x), lambda: mx4.quantize_pair(x), lambda: mx4.linear(x, w),
                 lambda: mx4.linear_grouped(x, w[None], torch.zeros(2, dtype=torch.int32)),
                 lambda: mx4.linear(x, w[:, :9]), lambda: mx4.linear_grouped(x, w, torch.zeros(2, dtype=torch.int32)),
                 lambda: mx4.empty_pair(torch.zeros(3)), lambda: mx4.empty_pair(torch.zeros(0, 3)),
                 lambda: mx4.MX4Tensor(torch.zeros(1, 3, 64, dtype=torch.uint8), torch.zeros(16, dtype=torch.uint8), (3, 64))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        mx4.matmul(x, w)


def test_step_list_refusals():
    p, g, m, v = torch.zeros(4, 8), torch.zeros(4, 8), torch.zeros(32), torch.zeros(32)

    class Copy:
        slabs, rows, cols, device, shape = 1, 8, 5, p.device, (8, 5)
        codes = scales = torch.zeros(1, dtype=torch.uint8)

    with pytest.raises(ValueError):
        B.TensorListMX4.from_tensors([p], [g], [m], [v], [(None, Copy)])
    with pytest.raises(ValueError):
        B.TensorListMX4.from_tensors([p.t()], [g], [m], [v], [None])
    with pytest.raises(ValueError):
        B.TensorListMX4.from_tensors([p], [g.bfloat16()], [m], [v], [None])
    with pytest.raises(ValueError):
        B.TensorListMX4.from_tensors([torch.zeros(32)], [torch.zeros(32)], [m], [v], [(None, None)])
    tl = B.TensorListMX4.from_tensors([p, v[:0]], [g, v[:0]], [m, v[:0]], [v, v[:0]], [None, None])
    assert tl.count == 2 and tl._arr[0].codes is None


def test_optimizer_refusals():
    ps = [torch.nn.Parameter(torch.zeros(4, 4)), torch.nn.Parameter(torch.zeros(4))]
    for kw in (dict(flatten=True), dict(capturable=True), dict(max_unorm=0.5), dict(lamb=True)):
        with pytest.raises(ValueError):
            optim.TwoStateOptimizer(ps, "adam", mx4=True, **kw)
    with pytest.raises(ValueError):
        optim.AdamW32bit(ps, mx4=[ps[1]])                        # one dimension
    with pytest.raises(ValueError):
        optim.AdamW32bit(ps, mx4=[torch.nn.Parameter(torch.zeros(2, 2))])      # not of this optimizer
    o = optim.AdamW32bit(ps, mx4=[ps[0]])
    with pytest.raises(ValueError):
        o.mx4_copies(ps[1])
    with pytest.raises(ValueError):
        optim.AdamW32bit(ps).mx4_copies(ps[0])
    o.refresh_mx4()                                              # no copies made yet: nothing to do
