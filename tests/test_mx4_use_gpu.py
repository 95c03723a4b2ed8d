"""How the 4-bit operators are used: kept copies, outputs that are changed in
place, sums into given tensors, and the report of waits that gave up."""
import ctypes

import pytest
import torch

from tests.mx4_support import close, product_bound, round_ref, turned_ref

pytestmark = pytest.mark.gpu


@pytest.fixture
def mx4():
    from elementwise_optimizer_b200 import binding, mx4 as m
    yield m
    n = ctypes.c_uint32()
    binding.check(binding.lib().opt2s_mx4_errors(ctypes.byref(n)), "opt2s_mx4_errors")
    assert n.value == 0


def normal(shape, seed, scale=1.0, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def offsets_of(counts):
    return torch.tensor([0] + counts, dtype=torch.int32).cumsum(0, dtype=torch.int32).cuda()


def test_copies_of_a_group_added_later(mx4):
    from elementwise_optimizer_b200 import optim
    a, b, foreign = (torch.nn.Parameter(normal((40, 96), s)) for s in (1, 2, 3))
    opt = optim.AdamW32bit([a], lr=1e-2, mx4=True)
    for p in (b, foreign):
        with pytest.raises(ValueError, match="not a parameter of this optimizer"):
            opt.mx4_copies(p)
    opt.add_param_group({"params": [b]})
    pair = opt.mx4_copies(b)
    a.grad, b.grad = torch.ones_like(a), torch.ones_like(b)
    opt.step()
    assert opt.mx4_copies(b) is pair
    for got, want in zip(pair, mx4.quantize_pair(b)):
        assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)


def test_a_step_between_forward_and_backward_is_noticed(mx4):
    """opt2s_step_mx4 writes the copies in place: a graph that saved them
    before must not use them, as after quantize_pair(out=)."""
    from elementwise_optimizer_b200 import binding as B
    w, grad, m, v = normal((40, 96), 11), normal((40, 96), 12), *(torch.zeros(40 * 96, device="cuda") for _ in range(2))
    pair = mx4.quantize_pair(w)
    tl = B.TensorListMX4.from_tensors([w], [grad], [m], [v], [pair])
    x = normal((9, 96), 13).requires_grad_()
    y = mx4.linear(x, w, copies=pair)
    mx4.opt2s_step_mx4(tl, B.make_hyper("adam", lr=0.1), 1)
    with pytest.raises(RuntimeError, match="inplace"):
        y.sum().backward()
    mx4.linear(x, w, copies=pair).sum().backward()
    assert torch.equal(x.grad, torch.autograd.grad(mx4.linear(x, w).sum(), x)[0])


def test_copies_first_asked_for_in_inference_mode(mx4):
    """An evaluation before the training: the copies that the optimizer keeps
    can be saved by a graph afterwards."""
    from elementwise_optimizer_b200 import optim
    w = torch.nn.Parameter(normal((40, 96), 21))
    opt = optim.AdamW32bit([w], lr=1e-2, mx4=True)
    x = normal((9, 96), 22).requires_grad_()
    with torch.inference_mode():
        want = mx4.linear(x, w, copies=opt.mx4_copies(w))
    for _ in range(2):
        y = mx4.linear(x, w, copies=opt.mx4_copies(w))
        assert torch.equal(y, mx4.linear(x, w)) and (want is None or torch.equal(y, want))
        want = None
        y.sum().backward()
        opt.step()
        opt.zero_grad()
        with torch.inference_mode():
            opt.refresh_mx4()


def test_copies_first_asked_for_under_capture(mx4):
    """A captured quantisation has not run when the capture ends, so what the
    optimizer would keep from then on holds no copies yet."""
    from elementwise_optimizer_b200 import optim
    w = torch.nn.Parameter(normal((40, 96), 23))
    opt = optim.AdamW32bit([w], lr=1e-2, mx4=True)
    x = normal((9, 96), 24)
    want = mx4.linear(x, w).detach()
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        x + 1
        with pytest.raises(RuntimeError, match="before the capture"):
            opt.mx4_copies(w)
    opt.mx4_copies(w)
    graph = torch.cuda.CUDAGraph()
    with torch.no_grad(), torch.cuda.graph(graph):
        y = mx4.linear(x, w, copies=opt.mx4_copies(w))
    graph.replay()
    assert torch.equal(y, want) and torch.equal(mx4.linear(x, w, copies=opt.mx4_copies(w)), want)


@pytest.mark.parametrize("shape", [(96,), (9, 96), (3, 4, 96), (0, 4, 96)])
def test_outputs_may_be_changed_in_place(mx4, shape):
    """A bias or a residual added in place, as to any layer's output."""
    w, bias = (normal(s, 31).requires_grad_() for s in ((40, 96), (40,)))
    x = normal(shape, 32).requires_grad_()
    dy = normal((*shape[:-1], 40), 33)
    y = mx4.linear(x, w)
    plain = y + bias
    want = torch.autograd.grad(plain, (x, w, bias), dy, retain_graph=True)
    y += bias
    assert torch.equal(y, plain)
    for a, b in zip(torch.autograd.grad(y, (x, w, bias), dy), want):
        assert torch.equal(a, b)
    served = mx4.project(x, mx4.quantize(w))
    plain = served + bias
    served += bias
    assert torch.equal(served, plain)
    assert torch.equal(torch.autograd.grad(served, bias, dy)[0], want[2])
    # the gradient too, as a leaf's
    mx4.linear(x, w).backward(dy)
    x.grad += bias.sum()
    assert x.grad.requires_grad


def test_the_error_count_waits_for_every_stream():
    """opt2s_mx4_errors speaks of all products in flight, those on streams
    that the legacy stream does not wait for included."""
    from elementwise_optimizer_b200 import binding
    n = ctypes.c_uint32()
    stream, done = torch.cuda.Stream(), torch.cuda.Event()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(200_000_000)               # 0.1 s
        done.record()
    assert not done.query()
    binding.check(binding.lib().opt2s_mx4_errors(ctypes.byref(n)), "opt2s_mx4_errors")
    assert done.query() and n.value == 0


@pytest.mark.parametrize("ctas,threads", [(1, 1), (1, 32), (3, 384), (300, 96)])
def test_a_wait_that_runs_out_counts_its_cta_once(testing_lib, ctas, threads):
    """A wait has a limit: each thread returns, and the error count grows by
    the CTAs that gave up, not by their threads."""
    from elementwise_optimizer_b200 import binding
    assert binding.testing_wait_runs_out(ctas, threads, 1000) == (ctas, ctas * threads)


def test_check_errors(mx4):
    w = mx4.quantize(normal((300, 8192), 71))
    mx4.project(normal((17, 8192), 72), w)
    mx4.check_errors()
    mx4.check_errors(w.device)


def test_layers_with_the_row_form_alone(mx4):
    """A program that serves keeps one form of a weight.  The other is needed
    for the input's gradient only."""
    w, ws = normal((40, 96), 81), normal((3, 40, 96), 82)
    x, off = normal((9, 96), 83), offsets_of([4, 0, 5])
    q, qs = mx4.quantize(w), mx4.quantize(ws)
    xg = x.clone().requires_grad_()
    assert torch.equal(mx4.linear(x, w, copies=(q, None)), mx4.linear(x, w))
    assert torch.equal(mx4.linear_grouped(x, ws, off, copies=(qs, None)), mx4.linear_grouped(x, ws, off))
    with torch.no_grad():
        assert torch.equal(mx4.linear(xg, w, copies=(q, None)), mx4.linear(x, w))
    wg = w.clone().requires_grad_()           # the weight's own gradient takes no copy
    dy = normal((9, 40), 84)
    got, = torch.autograd.grad(mx4.linear(x, wg, copies=(q, None)), wg, dy)
    assert torch.equal(got, torch.autograd.grad(mx4.linear(x, wg), wg, dy)[0])
    for call in (lambda: mx4.linear(xg, w, copies=(q, None)), lambda: mx4.linear_grouped(xg, ws, off, copies=(qs, None)),
                 lambda: mx4.linear(x, w, copies=(qs, None)), lambda: mx4.linear(x, w, copies=(mx4.quantize(w.t().contiguous()), None))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        mx4.linear(x, w, copies=(None, mx4.quantize_pair(w)[1]))


def added(before, y, tol, dtype):
    """(value, tolerance) of rounding before + s to `dtype`, s an fp32 sum
    within `tol` of y: the addition rounds to fp32 (2^-24 of a result of at
    most |before + y| + tol), and the result once more to `dtype`."""
    want = before + y
    tol = tol + 2.0 ** -24 * (want.abs() + tol)
    if dtype != torch.float32:
        tol = tol + torch.finfo(dtype).eps / 2 * (want.abs() + tol)
    return want, tol


def strided(shape, dtype, seed, wide):
    """(a random view of `shape` whose rows are further apart, its storage)."""
    store = normal((*shape[:-1], shape[-1] + wide), seed, dtype=dtype)
    return store[..., :shape[-1]], store


# the variants of the product: the swapped kernels (up to 16, 32 and 64 rows),
# whole and with the contraction cut over a cluster, single CTAs and pairs
@pytest.mark.parametrize("m,n,k", [(1, 40, 300), (16, 300, 8192), (17, 300, 8192), (30, 70, 200), (60, 131, 700), (50, 200, 8192),
                                   (100, 260, 520), (4000, 4090, 96)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("wide", [0, 13, 16])
def test_accumulate_in_every_variant(mx4, m, n, k, dtype, wide):
    a, b = normal((m, k), 41, 0.25), normal((n, k), 42, 0.25)
    out, store = strided((m, n), dtype, 43, wide)
    before = store.clone()
    mx4.matmul(mx4.quantize(a), mx4.quantize(b), out=out, accumulate=True)
    y, tol = product_bound(round_ref(a), round_ref(b), torch.float32)
    close(out, *added(before[..., :n].cpu().double(), y, tol, dtype))
    assert torch.equal(store[..., n:], before[..., n:])


@pytest.mark.parametrize("counts,extra", [([3, 0, 9, 1], 2), ([40, 0, 60], 0), ([300, 0, 129, 70], 5)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("wide", [0, 13])
def test_accumulate_grouped(mx4, counts, extra, dtype, wide):
    """Rows in no group stay as they were."""
    rows, n, k = sum(counts) + extra, 140, 520
    a, b = normal((rows, k), 51, 0.25), normal((len(counts), n, k), 52, 0.25)
    out, store = strided((rows, n), dtype, 53, wide)
    before = store.clone()
    mx4.matmul_grouped(mx4.quantize(a), mx4.quantize(b), offsets_of(counts), out=out, accumulate=True)
    av, bv, at = round_ref(a), round_ref(b), 0
    for e, c in enumerate(counts):
        s = slice(at, at + c)
        at += c
        y, tol = product_bound(av[s], bv[e], torch.float32)
        close(out[s], *added(before[s, :n].cpu().double(), y, tol, dtype))
    assert torch.equal(store[at:], before[at:]) and torch.equal(store[:, n:], before[:, n:])


@pytest.mark.parametrize("n,k", [(40, 96), (531, 300), (2050, 2100)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("wide", [0, 13])
def test_accumulate_expert_gradients(mx4, n, k, dtype, wide):
    """A second batch's weight gradients added to the first's: an expert
    without a token keeps what it has."""
    counts = [70, 0, 130, 1]
    dy, x, off = normal((201, n), 61, 0.25), normal((201, k), 62, 0.25), offsets_of(counts)
    out, store = strided((4, n, k), dtype, 63, wide)
    before = store.clone()
    mx4.matmul_ragged(mx4.quantize_pair(dy, offsets=off)[1], mx4.quantize_pair(x, offsets=off)[1], off, out=out, accumulate=True)
    at = 0
    for e, c in enumerate(counts):
        s = slice(at, at + c)
        at += c
        if not c:
            assert torch.equal(store[e], before[e])
            continue
        y, tol = product_bound(turned_ref(dy[s]), turned_ref(x[s]), torch.float32)
        close(out[e], *added(before[e, :, :k].cpu().double(), y, tol, dtype))
    assert torch.equal(store[..., k:], before[..., k:])


def test_stochastic_rounding_is_biased_where_it_saturates(mx4):
    """Over all 256 bytes the mean of a magnitude up to 6 times the scale is
    the value, to half a byte's step of its spacing; between 6 and 8 times the
    scale, where only a block's largest elements can lie, it is 6."""
    values = [0.1, 0.7, 1.3, 2.9, 4.5, 5.99, 6.0, 6.3, 7.0, 7.99]
    x = torch.zeros(256, 32)
    x[:, 0] = 4.0                             # with the others the block's scale is 1
    x[:, 1:1 + len(values)] = torch.tensor(values)
    x[:, 16:16 + len(values)] = -torch.tensor(values)
    r = torch.arange(256, dtype=torch.uint8)[:, None].expand(256, 32).contiguous()
    mean = mx4.quantize(x.cuda(), noise=r.cuda()).dequantize().double().cpu().mean(0)
    for i, value in enumerate(x[0, 1:1 + len(values)].double().tolist()):
        step = 0.5 if value < 2 else 1.0 if value < 4 else 2.0
        for got in (mean[1 + i].item(), -mean[16 + i].item()):
            if value <= 6.0:
                assert abs(got - value) <= step / 512 + 1e-12
            else:
                assert got == 6.0


def test_no_product_into_a_tensor_of_a_graph(mx4):
    """out= is not differentiated: written over, a tensor that requires grad
    would keep the gradient of what it held before.  As torch's own out=."""
    a, b = mx4.quantize(normal((9, 96), 91)), mx4.quantize(normal((40, 96), 92))
    leaf = torch.zeros(9, 40, device="cuda", requires_grad=True)
    for out in (leaf, leaf * 2):
        for accumulate in (False, True):
            version = out._version
            with pytest.raises(ValueError, match="requires grad"):
                mx4.matmul(a, b, out=out, accumulate=accumulate)
            assert out._version == version
    with torch.no_grad():
        assert torch.equal(mx4.matmul(a, b, out=leaf), mx4.matmul(a, b, torch.float32))


# (rows, columns, contraction): single CTAs' tiles and pairs', whole ones and partial ones
@pytest.mark.parametrize("m,n,k", [(128, 5, 64), (1217, 5, 33), (384, 132, 96), (384, 133, 200), (400, 136, 96), (4096, 4093, 64)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_columns_beside_an_output_stay(mx4, m, n, k, dtype):
    """Rows that start on 32 bytes and end off 16: what stands between them
    belongs to the caller, and there may be nothing behind the last."""
    a, b = normal((m, k), 101, 0.25), normal((n, k), 102, 0.25)
    ldd = (n + 15) // 16 * 16
    store = normal((m * ldd + 64,), 103, dtype=dtype)
    before, rows = store.clone(), store[:m * ldd].view(m, ldd)
    mx4.matmul(mx4.quantize(a), mx4.quantize(b), out=rows[:, :n])
    close(rows[:, :n], *product_bound(round_ref(a), round_ref(b), dtype))
    assert torch.equal(rows[:, n:], before[:m * ldd].view(m, ldd)[:, n:])
    assert torch.equal(store[m * ldd:], before[m * ldd:])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_columns_beside_grouped_outputs_stay(mx4, dtype):
    """The same for groups, and for the zeros of an expert without a token."""
    counts, n, k = [256, 0, 384], 133, 77
    rows, off = sum(counts), offsets_of(counts)
    x, w, dy = normal((rows, k), 111, 0.25), normal((3, n, k), 112, 0.25), normal((rows, n), 113, 0.25)
    y, dw = normal((rows, 144), 114, dtype=dtype), normal((3, n, 80), 115, dtype=dtype)
    y0, dw0 = y.clone(), dw.clone()
    mx4.matmul_grouped(mx4.quantize(x), mx4.quantize(w), off, out=y[:, :n])
    mx4.matmul_ragged(mx4.quantize_pair(dy, offsets=off)[1], mx4.quantize_pair(x, offsets=off)[1], off, out=dw[..., :k])
    assert torch.equal(y[:, n:], y0[:, n:]) and torch.equal(dw[..., k:], dw0[..., k:])
    at = 0
    for e, c in enumerate(counts):
        s = slice(at, at + c)
        at += c
        if not c:
            assert not dw[e, :, :k].any()
            continue
        close(y[s, :n], *product_bound(round_ref(x[s]), round_ref(w[e]), dtype))
        close(dw[e, :, :k], *product_bound(turned_ref(dy[s]), turned_ref(x[s]), dtype))


@pytest.mark.parametrize("counts,lead,behind", [([70, 0, 130], 3, 5), ([3, 0, 9, 1], 1, 2), ([300, 129], 40, 1)])
@pytest.mark.parametrize("noise", [False, True])
def test_rows_in_no_group_reach_nothing(mx4, counts, lead, behind, noise):
    """NaN and infinities in padding rows before and behind the groups: their
    outputs and gradients are zero, everything else as without them; and a NaN
    in one expert's token stays with that expert."""
    rows, n, k, tokens = lead + sum(counts) + behind, 140, 96, slice(lead, lead + sum(counts))
    x, dy, w = normal((rows, k), 121), normal((rows, n), 122), normal((len(counts), n, k), 123).requires_grad_()
    r = torch.randint(0, 256, (rows, n), dtype=torch.uint8).cuda() if noise else None
    off = offsets_of(counts) + lead

    def run(x, dy):
        x = x.clone().requires_grad_()
        y = mx4.linear_grouped(x, w, off, noise=r)
        return (y.detach(), *torch.autograd.grad(y, (x, w), dy))

    want = run(x, dy)
    for t in (x, dy):
        t[:lead], t[tokens.stop:] = float("nan"), float("inf")
    got = run(x, dy)
    for a, b in zip(got, want):
        assert torch.equal(a, b) and a.isfinite().all()
    for a in got[:2]:
        assert not a[:lead].any() and not a[tokens.stop:].any()
    x[lead, 5] = dy[lead, 7] = float("nan")          # the first expert's first token
    y, dx, dw = run(x, dy)
    for a in (y, dx):
        assert a[lead].isnan().all() and torch.equal(a[lead + 1:], want[0 if a is y else 1][lead + 1:])
    assert dw[0].isnan().any() and torch.equal(dw[1:], want[2][1:])
