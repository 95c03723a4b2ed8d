"""The microscaled 4-bit operators on the GPU against the plain 64-bit
implementation of mx4_support: quantisation bit for bit, products within the
bound of fp32 sums."""
import numpy as np
import pytest
import torch

from tests.mx4_support import close, encode_ref, product_bound, round_ref, turned_ref, unpack, up, values_ref

pytestmark = pytest.mark.gpu
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture
def mx4():
    from elementwise_optimizer_b200 import binding, mx4 as m
    yield m
    import ctypes
    n = ctypes.c_uint32()
    binding.check(binding.lib().opt2s_mx4_errors(ctypes.byref(n)), "opt2s_mx4_errors")
    assert n.value == 0


def gen(seed):
    return torch.Generator().manual_seed(seed)


def mixed(shape, dtype, seed, scale=1.0):
    """Normal values over some binades, with zeros and exact ties."""
    g = gen(seed)
    x = torch.randn(shape, generator=g) * torch.exp2(torch.randint(-3, 4, shape, generator=g).float())
    tie = torch.randint(0, 8, shape, generator=g)
    x = torch.where(tie == 0, torch.randint(-28, 29, shape, generator=g) * 0.25, x)
    x = torch.where(tie == 1, torch.zeros(()), x)
    return (x * scale).to(dtype).cuda()


def same_form(q, codes, scales):
    got_codes, got_scales, behind = unpack(q)
    codes, scales = codes.reshape(got_codes.shape), scales.reshape(got_scales.shape)
    np.testing.assert_array_equal(got_scales, scales)
    np.testing.assert_array_equal(got_codes, codes)
    assert not behind.any()


def check_pair(mx4, x, noise=None):
    q, qt = mx4.quantize_pair(x, noise=noise)
    xn = x.detach().cpu().double().numpy()
    nn = None if noise is None else noise.cpu().numpy()
    same_form(q, *encode_ref(xn, nn))
    same_form(qt, *encode_ref(np.swapaxes(xn, -1, -2), None if nn is None else np.swapaxes(nn, -1, -2)))
    return q, qt


# ---------------------------------------------------------------------------
# Quantisation
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 32), (3, 33), (32, 32), (128, 128), (129, 127), (5, 300), (300, 5),
                                       (257, 512)])
@pytest.mark.parametrize("noise", [False, True])
def test_quantize_pair_is_the_definition(mx4, rows, cols, dtype, noise):
    x = mixed((rows, cols), DTYPES[dtype], rows * 1000 + cols)
    r = torch.randint(0, 256, (rows, cols), generator=gen(7), dtype=torch.uint8).cuda() if noise else None
    check_pair(mx4, x, r)


def test_quantize_slabs_and_strides(mx4):
    x = mixed((3, 70, 161), torch.bfloat16, 1)
    check_pair(mx4, x)
    wide = mixed((40, 96), torch.float32, 2)
    view = wide[3:, 5:70]                     # rows 96 apart, base not 16-byte aligned
    q, qt = mx4.quantize_pair(view)
    same_form(q, *encode_ref(view.cpu().double().numpy()))
    same_form(qt, *encode_ref(view.t().cpu().double().numpy()))
    same = wide[:1].expand(33, 96)            # every row the same memory
    q, _ = mx4.quantize_pair(same)
    same_form(q, *encode_ref(same.cpu().double().numpy()))


def test_quantize_special_values(mx4):
    x = torch.zeros(8, 96)
    x[0, 5] = float("inf")
    x[1, 40] = float("nan")
    x[2, 70] = -float("inf")
    x[3, :32] = torch.finfo(torch.float32).max
    x[4, :32] = 2.0 ** -149                   # subnormal: scale 2^-127
    x[4, 32:64] = 2.0 ** -126 * 1.75
    x[5] = -0.0
    x[6, 3] = 7.9                             # saturates at 6 * 2^0
    x[6, 4] = 5.0                             # tie between 4 and 6: the even code, 4
    x[7, :7] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 4.0])
    q, qt = check_pair(mx4, x.cuda())
    v = q.dequantize()
    assert torch.isnan(v[0, :32]).all() and torch.isnan(v[1, 32:64]).all() and torch.isfinite(v[3:]).all()
    assert torch.equal(v[7, :7].cpu(), torch.tensor([0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0]))
    nan_rows = qt.dequantize().isnan().cpu()
    assert nan_rows.all(-1).nonzero().flatten().tolist() == [5, 40, 70] and int(nan_rows.sum()) == 3 * 8


def test_stochastic_rounding_is_unbiased_to_its_step(mx4):
    """All 256 bytes once on one value: the mean is the value to half a byte's
    step (1/512 of the spacing), from (r + 0.5)/256."""
    x = torch.full((256, 32), 1.3)
    x[:, 0] = 4.0                             # the block's scale is 1
    r = torch.arange(256, dtype=torch.uint8)[:, None].expand(256, 32).contiguous()
    v = mx4.quantize(x.cuda(), noise=r.cuda()).dequantize().double().cpu()
    assert set(v[:, 1].tolist()) == {1.0, 1.5}
    assert abs(v[:, 1:].mean().item() - float(np.float32(1.3))) <= 0.5 / 512 + 1e-12


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1), (5, 8), (33, 100), (2, 3, 136)])
def test_dequantize(mx4, shape, dtype):
    x = mixed(shape, torch.float32, 3)
    q = mx4.quantize(x)
    codes, scales, _ = unpack(q)
    want = torch.from_numpy(values_ref(codes, scales, shape[-1])).reshape(shape)
    got = q.dequantize(DTYPES[dtype])
    assert got.shape == want.shape and torch.equal(got.cpu(), want.to(DTYPES[dtype]))


def test_quantize_empty(mx4):
    q, qt = mx4.quantize_pair(torch.empty(0, 40, device="cuda"))
    assert q.rows == 0 and qt is None and q.dequantize().shape == (0, 40)


def offsets_of(counts):
    return torch.tensor(np.concatenate(([0], np.cumsum(counts))), dtype=torch.int32).cuda()


@pytest.mark.parametrize("counts", [[5], [0, 130, 1, 0, 300, 127, 128], [0, 0], [1] * 40])
@pytest.mark.parametrize("extra", [0, 9])
def test_quantize_grouped(mx4, counts, extra):
    rows, cols = sum(counts) + extra, 200
    if rows == 0:
        rows = 3
    x = mixed((rows, cols), torch.bfloat16, 5)
    q, qt = mx4.quantize_pair(x, offsets=offsets_of(counts))
    codes, scales = encode_ref(x.cpu().double().numpy())
    n = sum(counts)
    got_codes, got_scales, _ = unpack(q)
    np.testing.assert_array_equal(got_codes[0, :n], codes[:n])
    np.testing.assert_array_equal(got_scales[0, :n], scales[:n])
    t_codes, t_scales, _ = unpack(qt)
    want_c = np.zeros_like(t_codes[0])
    want_s = np.zeros_like(t_scales[0])
    at = row = 0
    for c in counts:
        if c:
            part_c, part_s = encode_ref(x[row:row + c].t().cpu().double().numpy())
            want_c[:, at:at + part_c.shape[1]] = part_c
            want_s[:, at // 32:at // 32 + part_s.shape[1]] = part_s
        at, row = at + up(c, 128), row + c
    np.testing.assert_array_equal(t_codes[0], want_c)
    np.testing.assert_array_equal(t_scales[0], want_s)


# ---------------------------------------------------------------------------
# Products
# ---------------------------------------------------------------------------

def gpu_close(got, a, b):
    """product_bound with the 64-bit reference on the GPU."""
    y, mag = a @ b.mT, a.abs() @ b.abs().mT
    tol = a.shape[-1] * 2.0 ** -23 * mag
    tol = tol + torch.finfo(got.dtype).eps / 2 * (y.abs() + tol)
    if got.dtype == torch.float16:
        tol = tol + 2.0 ** -25            # below 2^-14 fp16 values are 2^-24 apart: half a step, as in product_bound
    assert ((got.double() - y).abs() <= tol).all()


# every variant of the product over several rounds of its pipeline and, where
# the launch is persistent, of tiles: (rows, weight rows, columns)
LONG = [(2100, 4100, 2048), (1500, 3000, 3300), (16, 40000, 1536), (16, 300, 8192), (30, 20000, 2048), (30, 200, 16384),
        (60, 20100, 2048), (128, 40000, 1600), (100, 260, 9000), (3, 2048, 8192)]


@pytest.mark.parametrize("m,n,k", LONG)
def test_matmul_long(mx4, m, n, k):
    """With cold and warm caches, bit for bit the same every time."""
    g = torch.Generator(device="cuda").manual_seed(m + n + k)
    a, b = (mx4.quantize(torch.randn(r, k, generator=g, device="cuda")) for r in (m, n))
    flush = torch.empty(64 << 20, device="cuda")
    first = None
    for i in range(6):
        if i % 2 == 0:
            flush.normal_(generator=g)
        d = mx4.matmul(a, b, torch.float32 if i < 4 else torch.bfloat16)
        if first is None:
            first = d
            gpu_close(d, a.dequantize().double(), b.dequantize().double())
        assert torch.equal(d, first.to(d.dtype))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("groups,tokens,n,k", [(5, 3000, 700, 1500), (5, 3000, 528, 1040), (40, 1500, 520, 1300),
                                               (130, 100, 300, 2048)])
def test_grouped_long(mx4, groups, tokens, n, k, dtype):
    r = np.random.RandomState(groups)
    share = np.exp(1.5 * r.standard_normal(groups))
    counts = r.multinomial(tokens, share / share.sum()).tolist()
    g = torch.Generator(device="cuda").manual_seed(groups)
    x, dy = torch.randn(tokens, k, generator=g, device="cuda"), torch.randn(tokens, n, generator=g, device="cuda")
    w = mx4.quantize(torch.randn(groups, n, k, generator=g, device="cuda"))
    off = offsets_of(counts)
    xq, xt = mx4.quantize_pair(x, offsets=off)
    dt = mx4.quantize_pair(dy, offsets=off)[1]
    xv, wv, xtv, dtv = (t.dequantize().double() for t in (xq, w, xt, dt))
    flush = torch.empty(64 << 20, device="cuda")
    for i in range(3):
        flush.normal_(generator=g)
        y, dw = (torch.full(s, 7.0, dtype=DTYPES[dtype], device="cuda") for s in ((tokens + 3, n + 16), (groups * n, k + 16)))
        mx4.matmul_grouped(xq, w, off, out=y[:tokens, :n])
        mx4.matmul_ragged(dt, xt, off, out=dw.view(groups, n, k + 16)[..., :k])
        assert (y[tokens:] == 7).all() and (y[:, n:] == 7).all() and (dw[:, k:] == 7).all()
        y, dw = y[:tokens, :n], dw.view(groups, n, k + 16)[..., :k]
        at = col = 0
        for e, c in enumerate(counts):
            gpu_close(y[at:at + c], xv[at:at + c], wv[e])
            gpu_close(dw[e], dtv[:, col:col + c], xtv[:, col:col + c])
            at, col = at + c, col + up(c, 128)


def operand(mx4, rows, cols, seed, slabs=None, dtype=torch.float32):
    x = mixed((rows, cols) if slabs is None else (slabs, rows, cols), dtype, seed, 0.25)
    return x, mx4.quantize(x)


@pytest.mark.parametrize("m,n,k", [(128, 128, 64), (128, 256, 128), (1, 8, 32), (1, 128, 256), (16, 300, 1024),
                                   (17, 40, 40), (33, 129, 700), (64, 512, 2048), (65, 96, 96), (200, 100, 130),
                                   (300, 520, 1000), (1, 2048, 4100), (515, 700, 33)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_matmul(mx4, m, n, k, dtype):
    a, qa = operand(mx4, m, k, m + n)
    b, qb = operand(mx4, n, k, n + k + 1)
    y, tol = product_bound(round_ref(a), round_ref(b), DTYPES[dtype])
    close(mx4.matmul(qa, qb, DTYPES[dtype]), y, tol)


@pytest.mark.parametrize("counts", [[5], [0, 130, 1, 0, 300, 127, 128], [3, 0, 2, 9], [40, 10, 0, 60], [1] * 40, [0, 0]])
@pytest.mark.parametrize("extra", [0, 9])
@pytest.mark.parametrize("n,k", [(40, 96), (300, 520)])
def test_matmul_grouped(mx4, counts, extra, n, k):
    rows = max(1, sum(counts) + extra)
    a, qa = operand(mx4, rows, k, 11)
    b, qb = operand(mx4, n, k, 12, slabs=len(counts))
    offsets = offsets_of(counts)
    got = mx4.matmul_grouped(qa, qb, offsets, torch.float32)
    av, bv = round_ref(a), round_ref(b)
    want, tol = torch.zeros(rows, n, dtype=torch.float64), torch.zeros(rows, n, dtype=torch.float64)
    at = 0
    for e, c in enumerate(counts):
        want[at:at + c], tol[at:at + c] = product_bound(av[at:at + c], bv[e], torch.float32)
        at += c
    close(got, want, tol)
    assert not got[at:].any()
    # into a given tensor: rows in no group stay as they were
    out = torch.full((rows, n), 7.0, device="cuda")
    mx4.matmul_grouped(qa, qb, offsets, out=out)
    assert torch.equal(out[:at], got[:at]) and (out[at:] == 7.0).all()


@pytest.mark.parametrize("counts", [[5], [0, 130, 1, 0, 300, 127, 128], [64, 0, 65], [0, 0]])
@pytest.mark.parametrize("n,k", [(40, 96), (131, 257)])
def test_matmul_ragged(mx4, counts, n, k):
    rows = max(1, sum(counts))
    dy, x = mixed((rows, n), torch.float32, 21, 0.25), mixed((rows, k), torch.float32, 22, 0.25)
    offsets = offsets_of(counts)
    a, b = mx4.quantize_pair(dy, offsets=offsets)[1], mx4.quantize_pair(x, offsets=offsets)[1]
    got = mx4.matmul_ragged(a, b, offsets, torch.float32)
    at = 0
    for e, c in enumerate(counts):
        if c:
            y, tol = product_bound(turned_ref(dy[at:at + c]), turned_ref(x[at:at + c]), torch.float32)
            close(got[e], y, tol)
        else:
            assert not got[e].any()
        at += c


def test_matmul_accumulate_and_strides(mx4):
    a, qa = operand(mx4, 70, 200, 31)
    b, qb = operand(mx4, 90, 200, 32)
    y, tol = product_bound(round_ref(a), round_ref(b), torch.float32)
    big = torch.randn(70, 123, generator=gen(3)).cuda()
    before = big.clone()
    out = big[:, 5:95]                        # rows 123 apart, base not 16-byte aligned
    mx4.matmul(qa, qb, out=out, accumulate=True)
    want = before[:, 5:95].cpu().double() + y
    close(out, want, tol + 2.0 ** -23 * (want.abs() + before[:, 5:95].cpu().abs()))
    assert torch.equal(big[:, :5], before[:, :5]) and torch.equal(big[:, 95:], before[:, 95:])
    for dtype in (torch.bfloat16, torch.float16):
        y, tol = product_bound(round_ref(a), round_ref(b), dtype)
        out = torch.ones(70, 90, dtype=dtype, device="cuda")
        mx4.matmul(qa, qb, out=out, accumulate=True)
        close(out, y + 1, tol + torch.finfo(dtype).eps)      # 1 + y rounds relative to at most |y| + 1


def test_nan_block_reaches_only_its_row_and_column(mx4):
    a, b = mixed((140, 256), torch.float32, 41), mixed((150, 256), torch.float32, 42)
    a[7, 100] = float("nan")
    b[133, 3] = float("inf")
    d = mx4.matmul(mx4.quantize(a), mx4.quantize(b), torch.float32)
    bad = torch.zeros(140, 150, dtype=torch.bool)
    bad[7] = True
    bad[:, 133] = True
    assert torch.equal(d.isnan().cpu(), bad)


# ---------------------------------------------------------------------------
# Layers
# ---------------------------------------------------------------------------

def layer_ref(x, w, dy, noise=None):
    """(y, dx, dw) of the layer in 64 bits, each with its operands' magnitudes."""
    return ((round_ref(x), round_ref(w)), (round_ref(dy, noise), turned_ref(w)), (turned_ref(dy, noise), turned_ref(x)))


@pytest.mark.parametrize("lead,n,k", [((1,), 48, 64), ((3, 7), 100, 70), ((130,), 260, 129), ((600,), 300, 513)])
@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("f32", "f32"), ("f16", "f32")])
@pytest.mark.parametrize("noise", [False, True])
def test_linear(mx4, lead, n, k, dtype, wdtype, noise):
    x = mixed((*lead, k), DTYPES[dtype], 51, 0.25).requires_grad_()
    w = mixed((n, k), DTYPES[wdtype], 52, 0.25).requires_grad_()
    dy = mixed((*lead, n), DTYPES[dtype], 53, 0.25)
    r = torch.randint(0, 256, (*lead, n), generator=gen(8), dtype=torch.uint8).cuda() if noise else None
    for copies in (None, mx4.quantize_pair(w)):
        y = mx4.linear(x, w, copies=copies, noise=r)
        dx, dw = torch.autograd.grad(y, (x, w), dy)
        assert y.shape == (*lead, n) and y.dtype == x.dtype and dx.dtype == x.dtype and dw.dtype == w.dtype
        pairs = layer_ref(x.reshape(-1, k), w, dy.reshape(-1, n), None if r is None else r.reshape(-1, n))
        for got, (a, b) in zip((y.reshape(-1, n), dx.reshape(-1, k), dw), pairs):
            close(got, *product_bound(a, b, got.dtype))


def test_linear_gradient_is_that_of_the_straight_through_layer(mx4):
    """Against differences: with operands that 4 bits hold exactly the layer is
    linear, so the loss' central difference along a direction equals its
    gradient's product with it."""
    g = gen(61)
    x = torch.randint(-2, 3, (9, 64), generator=g).float().cuda()
    w = torch.randint(-2, 3, (33, 64), generator=g).float().cuda()
    dy = torch.randint(-2, 3, (9, 33), generator=g).float().cuda()
    for t in (x, w, dy):                      # every block of both forms has the largest magnitude 4 or 2
        t[0, :] = 2.0
        t[:, ::32] = 2.0
    x.requires_grad_()
    w.requires_grad_()
    dx, dw = torch.autograd.grad(mx4.linear(x, w), (x, w), dy)
    assert torch.equal(dx, dy @ w) and torch.equal(dw, dy.t() @ x)
    v = torch.zeros_like(w)
    v[3, 5] = 1.0
    with torch.no_grad():
        diff = ((mx4.linear(x, w + v) - mx4.linear(x, w - v)) * dy).sum() / 2
    assert abs(w[3, 5].item()) <= 2 and diff.item() == dw[3, 5].item()


def test_linear_gradient_of_one_operand_and_broadcast_gradient(mx4):
    x, w = mixed((40, 96), torch.float32, 71), mixed((50, 96), torch.float32, 72)
    xg, wg = x.clone().requires_grad_(), w.clone().requires_grad_()
    mx4.linear(xg, w).sum().backward()        # the gradient arrives as an expanded scalar
    mx4.linear(x, wg).sum().backward()
    ones = torch.ones(40, 50)
    _, dx, dw = layer_ref(x, w, ones)
    close(xg.grad, *product_bound(*dx, torch.float32))
    close(wg.grad, *product_bound(*dw, torch.float32))
    y = mx4.linear(x[:0].requires_grad_(), wg)
    assert y.shape == (0, 50)
    wg.grad = None
    y.sum().backward()
    assert not wg.grad.any()
    # a transposed input and a transposed gradient
    xt = x.t().contiguous().t().requires_grad_()
    gx, = torch.autograd.grad(mx4.linear(xt, w), (xt,), torch.ones(50, 40, device="cuda").t())
    assert torch.equal(gx, xg.grad)


@pytest.mark.parametrize("counts,extra", [([5], 0), ([0, 130, 1, 0, 60], 0), ([33, 0, 20], 4), ([0, 0], 2)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("noise", [False, True])
def test_linear_grouped(mx4, counts, extra, dtype, noise):
    rows, n, k = sum(counts) + extra, 140, 96
    x = mixed((rows, k), DTYPES[dtype], 81, 0.25).requires_grad_()
    w = mixed((len(counts), n, k), DTYPES[dtype], 82, 0.25).requires_grad_()
    dy = mixed((rows, n), DTYPES[dtype], 83, 0.25)
    r = torch.randint(0, 256, (rows, n), generator=gen(9), dtype=torch.uint8).cuda() if noise else None
    y = mx4.linear_grouped(x, w, offsets_of(counts), noise=r)
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    at = 0
    for e, c in enumerate(counts):
        s = slice(at, at + c)
        at += c
        if not c:
            assert not dw[e].any()
            continue
        pairs = layer_ref(x[s], w[e], dy[s], None if r is None else r[s])
        for got, (a, b) in zip((y[s], dx[s], dw[e]), pairs):
            close(got, *product_bound(a, b, got.dtype))
    assert not y[at:].any() and not dx[at:].any()


def test_project_matches_linear(mx4):
    x, w = mixed((2, 5, 96), torch.bfloat16, 91), mixed((50, 96), torch.bfloat16, 92)
    wq = mx4.quantize(w)
    assert torch.equal(mx4.project(x, wq), mx4.linear(x, w))
    assert mx4.project(x, wq, torch.float32).dtype == torch.float32
    ws = mixed((3, 50, 96), torch.bfloat16, 93)
    off = offsets_of([4, 0, 5])
    x2 = x.reshape(10, 96)
    assert torch.equal(mx4.project_grouped(x2, mx4.quantize(ws), off), mx4.linear_grouped(x2, ws, off))


@pytest.mark.parametrize("n,k", [(1, 32), (17, 100), (300, 2048), (40, 4100), (128, 131), (33, 32768), (5, 32769)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_project_one_row(mx4, n, k, dtype):
    """One row of up to 32,768 columns takes a kernel of its own: exact integer
    sums of each block, fp32 sums over the blocks."""
    x, w = mixed((1, k), DTYPES[dtype], 141, 0.25), mixed((n, k), torch.float32, 142, 0.25)
    y, tol = product_bound(round_ref(x), round_ref(w), DTYPES[dtype])
    close(mx4.project(x, mx4.quantize(w)), y, tol)
    wide = torch.empty(1, k + 3, dtype=x.dtype, device="cuda")[:, 1:k + 1].copy_(x)      # off 16 bytes
    assert torch.equal(mx4.project(wide, mx4.quantize(w)), mx4.project(x, mx4.quantize(w)))


@pytest.mark.parametrize("counts,extra", [([1, 0, 2, 1], 0), ([0, 7, 0, 0], 1), ([0, 0, 0], 2), ([3, 3, 0, 0, 0], 3)])
def test_project_grouped_few_rows(mx4, counts, extra):
    rows, n, k = sum(counts) + extra, 70, 260
    x, w = mixed((rows, k), torch.bfloat16, 151, 0.25), mixed((len(counts), n, k), torch.float32, 152, 0.25)
    got = mx4.project_grouped(x, mx4.quantize(w), offsets_of(counts), torch.float32)
    at = 0
    for e, c in enumerate(counts):
        if c:
            close(got[at:at + c], *product_bound(round_ref(x[at:at + c]), round_ref(w[e]), torch.float32))
        at += c
    assert not got[at:].any()


@pytest.mark.parametrize("rows", [1, 3])
def test_scales_at_both_ends_and_nan(mx4, rows):
    """Scales at both ends of their range, and blocks that are NaN."""
    w = torch.zeros(3, 64)
    w[0, :32], w[1, 40], w[2, 3] = 2.0 ** -126, 1.0, 1.0
    for x0, bad in ((2.0 ** 125, False), (2.0 ** -100, True)):       # 32 * 2^-1 through scales 2^123 and 2^-127
        x = torch.zeros(rows, 64)
        x[0, :32] = x0
        if bad:
            x[0, 40] = float("nan")
        got = mx4.project(x.cuda(), mx4.quantize(w.cuda())).cpu()
        want = round_ref(x) @ round_ref(w).mT
        assert torch.equal(got.isnan(), want.isnan()) and got[0].isnan().all() == bad
        if not bad:
            assert torch.equal(got, want.float()) and got[0, 0].item() == 16.0


# ---------------------------------------------------------------------------
# How they are called
# ---------------------------------------------------------------------------

def test_refusals(mx4):
    """Arguments that do not fit together, on the GPU's tensors."""
    from elementwise_optimizer_b200 import Opt2sError
    x, w = mixed((6, 96), torch.float32, 161), mixed((10, 96), torch.float32, 162)
    ws = mixed((2, 10, 96), torch.float32, 163)
    xq, wq, wsq = mx4.quantize(x), mx4.quantize(w), mx4.quantize(ws)
    off = offsets_of([2, 4])
    wide = torch.empty(6, 20, device="cuda")
    bad = [lambda: mx4.quantize(x[0]), lambda: mx4.quantize(x[None, None]), lambda: mx4.quantize(x.t()),
           lambda: mx4.quantize(x[:, :0]), lambda: mx4.quantize(ws[:0]),
           lambda: mx4.quantize(x, noise=torch.zeros(6, 95, dtype=torch.uint8, device="cuda")),
           lambda: mx4.quantize(x, noise=torch.zeros(6, 96, device="cuda")),
           lambda: mx4.quantize_pair(x, offsets=off.long()), lambda: mx4.quantize_pair(x, offsets=off[:1]),
           lambda: mx4.quantize_pair(x, offsets=off.cpu()), lambda: mx4.quantize_pair(ws, offsets=off),
           lambda: mx4.quantize_pair(x, out=mx4.empty_pair(w)),
           lambda: mx4.quantize_pair(x, offsets=torch.zeros(1026, dtype=torch.int32, device="cuda")),
           lambda: mx4.matmul(xq, mx4.quantize(w[:, :95])), lambda: mx4.matmul(xq, wsq), lambda: mx4.matmul(wsq, xq),
           lambda: mx4.matmul(xq, wq, accumulate=True), lambda: mx4.matmul(xq, wq, out=wide),
           lambda: mx4.matmul(xq, wq, dtype=torch.float32, out=wide[:, :10].bfloat16()),
           lambda: mx4.matmul(xq, wq, out=wide[:, ::2]), lambda: mx4.matmul_grouped(xq, wsq, offsets_of([1, 2, 3])),
           lambda: mx4.matmul_grouped(xq, wq, off), lambda: mx4.matmul_ragged(xq, wq, off),
           lambda: mx4.project(x[:, :95], wq), lambda: mx4.project(x, wsq), lambda: mx4.project_grouped(x, wq, off),
           lambda: mx4.linear(x, ws), lambda: mx4.linear(x, w.cpu()), lambda: mx4.linear(x, w, copies=mx4.quantize_pair(x)),
           lambda: mx4.linear(x, w, noise=torch.zeros(6, 9, dtype=torch.uint8, device="cuda")),
           lambda: mx4.linear_grouped(x, ws, offsets_of([6])), lambda: mx4.linear_grouped(x[None], ws, off),
           lambda: mx4.linear(x, w[:0])]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    for call in (lambda: mx4.quantize(x.double()), lambda: mx4.linear(x.int(), w), lambda: mx4.matmul(x, wq),
                 lambda: mx4.matmul(xq, wq, dtype=torch.float64), lambda: xq.dequantize(torch.int8)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(Opt2sError, match="ALIAS"):            # the output in an operand's memory
        mx4.matmul(xq, wq, out=xq.codes.view(torch.bfloat16).flatten()[:60].view(6, 10))
    # a copy written between forward and backward, and a gradient of the gradient
    xg = x.clone().requires_grad_()
    pair = mx4.quantize_pair(w)
    y = mx4.linear(xg, w, copies=pair)
    mx4.quantize_pair(w * 2, out=pair)
    with pytest.raises(RuntimeError, match="inplace"):
        y.sum().backward()
    y = mx4.linear(xg, w)
    with pytest.raises(NotImplementedError):
        torch.autograd.grad(y, xg, torch.ones_like(y).requires_grad_(), create_graph=True)


def test_no_gradient_of_a_gradient_is_lost(mx4):
    """dx depends on the weight whether or not dy asks for a gradient."""
    x, w = (mixed(s, torch.float32, 221).requires_grad_() for s in ((4, 64), (8, 64)))
    y = mx4.linear(x, w)
    with pytest.raises(NotImplementedError):
        torch.autograd.grad(y, x, torch.ones_like(y), create_graph=True)


def test_as_many_groups_as_there_may_be(mx4):
    r = np.random.RandomState(3)
    counts = r.multinomial(700, np.full(1024, 1 / 1024)).tolist()
    x, w, dy = mixed((700, 64), torch.float32, 201, 0.25), mixed((1024, 16, 64), torch.float32, 202, 0.25), \
        mixed((700, 16), torch.float32, 203, 0.25)
    off = offsets_of(counts)
    x.requires_grad_()
    w.requires_grad_()
    y = mx4.linear_grouped(x, w, off)
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    xv, wv, dv, wt = round_ref(x), round_ref(w), round_ref(dy), turned_ref(w)
    at = 0
    for e, c in enumerate(counts):
        s = slice(at, at + c)
        at += c
        close(y[s], *product_bound(xv[s], wv[e], torch.float32))
        close(dx[s], *product_bound(dv[s], wt[e], torch.float32))
        if c and e % 16 == 0:
            close(dw[e], *product_bound(turned_ref(dy[s]), turned_ref(x[s]), torch.float32))
        assert c or not dw[e].any()


def test_inference_mode_and_a_graph_used_twice(mx4):
    x, w = mixed((9, 96), torch.float32, 211), mixed((40, 96), torch.float32, 212)
    want = mx4.linear(x, w)
    with torch.inference_mode():
        pair = mx4.quantize_pair(w)
        assert torch.equal(mx4.linear(x, w), want) and torch.equal(mx4.linear(x, w, copies=pair), want)
        assert torch.equal(mx4.project(x, pair[0]), want)
        mx4.quantize_pair(w, out=pair)
        mx4.matmul(mx4.quantize(x), pair[0], out=torch.empty(9, 40, device="cuda"))
    d = torch.empty(9, 40, device="cuda")
    before = d._version
    mx4.matmul(mx4.quantize(x), pair[0], out=d)
    assert d._version > before
    xg = x.clone().requires_grad_()
    y = mx4.linear(xg, w)
    a, = torch.autograd.grad(y, xg, torch.ones_like(y), retain_graph=True)
    b, = torch.autograd.grad(y, xg, torch.ones_like(y))
    assert torch.equal(a, b)
    # checkpointing runs the forward again
    from torch.utils.checkpoint import checkpoint
    c, = torch.autograd.grad(checkpoint(lambda t: mx4.linear(t, w), xg, use_reentrant=False), xg, torch.ones_like(y))
    assert torch.equal(a, c)


@pytest.mark.parametrize("need", [(True, True), (True, False), (False, True)])
def test_empty_batch_of_experts(mx4, need):
    x = torch.empty(0, 96, device="cuda", requires_grad=need[0])
    w = mixed((3, 40, 96), torch.float32, 171).requires_grad_(need[1])
    y = mx4.linear_grouped(x, w, offsets_of([0, 0, 0]))
    assert y.shape == (0, 40)
    y.sum().backward()
    assert (x.grad is not None and x.grad.shape == x.shape) == need[0]
    assert not need[1] or (w.grad.shape == w.shape and not w.grad.any())


def test_one_dimensional_and_deep_inputs(mx4):
    x, w = mixed((96,), torch.float32, 181).requires_grad_(), mixed((40, 96), torch.float32, 182)
    y = mx4.linear(x, w)
    assert y.shape == (40,) and mx4.project(x, mx4.quantize(w)).shape == (40,)
    gx, = torch.autograd.grad(y, x, torch.ones(40, device="cuda"))
    gr, = torch.autograd.grad(mx4.linear(x[None, None], w), x, torch.ones(1, 1, 40, device="cuda"))
    assert gx.shape == (96,) and torch.equal(gx, gr)


def test_past_32_bits(mx4):
    """A source of 2^32 and some elements, and an output of as many."""
    rows, cols = 66000, 65536
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    x.normal_(generator=g)
    q, qt = mx4.quantize_pair(x)
    tail = x[-3:].cpu()
    v = round_ref(tail)
    cp = cols // 2
    codes, scales = encode_ref(tail.double().numpy())
    raw = q.codes[0, -3:].cpu().numpy()
    np.testing.assert_array_equal(np.stack((raw & 15, raw >> 4), -1).reshape(3, cols), codes)
    assert q.codes.shape[-1] == cp
    raw = qt.codes[0, -2:].cpu().numpy()
    codes, _ = encode_ref(x[:, -2:].t().cpu().double().numpy())
    np.testing.assert_array_equal(np.stack((raw & 15, raw >> 4), -1).reshape(2, -1)[:, :rows], codes[:, :rows])
    got = q.dequantize(torch.bfloat16)
    assert torch.equal(got[-3:].cpu().double(), v)
    del got, qt, x
    a = mx4.quantize(mixed((rows, 64), torch.float32, 191))
    b = mx4.quantize(mixed((cols, 64), torch.float32, 192))
    d = mx4.matmul(a, b)
    want = a.dequantize()[-5:].double().cpu() @ b.dequantize()[-300:].double().cpu().mT
    close(d[-5:, -300:], want, want.abs() * 2.0 ** -8 + 64 * 2.0 ** -23 * (a.dequantize()[-5:].double().abs().cpu()
                                                                         @ b.dequantize()[-300:].double().abs().cpu().mT))


def test_offsets_out_of_range_stay_in_bounds(mx4):
    """Clamped to the rows and to be non-decreasing: no access out of range,
    and the groups that remain are right."""
    x = mixed((50, 64), torch.float32, 101)
    w = mixed((4, 40, 64), torch.float32, 102)
    bad = torch.tensor([-7, 20, 10, 90, 60], dtype=torch.int32).cuda()       # as 0, 20, 20, 50, 50
    good = torch.tensor([0, 20, 20, 50, 50], dtype=torch.int32).cuda()
    xq, wq = mx4.quantize(x), mx4.quantize(w)
    assert torch.equal(mx4.matmul_grouped(xq, wq, bad), mx4.matmul_grouped(xq, wq, good))
    for a, b in zip(mx4.quantize_pair(x, offsets=bad), mx4.quantize_pair(x, offsets=good)):
        assert torch.equal(a.dequantize(), b.dequantize())


def test_other_stream_and_repeat_are_bitwise_equal(mx4):
    x, w = mixed((300, 512), torch.bfloat16, 111), mixed((400, 512), torch.bfloat16, 112)
    want = mx4.linear(x, w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = [mx4.linear(x, w) for _ in range(3)]
    s.synchronize()
    assert all(torch.equal(g, want) for g in got)


def test_two_streams_at_once(mx4):
    xs = [mixed((m, 1024), torch.bfloat16, 120 + m) for m in (5, 40, 200)]
    w = mx4.quantize(mixed((640, 1024), torch.bfloat16, 121))
    want = [mx4.project(x, w) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[] for _ in xs]
    for _ in range(20):
        for i, (s, x) in enumerate(zip(streams, xs)):
            with torch.cuda.stream(s):
                got[i].append(mx4.project(x, w))
    torch.cuda.synchronize()
    for g, y in zip(got, want):
        assert all(torch.equal(v, y) for v in g)


def test_every_kernel_at_once(mx4):
    """Products of all variants, quantisations and a one-row product on five
    streams together, as often as they fit: the same bits as alone."""
    g = torch.Generator(device="cuda").manual_seed(5)
    xs = [torch.randn(m, 2048, generator=g, device="cuda").bfloat16() for m in (1, 12, 30, 60, 120, 2100)]
    w = mx4.quantize(torch.randn(4100, 2048, generator=g, device="cuda"))
    want = [(mx4.project(x, w), mx4.quantize_pair(x)[1].codes) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(5)]
    got = []
    for i in range(40):
        with torch.cuda.stream(streams[i % 5]):
            k = i * 7 % len(xs)
            got.append((k, mx4.project(xs[k], w), mx4.quantize_pair(xs[k])[1].codes))
    torch.cuda.synchronize()
    for k, y, codes in got:
        assert torch.equal(y, want[k][0]) and torch.equal(codes, want[k][1])


def test_captured_forward_and_backward(mx4):
    """A layer's forward and backward in a CUDA graph, replayed on new inputs,
    beside a second captured graph."""
    x = mixed((70, 96), torch.float32, 131).requires_grad_()
    w = mixed((2, 50, 96), torch.float32, 132).requires_grad_()
    off = offsets_of([30, 35])
    dy = mixed((70, 50), torch.float32, 133)

    def step():
        y = mx4.linear_grouped(x, w, off)
        return (y.detach(), *torch.autograd.grad(y, (x, w), dy))

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, out))
    for seed in (134, 135):
        with torch.no_grad():
            x.copy_(mixed((70, 96), torch.float32, seed))
            off.copy_(offsets_of([seed - 130, 40]))
        want = [t.clone() for t in step()]
        for g, out in graphs:
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want))
