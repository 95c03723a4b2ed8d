"""The step that writes 4-bit copies: params and states bit for bit as
opt2s_step leaves them, copies bit for bit the quantisation of the new params;
and a small model trained through the 4-bit products."""
import pytest
import torch

from tests.mx4_support import close, product_bound, turned_ref

pytestmark = pytest.mark.gpu
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def collection(shapes, dtypes, algo, seed, shift=0):
    """Tensors (param, grad, state1, state2); shift > 0: each array starts
    that many elements into its storage."""
    g = torch.Generator().manual_seed(seed)

    def make(shape, dtype, scale, square=False, twice=False):
        n = torch.Size(shape).numel() * (2 if twice else 1)
        x = torch.randn(n + shift, generator=g) * scale
        x = (x.square() if square else x).to(dtype).cuda()[shift:]
        return x if twice else x.view(shape)

    out = []
    for i, shape in enumerate(shapes):
        dt = DTYPES[dtypes[i % len(dtypes)]]
        p, gr = make(shape, dt, 1.0), make(shape, dt, 1e-2)
        gr.view(-1)[::7] = 0.0
        out.append((p, gr, make(shape, torch.float32, 1e-3, twice=algo == "ademamix").reshape(-1),
                    make(shape, torch.float32, 1e-2, square=True).reshape(-1)))
    return out


def clones(ts, shift):
    def one(x):
        if not shift:
            return x.clone()
        y = torch.empty(x.numel() + shift, dtype=x.dtype, device=x.device)[shift:].view(x.shape)
        return y.copy_(x)
    return [tuple(one(x) for x in t) for t in ts]


SHAPES = [(1, 1), (5,), (33, 64), (128, 128), (2, 70, 136), (129, 100), (1, 257), (300, 31), (9000,), (257, 200), (0, 4), (1,)]


@pytest.mark.parametrize("algo", ["adam", "ademamix"])
@pytest.mark.parametrize("skip", [False, True])
@pytest.mark.parametrize("dtypes", [["f32"], ["bf16"], ["f16"], ["f32", "bf16", "f16"]])
@pytest.mark.parametrize("shift", [0, 1])
def test_step_mx4_is_step_and_quantise(algo, skip, dtypes, shift):
    from elementwise_optimizer_b200 import binding as B, mx4
    a = collection(SHAPES, dtypes, algo, 1, shift)
    b = clones(a, shift)
    copies = [mx4.empty_pair(t[0]) if t[0].dim() > 1 and t[0].numel() else None for t in a]
    for i, c in enumerate(copies):            # leave out one form of some
        if c is not None and i % 4 == 1:
            copies[i] = (c[0], None)
        if c is not None and i % 4 == 2:
            copies[i] = (None, c[1])
    h = B.make_hyper(algo, lr=1e-2, weight_decay=0.1, beta3=0.9999, alpha=5.0, skip_zeros=skip)
    plain = B.TensorList.from_tensors(*zip(*b))
    with_copies = B.TensorListMX4.from_tensors(*zip(*a), copies)
    n0 = B.launch_count()
    for t in (1, 2, 3):
        B.opt2s_step_mx4(with_copies, h, t)
    assert B.launch_count() - n0 == 3
    for t in (1, 2, 3):
        B.opt2s_step(plain, h, t)
    for x, y in zip(a, b):
        for k in (0, 2, 3):
            assert torch.equal(x[k], y[k])
        assert torch.equal(x[1], y[1])        # gradients unchanged
    for (p, *_), c in zip(a, copies):
        if c is not None:
            for got, want in zip(c, mx4.quantize_pair(p)):
                if got is not None:
                    assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)


def test_step_mx4_many_tensors():
    """More records than one launch takes."""
    from elementwise_optimizer_b200 import binding as B, mx4
    shapes = [(1 + i % 5, 3 + i % 40) if i % 3 else (1 + i % 90,) for i in range(600)]
    a = collection(shapes, ["f32", "bf16"], "adam", 2)
    b = clones(a, 0)
    copies = [mx4.empty_pair(t[0]) if t[0].dim() > 1 else None for t in a]
    h = B.make_hyper("adamw", weight_decay=0.01)
    n0 = B.launch_count()
    B.opt2s_step_mx4(B.TensorListMX4.from_tensors(*zip(*a), copies), h, 1)
    assert B.launch_count() - n0 == 3
    B.opt2s_step(B.TensorList.from_tensors(*zip(*b)), h, 1)
    for x, y in zip(a, b):
        assert all(torch.equal(u, v) for u, v in zip(x, y))
    for (p, *_), c in zip(a, copies):
        if c is not None:
            assert all(torch.equal(g.codes, w.codes) and torch.equal(g.scales, w.scales)
                       for g, w in zip(c, mx4.quantize_pair(p)))


def test_step_mx4_captured():
    from elementwise_optimizer_b200 import binding as B, mx4
    a = collection([(130, 96), (77,)], ["bf16"], "adam", 3)
    b = clones(a, 0)
    copies = [mx4.empty_pair(a[0][0]), None]
    h = B.make_hyper("adamw", lr=1e-2)
    tl, plain = B.TensorListMX4.from_tensors(*zip(*a), copies), B.TensorList.from_tensors(*zip(*b))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.opt2s_step_mx4(tl, h, 4)
    for _ in range(3):
        g.replay()
        B.opt2s_step(plain, h, 4)
    torch.cuda.synchronize()
    for x, y in zip(a, b):
        assert all(torch.equal(u, v) for u, v in zip(x, y))
    assert torch.equal(copies[0][1].codes, mx4.quantize_pair(a[0][0])[1].codes)


def test_optimizer_keeps_copies():
    """AdamW32bit(mx4=...) steps as without copies and its copies follow the
    parameters; a replaced gradient tensor and refresh_mx4 included."""
    from elementwise_optimizer_b200 import mx4, optim
    g = torch.Generator().manual_seed(5)
    ps = [torch.nn.Parameter(torch.randn(s, generator=g).cuda()) for s in [(64, 96), (3, 40, 70), (50,)]]
    qs = [torch.nn.Parameter(p.detach().clone()) for p in ps]
    opt, ref = optim.AdamW32bit(ps, lr=1e-2, mx4=True), optim.AdamW32bit(qs, lr=1e-2)
    first = [opt.mx4_copies(p) for p in ps[:2]]
    for step in range(4):
        for p, q in zip(ps, qs):
            p.grad = torch.randn(p.shape, generator=g).cuda()
            q.grad = p.grad.clone()
        opt.step()
        ref.step()
        assert all(torch.equal(p, q) for p, q in zip(ps, qs))
        for p, pair in zip(ps[:2], first):
            assert opt.mx4_copies(p) is pair
            for got, want in zip(pair, mx4.quantize_pair(p)):
                assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)
    with torch.no_grad():
        ps[0].mul_(3.0)
    opt.refresh_mx4()
    assert torch.equal(first[0][0].codes, mx4.quantize(ps[0]).codes)
    with pytest.raises(ValueError):
        opt.mx4_copies(ps[2])


def test_model_trained_through_copies():
    """Three steps of a two-layer model with experts: the products read the
    copies that the step writes, their gradients are the formula's, and a run
    without kept copies gives the same bits."""
    from elementwise_optimizer_b200 import mx4, optim
    shapes = [(96, 64), (3, 80, 96)]
    off = torch.tensor([0, 20, 20, 50], dtype=torch.int32).cuda()

    def run(keep):
        gg = torch.Generator().manual_seed(7)
        ws = [torch.nn.Parameter((torch.randn(s, generator=gg) * 0.1).cuda()) for s in shapes]
        opt = optim.AdamW32bit(ws, lr=1e-2, mx4=ws if keep else False)
        copies = (lambda w: opt.mx4_copies(w)) if keep else (lambda w: None)
        for _ in range(3):
            x = torch.randn(50, 64, generator=gg).cuda()
            h = torch.relu(mx4.linear(x, ws[0], copies=copies(ws[0])))
            y = mx4.linear_grouped(h, ws[1], off, copies=copies(ws[1]))
            y.square().mean().backward()
            opt.step()
            last = (x, h.detach(), y.detach(), [w.grad.clone() for w in ws])
            opt.zero_grad()
        return ws, last

    (wa, a), (wb, b) = run(True), run(False)
    assert all(torch.equal(u, v) for u, v in zip(wa, wb))
    assert torch.equal(a[2], b[2]) and all(torch.equal(u, v) for u, v in zip(a[3], b[3]))
    # the last step's expert gradient against the formula
    x, h, y, grads = a
    dy = (2.0 * y / y.numel()).cpu()
    for e, s in ((0, slice(0, 20)), (2, slice(20, 50))):
        close(grads[1][e], *product_bound(turned_ref(dy[s]), turned_ref(h[s]), torch.float32))
    assert not grads[1][1].any()
