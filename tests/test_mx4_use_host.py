"""How the 4-bit copies are kept and handed out, without a GPU."""
import pytest
import torch

from elementwise_optimizer_b200 import optim


def test_copies_only_of_the_optimizers_own_parameters():
    """A tensor that no step of this optimizer writes has no copies here,
    whatever its dimensions: they would go stale unnoticed."""
    own, foreign = (torch.nn.Parameter(torch.zeros(4, 4)) for _ in range(2))
    for mx4 in (True, [own]):
        opt = optim.AdamW32bit([own], mx4=mx4)
        with pytest.raises(ValueError, match="not a parameter of this optimizer"):
            opt.mx4_copies(foreign)
        with pytest.raises(ValueError, match="not a parameter of this optimizer"):
            opt.mx4_copies(own.detach())
        assert not opt._mx4_pairs


def test_the_step_tells_autograd_that_it_wrote_the_copies(monkeypatch):
    """Called by itself as by an optimizer; a step that fails writes nothing."""
    from types import SimpleNamespace

    from elementwise_optimizer_b200 import binding as B
    p, g, m, v = torch.zeros(4, 8), torch.zeros(4, 8), torch.zeros(32), torch.zeros(32)

    def form(rows, cols):
        return SimpleNamespace(slabs=1, rows=rows, cols=cols, shape=(rows, cols), device=p.device,
                               codes=torch.zeros(rows, 64, dtype=torch.uint8), scales=torch.zeros(16, dtype=torch.uint8))

    pair = (form(4, 8), form(8, 4))
    tl = B.TensorListMX4.from_tensors([p], [g], [m], [v], [pair])
    library = B.lib()
    status = 0

    class Fake:
        opt2s_error_string, opt2s_last_cuda_error = library.opt2s_error_string, library.opt2s_last_cuda_error

        @staticmethod
        def opt2s_step_mx4(*args):
            return status

    monkeypatch.setattr(B, "lib", lambda: Fake)
    monkeypatch.setattr(B, "_stream_handle", lambda stream: None)
    before = [f.codes._version for f in pair]
    B.opt2s_step_mx4(tl, B.make_hyper("adam"), 1)
    assert [f.codes._version for f in pair] == [n + 1 for n in before]
    status = -1
    with pytest.raises(B.Opt2sError):
        B.opt2s_step_mx4(tl, B.make_hyper("adam"), 1)
    assert [f.codes._version for f in pair] == [n + 1 for n in before]


def test_kept_copies_are_no_inference_tensors(monkeypatch):
    """A graph may save them, wherever they were first asked for."""
    from elementwise_optimizer_b200 import mx4
    monkeypatch.setattr(mx4, "quantize_pair", lambda p: (torch.empty(1), torch.empty(1)))
    own = torch.nn.Parameter(torch.zeros(4, 4))
    opt = optim.AdamW32bit([own], mx4=True)
    with torch.inference_mode():
        pair = opt.mx4_copies(own)
        assert torch.empty(1).is_inference()
    assert not any(t.is_inference() for t in pair) and opt.mx4_copies(own) is pair


def test_check_errors(monkeypatch):
    """The library's count of waits that gave up, as an exception."""
    import contextlib

    from elementwise_optimizer_b200 import binding as B, mx4
    library, found, entered = B.lib(), 0, []

    class Fake:
        opt2s_error_string, opt2s_last_cuda_error = library.opt2s_error_string, library.opt2s_last_cuda_error

        @staticmethod
        def opt2s_mx4_errors(count):
            count._obj.value = max(found, 0)
            return min(found, 0)

    monkeypatch.setattr(B, "lib", lambda: Fake)
    monkeypatch.setattr(torch.cuda, "device", lambda d: entered.append(d) or contextlib.nullcontext())
    assert mx4.check_errors() is None and mx4.check_errors("cuda:1") is None
    assert entered == [None, "cuda:1"]
    found = 3
    with pytest.raises(RuntimeError, match="3 CTAs"):
        mx4.check_errors()
    found = -4
    with pytest.raises(B.Opt2sError):
        mx4.check_errors()


def test_no_storage_for_copies_outside_a_cuda_device():
    """The step writes what empty_pair gives by its address."""
    from elementwise_optimizer_b200 import mx4
    with pytest.raises(ValueError, match="CUDA"):
        mx4.empty_pair(torch.zeros(4, 8))


def test_no_stride_leaves_the_address_space():
    """Rows or slabs so far apart that their span overflows are refused, not
    compared with the other operands as whatever is left of it."""
    import ctypes

    from elementwise_optimizer_b200 import binding as B
    L, base = B.lib(), 1 << 40
    rows, far = 1 << 22, 1 << 40

    def matrix(slabs, rows, cols, at):
        return B.opt2s_mx4(base + at, base + at + (1 << 36), slabs, rows, cols)

    for slabs, n, row_stride, slab_stride in ((1, rows, far, 0), (60000, 4, 8, far)):
        s = B.opt2s_mx4_source(base, None, slabs, n, 8, row_stride, slab_stride, B.OPT2S_F32, 0)
        q = matrix(slabs, n, 8, 1 << 38)
        assert L.opt2s_mx4_quantize(ctypes.byref(s), ctypes.byref(q), None, None, 0, None) == -1
    a, b = matrix(1, rows, 256, 1 << 38), matrix(1, 10, 256, 1 << 39)
    assert L.opt2s_mx4_matmul(ctypes.byref(a), ctypes.byref(b), base, far, B.OPT2S_F32, 0, None) == -1
