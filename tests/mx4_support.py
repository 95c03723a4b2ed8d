"""Plain 64-bit implementation of the microscaled 4-bit operators, for the
tests: numpy and torch on the CPU, straight from the definitions, nothing
shared with the library."""
import numpy as np
import torch

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def up(n, k):
    return (n + k - 1) // k * k


def encode_ref(x, noise=None):
    """(codes, scale bytes) of blocks of 32 along the last axis of x; codes
    uint8 one per element, padded to whole blocks with code 0."""
    x = np.asarray(x, np.float64)
    cols = x.shape[-1]
    pad = up(cols, 32)
    b = np.zeros((*x.shape[:-1], pad))
    b[..., :cols] = x
    b = b.reshape(*x.shape[:-1], pad // 32, 32)
    with np.errstate(invalid="ignore"):
        amax = np.abs(b).max(-1)
    dead = ~np.isfinite(amax)
    _, e = np.frexp(np.where(dead | (amax == 0), 1.0, amax))
    e = np.where(amax == 0, -127, np.maximum(e - 1 - 2, -127))
    a = np.minimum(np.abs(np.where(dead[..., None], 0.0, b)) / np.exp2(e.astype(np.float64))[..., None], 6.0)
    if noise is None:
        mid = (LEVELS[1:] + LEVELS[:-1]) / 2
        codes = np.zeros(a.shape, np.int64)
        for i, m in enumerate(mid):          # a tie goes to the even code
            codes += (a >= m) if (i + 1) % 2 == 0 else (a > m)
    else:
        n = np.zeros((*x.shape[:-1], pad))
        n[..., :cols] = noise
        u = (n.reshape(a.shape) + 0.5) / 256
        lo = np.clip(np.searchsorted(LEVELS, a, side="right") - 1, 0, 6)
        codes = lo + ((a - LEVELS[lo]) / (LEVELS[lo + 1] - LEVELS[lo]) > u)
    codes = codes + 8 * np.signbit(b)
    codes = np.where(dead[..., None], 0, codes).astype(np.uint8).reshape(*x.shape[:-1], pad)
    return codes, np.where(dead, 255, e + 127).astype(np.uint8)


def values_ref(codes, scales, cols):
    """The float64 values of codes (one per element) and block scale bytes."""
    v = np.where(codes >= 8, -1.0, 1.0) * LEVELS[codes % 8]
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    v = v.reshape(*scales.shape, 32) * s[..., None]
    return v.reshape(codes.shape)[..., :cols]


def round_ref(x, noise=None):
    """x through 4 bits, blocks along the last axis (torch float64, CPU)."""
    x = x.detach().cpu().double().numpy()
    codes, scales = encode_ref(x, None if noise is None else noise.cpu().numpy())
    return torch.from_numpy(np.ascontiguousarray(values_ref(codes, scales, x.shape[-1])))


def turned_ref(x, noise=None):
    """The transposed form's values: blocks down the columns."""
    return round_ref(x.detach().mT.contiguous(), None if noise is None else noise.mT.contiguous())


def unpack(q):
    """(codes one per element [slabs, rows, up(cols, 32)], scale bytes [slabs,
    rows, blocks], the padding's codes) of an MX4Tensor's storage."""
    cp = up(q.cols, 128)
    raw = q.codes.cpu().numpy().reshape(q.slabs, q.rows, cp // 2)
    codes = np.stack((raw & 15, raw >> 4), -1).reshape(q.slabs, q.rows, cp)
    s = q.scales.cpu().numpy().reshape(cp // 128, q.slabs, up(q.rows, 4), 4)[:, :, :q.rows]
    s = s.transpose(1, 2, 0, 3).reshape(q.slabs, q.rows, cp // 32)
    n = up(q.cols, 32)
    return codes[..., :n], s[..., :n // 32], codes[..., n:]


def product_bound(a, b, dtype):
    """(values, tolerance) of a @ b.mT in 64 bits.  The products of E2M1 values
    and their power-of-two scales are exact in fp32; each of the K additions
    may lose up to one ulp of a partial sum (2^-23 of at most sum |a||b|), and
    the result is rounded once to `dtype` (half an ulp; in fp16 also half the
    smallest subnormal)."""
    y = a @ b.mT
    mag = a.abs() @ b.abs().mT
    tol = a.shape[-1] * 2.0 ** -23 * mag
    tol = tol + torch.finfo(dtype).eps / 2 * (y.abs() + tol)
    return y, tol + (2.0 ** -25 if dtype == torch.float16 else 0.0)


def close(got, want, tol):
    """Elementwise |got - want| <= tol, with a readable failure."""
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (got.shape, want.shape)
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}: " \
        f"{got[tuple(bad.nonzero()[0])]} for {want[tuple(bad.nonzero()[0])]}"
