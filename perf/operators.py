"""Cases of the microscaled 4-bit operators: quantisation, the products of
4-bit operands (plain and grouped), the linear layers trained through them,
and the optimizer step that writes the 4-bit copies those layers read.

The format is MXFP4 (OCP Microscaling Formats v1.0): blocks of 32 elements
along the contraction axis, one E8M0 scale 2^(floor(log2 amax) - 2) a block,
E2M1 elements.  A 4-bit matrix of R rows and C columns (slabs of them for
grouped weights) is held as
    codes   uint8 [slabs, R, Cp/2]      two elements a byte, the lower index in the low nibble,
                                        Cp = C rounded up to 128, zeros behind C
    scales  uint8 [Cp/128, slabs, Rp, 4]  biased exponents, Rp = R rounded up to 4.

With ``own`` false run() computes the plain form with elementary torch
operations in 32 bits; with ``own`` true it makes the framework's calls.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BLOCK = 32

# AdamW and AdEMAMix settings of this repository's transformer-shaped workload.
HYPER = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "weight_decay": 0.1, "beta3": 0.9999,
         "alpha": 5.0}
STEP = 10

# The tensors of a collection, "rows x cols" or "n" for one without a copy.
SMALL = "64x33,100x64,1x257,64,33"
LAYER = "2048x2048,2048x2048,2048x2048,2048x2048,8192x2048,2048x8192,2048,2048,8192,2048"


def listed():
    return [
        # one token's hidden state before a 4-bit product: launch latency
        {"name": "quantize one token", "op": "quantize", "rows": 1, "cols": 2048, "dtype": "bf16", "noise": False},
        # a ragged fp32 matrix, both axes odd
        {"name": "quantize odd f32", "op": "quantize", "rows": 1777, "cols": 1001, "dtype": "f32", "noise": False},
        # the output gradient of a wide layer, stochastically rounded
        {"name": "quantize gradient", "op": "quantize", "rows": 4096, "cols": 8192, "dtype": "bf16", "noise": True},
        # serving: one token through the up projection
        {"name": "project one token", "op": "project", "tokens": 1, "cols": 2048, "rows": 8192, "dtype": "bf16",
         "groups": 0, "spread": 0.0},
        # serving: a small odd batch through the down projection
        {"name": "project small batch", "op": "project", "tokens": 17, "cols": 8192, "rows": 2048, "dtype": "f16",
         "groups": 0, "spread": 0.0},
        # a long prompt through the up projection
        {"name": "project prompt", "op": "project", "tokens": 8192, "cols": 2048, "rows": 8192, "dtype": "bf16",
         "groups": 0, "spread": 0.0},
        # serving: a few tokens spread over sixteen experts, some of them without any
        {"name": "project experts few", "op": "project", "tokens": 24, "cols": 2048, "rows": 2048, "dtype": "bf16",
         "groups": 16, "spread": 1.0},
        # forward and backward of the up projection at a training batch
        {"name": "train layer", "op": "train", "tokens": 4096, "cols": 2048, "rows": 8192, "dtype": "bf16",
         "wdtype": "bf16", "groups": 0, "spread": 0.0, "noise": True},
        # forward and backward with odd sizes everywhere and fp32 weights
        {"name": "train odd", "op": "train", "tokens": 999, "cols": 1000, "rows": 531, "dtype": "f32", "wdtype": "f32",
         "groups": 0, "spread": 0.0, "noise": False},
        # forward and backward of eight experts with unequal loads
        {"name": "train experts", "op": "train", "tokens": 8192, "cols": 2048, "rows": 2048, "dtype": "bf16",
         "wdtype": "bf16", "groups": 8, "spread": 1.0, "noise": True},
        # a handful of small tensors: launch latency
        {"name": "step small", "op": "step", "tensors": SMALL, "dtype": "f32", "algo": "adam"},
        # one transformer layer of this repository's AdEMAMix workload
        {"name": "step layer", "op": "step", "tensors": LAYER, "dtype": "bf16", "algo": "ademamix"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "project", "train", "step"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    if op == "quantize":
        rows, cols = _log(rng, 1, 4096), _log(rng, 32, 8192)
        return {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "noise": rng.random() < 0.5}
    if op == "step":
        shapes = ["%dx%d" % (_log(rng, 1, 2048), _log(rng, 1, 4096)) for _ in range(rng.randint(1, 5))]
        shapes += ["%d" % _log(rng, 1, 8192) for _ in range(rng.randint(0, 4))]
        return {"op": op, "tensors": ",".join(shapes), "dtype": dtype, "algo": rng.choice(["adam", "ademamix"])}
    groups = rng.choice([0, 0, rng.randint(1, 24)])
    top = 4096 if op == "project" else 2048
    case = {"op": op, "tokens": _log(rng, 1, top), "cols": _log(rng, 32, 2048 if groups else 4096),
            "rows": _log(rng, 32, 2048 if groups else 8192), "dtype": dtype, "groups": groups,
            "spread": round(rng.uniform(0.0, 2.0), 3)}
    if op == "train":
        case["wdtype"] = rng.choice([dtype, "f32"])
        case["noise"] = rng.random() < 0.5
    return case


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _up(n, k):
    return (n + k - 1) // k * k


def _normal(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def _activations(gen, rows, cols, dtype):
    """Normal values with a few large channels and, among many rows, an all-zero one."""
    x = torch.randn((rows, cols), generator=gen, device="cuda")
    x *= torch.exp2(torch.randint(0, 64, (1, cols), generator=gen, device="cuda").sub_(58).clamp_(min=0).float())
    if rows > 4:
        x[rows // 2] = 0
    return x.to(dtype)


def _gradients(gen, rows, cols, dtype):
    """Small values whose size differs from row to row."""
    size = torch.exp2(torch.randint(-12, -4, (rows, 1), generator=gen, device="cuda").float())
    return (torch.randn((rows, cols), generator=gen, device="cuda") * size).to(dtype)


def _packed(gen, slabs, rows, cols):
    """A 4-bit matrix as a serving program has loaded it: (codes, scales)."""
    cp, rp = _up(cols, 128), _up(rows, 4)
    codes = torch.randint(0, 256, (slabs, rows, cp // 2), generator=gen, device="cuda", dtype=torch.uint8)
    codes[..., (cols + 1) // 2:] = 0
    if cols % 2:
        codes[..., cols // 2] &= 15
    scales = torch.randint(115, 120, (cp // 128, slabs, rp, 4), generator=gen, device="cuda", dtype=torch.uint8)
    flat = scales.permute(1, 2, 0, 3).reshape(slabs, rp, cp // 32).clone()
    flat[:, rows:] = 0
    flat[..., (cols + 31) // 32:] = 0
    return codes, flat.view(slabs, rp, cp // 128, 4).permute(2, 0, 1, 3).contiguous()


def _counts(seed, tokens, groups, spread):
    """Rows of each group: uneven shares, one group empty where there are several."""
    r = np.random.RandomState(seed % (2 ** 31))
    share = np.exp(spread * r.standard_normal(groups))
    if groups > 2:
        share[r.randint(groups)] = 0.0
    return r.multinomial(tokens, share / share.sum()).tolist()


def _shapes(case):
    return [tuple(int(v) for v in t.split("x")) for t in case["tensors"].split(",")]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    state = {"case": case}
    if case["op"] == "quantize":
        state["x"] = _gradients(gen, case["rows"], case["cols"], dtype) if case["noise"] else \
            _activations(gen, case["rows"], case["cols"], dtype)
        state["noise"] = torch.randint(0, 256, (case["rows"], case["cols"]), generator=gen, device="cuda",
                                       dtype=torch.uint8) if case["noise"] else None
        return state
    if case["op"] == "step":
        state["tensors"] = []
        for shape in _shapes(case):
            t = {"param": _normal(gen, shape, dtype, 0.05), "grad": _normal(gen, shape, dtype, 1e-2)}
            m = torch.randn((2 if case["algo"] == "ademamix" else 1, *shape), generator=gen, device="cuda") * 1e-3
            t["state1"] = m.reshape(-1)
            t["state2"] = (torch.randn(shape, generator=gen, device="cuda").square_() * 1e-4).reshape(-1)
            state["tensors"].append(t)
        state["bc"] = [torch.full((), v, device="cuda") for v in _corrections()]
        return state
    tokens, cols, rows, groups = case["tokens"], case["cols"], case["rows"], case["groups"]
    state["x"] = _activations(gen, tokens, cols, dtype)
    if groups:
        state["counts"] = _counts(seed, tokens, groups, case["spread"])
        state["offsets"] = torch.tensor([0] + np.cumsum(state["counts"]).tolist(), dtype=torch.int32, device="cuda")
    if case["op"] == "project":
        state["codes"], state["scales"] = _packed(gen, max(1, groups), rows, cols)
        return state
    shape = (groups, rows, cols) if groups else (rows, cols)
    state["w"] = _normal(gen, shape, DTYPES[case["wdtype"]], 0.02).requires_grad_()
    state["x"].requires_grad_()
    state["dy"] = _gradients(gen, tokens, rows, dtype)
    state["noise"] = torch.randint(0, 256, (tokens, rows), generator=gen, device="cuda", dtype=torch.uint8) \
        if case["noise"] else None
    return state


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------

def _round(x, noise=None):
    """The values that x stands for in 4 bits, fp32, blocks along the last axis."""
    cols = x.shape[-1]
    pad = _up(cols, BLOCK) - cols
    b = torch.nn.functional.pad(x.float(), (0, pad)).unflatten(-1, (-1, BLOCK))
    amax = b.abs().amax(-1, keepdim=True)
    exponent = (amax.view(torch.int32) >> 23).sub_(129).clamp_(min=-127)
    inverse = ((127 - exponent) << 23).view(torch.float32)          # 2^-exponent, a normal number
    a = (b.abs() * inverse).clamp_(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    if noise is None:
        q = torch.round(a / step)
    else:
        u = (torch.nn.functional.pad(noise, (0, pad)).unflatten(-1, (-1, BLOCK)).float() + 0.5) / 256
        low = torch.floor(a / step)
        q = low + (a / step - low > u)
    v = torch.copysign(q * step, b) / inverse
    v = torch.where(torch.isfinite(amax), v, torch.nan)
    return v.flatten(-2)[..., :cols]


def _unpack(codes, scales, cols):
    """The values of a packed matrix, fp32 [slabs, rows, cols]."""
    slabs, rows, half = codes.shape
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    s = scales[:, :, :rows].permute(1, 2, 0, 3).reshape(slabs, rows, 2 * half // BLOCK)
    power = ((s.int() + 1) << 23).view(torch.float32) * 0.5         # 2^(s - 127), exactly
    v = table[q].unflatten(-1, (-1, BLOCK)) * power[..., None]
    return v.flatten(-2)[..., :cols]


def _turned(x, noise=None):
    """The values of x in blocks down its columns, returned transposed."""
    return _round(x.transpose(-1, -2).contiguous(), None if noise is None else noise.t().contiguous())


def _f32(v):
    return float(np.float32(v))


def _corrections():
    """1 - beta1^t and 1 - beta2^t of the step, in 64 bits, of the fp32 betas."""
    return [_f32(1.0 - _f32(HYPER[k]) ** STEP) for k in ("beta1", "beta2")]


def _moment(old, beta, g):
    return old * _f32(beta) + g * float(np.float32(1) - np.float32(beta))


def _step_plain(state, t):
    """One AdamW or AdEMAMix update of one tensor, each operation rounded to fp32."""
    mix = state["case"]["algo"] == "ademamix"
    g, p = t["grad"].float().reshape(-1), t["param"].float().reshape(-1)
    n = g.numel()
    m = _moment(t["state1"][:n], HYPER["beta1"], g)
    gg = g * float(np.float32(1) - np.float32(HYPER["beta2"])) * g
    v = t["state2"] * _f32(HYPER["beta2"]) + gg
    num = m / state["bc"][0]
    t["state1"][:n] = m
    if mix:
        m2 = _moment(t["state1"][n:], HYPER["beta3"], g)
        num = num + m2 * _f32(HYPER["alpha"])
        t["state1"][n:] = m2
    t["state2"].copy_(v)
    den = torch.sqrt(v / state["bc"][1]) + _f32(HYPER["eps"])
    decay = _f32(1.0 - _f32(HYPER["lr"]) * _f32(HYPER["weight_decay"]))
    p = p * decay - num / den * _f32(HYPER["lr"])
    t["param"].copy_(p.view(t["param"].shape))
    return t["param"]


def _run_plain(state):
    case = state["case"]
    if case["op"] == "quantize":
        return [_round(state["x"], state["noise"]).bfloat16(), _turned(state["x"], state["noise"]).bfloat16()]
    if case["op"] == "step":
        for t in state["tensors"]:
            _step_plain(state, t)
        return _step_outputs(state, [(_round(t["param"]).bfloat16(), _turned(t["param"]).bfloat16())
                                     for t in state["tensors"] if t["param"].dim() == 2])
    dtype = DTYPES[case["dtype"]]
    groups = case["groups"]
    parts = state["counts"] if groups else [case["tokens"]]
    if case["op"] == "project":
        w = _unpack(state["codes"], state["scales"], case["cols"])
        return torch.cat([x @ e.t() for x, e in zip(_round(state["x"]).split(parts), w)]).to(dtype)
    x, dy, w = state["x"].detach(), state["dy"], state["w"].detach()
    wide = w if groups else w[None]
    y = torch.cat([a @ e.t() for a, e in zip(_round(x).split(parts), _round(wide))])
    dx = torch.cat([a @ e.t() for a, e in zip(_round(dy, state["noise"]).split(parts), _turned(wide))])
    noise = [None] * len(parts) if state["noise"] is None else state["noise"].split(parts)
    dw = torch.stack([_turned(d, r) @ _turned(a).t() if len(d) else torch.zeros_like(w[0], dtype=torch.float32)
                      for d, r, a in zip(dy.split(parts), noise, x.split(parts))])
    return {"y": y.to(dtype), "dx": dx.to(dtype), "dw": dw.view(w.shape).to(w.dtype)}


def _step_outputs(state, copies):
    names = ("param", "state1", "state2")
    return {"tensors": [[t[k] for k in names] for t in state["tensors"]], "copies": [list(c) for c in copies]}


# ---------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------

def _run_own(state):
    from elementwise_optimizer_b200 import binding, mx4
    case = state["case"]
    if case["op"] == "quantize":
        q, qt = mx4.quantize_pair(state["x"], noise=state["noise"])
        return [q.dequantize(torch.bfloat16), qt.dequantize(torch.bfloat16)]
    if case["op"] == "step":
        if "list" not in state:          # the descriptor and the copies that a program keeps between steps
            ts = state["tensors"]
            state["copies"] = [mx4.empty_pair(t["param"]) if t["param"].dim() == 2 else None for t in ts]
            state["list"] = mx4.TensorListMX4.from_tensors(
                [t["param"] for t in ts], [t["grad"] for t in ts], [t["state1"] for t in ts],
                [t["state2"] for t in ts], state["copies"])
            state["hyper"] = binding.make_hyper(case["algo"], **HYPER)
        mx4.opt2s_step_mx4(state["list"], state["hyper"], STEP)
        return _step_outputs(state, [[q.dequantize(torch.bfloat16) for q in c]
                                     for c in state["copies"] if c is not None])
    if case["op"] == "project":
        wq = mx4.MX4Tensor(state["codes"], state["scales"], (case["rows"], case["cols"]))
        if case["groups"]:
            return mx4.project_grouped(state["x"], wq, state["offsets"])
        return mx4.project(state["x"], wq)
    if case["groups"]:
        y = mx4.linear_grouped(state["x"], state["w"], state["offsets"], noise=state["noise"])
    else:
        y = mx4.linear(state["x"], state["w"], noise=state["noise"])
    dx, dw = torch.autograd.grad(y, (state["x"], state["w"]), state["dy"])
    return {"y": y.detach(), "dx": dx, "dw": dw}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    size = {"f32": 4, "f16": 2, "bf16": 2}
    packed = 0.5 + 1 / 32
    if case["op"] == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (size[case["dtype"]] + int(case["noise"]) + 2 * packed + 4), "flops": 0}
    if case["op"] == "step":
        b = 0.0
        for shape in _shapes(case):
            n = math.prod(shape)
            b += n * (3 * size[case["dtype"]] + (24 if case["algo"] == "ademamix" else 16))
            b += n * (2 * packed + 4) if len(shape) == 2 else 0
        return {"bytes": b, "flops": 0}
    t, c, r, g = case["tokens"], case["cols"], case["rows"], max(1, case["groups"])
    if case["op"] == "project":
        live = min(g, t)
        return {"bytes": size[case["dtype"]] * t * (c + r) + live * r * c * packed, "flops": 2.0 * t * r * c}
    b = size[case["dtype"]] * 2 * t * (c + r) + 2 * size[case["wdtype"]] * g * r * c + int(case["noise"]) * t * r
    return {"bytes": b, "flops": 6.0 * t * r * c}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _two_to(e):
    """2^e in 64 bits, from its bit pattern (pow need not be exact on the GPU)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _grid64(x, noise=None):
    """x in 4 bits from the definition: the scale by frexp, the element by
    comparing with the borders between neighbours (ties to the even code)."""
    x = x.detach().double()
    cols = x.shape[-1]
    shape = (*x.shape[:-1], _up(cols, BLOCK) // BLOCK, BLOCK)
    b = x.new_zeros((*x.shape[:-1], _up(cols, BLOCK)))
    b[..., :cols] = x
    b = b.reshape(shape)
    amax = b.abs().max(-1, keepdim=True).values
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 3, torch.full_like(amax, -127, dtype=torch.int32))
    scale = _two_to(e.clamp(min=-127))
    a = b.abs() / scale
    levels = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    out = torch.zeros_like(a)
    if noise is not None:
        u = b.new_zeros((*x.shape[:-1], shape[-2] * BLOCK))
        u[..., :cols] = noise.double()
        u = (u.reshape(shape) + 0.5) / 256
    for code in range(1, 8):
        lo, hi = levels[code - 1], levels[code]
        if noise is None:
            border = (lo + hi) / 2
            up = a >= border if code % 2 == 0 else a > border
        else:
            up = (a - lo) / (hi - lo) > u
        out = torch.where(up, torch.full_like(out, hi), out)
    out = out * torch.sign(b) * scale
    return out.reshape(*x.shape[:-1], -1)[..., :cols]


def _grid64_down(x, noise=None):
    return _grid64(x.detach().mT.contiguous(), None if noise is None else noise.mT.contiguous())


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "quantize":
        return [_grid64(state["x"], state["noise"]), _grid64_down(state["x"], state["noise"])]
    if case["op"] == "step":
        h = {k: float(np.float32(v)) for k, v in HYPER.items()}
        tensors, copies = [], []
        for t in state["tensors"]:
            g, p = t["grad"].double().flatten(), t["param"].double().flatten()
            n = g.numel()
            m = h["beta1"] * t["state1"][:n].double() + (1 - h["beta1"]) * g
            v = h["beta2"] * t["state2"].double() + (1 - h["beta2"]) * g ** 2
            first, upd = m, m / (1 - h["beta1"] ** STEP)
            if case["algo"] == "ademamix":
                m2 = h["beta3"] * t["state1"][n:].double() + (1 - h["beta3"]) * g
                first, upd = torch.cat((m, m2)), upd + h["alpha"] * m2
            upd = upd / ((v / (1 - h["beta2"] ** STEP)).sqrt() + h["eps"])
            p = (p * (1 - h["lr"] * h["weight_decay"]) - h["lr"] * upd).view(t["param"].shape)
            tensors.append([p, first, v])
            if p.dim() == 2:             # the copies are those of the stored param: no value of their own in 64 bits
                copies.append([None, None])
        return {"tensors": tensors, "copies": copies}
    groups = case["groups"]
    parts = state["counts"] if groups else [case["tokens"]]
    starts = np.cumsum([0] + parts)
    if case["op"] == "project":
        x = _grid64(state["x"])
        codes, scales = state["codes"].long(), state["scales"].long()
        y = []
        levels = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
        for e in range(max(1, groups)):
            at = torch.arange(case["cols"], device="cuda")
            nibble = torch.where(at % 2 == 0, codes[e][:, at // 2] % 16, codes[e][:, at // 2] // 16)
            w = levels[nibble % 8] * torch.where(nibble < 8, 1.0, -1.0)
            w = w * _two_to(scales[at // 128, e, :case["rows"], (at // 32) % 4].t() - 127)
            y.append(x[starts[e]:starts[e + 1]] @ w.t())
        return torch.cat(y)
    x, dy, w, noise = state["x"], state["dy"], state["w"], state["noise"]
    wide = w if groups else w[None]
    xq, dq, wq, wt = _grid64(x), _grid64(dy, noise), _grid64(wide), _grid64_down(wide)
    y, dx, dw = [], [], []
    for e in range(len(parts)):
        s = slice(starts[e], starts[e + 1])
        y.append(xq[s] @ wq[e].t())
        dx.append(dq[s] @ wt[e].t())
        if parts[e]:
            down = _grid64_down(dy[s], None if noise is None else noise[s])
            dw.append(down @ _grid64_down(x[s]).t())
        else:
            dw.append(torch.zeros_like(wq[e]))
    return {"y": torch.cat(y), "dx": torch.cat(dx), "dw": torch.stack(dw).view(w.shape)}
