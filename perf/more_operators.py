"""Measured cases of the gated projections and of the 4-bit weights.

``own`` selects what ``run`` computes: the plain form (elementary torch
operations in fp32, rounded once at the end) or this package's kernels.

  gated     gated_linear: h = act(x Wg^T) * (x Wu^T), the first half of a gated
            feed-forward block; with ``train`` also its backward pass (the
            gradients of x and of the weights), from the saved projections or,
            with ``again``, from projections computed again.
  w4_quant  w4_quant, then w4_dequant: weights brought to 4 bits with a scale
            (and zero point) per group, and the values that they stand for.
  w4        w4_linear: y = x W^T with 4-bit weights, from one row to many.
  w4_gated  w4_gated_linear: the gated projections with 4-bit weights.
"""
import math

import torch

own = False

DEV = "cuda"


# --------------------------------------------------------------------------
# cases

def listed():
    return [
        # one decoding sequence through a Llama-3-8B-sized block
        {"name": "gated_t1_4096_14336", "op": "gated", "tokens": 1, "k": 4096, "i": 14336,
         "dtype": "bfloat16", "act": "silu", "train": False, "again": False, "pad": 0},
        # a ragged batch of short prompts, every size odd, x a slice of a wider matrix
        {"name": "gated_t515_1000_2731", "op": "gated", "tokens": 515, "k": 1000, "i": 2731,
         "dtype": "float16", "act": "gelu", "train": False, "again": False, "pad": 3},
        # prefill through a DeepSeek-V3-sized dense block
        {"name": "gated_t4096_7168_18432", "op": "gated", "tokens": 4096, "k": 7168, "i": 18432,
         "dtype": "bfloat16", "act": "silu", "train": False, "again": False, "pad": 0},
        # a training step's block, projections saved
        {"name": "gated_train_t4096_4096_14336", "op": "gated", "tokens": 4096, "k": 4096,
         "i": 14336, "dtype": "bfloat16", "act": "silu", "train": True, "again": False, "pad": 0},
        # training on a ragged batch with the projections computed again
        {"name": "gated_train_t1003_1536_4099", "op": "gated", "tokens": 1003, "k": 1536,
         "i": 4099, "dtype": "float16", "act": "gelu_tanh", "train": True, "again": True, "pad": 8},
        # a router-sized slice of weights: latency of the loading path
        {"name": "w4_quant_256_1536", "op": "w4_quant", "n": 256, "k": 1536, "group": 32,
         "zeros": True, "dtype": "float16"},
        # a large projection on load
        {"name": "w4_quant_18432_7168", "op": "w4_quant", "n": 18432, "k": 7168, "group": 128,
         "zeros": False, "dtype": "bfloat16"},
        # one decoding sequence, the down projection of a Llama-3-8B-sized block
        {"name": "w4_t1_14336_4096", "op": "w4", "tokens": 1, "k": 14336, "n": 4096, "group": 128,
         "zeros": False, "dtype": "bfloat16", "pad": 0},
        # a decode batch, an odd number of outputs, zero points and short groups
        {"name": "w4_t37_7168_2111", "op": "w4", "tokens": 37, "k": 7168, "n": 2111, "group": 64,
         "zeros": True, "dtype": "float16", "pad": 8},
        # prefill on the same 4-bit weights
        {"name": "w4_t2048_7168_18432", "op": "w4", "tokens": 2048, "k": 7168, "n": 18432,
         "group": 128, "zeros": True, "dtype": "bfloat16", "pad": 0},
        # one decoding sequence through the gated projections in 4 bits
        {"name": "w4_gated_t1_4096_14336", "op": "w4_gated", "tokens": 1, "k": 4096, "i": 14336,
         "group": 128, "zeros": False, "dtype": "bfloat16", "act": "silu", "pad": 0},
        # a large decode batch with zero points
        {"name": "w4_gated_t128_4096_14336", "op": "w4_gated", "tokens": 128, "k": 4096,
         "i": 14336, "group": 64, "zeros": True, "dtype": "float16", "act": "silu", "pad": 0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng):
    """A layer's width: a usual one, or any other, odd ones among them."""
    if rng.random() < 0.4:
        return _log_int(rng, 50, 18432)
    return rng.choice([512, 576, 1024, 1536, 2048, 4096, 5120, 7168, 14336, 18432])


def _tokens(rng, most):
    """Rows of a batch: decode batches as often as longer ones."""
    most = max(1, int(most))
    if rng.random() < 0.5:
        return min(rng.randint(1, 64), most)
    return min(_log_int(rng, 1, 8192), most)


def draw(rng):
    op = rng.choice(["gated", "gated", "w4_quant", "w4", "w4_gated"])
    c = {"op": op, "dtype": rng.choice(["bfloat16", "float16"])}
    if op == "gated":
        k, i = _width(rng), _width(rng)
        train = rng.random() < 0.5
        most = 4096 * (4096 * 14336 if train else 7168 * 18432) // (k * i)
        return {**c, "tokens": _tokens(rng, most), "k": k, "i": i, "train": train,
                "act": rng.choice(["silu", "gelu", "gelu_tanh"]),
                "again": train and rng.random() < 0.4, "pad": rng.choice([0, 0, 3, 8, 128])}
    group = rng.choice([32, 64, 128])
    k = group * max(1, _width(rng) // group)
    c = {**c, "k": k, "group": group, "zeros": rng.random() < 0.5}
    if op == "w4_quant":
        return {**c, "n": max(1, min(_width(rng), 18432 * 7168 // k))}
    c["pad"] = rng.choice([0, 0, 3, 8, 128])
    if op == "w4":
        n = _width(rng)
        return {**c, "n": n, "tokens": _tokens(rng, 2048 * 7168 * 18432 // (k * n))}
    i = _width(rng)
    return {**c, "i": i, "tokens": _tokens(rng, 128 * 4096 * 14336 // (k * i)),
            "act": rng.choice(["silu", "gelu", "gelu_tanh"])}


# --------------------------------------------------------------------------
# inputs

def _randn(g, *shape):
    return torch.randn(*shape, device=DEV, generator=g)


def _activations(g, tokens, k, pad, dtype):
    """Rows after a norm: a few channels much larger than the others; with
    ``pad`` a column slice of a wider matrix."""
    loud = torch.where(torch.rand(k, device=DEV, generator=g) < 0.005, 8.0, 1.0)
    wide = torch.zeros(tokens, k + pad, device=DEV, dtype=dtype)
    wide[:, :k] = (_randn(g, tokens, k) * loud).to(dtype)
    return wide[:, :k]


def _weights(g, n, k, dtype):
    return (_randn(g, n, k) / math.sqrt(k)).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed * 6007 + 29)
    c = dict(case)
    t = getattr(torch, c["dtype"])
    if c["op"] == "w4_quant":
        c["w"] = _weights(g, c["n"], c["k"], t)
        return c
    c["x"] = _activations(g, c["tokens"], c["k"], c["pad"], t)
    if c["op"] == "gated":
        c["w"] = _weights(g, 2 * c["i"], c["k"], t)
        c["d_h"] = _randn(g, c["tokens"], c["i"]).to(t) if c["train"] else None
        return c
    rows = c["n"] if c["op"] == "w4" else 2 * c["i"]
    q, c["scale"], c["zero"] = _quant(_weights(g, rows, c["k"], t), c["group"], c["zeros"])
    c["codes"] = q[:, 0::2] | (q[:, 1::2] << 4)
    return c


# --------------------------------------------------------------------------
# the package's calls

def _own(s):
    import block_scaled_fp8_act_amd as fb
    if s["op"] == "gated":
        if not s["train"]:
            return fb.gated_linear(s["x"], s["w"], act=s["act"])
        if s["again"]:
            h, gate_up = fb.gated_linear(s["x"], s["w"], act=s["act"]), None
        else:
            h, gate_up = fb.gated_linear(s["x"], s["w"], act=s["act"], save=True)
        return h, *fb.gated_linear_backward(s["d_h"], s["x"], s["w"], gate_up, act=s["act"])
    if s["op"] == "w4_quant":
        codes, scale, zeros = fb.w4_quant(s["w"], group=s["group"], zeros=s["zeros"])
        w = fb.w4_dequant(codes, scale, zeros)
        return (w, scale, zeros) if s["zeros"] else (w, scale)
    if s["op"] == "w4":
        return fb.w4_linear(s["x"], s["codes"], s["scale"], s["zero"])
    return fb.w4_gated_linear(s["x"], s["codes"], s["scale"], s["zero"], act=s["act"])


# --------------------------------------------------------------------------
# the plain form

def _act(g, act):
    """act(g) and its derivative."""
    if act == "gelu":
        phi = torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))
        cdf = 0.5 * torch.erfc(g * -math.sqrt(0.5))
        return g * cdf, cdf + g * phi
    if act == "silu":
        z, dz = g, 1.0
    else:    # gelu_tanh: g (1 + tanh(z / 2)) / 2 = g / (1 + e^-z)
        c = 2.0 * math.sqrt(2.0 / math.pi)
        z, dz = c * (g + 0.044715 * g * g * g), c * (1.0 + 3 * 0.044715 * g * g)
    s = 1.0 / (1.0 + torch.exp(-z))
    return g * s, s + g * s * (1.0 - s) * dz


def _plain_gated(s):
    x, w, i, t = s["x"].float(), s["w"].float(), s["i"], s["w"].dtype
    gu = x @ w.t()
    g, u = gu[:, :i], gu[:, i:]
    a, da = _act(g, s["act"])
    h = (a * u).to(t)
    if not s["train"]:
        return h
    d = s["d_h"].float()
    dgu = torch.cat([d * u * da, d * a], 1)
    return h, (dgu @ w).to(t), (dgu.t() @ x).to(t)


def _quant(w, group, zeros):
    """Codes 0..15 (one a byte), scales in the weights' type, zero points."""
    n, k = w.shape
    v = w.float().view(n, k // group, group)
    if zeros:
        lo, hi = v.amin(2).clamp(max=0.0), v.amax(2).clamp(min=0.0)
        scale = ((hi - lo) / 15.0).to(w.dtype)
    else:
        scale = (v.abs().amax(2) / 7.0).to(w.dtype)
    step = scale.double()
    inv = lambda a: torch.where(step > 0, a, 0.0)  # noqa: E731
    if zeros:
        zero = inv(torch.round(-lo.double() / step)).clamp(0, 15)
    else:
        zero = torch.full_like(step, 8.0)
    q = torch.empty(n, k // group, group, dtype=torch.uint8, device=w.device)
    for r in range(0, n, 4096):       # (in 64 bits: quotients next to a border)
        e = scale[r:r + 4096, :, None].double()
        z = torch.where(e > 0, torch.round(v[r:r + 4096].double() / e), 0.0)
        q[r:r + 4096] = (z + zero[r:r + 4096, :, None]).clamp(0, 15).to(torch.uint8)
    return q.view(n, k), scale, zero.to(torch.uint8) if zeros else None


def _values(q, scale, zero, group):
    """What codes (one a byte) stand for, in 32 bits."""
    n, k = q.shape
    v = q.view(n, k // group, group).float()
    v = v - (8.0 if zero is None else zero[:, :, None].float())
    return (v * scale[:, :, None].float()).view(n, k)


def _plain_w4_quant(s):
    q, scale, zero = _quant(s["w"], s["group"], s["zeros"])
    w = _values(q, scale, zero, s["group"]).to(s["w"].dtype)
    return (w, scale, zero) if s["zeros"] else (w, scale)


def _plain_w4(s):
    q = torch.stack([s["codes"] & 15, s["codes"] >> 4], 2).flatten(1)
    y = s["x"].float() @ _values(q, s["scale"], s["zero"], s["group"]).t()
    if s["op"] == "w4_gated":
        y = _act(y[:, :s["i"]], s["act"])[0] * y[:, s["i"]:]
    return y.to(s["x"].dtype)


def run(state):
    if own:
        return _own(state)
    return {"gated": _plain_gated, "w4_quant": _plain_w4_quant, "w4": _plain_w4,
            "w4_gated": _plain_w4}[state["op"]](state)


# --------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "gated":
        t, k, i = c["tokens"], c["k"], c["i"]
        bytes_ = 2 * (t * k + 2 * i * k + t * i)
        if not c["train"]:
            return {"bytes": bytes_, "flops": 4 * t * k * i}
        # d_h in; the gradients of x and of the weights out
        return {"bytes": bytes_ + 2 * (t * i + t * k + 2 * i * k), "flops": 12 * t * k * i}
    k, group = c["k"], c["group"]
    rows = 2 * c["i"] if c["op"] == "w4_gated" else c["n"]
    packed = rows * k // 2 + rows * (k // group) * (3 if c["zeros"] else 2)
    if c["op"] == "w4_quant":     # weights in, codes out; codes in, values out
        return {"bytes": 4 * rows * k + 2 * packed, "flops": 4 * rows * k}
    t, out = c["tokens"], c["i"] if c["op"] == "w4_gated" else c["n"]
    return {"bytes": packed + 2 * t * (k + out), "flops": 2 * t * k * rows}


# --------------------------------------------------------------------------
# the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"gated": _exact_gated, "w4_quant": _exact_quant, "w4": _exact_w4,
            "w4_gated": _exact_w4}[s["op"]](s)


def _glu64(gu, act):
    g, u = gu.chunk(2, dim=1)
    if act == "silu":
        return torch.nn.functional.silu(g) * u
    return torch.nn.functional.gelu(g, approximate="tanh" if act == "gelu_tanh" else "none") * u


def _exact_gated(s):
    x, w = s["x"].double(), s["w"].double()
    if not s["train"]:
        return _glu64(x @ w.t(), s["act"])
    x.requires_grad_()
    w.requires_grad_()
    h = _glu64(x @ w.t(), s["act"])
    dx, dw = torch.autograd.grad(h, (x, w), s["d_h"].double())
    return h.detach(), dx, dw


def _exact_quant(s):
    """Per group: scale = T(fl32(range / steps)), T the weights' type; codes the
    nearest (ties to even) whole numbers of scales, held in 4 bits."""
    w, t = s["w"].double(), s["w"].dtype
    n, k = w.shape
    w = w.reshape(-1, s["group"])
    if s["zeros"]:
        least = torch.minimum(w.min(1).values, torch.zeros((), device=DEV, dtype=torch.float64))
        most = torch.maximum(w.max(1).values, torch.zeros((), device=DEV, dtype=torch.float64))
        step = ((most - least).float().double() / 15).float().to(t).double()
        there = step > 0
        zero = torch.zeros_like(step)
        zero[there] = (-least[there] / step[there]).round().clamp(0, 15)
        first, last = -zero, 15 - zero
    else:
        step = (w.abs().max(1).values / 7).float().to(t).double()
        there = step > 0
        zero = None
        first, last = torch.full_like(step, -8.0), torch.full_like(step, 7.0)
    steps = torch.zeros_like(w)
    steps[there] = (w[there] / step[there, None]).round()
    steps = torch.minimum(torch.maximum(steps, first[:, None]), last[:, None])
    out = (steps * step[:, None]).view(n, k), step.view(n, -1)
    return out if zero is None else (*out, zero.to(torch.uint8).view(n, -1))


def _exact_w4(s):
    n, half = s["codes"].shape
    w = torch.empty(n, 2 * half, device=DEV, dtype=torch.float64)
    w[:, ::2] = (s["codes"] % 16).double()
    w[:, 1::2] = (s["codes"] // 16).double()
    per = lambda p: p.double().repeat_interleave(s["group"], 1)  # noqa: E731
    w -= 8.0 if s["zero"] is None else per(s["zero"])
    w *= per(s["scale"])
    y = s["x"].double() @ w.t()
    return y if s["op"] == "w4" else _glu64(y, s["act"])
