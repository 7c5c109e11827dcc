"""Measured cases of the routing, row-grouping, combining and adapter operators.

``own`` selects what ``run`` computes: the plain form (elementary torch
operations in fp32, rounded once at the end) or this package's kernels.

  route    moe_route / moe_route_backward: the top-k experts of each token,
           their softmax weights, the rows each expert gets and the balance
           loss; with ``train`` also the gradient of the logits.
  group    group_rows: rows listed by group (stable), their positions, and the
           groups' offsets, as the grouped GEMM takes them.
  combine  moe_combine / moe_combine_backward: a token's weighted sum over its
           experts' output rows, added to the shared expert's output; with
           ``train`` the gradients of the rows and of the weights.
  lora     lora_add: low-rank adapters of many requests, one per row at most,
           added to a shared projection's output.
"""
import math

import torch

own = False

DEV = "cuda"


# --------------------------------------------------------------------------
# cases

def listed():
    return [
        # one decode step of 16 sequences through a wide router, serving only
        {"name": "route_decode_t16_e256", "op": "route", "tokens": 16, "experts": 256, "k": 8,
         "dtype": "float32", "renorm": True, "masked": False, "closed": 0, "train": False},
        # the MoE share's own batch: 4096 tokens to 8 of 32 experts, uneven
        # popularity, balance loss and gradient as in a training step
        {"name": "route_train_t4096_e32", "op": "route", "tokens": 4096, "experts": 32, "k": 8,
         "dtype": "float32", "renorm": True, "masked": False, "closed": 0, "train": True},
        # a padded odd batch in bf16, four experts closed, weights not renormalised
        {"name": "route_train_t5003_e60", "op": "route", "tokens": 5003, "experts": 60, "k": 4,
         "dtype": "bfloat16", "renorm": False, "masked": True, "closed": 4, "train": True},
        # a large training batch through a wide router
        {"name": "route_train_t131072_e256", "op": "route", "tokens": 131072, "experts": 256, "k": 8,
         "dtype": "float32", "renorm": True, "masked": True, "closed": 0, "train": True},
        # the rows of one decode step (16 tokens, 8 experts each)
        {"name": "group_r128_g256", "op": "group", "rows": 128, "groups": 256, "dropped": 0.0},
        # the rows of a large prefill batch, some of them padding
        {"name": "group_r1048576_g256", "op": "group", "rows": 1048576, "groups": 256,
         "dropped": 0.05},
        # a decode step's outputs back to its tokens, no shared expert
        {"name": "combine_t16_n7168", "op": "combine", "tokens": 16, "k": 8, "n": 7168,
         "base": False, "dropped": 0.0, "train": False},
        # the MoE share's 32768 rows back to 4096 tokens, forward and backward
        {"name": "combine_train_t4096_n7168", "op": "combine", "tokens": 4096, "k": 8, "n": 7168,
         "base": True, "dropped": 0.02, "train": True},
        # decode: 16 sequences, an adapter each, beside a 4096 x 4096 projection
        {"name": "lora_decode_t16_4096", "op": "lora", "tokens": 16, "requests": 16, "k": 4096,
         "n": 4096, "rank": 16, "adapters": 16, "bare": 0.0},
        # a mixed batch of short chunks and single tokens, some without adapter
        {"name": "lora_mixed_t515_7168_1536", "op": "lora", "tokens": 515, "requests": 80,
         "k": 7168, "n": 1536, "rank": 64, "adapters": 32, "bare": 0.2},
        # prefill of a few long prompts beside an MLP up projection
        {"name": "lora_prefill_t8192_7168_18432", "op": "lora", "tokens": 8192, "requests": 10,
         "k": 7168, "n": 18432, "rank": 32, "adapters": 8, "bare": 0.1},
        # prefill beside a down projection, larger ranks, an odd number of rows
        {"name": "lora_prefill_t4099_14336_4096", "op": "lora", "tokens": 4099, "requests": 7,
         "k": 14336, "n": 4096, "rank": 128, "adapters": 5, "bare": 0.0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng):
    """A layer's width: a usual one, or any other, odd ones among them."""
    if rng.random() < 0.4:
        return _log_int(rng, 50, 16384)
    return rng.choice([64, 512, 576, 1024, 1536, 2048, 4096, 7168, 14336, 18432])


def draw(rng):
    op = rng.choice(["route", "group", "combine", "lora"])
    if op == "route":
        experts = _log_int(rng, 4, 512)
        return {"op": op, "tokens": min(_log_int(rng, 1, 131072), 131072 * 256 // experts),
                "experts": experts, "k": rng.randint(1, min(experts, 10)),
                "dtype": rng.choice(["float32", "bfloat16"]), "renorm": rng.random() < 0.5,
                "masked": rng.random() < 0.5, "closed": rng.randint(0, experts // 8),
                "train": rng.random() < 0.6}
    if op == "group":
        return {"op": op, "rows": _log_int(rng, 1, 1048576), "groups": _log_int(rng, 1, 1024),
                "dropped": rng.choice([0.0, 0.05, 0.5])}
    if op == "combine":
        n, k = _width(rng), rng.randint(1, 10)
        most = 4096 * 7168 * (8 + 1) // (n * (k + 1))    # the largest listed case's bytes
        return {"op": op, "tokens": min(_log_int(rng, 1, 16384), most), "k": k,
                "n": n, "base": rng.random() < 0.5, "dropped": rng.choice([0.0, 0.02, 0.3]),
                "train": rng.random() < 0.5}
    k = rng.choice([128, 512, 896, 1536, 2048, 4096, 5120, 7168, 14336, 16384])
    n = _width(rng)
    rank, adapters = 8 * _log_int(rng, 1, 16), _log_int(rng, 1, 32)
    # within the listed cases' largest bytes and plain products
    most = min(8192, 8192 * 256 * 25600 // (adapters * rank * (k + n)),
               8192 * (7168 + 2 * 18432) // (k + 2 * n))
    tokens = min(_log_int(rng, 1, 8192), most)
    requests = rng.randint(1, tokens) if tokens <= 64 else _log_int(rng, 1, min(tokens, 256))
    return {"op": op, "tokens": tokens, "requests": requests, "k": k, "n": n, "rank": rank,
            "adapters": adapters, "bare": rng.choice([0.0, 0.2])}


# --------------------------------------------------------------------------
# inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed * 7919 + 13)


def _randn(g, *shape):
    return torch.randn(*shape, device=DEV, generator=g)


def _rand(g, *shape):
    return torch.rand(*shape, device=DEV, generator=g)


def _group_ids(g, rows, groups, dropped):
    """Group of each row with uneven (Zipf 1.1) popularity, -1 where dropped."""
    popular = torch.arange(1, groups + 1, device=DEV, dtype=torch.float32).pow(-1.1).cumsum(0)
    ids = torch.searchsorted(popular / popular[-1], _rand(g, rows)).clamp(max=groups - 1)
    return torch.where(_rand(g, rows) < dropped, -1, ids).to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    if c["op"] == "route":
        T, E, k = c["tokens"], c["experts"], c["k"]
        popular = -0.5 * torch.arange(1, E + 1, device=DEV, dtype=torch.float32).log()
        logits = _randn(g, T, E) * 1.5 + popular[torch.randperm(E, device=DEV, generator=g)]
        if c["closed"]:
            shut = torch.randperm(E, device=DEV, generator=g)[:c["closed"]]
            logits[:, shut] = -math.inf
        c["logits"] = logits.to(getattr(torch, c["dtype"]))
        c["mask"] = None
        if c["masked"]:   # padding rows hold whatever was there
            c["mask"] = _rand(g, T) >= 0.1
            c["logits"][~c["mask"]] = math.nan
        c["coef"] = 0.01 if c["train"] else None
        c["d_weights"] = _randn(g, T, k) * 0.1
        c["d_loss"] = torch.ones((), device=DEV)
    elif c["op"] == "group":
        c["ids"] = _group_ids(g, c["rows"], c["groups"], c["dropped"])
    elif c["op"] == "combine":
        T, k, n = c["tokens"], c["k"], c["n"]
        kept = _rand(g, T * k) >= c["dropped"]
        place = torch.argsort(_rand(g, T * k) + (~kept) * 2.0)   # kept slots first, then dropped
        positions = torch.empty_like(place)
        positions[place] = torch.arange(T * k, device=DEV)
        c["positions"] = torch.where(kept, positions, -1).to(torch.int32).view(T, k)
        c["offsets"] = kept.sum(dtype=torch.int32).view(1)
        c["y"] = _randn(g, T * k, n).to(torch.bfloat16)
        c["y"][torch.arange(T * k, device=DEV) >= c["offsets"]] = math.nan   # rows no expert wrote
        c["weights"] = torch.softmax(_randn(g, T, k), 1)
        c["base_out"] = _randn(g, T, n).to(torch.bfloat16) if c["base"] else None
        c["d_out"] = _randn(g, T, n).to(torch.bfloat16)
    else:
        T, K, N, r, L = c["tokens"], c["k"], c["n"], c["rank"], c["adapters"]
        # consecutive rows per request; single tokens are requests of length one
        cuts = torch.randperm(T, device=DEV, generator=g)[:c["requests"] - 1].sort().values
        which = torch.bucketize(torch.arange(T, device=DEV), cuts, right=True)
        who = torch.randint(0, L, (c["requests"] + 1,), device=DEV, generator=g)
        if c["requests"] <= L:     # an adapter of its own for each request
            who[:-1] = torch.randperm(L, device=DEV, generator=g)[:c["requests"]]
        who = torch.where(_rand(g, who.numel()) < c["bare"], -1, who)
        c["ids"] = who[which].to(torch.int32)
        c["x"] = _randn(g, T, K).to(torch.bfloat16)
        c["base"] = _randn(g, T, N).to(torch.bfloat16)
        c["a"] = (_randn(g, L, r, K) / math.sqrt(K)).to(torch.bfloat16)
        c["b"] = (_randn(g, L, N, r) / math.sqrt(r)).to(torch.bfloat16)
        c["scale"] = 0.25 + _rand(g, L)
        c["out"] = torch.empty_like(c["base"])
    return c


# --------------------------------------------------------------------------
# the package's calls

def _own(s):
    import block_scaled_fp8_act_amd as fb
    if s["op"] == "route":
        r = fb.moe_route(s["logits"], s["k"], mask=s["mask"], renormalize=s["renorm"],
                         loss_coef=s["coef"])
        if not s["train"]:
            return r.ids, r.weights, r.counts
        d = fb.moe_route_backward(s["logits"], r, d_weights=s["d_weights"], d_loss=s["d_loss"])
        return r.ids, r.weights, r.counts, r.loss, d
    if s["op"] == "group":
        r = fb.group_rows(s["ids"], s["groups"])
        return r.order, r.positions, r.offsets
    if s["op"] == "combine":
        out = fb.moe_combine(s["y"], s["weights"], s["positions"], base=s["base_out"])
        if not s["train"]:
            return out
        return out, *fb.moe_combine_backward(s["d_out"], s["y"], s["weights"], s["positions"],
                                             s["offsets"])
    return fb.lora_add(s["base"], s["x"], s["a"], s["b"], s["ids"], scale=s["scale"],
                       out=s["out"])


# --------------------------------------------------------------------------
# the plain form

def _plain_route(s):
    T, E, k = s["tokens"], s["experts"], s["k"]
    l = s["logits"].float()
    if s["mask"] is not None:
        l = torch.where(s["mask"][:, None], l, -math.inf)
    top, at = torch.sort(l, dim=1, descending=True, stable=True)   # ties to the lowest expert
    top, at = top[:, :k], at[:, :k]
    live = top[:, :1] > -math.inf
    chosen = top > -math.inf
    ids = torch.where(chosen, at, -1).to(torch.int32)
    peak = torch.where(live, top[:, :1], 0.0)
    whole = torch.exp(l - peak)
    total = torch.where(live, whole.sum(1, keepdim=True), 1.0)
    p = whole / total
    w = torch.exp(top - peak)
    w = w / (torch.where(live, w.sum(1, keepdim=True), 1.0) if s["renorm"] else total)
    counts = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    counts.scatter_add_(0, torch.where(chosen, at, E).reshape(-1),
                        torch.ones(T * k, dtype=torch.int32, device=DEV))
    counts = counts[:E]
    if not s["train"]:
        return ids, w, counts
    n = live.sum().clamp(min=1).float()
    share = counts.float() * (s["coef"] * E / k) / (n * n)
    loss = (share * p.sum(0)).sum()
    dp = share * s["d_loss"]
    d = p * (dp - (p * dp).sum(1, keepdim=True))
    dw = torch.where(chosen, s["d_weights"], 0.0)
    back = (w * dw).sum(1, keepdim=True)
    if s["renorm"]:
        d.scatter_add_(1, at, w * (dw - back))
    else:
        d = (d - p * back).scatter_add_(1, at, w * dw)
    return ids, w, counts, loss, d.to(s["logits"].dtype)


def _plain_group(s):
    R, G = s["rows"], s["groups"]
    key = torch.where((s["ids"] >= 0) & (s["ids"] < G), s["ids"], G)
    key, order = torch.sort(key, stable=True)
    positions = torch.empty(R, dtype=torch.int32, device=DEV)
    positions[order] = torch.where(key < G, torch.arange(R, dtype=torch.int32, device=DEV), -1)
    offsets = torch.searchsorted(key, torch.arange(G + 1, dtype=torch.int32, device=DEV))
    return order.to(torch.int32), positions, offsets.to(torch.int32)


def _plain_combine(s):
    R, T = s["y"].shape[0], s["tokens"]
    pos = s["positions"].long()
    kept = pos >= 0
    rows = torch.where(kept[:, :, None], s["y"][pos.clamp(min=0)].float(), 0.0)
    out = (rows * s["weights"][:, :, None]).sum(1)
    if s["base_out"] is not None:
        out = out + s["base_out"].float()
    out = out.to(torch.bfloat16)
    if not s["train"]:
        return out
    d = s["d_out"].float()[:, None, :]
    dw = (rows * d).sum(2)
    dy = torch.zeros(R + 1, s["n"], dtype=torch.bfloat16, device=DEV)
    dy[torch.where(kept, pos, R).reshape(-1)] = (d * s["weights"][:, :, None]).to(
        torch.bfloat16).view(T * s["k"], -1)
    return out, dy[:R], dw


def _plain_lora(s):
    T, K, N, r, L = s["tokens"], s["k"], s["n"], s["rank"], s["adapters"]
    # every adapter's first product, those of other rows' adapters masked out
    h = (s["x"].float() @ s["a"].float().view(L * r, K).t()).view(T, L, r)
    mine = torch.arange(L, device=DEV)[None, :] == s["ids"][:, None]
    h = torch.where(mine[:, :, None], h * s["scale"][None, :, None], 0.0).view(T, L * r)
    delta = h @ s["b"].float().permute(0, 2, 1).reshape(L * r, N)
    s["out"].copy_(s["base"].float() + delta)
    return s["out"]


def run(state):
    if own:
        return _own(state)
    return {"route": _plain_route, "group": _plain_group, "combine": _plain_combine,
            "lora": _plain_lora}[state["op"]](state)


# --------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "route":
        T, E, k = c["tokens"], c["experts"], c["k"]
        size = 4 if c["dtype"] == "float32" else 2
        bytes_ = T * E * size + T * k * 8 + E * 4 + (T if c["masked"] else 0)
        flops = 5 * T * E
        if c["train"]:    # the gradient: logits and weight gradients in, logit gradients out
            bytes_ += 2 * T * E * size + T * k * 12
            flops += 8 * T * E
        return {"bytes": bytes_, "flops": flops}
    if c["op"] == "group":
        return {"bytes": 12 * c["rows"] + 4 * (c["groups"] + 1), "flops": 0}
    if c["op"] == "combine":
        T, k, n = c["tokens"], c["k"], c["n"]
        kept = T * k * (1 - c["dropped"])
        bytes_ = 2 * n * (kept + T * (2 if c["base"] else 1)) + 8 * T * k
        flops = 2 * kept * n
        if c["train"]:
            bytes_ += 2 * n * (kept + T + T * k) + 12 * T * k
            flops += 3 * kept * n
        return {"bytes": bytes_, "flops": flops}
    T, K, N, r = c["tokens"], c["k"], c["n"], c["rank"]
    used = min(c["adapters"], c["requests"])
    worn = T * (1 - c["bare"])
    return {"bytes": 2 * worn * K + 4 * T * N + 2 * used * r * (K + N) + 4 * T,
            "flops": 2 * worn * r * (K + N)}


# --------------------------------------------------------------------------
# the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "group": _exact_group, "combine": _exact_combine,
            "lora": _exact_lora}[s["op"]](s)


def _exact_route(s):
    T, E, k = s["tokens"], s["experts"], s["k"]
    z = s["logits"].double()
    if s["mask"] is not None:
        z[~s["mask"]] = -math.inf
    rest = z.clone()
    ids, weights = [], []
    grid = torch.arange(E, device=DEV)
    for _ in range(k):      # the largest left, the lowest index among equals
        m = rest.amax(1, keepdim=True)
        i = torch.where(rest == m, grid, E).amin(1, keepdim=True)
        ids.append(torch.where(m > -math.inf, i, -1))
        weights.append(m)
        rest.scatter_(1, i, -math.inf)
    ids, weights = torch.cat(ids, 1), torch.cat(weights, 1)
    live = ids[:, 0] >= 0
    norm = torch.logsumexp(weights if s["renorm"] else z, 1, keepdim=True)
    w = torch.where(ids >= 0, torch.exp(weights - norm), 0.0)
    counts = (ids.reshape(-1, 1) == grid).sum(0).to(torch.int32) if T * k * E < 1 << 28 else \
        torch.bincount(ids[ids >= 0].long(), minlength=E).to(torch.int32)
    if not s["train"]:
        return ids.to(torch.int32), w, counts
    p = torch.zeros_like(z)
    p[live] = torch.softmax(z[live], 1)
    n = max(int(live.sum()), 1)
    loss = s["coef"] * (counts.double() * E / (k * n) * (p.sum(0) / n)).sum()
    g = s["d_loss"].double() * s["coef"] * counts.double() * E / (k * n) / n     # dL/dp
    gp = g.expand(T, E).clone()
    dw = torch.where(ids >= 0, s["d_weights"].double(), 0.0)
    safe = ids.clamp(min=0).long()
    if s["renorm"]:
        d = torch.zeros_like(z).scatter_add_(1, safe, w * (dw - (w * dw).sum(1, keepdim=True)))
    else:
        gp.scatter_add_(1, safe, dw)
        d = torch.zeros_like(z)
    d += p * (gp - (p * gp).sum(1, keepdim=True))
    return ids.to(torch.int32), w, counts, loss, d


def _exact_group(s):
    ids = s["ids"].cpu().numpy()
    R, G = s["rows"], s["groups"]
    key = [int(i) if 0 <= i < G else G for i in ids]
    order = sorted(range(R), key=key.__getitem__)
    positions = [-1] * R
    offsets = [0] * (G + 1)
    for at, row in enumerate(order):
        if key[row] < G:
            positions[row] = at
            offsets[key[row] + 1] += 1
    for g in range(G):
        offsets[g + 1] += offsets[g]
    as_int = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return as_int(order), as_int(positions), as_int(offsets)


def _exact_combine(s):
    T, k, n = s["tokens"], s["k"], s["n"]
    out = torch.zeros(T, n, dtype=torch.float64, device=DEV)
    if s["base_out"] is not None:
        out += s["base_out"]
    dy = torch.zeros(s["y"].shape[0], n, dtype=torch.float64, device=DEV)
    dw = torch.zeros(T, k, dtype=torch.float64, device=DEV)
    for j in range(k):
        kept = (s["positions"][:, j] >= 0).nonzero()[:, 0]
        rows = s["positions"][kept, j].long()
        w = s["weights"][kept, j].double()[:, None]
        out[kept] += w * s["y"][rows]
        if s["train"]:
            d = s["d_out"][kept].double()
            dw[kept, j] = (d * s["y"][rows]).sum(1)
            dy[rows] = w * d
    return (out, dy, dw) if s["train"] else out


def _exact_lora(s):
    out = s["base"].double()
    for g in s["ids"].unique().tolist():
        if g < 0:
            continue
        rows = (s["ids"] == g).nonzero()[:, 0]
        h = s["x"][rows].double() @ s["a"][g].double().t().contiguous()
        out[rows] += s["scale"][g].double() * (h @ s["b"][g].double().t().contiguous())
    return out
