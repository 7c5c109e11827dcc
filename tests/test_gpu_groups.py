"""Rows by group (exact) and the weighted return of the experts' rows, against
the binary64 oracle.

Tolerances: combine adds k + 1 fp32 terms, so (k + 1) 2^-24 of their
magnitudes, and rounds once to bf16 (half a unit of its 8
significant bits: 2^-8 of the result); a weight gradient
adds N products, at most N / 256 + 8 one after another in a lane and 10 across
lanes and waves.  d_y is one fp32 product rounded to bf16: equal bits."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_act_amd as fb
from gpu_helpers import dev, say
from oracle import routing as orr

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("R", [0, 1, 2, 63, 64, 65, 128, 1000, 1024, 1025, 8191, 8192, 8193, 20000,
                               131073])
@pytest.mark.parametrize("G", [1, 2, 31, 256, 1024])
def test_group_rows(R, G):
    say("group", R, G)
    r = np.random.default_rng(R * 7 + G)
    ids = np.minimum(r.geometric(3.0 / (G + 2), R) - 1, G - 1).astype(np.int32)
    if R > 2:
        out = r.random(R) < 0.1
        ids[out] = r.choice([-1, G, -2 ** 31, 2 ** 31 - 1, G + 7], int(out.sum()))
    g = fb.group_rows(torch.from_numpy(ids).to(dev()), G)
    torch.cuda.synchronize()
    key = np.where((ids >= 0) & (ids < G), ids, G)
    order = np.argsort(key, kind="stable").astype(np.int32)
    offsets = np.searchsorted(key[order], np.arange(G + 1)).astype(np.int32)
    positions = np.empty(R, np.int32)
    positions[order] = np.where(key[order] < G, np.arange(R), -1)
    if R <= 200:
        for a, b in zip(orr.group_rows(ids, G), (order, positions, offsets)):
            assert np.array_equal(a, b)
    assert np.array_equal(g.offsets.cpu().numpy(), offsets)
    assert np.array_equal(g.order.cpu().numpy(), order)
    assert np.array_equal(g.positions.cpu().numpy(), positions)


@pytest.mark.parametrize("value", [-1, 0, 6])
def test_group_rows_all_in_one(value):
    ids = torch.full((5000, 2), value, dtype=torch.int32, device=dev())
    g = fb.group_rows(ids, 7)
    assert g.positions.shape == (5000, 2)
    assert torch.equal(g.order.cpu(), torch.arange(10000, dtype=torch.int32))
    assert int(g.offsets[7]) == (0 if value < 0 else 10000)


def places(seed, T, k, R, dropped):
    """Distinct rows for the kept slots, the first ones of y."""
    r = np.random.default_rng(seed)
    pos = np.full(T * k, -1, np.int32)
    kept = r.permutation(T * k)[:int(round(T * k * (1 - dropped)))]
    kept = kept[:R]
    pos[kept] = r.permutation(len(kept))
    return pos.reshape(T, k), len(kept)


@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (1, 8, 7168), (3, 2, 7), (16, 8, 512), (5, 3, 513),
                                   (4, 32, 2049), (33, 6, 1000), (7, 9, 4096), (2, 5, 8191),
                                   (300, 4, 72)])
@pytest.mark.parametrize("base", [False, True])
@pytest.mark.parametrize("dropped", [0.0, 0.4, 1.0])
def test_combine(T, k, N, base, dropped):
    say("combine", T, k, N, base, dropped)
    r = np.random.default_rng(T * k + N)
    R = T * k + 3
    pos, used = places(N, T, k, R, dropped)
    y = torch.from_numpy(r.standard_normal((R, N)).astype(np.float32)).bfloat16()
    y[used:] = float("nan")                       # rows of no slot are not read
    w = r.random((T, k)).astype(np.float32)
    w[pos < 0] = np.nan                           # nor are the weights of dropped slots
    b = torch.from_numpy(r.standard_normal((T, N)).astype(np.float32)).bfloat16() if base else None
    b64 = None if b is None else b.double().numpy()
    want, mag = orr.combine(y.double().numpy(), w.astype(np.float64), pos, b64)
    wd, pd = torch.from_numpy(w).to(dev()), torch.from_numpy(pos).to(dev())
    bd = None if b is None else b.to(dev())
    got = fb.moe_combine(y.to(dev()), wd, pd, bd)
    tol = mag * (k + 1) * U + np.abs(want) * 2.0 ** -8 * 1.0001
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= tol)
    if base:                                      # in place
        fb.fp8blk_moe_combine(y.to(dev()), wd, pd, bd, bd)
        assert torch.equal(bd, got)


@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (1, 8, 7168), (3, 2, 7), (16, 8, 512), (5, 3, 513),
                                   (4, 32, 2049), (33, 9, 1000), (2, 5, 8191)])
@pytest.mark.parametrize("dropped", [0.0, 0.4, 1.0])
def test_combine_backward(T, k, N, dropped):
    say("combine backward", T, k, N, dropped)
    r = np.random.default_rng(T * k + N + 1)
    R = T * k + 3
    pos, used = places(N + 1, T, k, R, dropped)
    y = torch.from_numpy(r.standard_normal((R, N)).astype(np.float32)).bfloat16()
    y[used:] = float("nan")
    d = torch.from_numpy(r.standard_normal((T, N)).astype(np.float32)).bfloat16()
    w = torch.from_numpy(r.random((T, k)).astype(np.float32))
    used_d = torch.tensor([0, used], dtype=torch.int32, device=dev())
    dy, dw = fb.moe_combine_backward(d.to(dev()), y.to(dev()), w.to(dev()),
                                     torch.from_numpy(pos).to(dev()), used_d)
    want, mag = orr.combine_weight_gradient(d.double().numpy(), y.double().numpy(), pos)
    tol = mag * (N / 256 + 18) * U
    assert np.all(np.abs(dw.double().cpu().numpy() - want) <= tol)
    rows = torch.zeros(R, N, dtype=torch.bfloat16)
    kept = torch.from_numpy(pos >= 0)
    rows[torch.from_numpy(pos)[kept].long()] = (w[:, :, None] * d.float()[:, None, :])[kept].bfloat16()
    assert torch.equal(dy.cpu(), rows)


def test_combine_gradients_against_differences():
    """The sum is linear in each weight and in each row, so a difference of
    the forward in binary64 is the gradient itself."""
    T, k, N = 3, 4, 40
    r = np.random.default_rng(0)
    pos, used = places(2, T, k, T * k, 0.2)
    y = torch.from_numpy(r.standard_normal((T * k, N)).astype(np.float32)).bfloat16()
    d = torch.from_numpy(r.standard_normal((T, N)).astype(np.float32)).bfloat16()
    w = torch.from_numpy(r.random((T, k)).astype(np.float32))
    dy, dw = fb.moe_combine_backward(d.to(dev()), y.to(dev()), w.to(dev()),
                                     torch.from_numpy(pos).to(dev()),
                                     torch.tensor([used], dtype=torch.int32, device=dev()))
    y64, w64, d64 = y.double().numpy(), w.double().numpy(), d.double().numpy()
    value = lambda yy, ww: float(np.sum(d64 * orr.combine(yy, ww, pos)[0]))  # noqa: E731
    at = value(y64, w64)
    for i in range(T):
        for j in range(k):
            up = w64.copy()
            up[i, j] += 1.0
            diff = value(y64, up) - at
            assert abs(float(dw[i, j]) - diff) <= 1e-5 * (1 + abs(diff))
    for p in range(used):
        up = y64.copy()
        up[p, 7] += 1.0
        diff = value(up, w64) - at
        assert abs(float(dy[p, 7]) - diff) <= 2.0 ** -8 * abs(diff) + 1e-9


def test_combine_positions_out_of_range_add_nothing():
    y = torch.ones(4, 24, dtype=torch.bfloat16, device=dev())
    pos = torch.tensor([[4, 2 ** 31 - 1], [-5, 1]], dtype=torch.int32, device=dev())
    w = torch.full((2, 2), 2.0, device=dev())
    out = fb.moe_combine(y, w, pos)
    assert not out[0].any() and bool((out[1] == 2).all())


def test_combine_no_rows():
    none = torch.empty(0, 5, dtype=torch.bfloat16, device=dev())
    pos = torch.full((3, 2), -1, dtype=torch.int32, device=dev())
    w = torch.ones(3, 2, device=dev())
    assert not fb.moe_combine(none, w, pos).any()
    zero = torch.zeros(1, dtype=torch.int32, device=dev())
    dy, dw = fb.moe_combine_backward(torch.ones(3, 5, dtype=torch.bfloat16, device=dev()), none, w,
                                     pos, zero)
    assert dy.shape == (0, 5) and not dw.any()
    y = torch.ones(6, 5, dtype=torch.bfloat16, device=dev())
    dy, dw = fb.moe_combine_backward(none, y, w[:0], pos[:0], zero)
    assert not dy.any()
    assert fb.moe_combine(y, w[:0], pos[:0]).shape == (0, 5)


def test_group_and_combine_refusals():
    ids = torch.zeros(8, dtype=torch.int32, device=dev())
    for bad in (0, 1025):
        with pytest.raises(ValueError):
            fb.group_rows(ids, bad)
    with pytest.raises(TypeError):
        fb.group_rows(ids.long(), 4)
    with pytest.raises(ValueError):
        fb.group_rows(ids[::2], 4)
    y = torch.zeros(8, 16, dtype=torch.bfloat16, device=dev())
    w = torch.zeros(4, 2, device=dev())
    p = torch.zeros(4, 2, dtype=torch.int32, device=dev())
    with pytest.raises(TypeError):
        fb.moe_combine(y.float(), w, p)
    with pytest.raises(TypeError):
        fb.moe_combine(y, w, p.long())
    with pytest.raises(ValueError):
        fb.moe_combine(y, w, p[:3])
    with pytest.raises(ValueError):
        fb.moe_combine(y, w, p, base=y)
    with pytest.raises(ValueError):
        fb.moe_combine(y, torch.zeros(4, 33, device=dev()),
                       torch.zeros(4, 33, dtype=torch.int32, device=dev()))
    with pytest.raises(ValueError):
        fb.moe_combine_backward(y, y, w, p, ids)


@pytest.mark.parametrize("fmt", ["float", "ue8m0"])
@pytest.mark.parametrize("T", [1, 16, 150])
def test_moe_experts(T, fmt):
    """The whole path: each token's sum over its experts equals the experts'
    products called one by one on that token's quantized row (the grouped
    product takes the same rows, in another order), weighted and added in
    fp32; masked tokens keep the shared expert's output."""
    E, K, I, k = 6, 256, 128, 3
    r = np.random.default_rng(T)
    bf = lambda *s: torch.from_numpy(r.standard_normal(s).astype(np.float32)).bfloat16().to(dev())  # noqa: E731
    x, shared = bf(T, K), bf(T, K)
    up = [fb.weight_block_quant(bf(2 * I, K) * 0.05, fmt) for _ in range(E)]
    down = [fb.weight_block_quant(bf(K, I) * 0.05, fmt) for _ in range(E)]
    stack = lambda ws, i: torch.stack([w[i] for w in ws])  # noqa: E731
    mask = torch.from_numpy(r.random(T) < 0.8).to(dev())
    routing = fb.moe_route(bf(T, E), k, mask=mask)
    got = fb.moe_experts(x, routing, stack(up, 0), stack(up, 1), stack(down, 0), stack(down, 1), shared)
    rows = []
    for e in range(E):
        h = fb.block_gemm(*fb.act_quant_group(x, fmt), *up[e])
        rows.append(fb.block_gemm(*fb.swiglu_act_quant(h, fmt), *down[e]).double())
    ids = routing.ids.long()
    each = torch.stack(rows)[ids.clamp(min=0), torch.arange(T, device=dev())[:, None]]   # [T,k,K]
    terms = torch.where((ids >= 0)[:, :, None], each * routing.weights.double()[:, :, None], 0.0)
    want = shared.double() + terms.sum(1)
    # both GEMMs meet the same tolerance: 2^-8 of an element each, the products' spread beside it
    tol = 2.0 ** -8 * want.abs() + 2.0 ** -5 * terms.abs().sum(1) + 2.0 ** -7 * terms.abs().amax()
    assert bool(((got.double() - want).abs() <= tol).all())
    assert torch.equal(got[~mask], shared[~mask])
