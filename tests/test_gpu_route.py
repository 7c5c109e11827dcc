"""Routing, its balance loss and gradient against the binary64 oracle.

Tolerances (u = 2^-24).  A probability is a quotient of e^x terms, x = l - max:
x is rounded once (|x| u), the exponential and the quotient a few ulp, and the
sum of E positive terms is added at most 16 in a lane and 6 across lanes; so
|p - p^| <= p (40 + 2 |x|) u.  The loss adds T such terms per expert (at most
T / 32 + 32 one after another).  A gradient adds up terms whose magnitudes the
oracle sums (times the same relative bound, for the terms and for the sums
inside); a bf16 result is rounded once more (2^-8)."""
import math

import numpy as np
import pytest
import torch

import block_scaled_fp8_act_amd as fb
from gpu_helpers import dev, say
from oracle import routing as orr

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def make(seed, T, E, dtype, std=2.0, ties=False, closed=0, masked=0.0):
    r = np.random.default_rng(seed)
    l = r.standard_normal((T, E)).astype(np.float32) * std
    if ties:
        l = np.round(l)
    if closed:
        l[:, r.permutation(E)[:closed]] = -np.inf
    t = torch.from_numpy(l).to(dtype)
    mask = (r.random(T) >= masked) if masked else None
    if mask is not None:
        t[~torch.from_numpy(mask)] = float("nan")
    return t, mask


def check(t, k, mask=None, renorm=True, coef=0.01, seed=0, d_loss=0.7):
    T, E = t.shape
    l64 = t.double().numpy()
    m = None if mask is None else torch.from_numpy(mask).to(dev())
    r = fb.moe_route(t.to(dev()), k, mask=m, renormalize=renorm, loss_coef=coef)
    torch.cuda.synchronize()
    ids, w, counts, n, loss = orr.route(l64, k, mask, renorm, coef)
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    assert np.array_equal(r.counts.cpu().numpy(), counts)
    assert int(r.rows) == n
    live = ids >= 0
    peak = np.where(np.isnan(l64), -np.inf, l64).max(1)
    x = np.zeros_like(w)
    rows = np.nonzero(live)
    x[rows] = np.abs(l64[rows[0], ids[rows]] - peak[rows[0]])
    assert np.all(np.abs(r.weights.cpu().numpy() - w) <= w * (40 + 2 * x) * U)
    fin = np.where(np.isfinite(l64), l64, np.nan)
    span = float(np.nanmax(np.nanmax(fin, 1, initial=0) - np.nanmin(fin, 1, initial=0)))
    span = min(span, 110.0)     # e^-110 is below fp32
    rel = (40 + 2 * span + T / 32 + 32) * U
    assert abs(float(r.loss) - loss) <= abs(loss) * rel + 1e-30
    # gradient
    g = np.random.default_rng(seed + 99)
    dw = g.standard_normal((T, k)).astype(np.float32)
    dw_dev = torch.from_numpy(np.where(live, dw, np.nan)).to(dev())    # unused slots are not read
    d = fb.moe_route_backward(t.to(dev()), r, dw_dev, torch.tensor(d_loss, device=dev()))
    torch.cuda.synchronize()
    want, mag = orr.route_backward(l64, k, ids, counts, n, renorm, coef, dw, np.float32(d_loss))
    got = d.double().cpu().numpy()
    assert d.dtype == t.dtype
    tol = mag * (100 + 4 * span) * U + 1e-37
    if t.dtype == torch.bfloat16:
        tol = tol + np.abs(want) * 2.0 ** -8
    assert np.all(np.abs(got - want) <= tol), float(np.max(np.abs(got - want) / (tol + 1e-300)))
    return r, d


SHAPES = [(1, 1, 1), (1, 8, 8), (3, 5, 2), (16, 256, 8), (65, 32, 8), (64, 32, 8), (33, 60, 4),
          (130, 61, 3), (257, 64, 6), (100, 128, 8), (77, 129, 9), (40, 255, 16), (300, 256, 8),
          (50, 257, 17), (21, 512, 32), (9, 1000, 10), (7, 1021, 22), (130, 1024, 8)]


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [True, False])
def test_route(T, E, k, dtype, renorm):
    say("route", T, E, k, dtype, renorm)
    t, _ = make(T * 1000 + E, T, E, dtype)
    check(t, k, None, renorm)


@pytest.mark.parametrize("E", [6, 60, 128, 250, 300, 777])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_ties_masks_and_closed_experts(E, dtype):
    """Ties go to the lowest expert; masked rows hold NaN; fewer experts open
    than k leaves slots empty."""
    t, mask = make(E, 150, E, dtype, ties=True, closed=E - 5, masked=0.3)
    r, d = check(t, min(E, 8), mask, renorm=E % 4 == 0)
    assert not np.any(d.float().cpu().numpy()[~mask])
    t, mask = make(E + 1, 150, E, dtype, ties=True, masked=0.3)
    check(t, min(E, 6), mask)


@pytest.mark.parametrize("renorm", [True, False])
def test_route_rows_without_any_open_expert(renorm):
    t, _ = make(5, 40, 24, torch.float32)
    t[3] = -math.inf
    t[17:20] = -math.inf
    t[25, 3:] = -math.inf
    check(t, 4, None, renorm)
    check(torch.full((9, 24), -math.inf), 4, None, renorm)
    check(t, 4, np.zeros(40, bool), renorm)


def test_route_lowest_finite_values():
    """Masks written as the type's lowest value: finite, so chosen only where
    nothing else is left; a row of nothing else is uniform."""
    for dtype in (torch.float32, torch.bfloat16):
        low = torch.finfo(dtype).min
        t, _ = make(8, 20, 16, dtype)
        t[:, 2:] = low
        t[5] = low
        check(t, 4, None, True)
        check(t, 4, None, False)


def test_route_signed_zero_is_a_tie():
    t = torch.tensor([[0.0, -0.0, 0.0, -1.0], [-0.0, 0.0, -0.0, 0.0]])
    r, _ = check(t, 3)
    assert r.ids.tolist() == [[0, 1, 2], [0, 1, 2]]


def test_route_without_loss_and_its_repeats():
    """Serving form: the same choice and weights without the loss; and the same
    bits on every call."""
    for T in (5, 64, 65, 3000):
        t, mask = make(T, T, 96, torch.float32, masked=0.1)
        x, m = t.to(dev()), torch.from_numpy(mask).to(dev())
        a = fb.moe_route(x, 8, mask=m, loss_coef=0.01)
        b = fb.moe_route(x, 8, mask=m)
        c = fb.moe_route(x, 8, mask=m, loss_coef=0.01)
        assert b.loss is None and b.rows is None
        for f in ("ids", "weights", "counts"):
            assert torch.equal(getattr(a, f), getattr(b, f)), f
        assert torch.equal(a.loss, c.loss)


def test_route_large_batch():
    """Many rows per wave, over several workgroups (the oracle in torch fp64)."""
    T, E, k = 40000, 160, 6
    t, _ = make(3, T, E, torch.float32)
    r = fb.moe_route(t.to(dev()), k, loss_coef=0.01)
    p = torch.softmax(t.double(), 1)
    order = torch.sort(t, dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(r.ids.cpu().long(), order)
    counts = torch.bincount(order.reshape(-1), minlength=E)
    assert torch.equal(r.counts.cpu().long(), counts)
    loss = 0.01 * float((counts * E / (k * T) * p.mean(0)).sum())
    assert abs(float(r.loss) - loss) <= loss * (100 + T / 32) * U
    d = fb.moe_route_backward(t.to(dev()), r, None, torch.ones(1, device=dev())).cpu().double()
    g = 0.01 * counts * E / (k * T) / T
    want = p * (g - (p * g).sum(1, keepdim=True))
    mag = p * (g + (p * g).sum(1, keepdim=True))
    assert bool(((d - want).abs() <= mag * 160 * U + 1e-37).all())


@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_against_differences(renorm):
    """Central differences of the oracle's value in binary64, step h = 2^-12:
    their own error is h^2 times the third derivative, which for softmax terms
    is below the term's magnitude."""
    T, E, k = 6, 20, 3
    t, _ = make(11, T, E, torch.float32)
    r = fb.moe_route(t.to(dev()), k, renormalize=renorm, loss_coef=0.5)
    dw = np.random.default_rng(1).standard_normal((T, k)).astype(np.float32)
    d = fb.moe_route_backward(t.to(dev()), r, torch.from_numpy(dw).to(dev()),
                              torch.tensor([2.0], device=dev())).double().cpu().numpy()
    l = t.double().numpy()
    ids, counts, n = r.ids.cpu().numpy(), r.counts.cpu().numpy(), int(r.rows)
    _, mag = orr.route_backward(l, k, ids, counts, n, renorm, 0.5, dw, 2.0)
    h = 2.0 ** -12
    for i in range(T):
        for j in range(E):
            up, dn = l.copy(), l.copy()
            up[i, j] += h
            dn[i, j] -= h
            diff = (orr.route_value(up, k, ids, counts, n, renorm, 0.5, dw, 2.0)
                    - orr.route_value(dn, k, ids, counts, n, renorm, 0.5, dw, 2.0)) / (2 * h)
            assert abs(d[i, j] - diff) <= mag[i, j] * (h * h + 160 * U) + 1e-9


def test_route_gradient_parts_alone():
    t, _ = make(12, 30, 40, torch.float32)
    r = fb.moe_route(t.to(dev()), 5, loss_coef=0.3)
    dw = torch.randn(30, 5, device=dev())
    dl = torch.tensor([1.5], device=dev())
    zero_w, zero_l = torch.zeros_like(dw), torch.zeros_like(dl)
    for a, b in (((dw, None), (dw, zero_l)), ((None, dl), (zero_w, dl))):
        x = fb.moe_route_backward(t.to(dev()), r, *a)
        y = fb.moe_route_backward(t.to(dev()), r, *b)
        assert torch.equal(x, y)
    assert not fb.moe_route_backward(t.to(dev()), r).any()


def test_route_no_rows():
    r = fb.moe_route(torch.empty(0, 12, device=dev()), 3, loss_coef=0.1)
    assert r.ids.shape == (0, 3) and int(r.counts.sum()) == 0 and int(r.rows) == 0
    assert float(r.loss) == 0.0
    assert fb.moe_route_backward(torch.empty(0, 12, device=dev()), r, torch.empty(0, 3, device=dev()),
                                 torch.ones(1, device=dev())).shape == (0, 12)


def test_route_refusals():
    x = torch.zeros(4, 8, device=dev())
    for bad in (0, 9):
        with pytest.raises(ValueError):
            fb.moe_route(x, bad)
    with pytest.raises(ValueError):
        fb.moe_route(torch.zeros(4, 64, device=dev()), 33)      # more than MAX_TOPK
    with pytest.raises(ValueError):
        fb.moe_route(torch.zeros(4, 1025, device=dev()), 2)     # more than MAX_GROUPS
    with pytest.raises(TypeError):
        fb.moe_route(x.half(), 2)
    with pytest.raises(ValueError):
        fb.moe_route(x.t(), 2)
    with pytest.raises(ValueError):
        fb.moe_route(x, 2, mask=torch.ones(5, dtype=torch.bool, device=dev()))
    with pytest.raises(ValueError):
        fb.moe_route(x.cpu(), 2)
    r = fb.moe_route(x, 2)
    with pytest.raises(ValueError):
        fb.moe_route_backward(x, r, torch.zeros(4, 3, device=dev()))
    with pytest.raises(ValueError):
        fb.moe_route_backward(torch.zeros(4, 9, device=dev()), r)
    with pytest.raises(ValueError):
        fb.moe_route_backward(x, r, d_loss=torch.ones(1, device=dev()))   # routed without the loss
