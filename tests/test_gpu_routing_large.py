"""Routing, row groups and combining at the large end (many rows per wave,
every launch shape, offsets past 32 bits), and all of the new operators under
graph capture."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_act_amd as fb
from gpu_helpers import dev, say
from test_gpu_route import check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R,G", [(1 << 20, 32), ((1 << 20) + 1, 300), (3_000_001, 7),
                                 (5_000_000, 1024)])
def test_group_rows_large(R, G):
    say("group", R, G)
    ids = torch.randint(-2, G + 2, (R,), dtype=torch.int32, device=dev(),
                        generator=torch.Generator(device=dev()).manual_seed(R))
    g = fb.group_rows(ids, G)
    key = torch.where((ids >= 0) & (ids < G), ids, G)
    sorted_key, order = torch.sort(key, stable=True)
    assert torch.equal(g.order.long(), order)
    offsets = torch.searchsorted(sorted_key, torch.arange(G + 1, dtype=torch.int32, device=dev()))
    assert torch.equal(g.offsets.long(), offsets)
    at = torch.empty_like(g.positions)
    at[order] = torch.where(sorted_key < G, torch.arange(R, dtype=torch.int32, device=dev()), -1)
    assert torch.equal(g.positions, at)


def test_combine_past_2_31_elements():
    T, k, N = 70000, 4, 8192
    y = torch.empty((T * k, N), dtype=torch.bfloat16, device=dev())
    last = torch.arange(T * k - 8, T * k, device=dev())
    y[last] = torch.arange(8, device=dev(), dtype=torch.float32)[:, None].bfloat16()
    pos = torch.full((T, k), -1, dtype=torch.int32, device=dev())
    pos[T - 2:] = last.view(2, 4).int()
    w = torch.ones((T, k), device=dev())
    out = fb.moe_combine(y, w, pos)
    assert bool((out[T - 2] == 6).all()) and bool((out[T - 1] == 22).all())
    assert not out[:T - 2].any()
    used = torch.tensor([T * k], dtype=torch.int32, device=dev())
    d = torch.ones((T, N), dtype=torch.bfloat16, device=dev())
    dy, dw = fb.moe_combine_backward(d, y, w, pos, used)
    assert bool((dy[last] == 1).all())
    assert torch.equal(dw[T - 2:].cpu(), torch.arange(8.0).view(2, 4) * N)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_past_2_31_elements(dtype):
    """The last rows of 2.2 million x 1000 logits, forward and backward."""
    T, E, k = 2_200_000, 1000, 4
    x = torch.full((T, E), -1.0, dtype=dtype, device=dev())
    x[T - 1, [3, 999, 500, 7]] = torch.tensor([4.0, 3.0, 2.0, 1.0], dtype=dtype, device=dev())
    r = fb.moe_route(x, k, loss_coef=1.0)
    assert r.ids[T - 1].tolist() == [3, 999, 500, 7]
    assert r.ids[T - 2].tolist() == [0, 1, 2, 3]
    assert int(r.rows) == T
    counts = torch.zeros(E, dtype=torch.int32)
    counts[:4] = T - 1
    for e in (3, 999, 500, 7):
        counts[e] += 1
    assert torch.equal(r.counts.cpu(), counts)
    dw = torch.zeros((T, k), device=dev())
    dw[T - 1] = torch.tensor([1.0, 0.0, 0.0, 0.0], device=dev())
    d = fb.moe_route_backward(x, r, dw)[T - 1].double().cpu()
    w = torch.softmax(torch.tensor([4.0, 3.0, 2.0, 1.0], dtype=torch.float64), 0)
    want = w * (torch.tensor([1.0, 0, 0, 0], dtype=torch.float64) - w[0])
    got = d[[3, 999, 500, 7]]
    assert torch.allclose(got, want, rtol=1e-5 if dtype == torch.float32 else 2.0 ** -8, atol=1e-7)
    assert int((d != 0).sum()) == 4


@pytest.mark.parametrize("E,k", [(256, 8), (250, 16), (60, 4), (17, 3), (8, 8), (700, 8)])
def test_route_equal_logits(E, k):
    """A row of equal logits chooses the first experts with equal weights."""
    for T in (5, 100, 3000):
        r = fb.moe_route(torch.full((T, E), 0.25, device=dev()), k)
        assert torch.equal(r.ids.cpu(), torch.arange(k, dtype=torch.int32).expand(T, k))
        assert bool((r.weights - 1.0 / k).abs().max() <= 64 * 2.0 ** -24 / k)


@pytest.mark.parametrize("E,k", [(24, 20), (40, 32), (100, 17), (131, 32), (256, 24), (253, 31)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_many_choices(E, k, dtype):
    """More than 16 choices among up to 256 experts, two slots a lane."""
    t, mask = make(E + k, 90, E, dtype, masked=0.2)
    check(t, k, mask, renorm=E % 2 == 0)
    t, _ = make(E, 90, E, dtype, ties=True)
    check(t, k)


@pytest.mark.parametrize("T", [40, 700])
def test_operators_under_graph_capture(T):
    """Routing to combining and an adapter, captured once and replayed with
    eager work in between: the eager bits every time."""
    E, k, N, K, r, L = 24, 4, 136, 256, 16, 3
    g = torch.Generator(device=dev()).manual_seed(T)
    rand = lambda *s: torch.randn(*s, device=dev(), generator=g)  # noqa: E731
    logits, dw, dl = rand(T, E), rand(T, k), torch.ones(1, device=dev())
    y, base, d_out = rand(T * k, N).bfloat16(), rand(T, N).bfloat16(), rand(T, N).bfloat16()
    x, a, b = rand(T, K).bfloat16(), rand(L, r, K).bfloat16(), rand(L, N, r).bfloat16()
    ids = (torch.arange(T, device=dev()) % (L + 1) - 1).int()

    def step():
        route = fb.moe_route(logits, k, loss_coef=0.01)
        d_logits = fb.moe_route_backward(logits, route, dw, dl)
        groups = fb.group_rows(route.ids, E)
        out = fb.moe_combine(y, route.weights, groups.positions, base)
        d_y, d_w = fb.moe_combine_backward(d_out, y, route.weights, groups.positions, groups.offsets)
        z = fb.lora_add(base, x, a, b, ids)
        return [route.ids, route.weights, route.counts, route.loss, d_logits, groups.order,
                groups.offsets, out, d_y, d_w, z]

    want = [t.clone() for t in step()]
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        step()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=s):
            got = step()
    torch.cuda.synchronize()
    for _ in range(4):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for i, (t, w) in enumerate(zip(got, want)):
            assert torch.equal(t, w), i
        step()                               # eager work between replays
        torch.cuda.synchronize()


def test_operators_on_another_stream():
    """Issued on a side stream, the operators run there: their inputs come from
    work queued on that stream just before."""
    T, E, k = 20000, 64, 4
    s = torch.cuda.Stream()
    x = torch.randn(T, E, device=dev())
    want = fb.moe_route(x * 2, k, loss_coef=1.0)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        z = x
        for _ in range(20):
            z = z * 1.0
        got = fb.moe_route(z * 2, k, loss_coef=1.0)
        groups = fb.group_rows(got.ids, E)
    s.synchronize()
    assert torch.equal(got.ids, want.ids) and torch.equal(got.loss, want.loss)
    assert int(groups.offsets[E]) == T * k
