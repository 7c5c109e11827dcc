"""moe_experts against its own parts: bit for bit the weighted return of the
grouped products on the quantized rows, and within one rounding of the binary64
sum of those products' rows.

Tolerance: k + 1 fp32 terms, (k + 1) 2^-24 of their magnitudes, and one rounding
to bf16, 2^-8 of the result.  The products' rows are the experts' own: a row of
the grouped product is the same row of the expert's product, whose accumulation
order may differ, so both within 2^-8 of an element and 2^-13 of the magnitudes
of its products (the products' tolerance), on the same codes."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_act_amd as fb
from gpu_helpers import dev, say
from oracle import routing as orr

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["float", "ue8m0"])
@pytest.mark.parametrize("T,E,k", [(1, 6, 3), (16, 6, 3), (150, 6, 3), (40, 32, 8), (300, 5, 1)])
@pytest.mark.parametrize("with_base", [False, True])
def test_moe_experts_is_its_parts(T, E, k, fmt, with_base):
    say("experts", T, E, k, fmt, with_base)
    K, I, N = 256, 128, 320
    r = np.random.default_rng(T + E)
    bf = lambda *s: torch.from_numpy(r.standard_normal(s).astype(np.float32)).bfloat16().to(dev())  # noqa: E731
    x, base = bf(T, K), bf(T, N) if with_base else None
    stack = lambda ws: tuple(torch.stack(t) for t in zip(*ws))  # noqa: E731
    up = stack([fb.weight_block_quant(bf(2 * I, K) * 0.05, fmt) for _ in range(E)])
    down = stack([fb.weight_block_quant(bf(N, I) * 0.05, fmt) for _ in range(E)])
    mask = torch.from_numpy(r.random(T) < 0.8).to(dev())
    routing = fb.moe_route(bf(T, E), k, mask=mask)
    got = fb.moe_experts(x, routing, *up, *down, base)

    groups = fb.group_rows(routing.ids, E)
    used = int(groups.offsets[E])
    rows = x[(groups.order // k).long()]
    h = fb.grouped_block_gemm(*fb.act_quant_group(rows, fmt), *up, groups.offsets)
    h_q, h_s = fb.swiglu_act_quant(h, fmt)
    y = fb.grouped_block_gemm(h_q, h_s, *down, groups.offsets)
    assert torch.equal(got, fb.moe_combine(y, routing.weights, groups.positions, base))

    pos = groups.positions.cpu().numpy()
    assert np.array_equal(pos >= 0, routing.ids.cpu().numpy() >= 0)
    y64 = torch.where(torch.arange(len(y), device=dev())[:, None] < used, y.double(), 0.0).cpu().numpy()
    want, mag = orr.combine(y64, routing.weights.double().cpu().numpy(), pos,
                            None if base is None else base.double().cpu().numpy())
    off = np.abs(got.double().cpu().numpy() - want)
    assert np.all(off <= mag * (k + 1) * 2.0 ** -24 + np.abs(want) * 2.0 ** -8 * 1.0001)

    # each row of y: the slot's expert's product of the slot's quantized row
    q = lambda t: t.view(torch.float8_e4m3fn).double()  # noqa: E731
    scale = lambda s: s.double() if fmt == "float" else torch.exp2(s.double() - 127.0)  # noqa: E731
    a = q(h_q) * scale(h_s).repeat_interleave(128, 1)
    at = groups.order[:used].cpu().numpy()
    expert = routing.ids.cpu().numpy().reshape(-1)[at]
    assert np.array_equal(expert, np.sort(expert))
    for e in range(E):
        mine = torch.from_numpy(np.flatnonzero(expert == e)).to(dev())
        w = q(down[0][e]) * scale(down[1][e]).repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)
        full = a[mine] @ w.t().contiguous()
        spread = a[mine].abs() @ w.abs().t().contiguous()
        assert bool(((y[mine].double() - full).abs() <= 2.0 ** -8 * full.abs() + 2.0 ** -13 * spread).all())
