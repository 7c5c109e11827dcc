"""Gated projections and 4-bit weights where byte offsets pass 32 bits: each of x,
the outputs, the saved factors, codes and weights is larger than 4 GiB in one case."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_act_amd as fb
from gpu_helpers import dev, say
from oracle import gated as og
from oracle import w4 as ow
from test_gpu_gated import factors_of, near
from test_gpu_gated import make as make_gated
from test_gpu_gated import n64
from test_gpu_w4 import make, on, product
from test_gpu_w4 import near as near_w4

pytestmark = pytest.mark.gpu
ROWS = 1_050_003


def spread(t):
    """t's rows as the first 3 and the last ones of ROWS, the others zero."""
    big = torch.zeros((ROWS, t.shape[1]), dtype=t.dtype, device=dev())
    big[:3], big[3 - len(t):] = t[:3].to(dev()), t[3:].to(dev())
    return big


def picked(t, n):
    """Those rows; the others are zero (checked)."""
    assert not bool(t[3:3 - n].any())
    return torch.cat([t[:3], t[3 - n:]])


@pytest.mark.parametrize("I,K", [(40, 2056), (1100, 24)])
def test_gated_rows_past_32_bits(I, K):
    """Rows of zeros have zero outputs, factors and gradients, and add nothing to d_W."""
    n = 73
    say("gated large", I, K)
    x, w, d = make_gated(I, n, I, K, "bfloat16")
    xd, wd, dd = spread(x), w.to(dev()), spread(d)
    h, saved = fb.gated_linear(xd, wd, save=True)
    near(picked(h, n), *og.forward(n64(x), n64(w), "silu", "bfloat16"), "h")
    f, e = og.factors(n64(x), n64(w), "silu")
    near(factors_of(picked(saved, n), I), f, e + og.KEPT * (np.abs(f) + e), "factors")
    for kept in (saved, None):
        dx, dw = fb.gated_linear_backward(dd, xd, wd, kept)
        vx, tx, vw, tw = og.backward(n64(d), n64(x), n64(w), "silu", "bfloat16", kept is not None)
        near(picked(dx, n), vx, tx, "d_x")
        near(dw, vw, tw, "d_w")


def test_w4_x_past_32_bits():
    n, N, K = 50, 72, 2048
    _, t, _ = make(1, N, K, 32, True, "bfloat16")
    x = torch.randn(n, K, generator=torch.Generator().manual_seed(2)).bfloat16()
    want, tol = product(x, t)
    say("w4 large x")
    near_w4(picked(fb.w4_linear(spread(x), *on(t)), n), want, tol, "bfloat16", "y")


@pytest.mark.parametrize("group", [32, 128])
def test_w4_weights_past_32_bits(group):
    N, K, D = 1_100_002, 8192, dev()
    g = torch.Generator(device=D).manual_seed(group)
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=D, generator=g)
    scale = (0.01 + torch.rand((N, K // group), device=D, generator=g)).bfloat16()
    zeros = torch.randint(0, 16, scale.shape, dtype=torch.uint8, device=D, generator=g)
    rows = torch.cat([torch.arange(5), torch.arange(N // 2 - 3, N // 2 + 3), torch.arange(N - 140, N)])
    part = tuple(t[rows.to(D)].cpu() for t in (codes, scale, zeros))
    say("w4 large", group)
    w = fb.w4_dequant(codes, scale, zeros)
    values = ow.values(part[0].numpy(), n64(part[1]), part[2].numpy(), group)
    assert torch.equal(w[rows.to(D)].cpu(), torch.from_numpy(values).bfloat16())
    back = fb.w4_quant(w, group, True)
    q, s, z = ow.quant(n64(w[rows.to(D)]), group, True, "bfloat16")
    assert torch.equal(back.codes[rows.to(D)].cpu(), torch.from_numpy(ow.pack(q)))
    assert torch.equal(back.scale[rows.to(D)].cpu(), torch.from_numpy(s).bfloat16())
    assert torch.equal(back.zeros[rows.to(D)].cpu(), torch.from_numpy(z))
    del w, back
    for M in (1, 20, 60):
        x = torch.randn(M, K, generator=torch.Generator().manual_seed(M)).bfloat16()
        say("w4 large", group, M)
        y = fb.w4_linear(x.to(D), codes, scale, zeros)
        want, tol = product(x, part)
        near_w4(y[:, rows.to(D)], want, tol, "bfloat16", "y")
        I = N // 2
        outs = torch.cat([torch.arange(5), torch.arange(I - 60, I)])
        gates, ups = (tuple(t[i.to(D)].cpu() for t in (codes, scale, zeros)) for i in (outs, outs + I))
        (gv, ge), (uv, ue) = product(x, gates), product(x, ups)
        a, _ = og.act(gv, "silu")
        want = a * uv
        tol = og.SLOPE * ge * np.abs(uv) + (np.abs(a) + og.SLOPE * ge) * ue + og.EVAL * np.abs(want)
        near_w4(fb.w4_gated_linear(x.to(D), codes, scale, zeros)[:, outs.to(D)], want, tol, "bfloat16", "h")
