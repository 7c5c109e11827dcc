"""The routing softmax far below a row's largest logit.

The logits are multiples of 1/16, so their differences x = l - max are exact in
fp32 and what is left is the exponential's own error, which does not grow with
|x| beyond 0.05 |x| u (u = 2^-24, the constant's rounding): 2 u of the hardware's
exponential, 1 u of its correction, and 5 u at |x| = 86.  The largest term is 1
and the others are below 2^-80, so their sum and its reciprocal are 1 exactly,
and the product with it is exact too: 8 u of a weight."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_act_amd as fb
from gpu_helpers import dev, say

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("E", [8, 32, 60, 128, 250, 256, 300, 1024])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [True, False])
def test_weights_far_below_the_peak(E, dtype, renorm):
    say("route far", E, dtype, renorm)
    T, k = 600, 8
    g = np.random.default_rng(E)
    x = torch.full((T, E), -float("inf"), dtype=torch.float64)
    for t in range(T):
        at = torch.from_numpy(g.permutation(E)[:k].copy())
        x[t, at] = -torch.from_numpy(g.permutation(np.arange(56 * 16, 86 * 16))[:k].copy() / 16.0)
        x[t, at[0]] = 0.0
    if dtype == torch.bfloat16:      # 8 bits: steps of 1/2 at these sizes
        x = torch.where(torch.isfinite(x), torch.round(x * 2) / 2, x)
    r = fb.moe_route(x.to(dtype).to(dev()), k, renormalize=renorm)
    ids, w = r.ids.cpu().long(), r.weights.double().cpu()
    assert bool((ids >= 0).all())
    want = torch.exp(torch.gather(x, 1, ids))
    off = ((w - want).abs() / want).max()
    assert bool(((w - want).abs() <= 8 * U * want).all()), float(off / U)


@pytest.mark.parametrize("E", [8, 60, 256, 1024])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_weights_at_the_ends(E, dtype):
    """Terms too small for fp32, the type's lowest value and -inf weigh 0; a NaN
    logit shows in the loss."""
    low = torch.finfo(dtype).min
    x = torch.tensor([0.0, -1.0, -150.0, -1e4, -1e30, 0.6 * low, low, -float("inf")]).to(dtype)
    x = torch.cat([x, torch.full((E - 8,), -float("inf"), dtype=dtype)])
    for top in (0.0, -3.0, 1e30, -0.9 * low):
        t = x.clone()
        t[0] = top
        p = torch.softmax(t.double(), 0)
        r = fb.moe_route(t.expand(70, E).contiguous().to(dev()), 7, renormalize=False, loss_coef=1.0)
        w = torch.zeros(70, E, dtype=torch.float64).scatter_(1, r.ids.cpu().long().clamp(min=0),
                                                             r.weights.cpu().double())
        assert bool(((w - p).abs() <= 40 * U * p + 2.0 ** -126).all())
        assert bool(torch.isfinite(r.loss))
        d = fb.moe_route_backward(t.expand(70, E).contiguous().to(dev()), r, torch.ones(70, 7, device=dev()),
                                  torch.ones(1, device=dev()))
        assert bool(torch.isfinite(d).all())
    t = x.expand(70, E).clone()
    t[7, 1] = float("nan")
    assert bool(torch.isnan(fb.moe_route(t.to(dev()), 2, loss_coef=1.0).loss))
