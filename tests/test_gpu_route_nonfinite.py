"""A gradient of the loss that is infinite or NaN (an overflowed loss scale)
reaches the routed rows alone: rows that were not routed get 0."""
import pytest
import torch

import block_scaled_fp8_act_amd as fb
from gpu_helpers import dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E", [8, 60, 256, 250, 512])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d_loss", [float("inf"), float("nan")])
@pytest.mark.parametrize("renorm", [True, False])
def test_rows_not_routed_get_zero(E, dtype, d_loss, renorm):
    T, k = 90, 3
    x = torch.randn(T, E, generator=torch.Generator().manual_seed(E)).to(dtype)
    mask = torch.arange(T) % 4 > 0
    x[~mask] = float("nan")
    x[5] = -float("inf")
    live = mask.clone()
    live[5] = False
    r = fb.moe_route(x.to(dev()), k, mask=mask.to(dev()), renormalize=renorm, loss_coef=0.1)
    d = fb.moe_route_backward(x.to(dev()), r, torch.ones(T, k, device=dev()),
                              torch.tensor(d_loss, device=dev())).cpu().float()
    assert not d[~live].any()
    assert not bool(torch.isfinite(d[live]).all())
