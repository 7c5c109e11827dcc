"""The range of dgu, which the gradients round to the type of x: past fp16's largest
number an infinity that shows, below half its smallest one zero; none of it in bf16."""
import pytest
import torch

import block_scaled_fp8_act_amd as fb
from gpu_helpers import dev

pytestmark = pytest.mark.gpu


def block(M, dtype):
    """I = 3, K = 8: g = 8 in every row and u = 4, 2^-5 and 1, so that dgu of the up
    rows is 8 d_h (SiLU of 8 is 8 less 0.003) and of the gates' 4, 2^-5 and 1 times
    d_h (SiLU's slope there is 1.002)."""
    x = torch.zeros(M, 8, dtype=dtype, device=dev())
    x[:, 0], x[:, 1] = 1.0, 0.5
    w = torch.zeros(6, 8, dtype=dtype, device=dev())
    w[:3, 0] = 8.0
    w[3:, 1] = torch.tensor([8.0, 2.0 ** -4, 2.0])
    return x, w


@pytest.mark.parametrize("saved", [False, True])
@pytest.mark.parametrize("M", [1, 4, 70])
def test_fp16_gradients_past_the_largest_number(M, saved):
    x, w = block(M, torch.float16)
    d = torch.ones(M, 3, dtype=torch.float16, device=dev())
    kept = fb.gated_linear(x, w, save=True)[1] if saved else None
    clean = fb.gated_linear_backward(d, x, w, kept)
    d[0, 1] = 30000.0                  # 8 times it is past 65504, 2^-5 times it is not
    dx, dw = fb.gated_linear_backward(d, x, w, kept)
    assert not bool(dx[0, :2].isfinite().any()) and torch.equal(dx[1:], clean[0][1:])
    assert not bool(dw[4, :2].isfinite().any()) and bool(dw[[0, 1, 2, 3, 5]].isfinite().all())
    xb, wb = block(M, torch.bfloat16)
    kb = fb.gated_linear(xb, wb, save=True)[1] if saved else None
    bx, bw = fb.gated_linear_backward(d.bfloat16(), xb, wb, kb)
    assert bool(bx.isfinite().all()) and bool(bw.isfinite().all())
    assert abs(float(bw[4, 0]) / (8 * 30000 + 8 * (M - 1)) - 1) < 2.0 ** -6


@pytest.mark.parametrize("saved", [False, True])
@pytest.mark.parametrize("M", [1, 4, 70])
def test_fp16_gradients_below_the_smallest_number(M, saved):
    x, w = block(M, torch.float16)
    kept = fb.gated_linear(x, w, save=True)[1] if saved else None
    d = torch.full((M, 3), 2.0 ** -21, dtype=torch.float16, device=dev())
    dw = fb.gated_linear_backward(d, x, w, kept)[1]
    # of the gates' rows 2^-19, 2^-26 (below half of 2^-24: zero) and 2^-21 a row of x
    assert float(dw[1].abs().max()) == 0.0
    for n, one in ((0, 2.0 ** -19), (2, 2.0 ** -21), (4, 2.0 ** -18)):
        # dgu within half of 2^-24, the sum within half a step
        assert abs(float(dw[n, 0]) - M * one) <= M * (2.0 ** -25 + 0.01 * one) + 2.0 ** -25
