"""Combine and its gradients over more tokens than one launch takes (a grid
holds fewer than 2^32 threads): the same sums for the last tokens as for the
first."""
import pytest
import torch

import block_scaled_fp8_act_amd as fb
from gpu_helpers import dev, say

pytestmark = pytest.mark.gpu


def test_combine_past_one_grid():
    T = (1 << 26) + 5
    say("combine", T)
    y = torch.tensor([[1.0], [2.0], [4.0]], dtype=torch.bfloat16, device=dev())
    pos = torch.remainder(torch.arange(T, dtype=torch.int32, device=dev()), 4)[:, None].sub_(1)
    w = torch.full((T, 1), 3.0, device=dev())
    out = fb.moe_combine(y, w, pos)
    want = torch.tensor([0.0, 3.0, 6.0, 12.0], dtype=torch.bfloat16, device=dev())
    assert torch.equal(out[:, 0].view(-1)[:T - 1].view(-1, 4), want.expand((T - 1) // 4, 4))
    assert float(out[T - 1, 0]) == float(want[(T - 1) % 4])


def test_combine_backward_past_one_grid():
    T, N = (1 << 24) + 5, 3
    say("combine backward", T)
    R = T + 2
    y = torch.ones(R, N, dtype=torch.bfloat16, device=dev())
    pos = torch.arange(T - 1, -1, -1, dtype=torch.int32, device=dev())[:, None]
    w = (torch.remainder(torch.arange(T, device=dev()), 8) + 1).float()[:, None]
    d = torch.full((T, N), 0.5, dtype=torch.bfloat16, device=dev())
    used = torch.tensor([T], dtype=torch.int32, device=dev())
    dy, dw = fb.moe_combine_backward(d, y, w, pos, used)
    assert bool((dw == 1.5).all())
    assert torch.equal(dy[:T], (w.flip(0) * 0.5).bfloat16().expand(T, N))
    assert not dy[T:].any()
