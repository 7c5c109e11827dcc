"""The feed-forward example runs, and its block's gradients are those of the formulas."""
import os
import sys

import pytest
import torch

from oracle import gated as og

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_ffn_example(act, capsys):
    import ffn_layer
    ffn_layer.main(["--tokens", "70", "--act", act])
    assert "served 70 tokens in 4 bits" in capsys.readouterr().out


@pytest.mark.parametrize("need_x", [False, True])
def test_ffn_gradients(need_x):
    """Through the autograd function, with the loss's gradient of h given: an expanded
    one, as a sum's is."""
    import ffn_layer
    block = ffn_layer.Block()
    n = lambda t: t.detach().cpu().double().numpy()  # noqa: E731
    x = torch.randn(40, ffn_layer.HIDDEN, device="cuda").bfloat16().requires_grad_(need_x)
    h = ffn_layer.GatedLinear.apply(x, block.up, block.act)
    d = torch.randn(1, ffn_layer.INTER, device="cuda").bfloat16().expand(40, -1)
    h.backward(d)
    vx, tx, vw, tw = og.backward(n(d), n(x), n(block.up), "silu", "bfloat16", True)
    assert (abs(n(block.up.grad) - vw) <= tw).all()
    assert (x.grad is not None) == need_x and (not need_x or (abs(n(x.grad) - vx) <= tx).all())
