"""The example runs, its output does not depend on the batch a token is served
in beyond the quantized products' rounding, and the balance loss falls."""
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def test_moe_layer_example(capsys):
    import moe_layer
    before, after = moe_layer.main(["--tokens", "150", "--requests", "9"])
    assert after < before
    assert "served 150 tokens" in capsys.readouterr().out


def test_masked_tokens_keep_the_shared_expert():
    import moe_layer
    layer = moe_layer.Layer()
    x = torch.randn(70, moe_layer.HIDDEN, device="cuda").bfloat16()
    none = torch.full((70,), -1, dtype=torch.int32, device="cuda")
    mask = torch.arange(70, device="cuda") % 3 > 0
    y, routing, _ = layer.forward(x, none, mask=mask)
    z, _, _ = layer.forward(x, none, mask=torch.zeros_like(mask))
    assert torch.equal(y[~mask], z[~mask])
    assert bool((routing.ids[~mask] == -1).all()) and not torch.equal(y[mask], z[mask])
