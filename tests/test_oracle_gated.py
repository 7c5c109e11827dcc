"""The gated projections' oracle against torch's binary64 autograd, on the CPU."""
import numpy as np
import pytest
import torch

from oracle import gated as og


@pytest.mark.parametrize("name,form", [("silu", None), ("gelu", "none"), ("gelu_tanh", "tanh")])
def test_oracle_gated(name, form):
    g = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, w, d = rnd(9, 7).requires_grad_(), (2 * rnd(12, 7)).requires_grad_(), rnd(9, 6)
    gate, u = (x @ w.t()).chunk(2, 1)
    a = torch.nn.functional.silu(gate) if form is None else torch.nn.functional.gelu(gate, approximate=form)
    gx, gw = torch.autograd.grad(a * u, (x, w), d)
    xn, wn = x.detach().numpy(), w.detach().numpy()
    h, _ = og.forward(xn, wn, name, "float16")
    vx, _, vw, _ = og.backward(d.numpy(), xn, wn, name, "float16", True)
    for got, want in ((h, (a * u).detach()), (vx, gx), (vw, gw)):
        assert np.abs(got - want.numpy()).max() < 1e-12
