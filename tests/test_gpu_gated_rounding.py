"""What separates the gradients from fp32's: one rounding of dgu to 16 bits, and their
own.  Against the formula with dgu rounded so, only their own is left."""
import pytest
import torch

import block_scaled_fp8_act_amd as fb
import large_tiles as lt
from gpu_helpers import dev, say

pytestmark = pytest.mark.gpu


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("M,I,K", [(2048, 1408, 1024), (1003, 2051, 776), (60, 700, 264)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("saved", [False, True])
@pytest.mark.parametrize("act", list(fb.ACTS))
def test_gradients_round_dgu_once(M, I, K, dtype, saved, act):
    """An error of one rounding is e, of two independent ones 1.41 e.  A factor kept in
    24 bits is off by up to 2^-16 of itself, 2^-17 on average, and moves dgu over a border
    of its rounding, fp16's step being 2^-11 of it or more, in at most 2^-6 of all cases;
    that costs a whole step, whose square is 12 e^2.  So e^2 grows by 12 2^-6 = 0.19 at
    most: 1.09 e in place of e, 1.48 e in place of 1.41 e; fp32 sums add far less."""
    g = torch.Generator(device=dev()).manual_seed(M)
    rnd = lambda *s: torch.randn(*s, device=dev(), generator=g)  # noqa: E731
    x, w, d = (t.to(dtype) for t in (rnd(M, K), rnd(2 * I, K) * K ** -0.5, rnd(M, I)))
    kept = fb.gated_linear(x, w, act, save=True)[1] if saved else None
    got = fb.gated_linear_backward(d, x, w, kept, act)
    x, w, d = x.double(), w.double(), d.double()
    gate, up, _, _ = lt.project(x, w)
    a, slope = lt.act(gate, act)
    dgu = torch.cat([d * up * slope, d * a], 1)
    once = dgu.to(dtype).double()
    for have, p, r, q, name in ((got[0], dgu, once, w, "d_x"), (got[1], dgu.t(), once.t(), x, "d_w")):
        exact, formula = p @ q, r @ q
        one = rel(formula.to(dtype), formula)
        say(name, "own rounding", one, "from the formula", rel(have, formula), "from binary64", rel(have, exact))
        assert rel(have, formula) <= 1.1 * one and rel(have, exact) <= 1.5 * one
