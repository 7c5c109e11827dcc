"""The activations' own precision: with g and u whole products of one term each, the
saved factors show act'(g) u and act(g) to their 24 bits."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_act_amd as fb
from gpu_helpers import dev, say
from large_tiles import act as act64
from test_gpu_gated import factors_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", list(fb.ACTS))
@pytest.mark.parametrize("M", [2, 100, 5000])
def test_activation_precision(act, M):
    """Gates from -13 to 7 (1, 0.75 and -0.5 times x; those of up to two rows go by a
    kernel of their own).  Half a step of 24 bits with 8 of exponent is 2^-16 of a value
    (one bit of sign, 8 of exponent, 15 kept of the significand beside its leading
    one); beside it act is held to 2^-20, and act', a sum of two terms of opposite sign,
    to 2^-20 of their magnitudes.  A logistic below fp32's normal numbers, 2^-126, counts
    as zero: its part of act and act' is at most 1 + |z'| times as much, 1 + 12 1.6 (1 +
    0.134 12^2) < 512 in the form by tanh, less in the others."""
    g = np.linspace(-13.0, 7.0, 5000)
    for first in ([0] if M == 5000 else range(0, 5000 - M, 437)):
        x = torch.ones(M, 2, dtype=torch.float16)
        x[:, 0] = torch.from_numpy(g[first:first + M])
        w = torch.tensor([[1.0, 0], [0.75, 0], [-0.5, 0], [0, 1], [0, 1], [0, 1]]).half()
        _, saved = fb.gated_linear(x.to(dev()), w.to(dev()), act, save=True)
        got = factors_of(saved, 3).double().numpy()
        v = x[:, :1].double().numpy() * np.array([[1.0, 0.75, -0.5]])
        a, slope = (t.numpy() for t in act64(torch.from_numpy(v), act))
        # the larger of the slope's two terms, the other the difference
        step = a / np.where(v == 0, 1, v)
        step[v == 0] = 0.5
        for name, have, want, size in (("act", got[:, 3:], a, np.abs(a)),
                                       ("act'", got[:, :3], slope, np.abs(step) + np.abs(slope - step))):
            off = np.abs(have - want) / (2.0 ** -16 * np.abs(want) + 2.0 ** -20 * size + 512 * 2.0 ** -126)
            say(act, M, first, name, "of the tolerance:", float(off.max()))
            assert off.max() <= 1.0, (act, name, v.flat[off.argmax()], float(off.max()))
