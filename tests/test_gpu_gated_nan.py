"""NaN gates of the gated projections stay visible in everything that they enter."""
import pytest
import torch

import block_scaled_fp8_act_amd as fb
from gpu_helpers import dev
from test_gpu_gated import factors_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", list(fb.ACTS))
@pytest.mark.parametrize("M", [1, 2, 9, 300])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_nan_gates(act, M, dtype):
    """A NaN gate makes h, both factors, dgu and with it the row of d_x NaN, and the
    gates' and ups' rows of d_w, but nothing of other rows and outputs."""
    I, K, nan = 5, 16, float("nan")
    g = torch.Generator().manual_seed(M)
    x, w, d = (torch.randn(*s, generator=g).to(dtype).to(dev()) for s in ((M, K), (2 * I, K), (M, I)))
    x[:, 3] = 1.0
    w[:, 3] = 0.0
    clean = fb.gated_linear(x, w, act)
    w[2, 3] = nan                       # the gate of output 2, in every row
    keep = [i for i in range(I) if i != 2]
    h, saved = fb.gated_linear(x, w, act, save=True)
    f = factors_of(saved, I)
    assert bool(h[:, 2].isnan().all()) and torch.equal(h[:, keep], clean[:, keep])
    assert bool(f[:, [2, 2 + I]].isnan().all()) and not bool(f[:, keep].isnan().any())
    rows, without = keep + [i + I for i in keep], torch.where(w.isnan(), 0, w)
    saved_without = fb.gated_linear(x, without, act, save=True)[1]
    for kept, other in ((saved, saved_without), (None, None)):
        dx, dw = fb.gated_linear_backward(d, x, w, kept, act)
        assert bool(dx.isnan().all()) and bool(dw[[2, 2 + I]].isnan().all())
        assert torch.equal(dw[rows], fb.gated_linear_backward(d, x, without, other, act)[1][rows])
