"""Infinite and NaN entries of B: the result is what fp32 products and sums of
the same values give, an infinity where the terms leave one and NaN where they
do not."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_act_amd as fb
from gpu_helpers import dev, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [4, 100, 4100])
@pytest.mark.parametrize("r", [8, 16, 24, 40, 64, 72, 136, 200])
def test_infinite_entries_of_b(T, r):
    say("lora infinite", T, r)
    K, N = 128, 40
    g = np.random.default_rng(r)
    x = torch.from_numpy(g.integers(1, 4, (T, K)).astype(np.float32))
    a = torch.from_numpy((g.integers(0, 10, (1, r, K)) == 0).astype(np.float32))
    a[0, :, 0] = 1                                  # h > 0, few bits: exact in bf16
    a[0, 1] *= 1.0 + 2.0 ** -7                      # one rank whose h takes more than bf16 holds
    a[0, 2] = 0                                     # and one whose h is zero
    b = torch.from_numpy(g.integers(-2, 3, (1, N, r)).astype(np.float32))
    inf = float("inf")
    b[0, 3, 0] = inf
    b[0, 4, r - 1] = -inf
    b[0, 5, 1] = inf
    b[0, 6, [0, r - 1]] = inf
    b[0, 7, 0], b[0, 7, r - 1] = inf, -inf          # NaN
    b[0, 8, 2] = inf                                # 0 times infinity: NaN
    b[0, 9, r - 1] = float("nan")
    x, a, b = (t.bfloat16() for t in (x, a, b))
    base = torch.ones(T, N).bfloat16()
    ids = torch.zeros(T, dtype=torch.int32)
    got = fb.lora_add(base.to(dev()), x.to(dev()), a.to(dev()), b.to(dev()), ids.to(dev())).cpu().float()
    h = x.double() @ a[0].double().t()
    terms = h[:, None, :] * b[0].double()[None, :, :]
    want = base.double() + terms.sum(2)
    assert bool(torch.isfinite(want[:, 10:]).all()) and bool((want[:, 3] == inf).all())
    bad = ~torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[bad & ~torch.isnan(want)].double(), want[bad & ~torch.isnan(want)])
    assert bool(torch.isfinite(got[~bad]).all())
    # an infinite h (of one row): infinite against positive entries, NaN against a
    # zero and against entries of both signs
    x[1, 0] = inf
    a[0, 2] = a[0, 0]
    b = torch.from_numpy(g.integers(1, 3, (1, N, r)).astype(np.float32)).bfloat16()
    b[0, 3, 4], b[0, 4, r - 1] = 0, -1
    got = fb.lora_add(base.to(dev()), x.to(dev()), a.to(dev()), b.to(dev()), ids.to(dev())).cpu().float()
    nan = torch.zeros(N, dtype=torch.bool)
    nan[3:5] = True
    assert torch.equal(torch.isnan(got[1]), nan) and bool((got[1][~nan] == inf).all())
    assert bool(torch.isfinite(got[torch.arange(T) != 1]).all())
