"""Adapters where only the first product's lower bits are left, on values that
every fp32 step holds exactly; so the result is the integers' one rounding to
bf16, bit for bit.

The first product is h = 2^22 + s with |s| < 2^10 (x and A are integers of at
most 8 bits, or 2^22), and a column of B takes one rank's h less another's: all
partial sums are integers below 2^24."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_act_amd as fb
from gpu_helpers import dev, say

pytestmark = pytest.mark.gpu


def make(seed, T, K, N, r, L):
    g = np.random.default_rng(seed)
    x = g.integers(-8, 9, (T, K)).astype(np.float32)
    a = np.zeros((L, r, K), np.float32)
    for l in range(L):
        for q in range(r):      # 100 terms of at most 8: |s| <= 800
            a[l, q, g.permutation(K - 1)[:100] + 1] = g.choice([-1, 1], 100)
    x[:, 0], a[:, :, 0] = 2.0 ** 22, 1
    b = np.zeros((L, N, r), np.float32)
    for l in range(L):
        for n in range(N):
            p, q = g.permutation(r)[:2]
            b[l, n, p], b[l, n, q] = 1, -1
    base = g.integers(-100, 101, (T, N)).astype(np.float32)
    return [torch.from_numpy(t).bfloat16() for t in (x, base, a, b)]


@pytest.mark.parametrize("T,L", [(1, 1), (16, 5), (64, 2), (65, 3), (300, 7), (4100, 2)])
@pytest.mark.parametrize("K,r", [(128, 8), (256, 16), (640, 24), (1536, 32), (384, 72), (256, 136),
                                 (256, 256)])
def test_first_product_keeps_its_bits(T, L, K, r):
    say("lora exact", T, L, K, r)
    N = 70
    x, base, a, b = make(T + r, T, K, N, r, L)
    ids = (np.arange(T) % (L + 1) - 1).astype(np.int32) if L > 1 else np.zeros(T, np.int32)
    scale = torch.tensor([0.5, 2.0, 1.0, 4.0, 0.25, 1.0, 2.0][:L])
    got = fb.lora_add(base.to(dev()), x.to(dev()), a.to(dev()), b.to(dev()),
                      torch.from_numpy(ids).to(dev()), scale.to(dev()))
    want = base.double()
    for g in range(L):
        rows = torch.from_numpy(np.flatnonzero(ids == g))
        h = x[rows].double() @ a[g].double().t()
        want[rows] += scale[g].double() * (h @ b[g].double().t())
    assert torch.equal(got.cpu(), want.float().bfloat16())
