"""Adapters beside large batches (64- and 128-row tiles, every rank's kernels) and
in matrices whose offsets pass 32 bits.  Tolerance as in test_gpu_lora."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_act_amd as fb
from gpu_helpers import dev, say
from test_gpu_lora import check, make, on

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("r", [8, 16, 24, 32, 40, 64, 72, 128, 136, 256])
@pytest.mark.parametrize("T,L", [(1100, 3), (4096, 3), (4200, 40)])
def test_lora_large_batch(T, L, r):
    say("lora large", T, L, r)
    K, N = 384, 206
    x, base, a, b, scale = make(T + r, T, K, N, r, L)
    g = np.random.default_rng(r)
    ids = np.repeat(g.integers(-1, L, T), g.integers(1, 60, T))[:T].astype(np.int32)
    got = fb.lora_add(on(base), on(x), on(a), on(b), torch.from_numpy(ids).to(dev()), on(scale))
    check(got, base, x, a, b, ids, scale)


@pytest.mark.parametrize("T", [3, 300, 4300])
def test_lora_rows_past_2_31_elements(T):
    """x, base and out are columns of matrices of T x ld with T * ld > 2^31."""
    K, N, r, L = 128, 70, 16, 2
    ld = (1 << 31) // (T - 1) + 256
    x, base, a, b, scale = make(T, T, K, N, r, L)
    ids = (np.arange(T) % (L + 1)).astype(np.int32)
    wide = torch.empty((T, ld), dtype=torch.bfloat16, device=dev())
    wide[:, :K] = on(x)
    wide[:, K:K + N] = on(base)
    y = wide[:, K:K + N]
    fb.lora_add(y, wide[:, :K], on(a), on(b), torch.from_numpy(ids).to(dev()), on(scale), out=y)
    check(y, base, x, a, b, ids, scale)
    assert torch.equal(wide[:, :K].cpu(), x)


@pytest.mark.parametrize("T", [2, 100])
def test_lora_adapters_past_2_31_elements(T):
    """The last of 40 adapters starts past 2^31 elements of B (and, at K =
    262144, of A)."""
    K, N, r, L = 262144, 262144, 256, 40
    a = torch.zeros((L, r, K), dtype=torch.bfloat16, device=dev())
    b = torch.zeros((L, N, r), dtype=torch.bfloat16, device=dev())
    a[L - 1, 5, K - 9] = 2.0
    b[L - 1, N - 3, 5] = 3.0
    x = torch.zeros((T, K), dtype=torch.bfloat16, device=dev())
    x[:, K - 9] = torch.arange(1, T + 1, device=dev()).bfloat16()
    ids = torch.full((T,), L - 1, dtype=torch.int32, device=dev())
    y = fb.lora_add(None, x, a, b, ids)
    want = (6.0 * x[:, K - 9].float()).bfloat16()
    assert torch.equal(y[:, N - 3], want)
    y[:, N - 3] = 0
    assert not y.any()


def test_lora_groups_serve_every_projection_of_a_batch():
    """One listing for projections of several widths; and a listing of other
    rows' order gives the same bits (the order within an adapter is its own)."""
    T, L = 700, 5
    ids = torch.from_numpy((np.arange(T) // 90 % (L + 1) - 1).astype(np.int32)).to(dev())
    groups = fb.group_rows(ids, L)
    for K, N, r in ((256, 96, 16), (512, 300, 64)):
        x, base, a, b, scale = make(K, T, K, N, r, L)
        args = (on(base), on(x), on(a), on(b), ids, on(scale))
        assert torch.equal(fb.lora_add(*args, groups=groups), fb.lora_add(*args))
