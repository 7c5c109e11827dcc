"""Infinities, NaN and the largest numbers in x: a row's result is what (q - z) x and fp32
sums give, however many rows share its batch."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_act_amd as fb
from gpu_helpers import dev, say
from oracle import gated as og
from oracle import w4 as ow
from test_gpu_w4 import make, n64, near, on

pytestmark = pytest.mark.gpu
DTYPES = {"bfloat16": torch.bfloat16, "float16": torch.float16}
ROWS = [1, 2, 3, 8, 17, 33, 48, 49, 130]     # single sequences, decode batches, tiles


def weights(seed, N, K, group, zeros, dtype):
    _, (codes, scale, z), _ = make(seed, N, K, group, zeros, dtype)
    q = ow.unpack(codes.numpy())
    zz = np.full(scale.shape, 8) if z is None else z.numpy()
    q[:, 40] = np.arange(N) % 16
    q[5, 40], q[11, 40] = zz[5, 40 // group], zz[11, 40 // group]     # q = z: 0 times an infinity
    return torch.from_numpy(ow.pack(q)), scale, z


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True)])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_w4_infinite_x(M, group, zeros, dtype):
    N, K = 38, 2432                          # (not a multiple of 2048)
    K = K // group * group
    t = weights(M, N, K, group, zeros, dtype)
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(M)).to(DTYPES[dtype])
    clean = fb.w4_linear(x.to(dev()), *on(t))
    bad = sorted({0, M // 2, M - 1})
    for i, r in enumerate(bad):
        x[r, 40] = (float("inf"), -float("inf"), float("nan"))[(i + M) % 3]
    say("w4 infinite", M, group, zeros, dtype)
    y = fb.w4_linear(x.to(dev()), *on(t))
    keep = [r for r in range(M) if r not in bad]
    assert torch.equal(y[keep], clean[keep])
    values = ow.values(t[0].numpy(), n64(t[1]), None if t[2] is None else t[2].numpy(), group)
    with np.errstate(invalid="ignore"):
        want = (n64(x)[bad][:, None, :] * values[None]).sum(2)
    assert np.isnan(want[:, [5, 11]]).all() and np.array_equal(n64(y)[bad], want, equal_nan=True)
    h = fb.w4_gated_linear(x.to(dev()), *on(t))
    i = N // 2
    with np.errstate(invalid="ignore", over="ignore"):
        g, u = want[:, :i], want[:, i:]
        wh = g / (1 + np.exp(-g)) * u        # (-inf / inf is NaN: SiLU's formula)
    assert torch.equal(h[keep], fb.w4_gated_linear(torch.where(x.isfinite(), x, 0).to(dev()), *on(t))[keep])
    assert np.array_equal(n64(h)[bad], wh, equal_nan=True)


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("zeros", [False, True])
def test_w4_largest_x(M, zeros):
    """2^124 once a group: 15 times it is finite in fp32, 16 times it is not."""
    N, K, group = 34, 256, 32
    _, (codes, scale, z), _ = make(M, N, K, group, zeros, "bfloat16")
    scale = (scale.float() * 2.0 ** -12).bfloat16()
    x = torch.zeros(M, K, dtype=torch.bfloat16)
    x[:, 7::group] = 2.0 ** 124 * torch.sign(torch.randn(M, K // group, generator=torch.Generator().manual_seed(1)))
    y = fb.w4_linear(x.to(dev()), *on((codes, scale, z)))
    want, tol = ow.product(n64(x), codes.numpy(), n64(scale), None if z is None else z.numpy(), group)
    near(y, want, tol, "bfloat16", "largest")
    assert np.abs(want).max() > 2.0 ** 100 and og.HALF["bfloat16"] == 2.0 ** -8


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("group,K", [(32, 96), (128, 14336)])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_w4_rows_of_every_kind_in_one_batch(M, group, K, dtype):
    """Finite rows, all NaN (as the unused rows of a padded batch), NaN beside an
    infinity, and infinities of both signs; x a slice with an odd stride."""
    N = 70
    t = weights(M, N, K, group, True, dtype)
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(M)).to(DTYPES[dtype])
    inf = float("inf")
    for r in range(M):
        kind = (r + M) % 5
        if kind == 1:
            x[r] = float("nan")
        elif kind == 2:
            x[r, 40], x[r, K - 1] = inf, float("nan")
        elif kind == 3:
            x[r, 3], x[r, K - 2] = inf, -inf
        elif kind == 4:
            x[r, K - 1] = -inf
    wide = torch.full((M, K + 3), float("nan"), dtype=x.dtype, device=dev())
    wide[:, :K] = x.to(dev())
    y = n64(fb.w4_linear(wide[:, :K], *on(t)))
    values = ow.values(t[0].numpy(), n64(t[1]), t[2].numpy(), group)
    for r in range(M):
        with np.errstate(invalid="ignore"):
            want = (n64(x)[r] * values).sum(1)
        if np.isfinite(want).all():
            want, tol = ow.product(n64(x)[r:r + 1], t[0].numpy(), n64(t[1]), t[2].numpy(), group)
            tol = tol + og.HALF[dtype] * (np.abs(want) + tol) + og.TINY[dtype]
            assert np.all(np.abs(y[r:r + 1] - want) <= tol), r
        else:
            assert np.array_equal(y[r], want, equal_nan=True), r
    h = n64(fb.w4_gated_linear(wide[:, :K], *on(t)))
    assert np.isnan(h[[(r + M) % 5 in (1, 2) for r in range(M)]]).all()
    assert np.isfinite(h[[(r + M) % 5 == 0 for r in range(M)]]).all()
