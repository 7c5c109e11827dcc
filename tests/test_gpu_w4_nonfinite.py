"""NaN and infinite weights stay visible through the 4-bit quantizer: the scale of
their group is NaN or infinite, in both forms, and the other groups are as without."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_act_amd as fb
from gpu_helpers import dev, say
from oracle import w4 as ow

pytestmark = pytest.mark.gpu
DTYPES = {"bfloat16": torch.bfloat16, "float16": torch.float16}
INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("bad", [[NAN], [-NAN], [INF], [-INF], [INF, -INF], [NAN, INF], [-INF, NAN]])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_w4_quant_nonfinite(bad, group, zeros, dtype):
    N, K = 9, 512
    w = torch.randn(N, K, generator=torch.Generator().manual_seed(group)).to(DTYPES[dtype])
    clean = fb.w4_quant(w.to(dev()), group, zeros)
    for row in range(1, N):                  # of row r, group r of however many there are
        first = row % (K // group) * group
        for i, v in enumerate(bad):
            w[row, first + (7 * row + 13 * i) % group] = v
    say("w4 non-finite", bad, group, zeros, dtype)
    got = fb.w4_quant(w.to(dev()), group, zeros)
    hit = torch.zeros(N, K // group, dtype=torch.bool, device=dev())
    rows = torch.arange(1, N, device=dev())
    hit[rows, rows % (K // group)] = True
    s = got.scale[hit]
    assert bool((s.isnan() if any(np.isnan(bad)) else s == INF).all())
    assert torch.equal(got.scale[~hit], clean.scale[~hit])
    codes, before = (t.codes.view(N, K // group, group // 2) for t in (got, clean))
    assert torch.equal(codes[~hit], before[~hit]) and bool((codes[hit] == (0 if zeros else 0x88)).all())
    if zeros:
        assert torch.equal(got.zeros[~hit], clean.zeros[~hit]) and not bool(got.zeros[hit].any())
    q, want, z = ow.quant(w.double().numpy(), group, zeros, dtype)
    assert np.array_equal(got.scale.double().cpu().numpy(), want, equal_nan=True)
    assert np.array_equal(got.codes.cpu().numpy(), ow.pack(q))
    back = fb.w4_dequant(*got).view(N, K // group, group)
    assert bool(back[hit].isnan().all()) and not bool(back[~hit].isnan().any())
    # and so does every product with them
    for M in (1, 2, 5, 20, 60):
        y = fb.w4_linear(torch.ones(M, K, dtype=w.dtype, device=dev()), *got)
        assert not bool(y[:, 1:].isfinite().any()) and bool(y[:, 0].isfinite().all())


@pytest.mark.parametrize("zeros", [False, True])
def test_w4_quant_range_past_fp32(zeros):
    """hi - lo of the largest finite bf16 weights of both signs is infinite in fp32; a
    magnitude alone is not."""
    w = torch.zeros(2, 64, dtype=torch.bfloat16)
    w[:, 5] = torch.finfo(torch.bfloat16).max
    w[0, 9] = -torch.finfo(torch.bfloat16).max
    got = fb.w4_quant(w.to(dev()), 64, zeros)
    assert got.scale.isfinite().tolist() == [[not zeros], [True]]
    q, want, _ = ow.quant(w.double().numpy(), 64, zeros, "bfloat16")
    assert np.array_equal(got.scale.double().cpu().numpy(), want)
    assert np.array_equal(got.codes.cpu().numpy(), ow.pack(q))
