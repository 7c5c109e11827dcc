"""Low-rank adapters of many requests against the binary64 oracle.

Tolerance: the first product's fp32 sums add at most K / 64 + 64 terms one
after another, h enters the second with 16 significant bits (2^-16 of the
terms' magnitudes), and the result is rounded once to bf16
(8 significant bits: 2^-8)."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_act_amd as fb
import synth
from gpu_helpers import dev, say, to_dev_bf16
from oracle import adapters as oa

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def make(seed, T, K, N, r, L):
    g = np.random.default_rng(seed)
    bf = lambda *s: torch.from_numpy(g.standard_normal(s).astype(np.float32)).bfloat16()  # noqa: E731
    x, base = bf(T, K), bf(T, N)
    a, b = bf(L, r, K) * K ** -0.5, bf(L, N, r) * r ** -0.5
    scale = torch.from_numpy(g.uniform(0.2, 2.0, L).astype(np.float32))
    return x, base, a, b, scale


def check(got, base, x, a, b, ids, scale):
    K, r = x.shape[1], a.shape[1]
    n = lambda t: None if t is None else t.double().numpy()  # noqa: E731
    want, mag = oa.lora_add(n(base), n(x), n(a), n(b), ids, n(scale))
    tol = mag * (2.0 ** -16 + (K / 64 + 64 + r) * U) + np.abs(want) * 2.0 ** -8 * 1.0001
    off = np.abs(got.double().cpu().numpy() - want)
    assert np.all(off <= tol), float(np.max(off / (tol + 1e-300)))


def on(t):
    return None if t is None else t.to(dev())


SHAPES = [(1, 128, 1, 8, 1), (1, 4096, 4096, 16, 3), (16, 4096, 1024, 16, 16), (17, 256, 77, 8, 2),
          (64, 512, 300, 24, 5), (63, 1024, 513, 40, 64), (65, 512, 300, 32, 5), (80, 128, 63, 72, 1),
          (130, 896, 1030, 64, 7), (515, 1536, 256, 128, 100), (300, 640, 511, 256, 3),
          (257, 256, 64, 136, 300), (1200, 256, 192, 16, 2), (40, 7168, 576, 200, 3)]


@pytest.mark.parametrize("T,K,N,r,L", SHAPES)
@pytest.mark.parametrize("bare", [0.0, 0.3])
def test_lora_add(T, K, N, r, L, bare):
    say("lora", T, K, N, r, L, bare)
    x, base, a, b, scale = make(T + K, T, K, N, r, L)
    g = np.random.default_rng(T)
    ids = g.integers(0, L, T).astype(np.int32)
    ids[g.random(T) < bare] = -1
    if bare and T > 3:
        ids[1], ids[2] = L, 2 ** 31 - 1
    none = (ids < 0) | (ids >= L)
    x[torch.from_numpy(none)] = float("nan")       # rows without adapter are not read
    ids_d = torch.from_numpy(ids).to(dev())
    got = fb.lora_add(on(base), on(x), on(a), on(b), ids_d, on(scale))
    clean = torch.where(torch.from_numpy(none)[:, None], torch.zeros_like(x), x)
    check(got, base, clean, a, b, ids, scale)
    assert torch.equal(got.cpu()[none], base[none])
    # the rows listed beforehand, in place, and again: the same bits
    groups = fb.group_rows(ids_d, L)
    assert torch.equal(fb.lora_add(on(base), on(x), on(a), on(b), ids_d, on(scale), groups), got)
    y = on(base)
    assert fb.lora_add(y, on(x), on(a), on(b), ids_d, on(scale), out=y) is y
    assert torch.equal(y, got)
    # without a base and without scales
    check(fb.lora_add(None, on(x), on(a), on(b), ids_d), None, clean, a, b, ids, None)


@pytest.mark.parametrize("T", [5, 64, 65, 200])
@pytest.mark.parametrize("which", ["one", "none", "runs"])
def test_lora_adapter_patterns(T, which):
    L, K, N, r = 6, 384, 150, 16
    x, base, a, b, scale = make(T, T, K, N, r, L)
    ids = {"one": np.full(T, 4), "none": np.full(T, -1),
           "runs": np.sort(np.random.default_rng(T).integers(-1, L, T))[::-1]}[which]
    ids = np.ascontiguousarray(ids).astype(np.int32)
    got = fb.lora_add(on(base), on(x), on(a), on(b), torch.from_numpy(ids).to(dev()), on(scale))
    check(got, base, x, a, b, ids, scale)
    if which == "none":
        assert torch.equal(got.cpu(), base)


@pytest.mark.parametrize("T", [9, 150])
@pytest.mark.parametrize("N,pad", [(128, 64), (129, 7), (100, 1)])
def test_lora_column_slices(T, N, pad):
    """x, base and out as column slices of wider matrices (a fused
    projection's parts); what lies beside them is not touched."""
    L, K, r = 3, 256, 32
    x, base, a, b, scale = make(T + N, T, K, N, r, L)
    ids = (np.arange(T) % (L + 1) - 1).astype(np.int32)
    wide_x = torch.full((T, K + 24), 7.0, dtype=torch.bfloat16, device=dev())
    wide_y = torch.full((T, N + pad), 3.0, dtype=torch.bfloat16, device=dev())
    wide_x[:, 8:8 + K] = on(x)
    wide_y[:, :N] = on(base)
    y = wide_y[:, :N]
    fb.lora_add(y, wide_x[:, 8:8 + K], on(a), on(b), torch.from_numpy(ids).to(dev()), on(scale), out=y)
    check(y, base, x, a, b, ids, scale)
    assert bool((wide_y[:, N:] == 3).all())
    out = torch.full((T, N + pad), 5.0, dtype=torch.bfloat16, device=dev())
    fb.lora_add(on(base), wide_x[:, 8:8 + K], on(a), on(b), torch.from_numpy(ids).to(dev()), on(scale),
                out=out[:, :N])
    assert torch.equal(out[:, :N], y) and bool((out[:, N:] == 5).all())


def test_lora_infinite_first_product_stays_in_its_row():
    """An overflowing x A^T gives infinities or NaN in its own row alone."""
    x, base, a, b, _ = make(1, 20, 128, 70, 8, 1)
    ids = torch.zeros(20, dtype=torch.int32, device=dev())
    clean = fb.lora_add(on(base), on(x), on(a), on(b), ids)
    x[7] = 3e38
    a2 = a.clone()
    got = fb.lora_add(on(base), on(x), on(a2), on(b), ids)
    rest = torch.arange(20) != 7
    assert torch.equal(got.cpu()[rest], clean.cpu()[rest])
    assert not bool(torch.isfinite(got[7]).all())
    x[7] = 0.0
    x[7, 0] = float("inf")
    b1 = torch.ones_like(b)
    a2[:, :, 0] = 1.0
    got = fb.lora_add(on(base), on(x), on(a2), on(b1), ids)
    assert bool((got[7] == float("inf")).all())      # inf, not NaN from a split of it


def test_lora_no_rows_or_columns():
    x, base, a, b, _ = make(2, 4, 128, 16, 8, 2)
    ids = torch.zeros(4, dtype=torch.int32, device=dev())
    assert fb.lora_add(on(base)[:0], on(x)[:0], on(a), on(b), ids[:0]).shape == (0, 16)
    assert fb.lora_add(on(base)[:, :0], on(x), on(a), on(b)[:, :0].contiguous(), ids).shape == (4, 0)


def test_lora_on_another_stream():
    x, base, a, b, scale = make(3, 100, 512, 256, 16, 4)
    ids = torch.from_numpy((np.arange(100) % 4).astype(np.int32)).to(dev())
    args = (on(base), on(x), on(a), on(b), ids, on(scale))
    want = fb.lora_add(*args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = [fb.lora_add(*args) for _ in range(3)]
    s.synchronize()
    assert all(torch.equal(g, want) for g in got)


@pytest.mark.parametrize("M", [3, 16, 130])
def test_lora_linear(M):
    """The FP8 layer with its adapters: the layer's output, then lora_add."""
    N, K, L, r = 320, 512, 4, 16
    w_q, w_s = fb.weight_block_quant(to_dev_bf16(synth.normal_bf16(4, (N, K), 0.02)))
    x, _, a, b, scale = make(M, M, K, N, r, L)
    ids = torch.from_numpy((np.arange(M) % (L + 1) - 1).astype(np.int32)).to(dev())
    y = fb.linear(on(x), w_q, w_s)
    got = fb.lora_linear(on(x), w_q, w_s, on(a), on(b), ids, on(scale))
    assert torch.equal(got, fb.lora_add(y, on(x), on(a), on(b), ids, on(scale)))
    check(got, y.cpu(), x, a, b, ids.cpu().numpy(), scale)


def test_lora_refusals():
    x, base, a, b, scale = (on(t) for t in make(2, 4, 256, 16, 8, 2))
    ids = torch.zeros(4, dtype=torch.int32, device=dev())
    for bad in (7, 12, 264):
        with pytest.raises(ValueError):
            fb.lora_add(base, x, torch.zeros(2, bad, 256, dtype=torch.bfloat16, device=dev()),
                        torch.zeros(2, 16, bad, dtype=torch.bfloat16, device=dev()), ids)
    with pytest.raises(ValueError):
        fb.lora_add(base, x[:, :200], a[:, :, :200].contiguous(), b, ids)     # K % 128
    with pytest.raises(TypeError):
        fb.lora_add(base, x.float(), a, b, ids)
    with pytest.raises(TypeError):
        fb.lora_add(base, x, a, b, ids.long())
    with pytest.raises(ValueError):
        fb.lora_add(base, x, a, b, ids[:3])
    with pytest.raises(ValueError):
        fb.lora_add(base, x, a, b[:, :, :4].contiguous(), ids)
    with pytest.raises(ValueError):
        fb.lora_add(base.t().contiguous().t(), x, a, b, ids)
    with pytest.raises(ValueError):
        fb.lora_add(base[:, :8], x, a, b, ids)
    with pytest.raises(ValueError):
        fb.lora_add(base, x, a, b, ids, scale[:1])
    with pytest.raises(ValueError):
        fb.lora_add(base, x, a, b, ids, groups=fb.group_rows(ids, 3))
    with pytest.raises(fb.Fp8BlkError):
        fb.lora_add(base, x[:, 1:129], a[:, :, :128].contiguous(), b, ids)    # x's base at 2 bytes
