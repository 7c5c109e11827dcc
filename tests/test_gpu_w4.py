"""4-bit weights: codes, scales and zero points equal to the oracle's, and the
products within its tolerance (fp32 sums of products with the codes, one rounding
of the result; the gated form's own beside them).  No weight is rounded."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_act_amd as fb
from gpu_helpers import dev, say
from oracle import gated as og
from oracle import w4 as ow

pytestmark = pytest.mark.gpu
DTYPES = {"bfloat16": torch.bfloat16, "float16": torch.float16}


def rnd(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def n64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def make(seed, rows, K, group, zeros, dtype):
    """Weights of uneven groups, quantized by the oracle: (codes, scale, zeros) on
    the CPU and W in binary64."""
    w = rnd(seed, rows, K) * (0.5 + 2 * torch.rand(rows, 1, generator=torch.Generator().manual_seed(seed)))
    w = (w * K ** -0.5 + (0.3 * K ** -0.5 if zeros else 0.0)).to(DTYPES[dtype])
    q, s, z = ow.quant(n64(w), group, zeros, dtype)
    codes, z = ow.pack(q), (z if zeros else None)
    t = (torch.from_numpy(codes), torch.from_numpy(s).to(DTYPES[dtype]),
         None if z is None else torch.from_numpy(z))
    return w, t, ow.values(codes, s, z, group)


def on(ts):
    return tuple(None if t is None else t.to(dev()) for t in ts)


@pytest.mark.parametrize("N,K", [(1, 128), (3, 256), (129, 1024), (64, 7168), (2111, 384)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_w4_quant(N, K, group, zeros, dtype):
    w, (codes, scale, z), values = make(N + K, N, K, group, zeros, dtype)
    if N > 2:
        w[1] = 0
        w[2, :group] = w[2, :group].abs()
        q, s, zz = ow.quant(n64(w), group, zeros, dtype)
        codes, scale = torch.from_numpy(ow.pack(q)), torch.from_numpy(s).to(w.dtype)
        z = torch.from_numpy(zz) if zeros else None
        values = ow.values(ow.pack(q), s, zz, group)
    got = fb.w4_quant(w.to(dev()), group, zeros)
    assert torch.equal(got.scale.cpu(), scale) and torch.equal(got.codes.cpu(), codes)
    assert (got.zeros is None) == (not zeros) and (not zeros or torch.equal(got.zeros.cpu(), z))
    back = fb.w4_dequant(*got)
    assert torch.equal(back.cpu(), torch.from_numpy(values).to(w.dtype))


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_w4_quant_ties_and_extremes(zeros, dtype):
    """Weights that are half whole numbers of scales, of every magnitude of the
    type, tiny ones whose scales underflow among them."""
    g = np.random.default_rng(1)
    rows = []
    lo, hi = (-126, 120) if dtype == "bfloat16" else (-24, 11)
    for e in range(lo, hi):
        v = g.integers(-15, 16, 32) * 0.5
        v[0] = 7.0
        if zeros:
            v[1] = -8.0
        rows.append(v * 2.0 ** e)
    w = torch.from_numpy(np.stack(rows)).to(DTYPES[dtype])
    q, s, z = ow.quant(n64(w), 32, zeros, dtype)
    got = fb.w4_quant(w.to(dev()), 32, zeros)
    assert torch.equal(got.scale.cpu(), torch.from_numpy(s).to(w.dtype))
    assert np.array_equal(ow.unpack(got.codes.cpu().numpy()), q)
    assert not zeros or np.array_equal(got.zeros.cpu().numpy(), z)


def near(got, want, tol, dtype, what):
    tol = tol + og.HALF[dtype] * (np.abs(want) + tol) + og.TINY[dtype]
    got = n64(got)
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(),
                           float(np.max(np.abs(got - want) / tol)))


def product(x, t):
    """The oracle's x W^T of 4-bit weights t, and its tolerance."""
    codes, s, z = n64(t[0]).astype(np.uint8), n64(t[1]), n64(t[2])
    return ow.product(n64(x), codes, s, z, 2 * codes.shape[1] // s.shape[1])


def check(x, t, act, dtype, on_dev=None):
    xd = x.to(dev()) if on_dev is None else on_dev
    y, tol = product(x, t)
    t = on(t)
    near(fb.w4_linear(xd, *t), y, tol, dtype, "linear")
    if y.shape[1] % 2 == 0:
        i = y.shape[1] // 2
        a, _ = og.act(y[:, :i], act)
        eg, eu = og.SLOPE * tol[:, :i], tol[:, i:]
        h = a * y[:, i:]
        near(fb.w4_gated_linear(xd, *t, act=act), h,
             eg * np.abs(y[:, i:]) + (np.abs(a) + eg) * eu + og.EVAL * np.abs(h), dtype, "gated")


SIZES = [(1, 2, 32), (1, 130, 128), (1, 4096, 512), (2, 77, 1024), (3, 64, 4096), (4, 514, 2176), (5, 66, 320),
         (7, 128, 640), (8, 34, 14336), (9, 200, 256), (16, 256, 1536), (17, 62, 2048), (31, 1026, 96),
         (33, 300, 544), (48, 64, 7168), (64, 512, 384), (65, 190, 1056), (130, 258, 192), (300, 600, 608)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_w4_products(M, N, K, zeros, dtype):
    for group in (32, 64, 128):
        if K % group == 0:
            act = list(fb.ACTS)[(M + N) % 3]
            say("w4", M, N, K, group, zeros, dtype, act)
            _, t, _ = make(M + N + K, N, K, group, zeros, dtype)
            check(rnd(M, M, K).to(DTYPES[dtype]), t, act, dtype)


@pytest.mark.parametrize("M", [1, 3, 20, 140])
@pytest.mark.parametrize("pad", [8, 3, 1])
def test_w4_rows_of_a_wider_matrix(M, pad):
    N, K = 70, 160
    _, t, _ = make(M, N, K, 32, True, "float16")
    x = rnd(M + 1, M, K).half()
    wide = torch.full((M, K + 8 + pad), float("nan"), dtype=torch.float16, device=dev())
    wide[:, 8:8 + K] = x.to(dev())
    check(x, t, "gelu", "float16", on_dev=wide[:, 8:8 + K])


@pytest.mark.parametrize("M", [1, 4, 12, 64, 200])
def test_w4_outlier_under_a_zero_weight(M):
    """A channel 2^12 times the others whose weight is zero (q = z) in every row:
    what is left of it must not drown the rest (fp32 sums of the products with the
    codes themselves would leave 2^12 15 2^-24 per term)."""
    N, K = 32, 256
    _, t, _ = make(5, N, K, 64, True, "bfloat16")
    q = ow.unpack(t[0].numpy())
    z = t[2].numpy()
    q[:, 70] = z[:, 1]
    q[:, 200] = z[:, 3]
    t = (torch.from_numpy(ow.pack(q)), t[1], t[2])
    x = rnd(M, M, K)
    x[:, 70] = 4096.0
    x[:, 200] = -4096.0
    x = x.bfloat16()
    got = n64(fb.w4_linear(x.to(dev()), *on(t)))
    want, _ = product(x, t)
    # fp32 sums: the outlier's product with codes up to 31 (q and a bias) may pass
    # through them, a few additions' rounding (2^-24 each) of it stays behind
    left = 64 * 2.0 ** -24 * 31 * 4096 * np.abs(n64(t[1])).max()
    values = ow.values(t[0].numpy(), n64(t[1]), z, 64)
    tol = (np.abs(n64(x)) @ np.abs(values).T) * 300 * 2.0 ** -23 + left
    assert np.all(np.abs(got - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol))


# (the last: columns of whole rounds of tiles, then the others)
@pytest.mark.parametrize("M,N,K", [(2100, 6200, 192), (600, 5120, 1024), (2100, 7682, 2048)])
def test_w4_large_tiles(M, N, K):
    g = torch.Generator(device=dev()).manual_seed(M)
    w = (torch.randn(N, K, device=dev(), generator=g) * K ** -0.5).bfloat16()
    x = torch.randn(M, K, device=dev(), generator=g).bfloat16()
    t = fb.w4_quant(w, 64, True)
    q = torch.stack([t.codes & 15, t.codes >> 4], 2).flatten(1).double()
    v = (q - t.zeros.double().repeat_interleave(64, 1)) * t.scale.double().repeat_interleave(64, 1)
    y = x.double() @ v.t()
    # the result's rounding (half a step, 2^-8 in any norm), and fp32 sums
    for got, want in ((fb.w4_linear(x, *t), y),
                      (fb.w4_gated_linear(x, *t), torch.nn.functional.silu(y[:, :N // 2]) * y[:, N // 2:])):
        assert float((got.double() - want).norm() / want.norm()) < 2.0 ** -8


def test_w4_nothing_to_do():
    x = torch.ones(4, 64, dtype=torch.float16, device=dev())
    q = fb.w4_quant(torch.ones(0, 64, dtype=torch.float16, device=dev()), 32)
    assert q.codes.shape == (0, 32) and fb.w4_dequant(*q).shape == (0, 64)
    assert fb.w4_linear(x, *q).shape == (4, 0) and fb.w4_gated_linear(x, *q).shape == (4, 0)
    q = fb.w4_quant(torch.ones(6, 64, dtype=torch.float16, device=dev()), 32)
    assert fb.w4_linear(x[:0], *q).shape == (0, 6) and fb.w4_gated_linear(x[:0], *q).shape == (0, 3)


@pytest.mark.parametrize("M", [1, 6, 40, 150])
def test_w4_on_another_stream_and_in_a_graph(M):
    D = dev()
    _, t, _ = make(2, 96, 512, 128, True, "bfloat16")
    t = on(t)
    x = rnd(M, M, 515).bfloat16().to(D)[:, :512]
    ref = fb.w4_linear(x, *t), fb.w4_gated_linear(x, *t)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = [(fb.w4_linear(x, *t), fb.w4_gated_linear(x, *t)) for _ in range(3)]
    s.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, ref))
    lib = fb.load_library()
    outs = torch.zeros_like(ref[0]), torch.zeros_like(ref[1])
    ws = [torch.empty(f(M, n, 512, 515), dtype=torch.uint8, device=D) for f, n in
          ((lib.fp8blk_w4_linear_workspace_bytes, 96), (lib.fp8blk_w4_gated_linear_workspace_bytes, 48))]
    g = torch.cuda.CUDAGraph()

    def step():
        fb.fp8blk_w4_linear(x, *t, outs[0], ws[0])
        fb.fp8blk_w4_gated_linear(x, *t, "silu", outs[1], ws[1])
    with torch.cuda.stream(s):
        step()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            step()
    for _ in range(3):
        for o in outs:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, r) for o, r in zip(outs, ref))
        fb.w4_linear(x * 2, *t)
        torch.cuda.synchronize()


@pytest.mark.parametrize("M", [1, 5, 33, 100])
def test_w4_leaves_what_is_past_its_outputs(M):
    D = dev()
    N, K = 38, 96
    _, t, _ = make(3, N, K, 32, True, "bfloat16")
    t = on(t)
    x = rnd(M, M, K).bfloat16().to(D)
    lib = fb.load_library()
    for call, cols, need in ((fb.fp8blk_w4_linear, N, lib.fp8blk_w4_linear_workspace_bytes(M, N, K, K)),
                             (lambda *a: fb.fp8blk_w4_gated_linear(*a[:4], "silu", *a[4:]), N // 2,
                              lib.fp8blk_w4_gated_linear_workspace_bytes(M, N // 2, K, K))):
        flat = torch.full((M * cols + 64,), 5.0, dtype=torch.bfloat16, device=D)
        work = torch.full((need + 64,), 9, dtype=torch.uint8, device=D)
        call(x, *t, flat[:M * cols].view(M, cols), work[:need])
        assert bool((flat[M * cols:] == 5).all()) and bool((work[need:] == 9).all())
    w = rnd(1, N, K).bfloat16().to(D)
    flats = [torch.full((n + 64,), 5, dtype=d, device=D) for n, d in
             ((N * K // 2, torch.uint8), (N * K // 32, torch.bfloat16), (N * K // 32, torch.uint8))]
    fb.fp8blk_w4_quant(w, flats[0][:-64].view(N, K // 2), flats[1][:-64].view(N, 3), flats[2][:-64].view(N, 3))
    assert all(bool((f[-64:] == 5).all()) for f in flats)


@pytest.mark.parametrize("M", [1, 16, 100])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_w4_feed_forward_block(M, dtype):
    """A decoding step's whole block in 4 bits: gated projections, then the down
    projection; and the 16-bit block on the dequantized weights beside it."""
    K, I = 256, 384
    _, up, _ = make(1, 2 * I, K, 64, False, dtype)
    _, down, _ = make(2, K, I, 128, True, dtype)
    x = rnd(M, M, K).to(DTYPES[dtype])
    check(x, up, "silu", dtype)
    xd, up, down = x.to(dev()), on(up), on(down)
    h = fb.w4_gated_linear(xd, *up)
    y, tol = product(h, down)
    near(fb.w4_linear(h, *down), y, tol, dtype, "down")
    h16 = fb.gated_linear(xd, fb.w4_dequant(*up))
    want, tol = og.forward(n64(x), n64(fb.w4_dequant(*up)), "silu", dtype)
    assert np.all(np.abs(n64(h16) - want) <= tol)


def test_w4_refusals():
    D = dev()
    w = torch.ones(6, 128, dtype=torch.bfloat16, device=D)
    q = fb.w4_quant(w, 64, True)
    x = torch.ones(4, 128, dtype=torch.bfloat16, device=D)
    for bad in (lambda: fb.w4_quant(w, 16), lambda: fb.w4_quant(w[:, :96].contiguous(), 64),
                lambda: fb.w4_quant(w[:, ::2], 32), lambda: fb.w4_quant(w[0], 32), lambda: fb.w4_quant(w.cpu()),
                lambda: fb.w4_dequant(q.codes, q.scale[:5], None),
                lambda: fb.w4_dequant(q.codes, q.scale.repeat(1, 4), None),      # groups of 16
                lambda: fb.w4_dequant(q.codes, q.scale, q.zeros[:, :1]),
                lambda: fb.w4_linear(x[:, :64], *q), lambda: fb.w4_linear(x[0], *q),
                lambda: fb.w4_linear(x.t().contiguous().t(), *q), lambda: fb.w4_linear(x.cpu(), *q),
                lambda: fb.w4_linear(x, q.codes, q.scale, q.zeros.cpu()),
                lambda: fb.w4_gated_linear(x, q.codes[:5], q.scale[:5], None),
                lambda: fb.w4_gated_linear(x, *q, act="tanh")):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: fb.w4_quant(w.float()), lambda: fb.w4_linear(x.half(), *q),
                lambda: fb.w4_linear(x, q.codes.to(torch.int8), q.scale),
                lambda: fb.w4_linear(x, q.codes, q.scale.float()),
                lambda: fb.w4_linear(x, q.codes, q.scale, q.zeros.float())):
        with pytest.raises(TypeError):
            bad()
