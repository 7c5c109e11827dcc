"""The gated projections and their gradients against the binary64 oracle, whose
tolerances count the library's roundings (fp32 sums, one rounding to the 16-bit
type of each result and of dgu, 24 bits of the factors where they are saved)."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_act_amd as fb
from gpu_helpers import dev, say
from oracle import gated as og

pytestmark = pytest.mark.gpu
DTYPES = {"bfloat16": torch.bfloat16, "float16": torch.float16}


def make(seed, M, I, K, dtype):
    g = torch.Generator().manual_seed(seed)
    t = DTYPES[dtype]
    x = torch.randn(M, K, generator=g).to(t)
    w = (torch.randn(2 * I, K, generator=g) * (2.0 / K ** 0.5)).to(t)
    d = torch.randn(M, I, generator=g).to(t)
    return x, w, d


def n64(t):
    return t.detach().cpu().double().numpy()


def near(got, want, tol, what):
    """Within tolerance; values that round past fp16's largest finite one, 65504
    (its next step would be 65536, so from 65520 on), are infinities."""
    past = 65520.0 if got.dtype == torch.float16 else np.inf
    got = n64(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    over = np.isinf(got) & (np.sign(got) == np.sign(want)) & (np.abs(want) + tol >= past)
    off = np.abs(np.where(over, want, got) - want)
    bad = ~(off <= tol) | (np.isfinite(got) & (np.abs(want) - tol > past))
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(),
                           float(np.max(np.where(bad, off / tol, 0))))


def factors_of(saved, I):
    """The saved bytes as fp32 [M,2I]: of each half the top 24 bits of its values."""
    M = saved.shape[0]
    b = saved.cpu().view(M, 2, -1, 3).to(torch.int32)[:, :, :I]
    return ((b[..., 0] << 8) | (b[..., 1] << 16) | (b[..., 2] << 24)).view(torch.float32).reshape(M, 2 * I)


def check(x, w, d, act, dtype, on=None):
    """Forward, and both backward forms; ``on``: x as the device holds it."""
    D = dev()
    xd = x.to(D) if on is None else on
    wd, dd = w.to(D), d.to(D)
    h, saved = fb.gated_linear(xd, wd, act=act, save=True)
    near(h, *og.forward(n64(x), n64(w), act, dtype), "h")
    assert torch.equal(fb.gated_linear(xd, wd, act=act), h)
    f, e = og.factors(n64(x), n64(w), act)
    near(factors_of(saved, w.shape[0] // 2), f, e + og.KEPT * (np.abs(f) + e), "factors")
    for kept in (saved, None):
        dx, dw = fb.gated_linear_backward(dd, xd, wd, kept, act=act)
        vx, tx, vw, tw = og.backward(n64(d), n64(x), n64(w), act, dtype, kept is not None)
        near(dx, vx, tx, "d_x")
        near(dw, vw, tw, "d_w")
        assert torch.equal(fb.gated_linear_backward(dd, xd, wd, kept, act=act, need_w=False)[0], dx)
        none, dw2 = fb.gated_linear_backward(dd, xd, wd, kept, act=act, need_x=False)
        assert none is None and torch.equal(dw2, dw)


SIZES = [(1, 1, 1), (1, 64, 64), (2, 3, 5), (3, 100, 128), (7, 257, 72), (8, 48, 1000), (9, 130, 520),
         (16, 64, 257), (17, 33, 65), (33, 127, 8), (64, 128, 128), (65, 70, 136), (128, 64, 192),
         (129, 130, 72), (300, 257, 200), (257, 700, 331), (513, 300, 136)]


@pytest.mark.parametrize("M,I,K", SIZES)
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_gated(M, I, K, dtype):
    act = list(fb.ACTS)[(M + I + K) % 3]
    say("gated", M, I, K, dtype, act)
    check(*make(M + I + K, M, I, K, dtype), act, dtype)


@pytest.mark.parametrize("act", list(fb.ACTS))
@pytest.mark.parametrize("M", [5, 200])
def test_gated_activations(act, M):
    check(*make(M, M, 96, 64, "bfloat16"), act, "bfloat16")
    check(*make(M + 1, M, 96, 64, "float16"), act, "float16")


@pytest.mark.parametrize("act", list(fb.ACTS))
def test_gated_far_arguments(act):
    """Gates from -3e4 to 3e4 (exponentials and cubes that overflow, slopes that
    vanish): finite results within tolerance."""
    M, I, K = 40, 24, 8
    x, w, d = make(3, M, I, K, "float16")
    scale = torch.logspace(-3, 4.4, M)[:, None]
    x = torch.zeros(M, K).to(torch.float16)
    x[:, :1] = scale.to(torch.float16)
    x[:, 1] = 1.0
    w[:, 2:] = 0
    w[:I, 0] = torch.linspace(-1, 1, I).to(torch.float16)
    w[:I, 1] = 0
    w[I:, 0] = 0
    say("gated far", act)
    check(x, w, d, act, "float16")


@pytest.mark.parametrize("M", [1, 6, 40, 140])
@pytest.mark.parametrize("pad", [8, 3, 1])
def test_gated_rows_of_a_wider_matrix(M, pad):
    I, K = 72, 120
    x, w, d = make(M + pad, M, I, K, "bfloat16")
    wide = torch.full((M, K + 8 + pad), float("nan"), dtype=torch.bfloat16, device=dev())
    wide[:, 8:8 + K] = x.to(dev())
    say("gated wide", M, pad)
    check(x, w, d, "silu", "bfloat16", on=wide[:, 8:8 + K])


def against_64(x, w, d, act, what, bound):
    """Large sizes: relative Frobenius error against binary64 on the device."""
    h, saved = fb.gated_linear(x, w, act=act, save=True)
    dx, dw = fb.gated_linear_backward(d, x, w, saved, act=act)
    x2, w2 = x.double().requires_grad_(), w.double().requires_grad_()
    g, u = (x2 @ w2.t()).chunk(2, 1)
    a = torch.nn.functional.silu(g) if act == "silu" else torch.nn.functional.gelu(g)
    want = a * u
    gx, gw = torch.autograd.grad(want, (x2, w2), d.double())
    for name, got, ref in (("h", h, want.detach()), ("d_x", dx, gx), ("d_w", dw, gw)):
        err = float((got.double() - ref).norm() / ref.norm())
        say(what, name, err)
        assert err < bound, (what, name, err)


# (the last two: columns of whole rounds of tiles, then the others, in all three products)
@pytest.mark.parametrize("M,I,K", [(3900, 1610, 96), (1000, 4100, 1032), (520, 13000, 264), (4000, 2203, 2056),
                                   (2100, 1500, 7904)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_large_tiles(M, I, K, act):
    """Grids of 256 x 256 tiles.  A result's own rounding leaves at most half a
    step (2^-8) of relative error in any norm, its dgu the same again; the saved
    factors and fp32 sums add far less."""
    g = torch.Generator(device=dev()).manual_seed(M)
    rnd = lambda *s: torch.randn(*s, device=dev(), generator=g).bfloat16()  # noqa: E731
    against_64(rnd(M, K), rnd(2 * I, K) * K ** -0.5, rnd(M, I), act, (M, I, K), 2.1 * 2.0 ** -8)


def test_gated_gradients_by_differences():
    """d_x and d_w against central differences of the library's own forward sum
    <h, d>, h in fp16 (2^-11): a step of 2^-3 along a random direction v moves
    <h, d> by 2^-3 <grad, v>."""
    M, I, K = 48, 40, 64
    x, w, d = make(11, M, I, K, "float16")
    D = dev()
    x, w, d = x.to(D), (w * 0.5).to(D), d.to(D)
    dx, dw = fb.gated_linear_backward(d, x, w)
    step = 2.0 ** -3
    for t, grad, other in ((x, dx, lambda v: fb.gated_linear(v, w)), (w, dw, lambda v: fb.gated_linear(x, v))):
        v = torch.sign(torch.randn(t.shape, generator=torch.Generator().manual_seed(5))).to(D).half() * step
        hi, lo = t + v, t - v            # rounded: the true step is their difference
        moved = (hi.double() - lo.double())
        rise = float(((other(hi).double() - other(lo).double()) * d.double()).sum())
        want = float((grad.double() * moved).sum())
        # third-order term of the difference, and the roundings of h
        size = float((other(t).double().abs() * d.double().abs()).sum())
        assert abs(rise - want) <= 0.05 * float((grad.double() * moved).abs().sum() ** 0.5 * size ** 0.5) + \
            2 * 2.0 ** -11 * size, (rise, want, size)


def test_gated_no_rows_or_outputs():
    D = dev()
    w = torch.ones(6, 16, dtype=torch.bfloat16, device=D)
    x = torch.ones(4, 16, dtype=torch.bfloat16, device=D)
    assert fb.gated_linear(x[:0], w).shape == (0, 3)
    h, f = fb.gated_linear(x, w[:0], save=True)
    assert h.shape == (4, 0) and f.shape == (4, 0) and fb.factor_row(3) == 24
    dx, dw = fb.gated_linear_backward(h[:0, :0].new_empty(0, 3), x[:0], w)
    assert dx.shape == (0, 16) and not dw.any() and dw.shape == (6, 16)
    dx, dw = fb.gated_linear_backward(h, x, w[:0])
    assert not dx.any() and dx.shape == (4, 16) and dw.shape == (0, 16)


def test_gated_leaves_what_is_past_its_outputs():
    """Outputs given by the caller, with guards behind them."""
    D = dev()
    M, I, K = 37, 19, 41
    x, w, d = (t.to(D) for t in make(4, M, I, K, "bfloat16"))

    def guarded(rows, cols, t=torch.bfloat16):
        flat = torch.full((rows * cols + 64,), 5, dtype=t, device=D)
        return flat, flat[:rows * cols].view(rows, cols)
    flats, outs = zip(*(guarded(*s) for s in ((M, I), (M, fb.factor_row(I), torch.uint8), (M, K), (2 * I, K))))
    lib = fb.load_library()
    n = lib.fp8blk_gated_linear_workspace_bytes(M, I, K, K)
    work = torch.full((n + 64,), 7, dtype=torch.uint8, device=D)
    fb.fp8blk_gated_linear(x, w, "silu", outs[0], outs[1], work[:n])
    assert bool((work[n:] == 7).all())
    n = lib.fp8blk_gated_linear_backward_workspace_bytes(M, I, K, K, 1, 1)
    work = torch.full((n + 64,), 7, dtype=torch.uint8, device=D)
    fb.fp8blk_gated_linear_backward(d, x, w, outs[1], "silu", outs[2], outs[3], work[:n])
    assert bool((work[n:] == 7).all())
    for f in flats:
        assert bool((f[-64:] == 5).all())
    h, saved = fb.gated_linear(x, w, save=True)
    dx, dw = fb.gated_linear_backward(d, x, w, saved)
    for a, b in zip(outs, (h, saved, dx, dw)):
        assert torch.equal(a, b)


def test_gated_on_another_stream():
    D = dev()
    x, w, d = (t.to(D) for t in make(6, 150, 130, 200, "float16"))
    want = fb.gated_linear(x, w), *fb.gated_linear_backward(d, x, w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = [(fb.gated_linear(x, w), *fb.gated_linear_backward(d, x, w)) for _ in range(3)]
    s.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))


@pytest.mark.parametrize("M", [1, 8, 50, 300])
def test_gated_graph(M):
    """Forward and backward captured, replayed with eager work in between."""
    D = dev()
    I, K = 96, 259
    x, w, d = (t.to(D) for t in make(8, M, I, K, "bfloat16"))
    outs = [torch.zeros(s, dtype=torch.bfloat16, device=D) for s in ((M, I), (M, K), (2 * I, K))]
    outs.insert(1, torch.zeros(M, fb.factor_row(I), dtype=torch.uint8, device=D))
    lib = fb.load_library()
    w1 = torch.empty(lib.fp8blk_gated_linear_workspace_bytes(M, I, K, K), dtype=torch.uint8, device=D)
    w2 = torch.empty(lib.fp8blk_gated_linear_backward_workspace_bytes(M, I, K, K, 1, 1), dtype=torch.uint8,
                     device=D)

    def step():
        fb.fp8blk_gated_linear(x, w, "gelu", outs[0], outs[1], w1)
        fb.fp8blk_gated_linear_backward(d, x, w, outs[1], "gelu", outs[2], outs[3], w2)
    step()
    torch.cuda.synchronize()
    ref = [o.clone() for o in outs]
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
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
        fb.gated_linear(x * 2, w)
        torch.cuda.synchronize()


def test_gated_refusals():
    D = dev()
    x = torch.ones(4, 32, dtype=torch.bfloat16, device=D)
    w = torch.ones(6, 32, dtype=torch.bfloat16, device=D)
    d = torch.ones(4, 3, dtype=torch.bfloat16, device=D)
    for bad in (lambda: fb.gated_linear(x, w, act="relu"), lambda: fb.gated_linear(x, w[:5]),
                lambda: fb.gated_linear(x[:, :16], w), lambda: fb.gated_linear(x.t(), w),
                lambda: fb.gated_linear(x, w[:, ::2]), lambda: fb.gated_linear(x[None], w),
                lambda: fb.gated_linear(x.cpu(), w.cpu()), lambda: fb.gated_linear(x, w.cpu()),
                lambda: fb.gated_linear(x[:, :0], w[:, :0]),
                lambda: fb.gated_linear(x[:1].expand(4, 32), w),
                lambda: fb.gated_linear_backward(d[:3], x, w), lambda: fb.gated_linear_backward(d, x, w, d.view(torch.uint8)),
                lambda: fb.gated_linear_backward(d.t(), x, w)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: fb.gated_linear(x.float(), w.float()), lambda: fb.gated_linear(x, w.half()),
                lambda: fb.gated_linear_backward(d.half(), x, w), lambda: fb.gated_linear_backward(d, x, w, d)):
        with pytest.raises(TypeError):
            bad()
    wide = torch.ones(4, 40, dtype=torch.bfloat16, device=D)
    with pytest.raises(fb.Fp8BlkError):
        fb.gated_linear(wide[:, 1:33], w)              # x's base at 2 bytes
    with pytest.raises(fb.Fp8BlkError):                # no workspace where one is needed
        fb.fp8blk_gated_linear(torch.ones(70, 33, dtype=torch.bfloat16, device=D),
                               torch.ones(6, 33, dtype=torch.bfloat16, device=D), "silu",
                               torch.empty(70, 3, dtype=torch.bfloat16, device=D), None)
