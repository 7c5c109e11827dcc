"""Products on 256 x 256 tiles, whole, in ranges of K and in two launches, every
output against binary64 within the oracle's tolerances.  That these sizes run on such
tiles is a test of its own on the host."""
import pytest
import torch

import block_scaled_fp8_act_amd as fb
import large_tiles as lt
from gpu_helpers import dev, say
from oracle import gated as og

pytestmark = pytest.mark.gpu
DTYPES = {"bfloat16": torch.bfloat16, "float16": torch.float16}


def near(got, want, tol, what):
    """Every element; the worst one's place and its share of the tolerance."""
    assert got.shape == want.shape, what
    off = (got.double() - want).abs() / tol
    bad = ~(off <= 1.0)
    say(what, "of the tolerance:", float(off.max()))
    assert not bool(bad.any()), (what, int(bad.sum()), bad.nonzero()[:3].tolist(), float(off.max()))


@pytest.mark.parametrize("size", [s for s, _ in lt.GATED])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_gated_on_large_tiles(size, dtype):
    M, I, K = size
    name = list(fb.ACTS)[(M + (dtype == "float16")) % 3]
    g = torch.Generator(device=dev()).manual_seed(M)
    rnd = lambda *s: torch.randn(*s, device=dev(), generator=g)  # noqa: E731
    x, w, d = (t.to(DTYPES[dtype]) for t in (rnd(M, K), rnd(2 * I, K) * (2.0 * K ** -0.5), rnd(M, I)))
    say("large tiles", size, dtype, name)
    h, saved = fb.gated_linear(x, w, name, save=True)
    assert torch.equal(fb.gated_linear(x, w, name), h)
    x64, w64, d64 = x.double(), w.double(), d.double()
    want, e = lt.gated(*lt.project(x64, w64), name)
    near(h, want, lt.rounded(want, e, dtype), "h")
    for kept in (saved, None):
        dx, dw = fb.gated_linear_backward(d, x, w, kept, name)
        vx, tx, vw, tw = lt.gated_backward(d64, x64, w64, name, dtype, kept is not None)
        near(dx, vx, tx, ("d_x", kept is not None))
        near(dw, vw, tw, ("d_w", kept is not None))


@pytest.mark.parametrize("size", [s for s, _ in lt.W4])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_w4_on_large_tiles(size, group, zeros, dtype):
    M, N, K = size
    g = torch.Generator(device=dev()).manual_seed(N + group)
    x = torch.randn(M, K, device=dev(), generator=g).to(DTYPES[dtype])
    t = fb.w4_quant((torch.randn(N, K, device=dev(), generator=g) * K ** -0.5).to(DTYPES[dtype]), group, zeros)
    name = list(fb.ACTS)[(M + group // 32) % 3]
    say("large tiles", size, group, zeros, dtype, name)
    y, e = lt.w4_product(x.double(), *t, group)
    near(fb.w4_linear(x, *t), y, lt.rounded(y, e, dtype), "linear")
    i = N // 2
    h, eh = lt.gated(y[:, :i], y[:, i:], e[:, :i], e[:, i:], name)
    near(fb.w4_gated_linear(x, *t, act=name), h, lt.rounded(h, eh, dtype), "gated")
