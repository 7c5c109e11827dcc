"""Argument checks of the 4-bit weights' entry points, without a GPU: bad
arguments give the documented status before the HIP runtime is touched (a good
call ends at the device check, 4), and the workspace sizes are host arithmetic."""
import pytest

from test_capi_routing_cpu import A, ALIGN, B, BIG, C, D, E_, F, MIS, NULL, NULL_, SHAPE, fits
from test_capi_routing_cpu import lib  # noqa: F401  (the fixture)


def quant(lib, w=A, kind=1, N=0, K=256, group=64, codes=B, s=C, z=D):  # noqa: F811
    return lib.fp8blk_w4_quant(w, kind, N, K, group, codes, s, z, NULL)


def dequant(lib, w=A, kind=1, N=0, K=256, group=64, codes=B, s=C, z=D):  # noqa: F811
    return lib.fp8blk_w4_dequant(codes, s, z, kind, N, K, group, w, NULL)


WEIGHTS = [(dict(N=4, codes=NULL), NULL_), (dict(N=4, s=NULL), NULL_),
           (dict(N=-1), SHAPE), (dict(N=1 << 31), SHAPE), (dict(N=4, K=0), SHAPE), (dict(N=4, K=96), SHAPE),
           (dict(N=4, K=(1 << 22) + 64), SHAPE), (dict(N=4, group=16), SHAPE), (dict(N=4, group=256), SHAPE),
           (dict(N=4, group=0), SHAPE), (dict(N=4, kind=0), SHAPE), (dict(N=4, kind=3), SHAPE),
           (dict(N=4, codes=MIS), ALIGN), (dict(N=4, s=MIS), ALIGN), (dict(N=4, z=MIS), ALIGN)]


@pytest.mark.parametrize("call", [quant, dequant])
@pytest.mark.parametrize("bad,want", WEIGHTS + [(dict(N=4, w=NULL), NULL_), (dict(N=4, w=MIS), ALIGN)])
def test_w4_quant_arguments(lib, call, bad, want):  # noqa: F811
    assert call(lib, **bad) == want


def linear(lib, x=A, ldx=None, kind=1, M=4, N=0, K=256, group=64, codes=B, s=C, z=D, y=E_, work=F,  # noqa: F811
           nbytes=BIG):
    return lib.fp8blk_w4_linear(x, K if ldx is None else ldx, codes, s, z, kind, group, M, N, K, y, work, nbytes,
                                NULL)


def gated(lib, x=A, ldx=None, kind=1, M=4, N=0, K=256, group=64, codes=B, s=C, z=D, y=E_, work=F,  # noqa: F811
          nbytes=BIG, act=0):
    return lib.fp8blk_w4_gated_linear(x, K if ldx is None else ldx, codes, s, z, kind, group, act, M, N, K, y, work,
                                      nbytes, NULL)


@pytest.mark.parametrize("call", [linear, gated])
@pytest.mark.parametrize("bad,want", WEIGHTS + [
    (dict(N=4, x=NULL), NULL_), (dict(N=4, y=NULL), NULL_), (dict(N=4, x=MIS), ALIGN), (dict(N=4, y=MIS), ALIGN),
    (dict(N=4, M=-1), SHAPE), (dict(N=4, M=1 << 31), SHAPE), (dict(N=4, ldx=255), SHAPE),
    (dict(N=4, ldx=(1 << 22) + 8), SHAPE), (dict(N=1 << 26, M=1 << 30), SHAPE), (dict(N=(1 << 26) + 1), SHAPE), (dict(N=1 << 28), SHAPE),
    (dict(N=4, M=300, ldx=257, work=NULL), NULL_), (dict(N=4, M=300, ldx=257, nbytes=16), SHAPE),
    (dict(N=4, M=300, ldx=257, work=MIS), ALIGN)])
def test_w4_product_arguments(lib, call, bad, want):  # noqa: F811
    assert call(lib, **bad) == want


def test_w4_good_calls(lib):  # noqa: F811
    assert gated(lib, N=4, act=3) == SHAPE and gated(lib, N=1 << 30) == SHAPE
    for call in (quant, dequant, linear, gated):
        assert fits(call(lib, N=0, codes=NULL, s=NULL, z=NULL))
    assert fits(linear(lib, N=4, M=0, x=NULL, codes=NULL, s=NULL, y=NULL, work=NULL, nbytes=0))


def test_w4_workspaces(lib):  # noqa: F811
    f, g = lib.fp8blk_w4_linear_workspace_bytes, lib.fp8blk_w4_gated_linear_workspace_bytes
    assert f(4096, 14336, 4096, 4096) == 0 and g(4096, 14336, 4096, 4096) == 0
    assert f(4096, 14336, 4096, 4099) >= 4096 * 4096 * 2
    assert f(0, 64, 64, 64) == 0 and g(4, 0, 64, 64) == 0 and f(4, -1, 64, 64) == 0 and g(4, 1 << 31, 64, 64) == 0
