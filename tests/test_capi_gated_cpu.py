"""Argument checks of the gated projections' entry points, without a GPU: bad
arguments give the documented status before the HIP runtime is touched (a good
call ends at the device check, 4), and the workspace sizes are host arithmetic."""
import pytest

from test_capi_routing_cpu import A, ALIGN, B, BIG, C, D, E_, F, G_, H, MIS, NULL, NULL_, SHAPE, fits
from test_capi_routing_cpu import lib  # noqa: F401  (the fixture)


def forward(lib, x=A, ldx=None, w=B, kind=1, act=0, M=0, I=64, K=64, h=C, f=NULL, work=F, nbytes=BIG):  # noqa: E741,F811
    return lib.fp8blk_gated_linear(x, K if ldx is None else ldx, w, kind, act, M, I, K, h, f, work, nbytes, NULL)


COMMON = [(dict(M=-1), SHAPE), (dict(M=1 << 31), SHAPE), (dict(M=4, I=-1), SHAPE), (dict(M=4, K=0), SHAPE),
          (dict(M=4, I=(1 << 21) + 1), SHAPE), (dict(M=4, K=(1 << 22) + 1), SHAPE), (dict(M=4, ldx=63), SHAPE),
          (dict(M=4, ldx=(1 << 22) + 1), SHAPE), (dict(M=4, kind=0), SHAPE), (dict(M=4, kind=3), SHAPE),
          (dict(M=4, act=3), SHAPE), (dict(M=4, act=-1), SHAPE),
          (dict(M=(1 << 31) - 1, I=1 << 21), SHAPE),      # a grid of 2^32 threads
          (dict(M=4, x=NULL), NULL_), (dict(M=4, w=NULL), NULL_),
          (dict(M=4, x=MIS), ALIGN), (dict(M=4, w=MIS), ALIGN), (dict(M=4, f=MIS), ALIGN)]


@pytest.mark.parametrize("bad,want", COMMON + [
    (dict(M=4, h=NULL), NULL_), (dict(M=4, h=MIS), ALIGN), (dict(M=100, K=63, work=NULL), NULL_),
    (dict(M=100, K=63, nbytes=64), SHAPE), (dict(M=100, K=63, work=MIS), ALIGN)])
def test_gated_arguments(lib, bad, want):  # noqa: F811
    assert forward(lib, **bad) == want


def backward(lib, d=G_, x=A, ldx=None, w=B, f=NULL, kind=2, act=0, M=0, I=64, K=64, dx=C, dw=D, work=F,  # noqa: E741,F811
             nbytes=BIG):
    return lib.fp8blk_gated_linear_backward(d, x, K if ldx is None else ldx, w, f, kind, act, M, I, K, dx, dw,
                                            work, nbytes, NULL)


@pytest.mark.parametrize("bad,want", COMMON + [
    (dict(M=4, d=NULL), NULL_), (dict(M=4, d=MIS), ALIGN), (dict(M=4, dx=MIS), ALIGN), (dict(M=4, dw=MIS), ALIGN),
    (dict(M=4, work=NULL), NULL_), (dict(M=4, nbytes=64), SHAPE), (dict(M=4, work=MIS), ALIGN)])
def test_gated_backward_arguments(lib, bad, want):  # noqa: F811
    assert backward(lib, **bad) == want


def test_gated_good_calls(lib):  # noqa: F811
    # nothing to do: no pointers needed
    assert fits(forward(lib, x=NULL, w=NULL, h=NULL, work=NULL, nbytes=0))
    assert fits(forward(lib, M=4, I=0, x=NULL, w=NULL, h=NULL, work=NULL, nbytes=0))
    assert fits(backward(lib, M=4, dx=NULL, dw=NULL, d=NULL, x=NULL, w=NULL, work=NULL, nbytes=0))


def test_gated_workspaces(lib):  # noqa: F811
    f = lib.fp8blk_gated_linear_workspace_bytes
    b = lib.fp8blk_gated_linear_backward_workspace_bytes
    assert f(4096, 14336, 4096, 4096) == 0            # read where they are
    assert f(512, 64, 100, 100) >= (512 + 128) * 104 * 2
    assert f(0, 64, 100, 100) == 0 and f(-1, 64, 64, 64) == 0 and b(4, 64, 64, 63, 1, 1) == 0
    assert b(4096, 14336, 4096, 4096, 1, 1) >= 4096 * 28672 * 2
    assert b(300, 64, 4096, 4096, 1, 1) >= b(300, 64, 4096, 4096, 0, 0) >= 300 * 128 * 2
