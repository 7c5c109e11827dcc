"""Argument checks of the routing, row-grouping, combining and adapter entry
points, without a GPU: bad arguments give the documented status before the
HIP runtime is touched (a good call ends at the device check, 4), and the
workspace sizes are host arithmetic."""
import os

import pytest

NULL, A, B, C, D, E_, F, G_, H = None, 0x10000, 0x20000, 0x30000, 0x40000, 0x50000, 0x60000, 0x70000, 0x80000
MIS, ODD = 0x10008, 0x10002      # 8- and 2-byte aligned: never dereferenced
BIG = 1 << 30
NULL_, SHAPE, ALIGN, DEVICE = 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    import block_scaled_fp8_act_amd as fb
    from block_scaled_fp8_act_amd import build
    if not os.path.exists(fb.lib_path()):
        build.build()
    return fb.load_library()


def fits(status):
    """Passed every argument check: no GPU here, or one that did the no-op."""
    return status in (0, DEVICE)


def route(lib, logits=A, kind=0, mask=NULL, T=0, E=8, k=2, ids=B, w=C, counts=D, rows=E_, loss=NULL,
          work=F, nbytes=BIG):
    return lib.fp8blk_moe_route(logits, kind, mask, T, E, k, 1, 0.0, ids, w, counts, rows, loss, work,
                                nbytes, NULL)


@pytest.mark.parametrize("bad,want", [
    (dict(T=4, logits=NULL), NULL_), (dict(T=4, ids=NULL), NULL_), (dict(T=4, w=NULL), NULL_),
    (dict(T=4, counts=NULL), NULL_), (dict(T=1000, work=NULL), NULL_),
    (dict(T=-1), SHAPE), (dict(T=1 << 31), SHAPE), (dict(T=4, E=0), SHAPE), (dict(T=4, E=1025), SHAPE),
    (dict(T=4, k=0), SHAPE), (dict(T=4, k=9), SHAPE), (dict(T=4, E=64, k=33), SHAPE),
    (dict(T=4, kind=2), SHAPE), (dict(T=1 << 30, E=64, k=2), SHAPE),   # T k over int32 slots
    (dict(T=1000, nbytes=16), SHAPE),
    (dict(T=4, logits=MIS), ALIGN), (dict(T=4, ids=ODD), ALIGN), (dict(T=4, w=ODD), ALIGN),
    (dict(T=4, counts=ODD), ALIGN), (dict(T=4, loss=ODD), ALIGN), (dict(T=1000, work=MIS), ALIGN),
])
def test_route_arguments(lib, bad, want):
    assert route(lib, **bad) == want


def back(lib, T=0, E=8, k=2, logits=A, kind=1, ids=B, w=C, counts=D, rows=E_, dw=F, dl=G_, out=H):
    return lib.fp8blk_moe_route_backward(logits, kind, T, E, k, 0, 0.0, ids, w, counts, rows, dw, dl,
                                         out, NULL)


@pytest.mark.parametrize("bad,want", [
    (dict(T=4, logits=NULL), NULL_), (dict(T=4, ids=NULL), NULL_), (dict(T=4, w=NULL), NULL_),
    (dict(T=4, counts=NULL), NULL_), (dict(T=4, rows=NULL), NULL_), (dict(T=4, out=NULL), NULL_),
    (dict(T=-4), SHAPE), (dict(T=4, k=9), SHAPE), (dict(T=4, kind=7), SHAPE),
    (dict(T=4, logits=MIS), ALIGN), (dict(T=4, out=MIS), ALIGN), (dict(T=4, dw=ODD), ALIGN),
    (dict(T=4, dl=ODD), ALIGN),
])
def test_route_backward_arguments(lib, bad, want):
    assert back(lib, **bad) == want


@pytest.mark.parametrize("args,want", [
    ((NULL, 4, 8, B, C, D, F, BIG), NULL_), ((A, 4, 8, NULL, C, D, F, BIG), NULL_),
    ((A, 4, 8, B, NULL, D, F, BIG), NULL_), ((A, 4, 8, B, C, NULL, F, BIG), NULL_),
    ((A, 1 << 20, 8, B, C, D, NULL, BIG), NULL_),
    ((A, -1, 8, B, C, D, F, BIG), SHAPE), ((A, 1 << 31, 8, B, C, D, F, BIG), SHAPE),
    ((A, 4, 0, B, C, D, F, BIG), SHAPE), ((A, 4, 1025, B, C, D, F, BIG), SHAPE),
    ((A, 1 << 20, 8, B, C, D, F, 64), SHAPE),
    ((ODD, 4, 8, B, C, D, F, BIG), ALIGN), ((A, 4, 8, ODD, C, D, F, BIG), ALIGN),
    ((A, 4, 8, B, C, ODD, F, BIG), ALIGN), ((A, 1 << 20, 8, B, C, D, MIS, BIG), ALIGN),
])
def test_group_rows_arguments(lib, args, want):
    assert lib.fp8blk_group_rows(*args, NULL) == want


def combine(lib, y=A, R=8, w=B, pos=C, base=NULL, T=4, k=2, N=16, out=D):
    return lib.fp8blk_moe_combine(y, R, w, pos, base, T, k, N, out, NULL)


@pytest.mark.parametrize("bad,want", [
    (dict(y=NULL), NULL_), (dict(w=NULL), NULL_), (dict(pos=NULL), NULL_), (dict(out=NULL), NULL_),
    (dict(T=-1), SHAPE), (dict(R=-1), SHAPE), (dict(N=-1), SHAPE), (dict(k=0), SHAPE),
    (dict(k=33), SHAPE), (dict(T=1 << 30, k=4), SHAPE), (dict(T=1 << 20, N=1 << 21), SHAPE),
    (dict(y=MIS), ALIGN), (dict(out=MIS), ALIGN), (dict(base=MIS), ALIGN), (dict(w=ODD), ALIGN),
    (dict(pos=ODD), ALIGN),
])
def test_combine_arguments(lib, bad, want):
    assert combine(lib, **bad) == want


@pytest.mark.parametrize("bad,want", [
    (dict(d=NULL), NULL_), (dict(y=NULL), NULL_), (dict(used=NULL), NULL_), (dict(dy=NULL), NULL_),
    (dict(dw=NULL), NULL_), (dict(k=33), SHAPE), (dict(N=-1), SHAPE), (dict(T=1 << 31), SHAPE),
    (dict(d=MIS), ALIGN), (dict(dy=MIS), ALIGN), (dict(used=ODD), ALIGN), (dict(dw=ODD), ALIGN),
])
def test_combine_backward_arguments(lib, bad, want):
    a = dict(d=A, y=B, R=8, w=C, pos=D, used=E_, T=4, k=2, N=16, dy=F, dw=G_)
    a.update(bad)
    assert lib.fp8blk_moe_combine_backward(a["d"], a["y"], a["R"], a["w"], a["pos"], a["used"], a["T"],
                                           a["k"], a["N"], a["dy"], a["dw"], NULL) == want


def lora(lib, base=A, ldb=64, x=B, ldx=128, a=C, b=D, ids=E_, scale=NULL, order=NULL, offsets=NULL,
         T=4, K=128, N=64, r=8, L=2, out=F, ldo=64, work=G_, nbytes=BIG):
    return lib.fp8blk_lora_add(base, ldb, x, ldx, a, b, ids, scale, order, offsets, T, K, N, r, L, out,
                               ldo, work, nbytes, NULL)


@pytest.mark.parametrize("bad,want", [
    (dict(x=NULL), NULL_), (dict(a=NULL), NULL_), (dict(b=NULL), NULL_), (dict(ids=NULL), NULL_),
    (dict(out=NULL), NULL_), (dict(work=NULL), NULL_), (dict(order=H), NULL_), (dict(offsets=H), NULL_),
    (dict(T=-1), SHAPE), (dict(T=1 << 31), SHAPE), (dict(K=100), SHAPE), (dict(K=0), SHAPE),
    (dict(N=-1), SHAPE), (dict(r=0), SHAPE), (dict(r=12), SHAPE), (dict(r=264), SHAPE),
    (dict(L=0), SHAPE), (dict(L=1025), SHAPE), (dict(ldx=127), SHAPE), (dict(ldb=63), SHAPE),
    (dict(ldo=63), SHAPE), (dict(out=A, ldo=65), SHAPE), (dict(nbytes=8), SHAPE),
    (dict(T=100000, ldx=1 << 30), SHAPE),
    (dict(T=1 << 26, N=1 << 14, ldb=1 << 14, ldo=1 << 14, nbytes=1 << 60), SHAPE),  # over one grid
    (dict(x=MIS), ALIGN), (dict(a=MIS), ALIGN), (dict(b=MIS), ALIGN), (dict(base=MIS), ALIGN),
    (dict(out=MIS), ALIGN), (dict(work=MIS), ALIGN), (dict(ids=ODD), ALIGN), (dict(scale=ODD), ALIGN),
    (dict(order=ODD, offsets=H), ALIGN),
])
def test_lora_arguments(lib, bad, want):
    assert lora(lib, **bad) == want


def test_good_arguments_reach_the_device_check(lib):
    assert fits(lib.fp8blk_moe_route_backward(NULL, 0, 0, 8, 2, 1, 0.0, *[NULL] * 7, NULL))
    assert fits(lib.fp8blk_moe_combine(NULL, 0, NULL, NULL, NULL, 0, 2, 16, NULL, NULL))
    assert fits(lib.fp8blk_moe_combine_backward(NULL, NULL, 0, NULL, NULL, NULL, 0, 2, 16, NULL, NULL, NULL))
    assert fits(lora(lib, T=0, x=NULL, out=NULL, base=NULL))


def test_workspace_sizes(lib):
    """0 where one workgroup does all; invalid sizes 0; never less for more rows."""
    assert lib.fp8blk_moe_route_workspace_bytes(16, 256) == 0
    assert lib.fp8blk_moe_route_workspace_bytes(131072, 256) > 0
    assert lib.fp8blk_group_rows_workspace_bytes(128, 256) == 0
    assert lib.fp8blk_group_rows_workspace_bytes(1 << 20, 256) > 0
    for f, args in ((lib.fp8blk_moe_route_workspace_bytes, [(-1, 8), (8, 0), (8, 1025), (1 << 31, 8)]),
                    (lib.fp8blk_group_rows_workspace_bytes, [(-1, 8), (8, 0), (8, 1025), (1 << 31, 8)]),
                    (lib.fp8blk_lora_add_workspace_bytes,
                     [(-1, 128, 8, 1, 0), (8, 100, 8, 1, 0), (8, 128, 12, 1, 0), (8, 128, 8, 0, 0),
                      (0, 128, 8, 1, 0), (1 << 31, 128, 8, 1, 0)])):
        for a in args:
            assert f(*a) == 0, a
    for T in (1, 16, 64, 65, 515, 8192, 1 << 20):
        plain = lib.fp8blk_lora_add_workspace_bytes(T, 4096, 16, 8, 0)
        listed = lib.fp8blk_lora_add_workspace_bytes(T, 4096, 16, 8, 1)
        assert listed >= 4 * T * 16
        assert plain == listed if T <= 64 else plain >= listed + 8 * T
