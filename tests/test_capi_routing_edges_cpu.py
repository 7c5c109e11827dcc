"""Edges of the adapter entry point's argument checks, without a GPU.  (A
misaligned pointer shows that the size checks passed: they come first, and
nothing runs.)"""
import pytest

from test_capi_routing_cpu import ALIGN, MIS, NULL, SHAPE, fits, lib, lora  # noqa: F401


def test_empty_batch_without_a_base(lib):
    """An empty tensor's pointer is NULL, and there is no base: not in place."""
    assert fits(lora(lib, T=0, x=NULL, out=NULL, base=NULL, ldb=0))
    assert fits(lora(lib, T=0, x=NULL, out=NULL, base=NULL, ldb=64, ldo=80))
    assert fits(lora(lib, T=4, N=0, base=NULL, ldb=0, out=NULL, work=NULL))


@pytest.mark.parametrize("T,L,N,r", [(64, 64, 1 << 25, 8), (1000, 1000, 1 << 23, 8),
                                     (1000, 1000, 1 << 22, 64)])
def test_one_grid(lib, T, L, N, r):
    """Sizes up to a launch's 2^32 threads pass, larger ones are refused."""
    size = lambda n: dict(T=T, L=L, N=n, r=r, ldb=n, ldo=n, nbytes=1 << 40, work=MIS)  # noqa: E731
    assert lora(lib, **size(N // 2)) == ALIGN
    assert lora(lib, **size(N * 4)) == SHAPE


def test_largest_batches_that_fit(lib):
    """tiles * (N + 256) < 2^31 and tiles * (r + 32) < 2^29 pass."""
    for T, L, r in ((64, 1, 8), (64, 64, 256), (65, 1, 8), (1000, 9, 40), (1000, 1000, 256),
                    (4095, 1024, 64), (1 << 20, 8, 256), (1 << 22, 1024, 8), (100_000_000, 3, 256),
                    (800_000_000, 1024, 8)):
        tiles = min(T, T // (16 if T <= 64 else 64) + L + 1)
        if tiles * (r + 32) >= 1 << 29:
            continue
        N = min(((1 << 31) - 1) // tiles - 256, (1 << 40) // (L * r), (1 << 40) // T)
        N = max(N, 1)
        assert lora(lib, T=T, L=L, N=N, r=r, ldb=N, ldo=N, nbytes=1 << 50, work=MIS) == ALIGN, (T, L, r)
