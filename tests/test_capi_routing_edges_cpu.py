"""Edges of the adapter entry point's argument checks, without a GPU."""
from test_capi_routing_cpu import NULL, fits, lib, lora  # noqa: F401


def test_empty_batch_without_a_base(lib):
    """An empty tensor's pointer is NULL, and there is no base: not in place."""
    assert fits(lora(lib, T=0, x=NULL, out=NULL, base=NULL, ldb=0))
    assert fits(lora(lib, T=0, x=NULL, out=NULL, base=NULL, ldb=64, ldo=80))
    assert fits(lora(lib, T=4, N=0, base=NULL, ldb=0, out=NULL, work=NULL))
