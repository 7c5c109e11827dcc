"""Buffers of a caller that are smaller than they look are refused before a
launch, which would write or read past them."""
import pytest
import torch

import block_scaled_fp8_act_amd as fb
from gpu_helpers import dev

pytestmark = pytest.mark.gpu


def looks_large():
    """One byte of memory behind 2^24 elements; and every other of 2^24."""
    yield torch.zeros(1, dtype=torch.uint8, device=dev()).expand(1 << 24)
    yield torch.zeros(1 << 24, dtype=torch.uint8, device=dev())[::2]


def test_workspaces_that_are_not_contiguous():
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev())  # noqa: E731
    f32 = lambda *s: torch.zeros(*s, device=dev())  # noqa: E731
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=dev())  # noqa: E731
    T, E, k = 5000, 16, 2
    for work in looks_large():
        with pytest.raises(ValueError, match="contiguous"):
            fb.fp8blk_moe_route(f32(T, E), None, True, 0.0, i32(T, k), f32(T, k), i32(E), None, None, work)
        with pytest.raises(ValueError, match="contiguous"):
            fb.fp8blk_group_rows(i32(T), i32(T), i32(T), i32(E + 1), work)
        with pytest.raises(ValueError, match="contiguous"):
            fb.fp8blk_lora_add(None, bf(70, 128), bf(2, 8, 128), bf(2, 16, 8), i32(70), None, None,
                               bf(70, 16), work)
    work = torch.zeros(1 << 24, dtype=torch.uint8, device=dev())
    fb.fp8blk_moe_route(f32(T, E), None, True, 0.0, i32(T, k), f32(T, k), i32(E), None, None, work)
    fb.fp8blk_group_rows(i32(T), i32(T), i32(T), i32(E + 1), work)
    fb.fp8blk_lora_add(None, bf(70, 128), bf(2, 8, 128), bf(2, 16, 8), i32(70), None, None, bf(70, 16), work)
    torch.cuda.synchronize()


@pytest.mark.parametrize("rows", [0, 2])
def test_routing_rows_is_one_value(rows):
    x = torch.randn(4, 8, device=dev())
    r = fb.moe_route(x, 2, loss_coef=0.1)
    r = r._replace(rows=torch.zeros(8, dtype=torch.int32, device=dev())[8 - rows:])
    one = torch.ones(1, device=dev())
    with pytest.raises(ValueError, match="rows"):
        fb.moe_route_backward(x, r, d_loss=one)
    with pytest.raises(ValueError, match="rows"):
        fb.fp8blk_moe_route_backward(x, r, None, one, torch.empty_like(x))
