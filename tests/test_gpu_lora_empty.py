"""Adapters of an empty batch or of no columns, with and without a base, the
rows listed or not."""
import pytest
import torch

import block_scaled_fp8_act_amd as fb
from gpu_helpers import dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("listed", [False, True])
@pytest.mark.parametrize("with_base", [False, True])
@pytest.mark.parametrize("T,N", [(0, 16), (4, 0), (70, 0), (0, 0)])
def test_lora_empty(T, N, with_base, listed):
    K, r, L = 128, 8, 2
    new = lambda *s: torch.ones(*s, dtype=torch.bfloat16, device=dev())  # noqa: E731
    ids = torch.zeros(T, dtype=torch.int32, device=dev())
    groups = fb.group_rows(ids, L) if listed else None
    base = new(T, N) if with_base else None
    got = fb.lora_add(base, new(T, K), new(L, r, K), new(L, N, r), ids, groups=groups)
    assert got.shape == (T, N)
    out, work = new(T, N), torch.empty(1 << 20, dtype=torch.uint8, device=dev())
    fb.fp8blk_lora_add(base, new(T, K), new(L, r, K), new(L, N, r), ids, None, groups, out, work)
