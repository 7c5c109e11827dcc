"""Row-wise quantization of more rows than one launch takes (a grid holds fewer
than 2^32 threads): the last rows get the codes and scales of the first."""
import pytest
import torch

import block_scaled_fp8_act_amd as fb
from gpu_helpers import dev, say

pytestmark = pytest.mark.gpu


def test_rowwise_quant_past_one_grid():
    R, K = (1 << 24) + 8, 128
    say("rowwise", R)
    few = torch.randn(8, K, device=dev(), generator=torch.Generator(device=dev()).manual_seed(1)).bfloat16()
    q, s = fb.rowwise_quant(few)
    x = few.repeat(R // 8, 1)
    qs, ss = fb.rowwise_quant(x)
    assert torch.equal(ss.view(-1, 8), s.expand(R // 8, 8))
    assert torch.equal(qs.view(-1, 8, K), q.expand(R // 8, 8, K))
