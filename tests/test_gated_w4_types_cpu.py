"""What is no tensor is a TypeError, as everywhere in the binding; without a GPU."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_act_amd as fb

T = torch.ones(4, 64, dtype=torch.bfloat16)
CODES, SCALE = torch.zeros(6, 32, dtype=torch.uint8), torch.ones(6, 1, dtype=torch.bfloat16)


@pytest.mark.parametrize("other", [None, [[1.0]], np.ones((4, 64), np.float16), 3])
def test_no_tensor_is_a_type_error(other):
    for call in (lambda: fb.gated_linear(other, T), lambda: fb.gated_linear(other, other),
                 lambda: fb.gated_linear_backward(T, other, T), lambda: fb.gated_linear_backward(other, other, T),
                 lambda: fb.fp8blk_gated_linear(other, T, "silu", T, None),
                 lambda: fb.fp8blk_gated_linear_backward(T, other, T, None, "silu", None, None),
                 lambda: fb.w4_quant(other), lambda: fb.w4_dequant(other, SCALE),
                 lambda: fb.w4_linear(other, other, SCALE), lambda: fb.w4_linear(T, other, SCALE),
                 lambda: fb.w4_gated_linear(T, other, other), lambda: fb.fp8blk_w4_linear(T, other, SCALE, None, T),
                 lambda: fb.fp8blk_w4_gated_linear(other, other, SCALE, None, "silu", T),
                 lambda: fb.fp8blk_w4_quant(T, other, SCALE, None)):
        with pytest.raises(TypeError):
            call()


def test_other_arguments_that_are_no_tensors(monkeypatch):
    """The arguments behind the first, of tensors that pass for a device's."""
    class OnDevice(torch.Tensor):
        is_cuda = True
        get_device = lambda self: 0  # noqa: E731
    x, codes, scale = (t.as_subclass(OnDevice) for t in (T, CODES, SCALE))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for other in (None, [[1.0]], 3):
        for call in (lambda: fb.gated_linear(x, other), lambda: fb.gated_linear_backward(other, x, x),
                     lambda: fb.w4_linear(other, codes, scale), lambda: fb.w4_linear(x, codes, other),
                     lambda: fb.w4_dequant(codes, other)):
            with pytest.raises(TypeError):
                call()
    for call in (lambda: fb.w4_linear(x, codes, scale, [1]), lambda: fb.w4_gated_linear(x, codes, scale, 3)):
        with pytest.raises(TypeError):
            call()
