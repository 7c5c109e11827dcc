"""moe_experts refuses a routing that does not belong to its rows or its
weights before anything is launched: rows past x would be read out of range,
and experts past the weights' would vanish from the sums."""
import pytest
import torch

import block_scaled_fp8_act_amd as fb

T, K, I, N, E, TOPK = 6, 256, 128, 384, 4, 2


class Reached(Exception):
    """The call got past its checks."""


@pytest.fixture(autouse=True)
def no_launch(monkeypatch):
    def stop(*a, **k):
        raise Reached
    for name in ("group_rows", "act_quant_group", "grouped_block_gemm", "swiglu_act_quant", "moe_combine"):
        monkeypatch.setattr(fb, name, stop)


def call(x=(T, K), tokens=T, experts=E, up=(E, 2 * I, K), down=(E, N, I), base=(T, N), counts=True):
    routing = fb.Routing(torch.zeros(tokens, TOPK, dtype=torch.int32), torch.zeros(tokens, TOPK),
                         torch.zeros(experts, dtype=torch.int32) if counts else None, None, None, 0.0, True)
    new = lambda s, d: torch.zeros(s, dtype=d)  # noqa: E731
    scales = lambda s: torch.zeros(s[0], -(-s[1] // 128), s[2] // 128)  # noqa: E731
    fb.moe_experts(new(x, torch.bfloat16), routing, new(up, torch.uint8), scales(up),
                   new(down, torch.uint8), scales(down), None if base is None else new(base, torch.bfloat16))


@pytest.mark.parametrize("bad,what", [
    (dict(x=(T - 1, K)), "rows"),                       # would be read past its end
    (dict(x=(T + 1, K), base=(T + 1, N)), "rows"),      # would be dropped
    (dict(tokens=T - 1), "rows"), (dict(tokens=0), "rows"),
    (dict(experts=E + 1), "experts"), (dict(experts=E - 1), "experts"),
    (dict(up=(E - 1, 2 * I, K)), "experts"), (dict(down=(E + 2, N, I)), "experts"),
    (dict(up=(E - 1, 2 * I, K), down=(E - 1, N, I)), "experts"),
    (dict(up=(E, 2 * I, 2 * K)), "K"), (dict(down=(E, N, 2 * I)), "gate_up"),
    (dict(base=(T, N + 1)), "base"), (dict(base=(T - 1, N)), "base"),
])
def test_refused_before_any_launch(bad, what):
    with pytest.raises(ValueError, match=what):
        call(**bad)


@pytest.mark.parametrize("good", [{}, dict(base=None), dict(x=(0, K), tokens=0, base=(0, N)),
                                  dict(counts=False)])
def test_matching_arguments_are_taken(good):
    with pytest.raises(Reached):
        call(**good)
