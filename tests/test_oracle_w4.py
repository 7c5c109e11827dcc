"""The 4-bit weights' oracle by hand, on the CPU."""
import numpy as np
import torch

from oracle import w4 as ow


def test_type_rounding():
    g = np.random.default_rng(0)
    v = (g.standard_normal(4000) * 2.0 ** g.integers(-30, 15, 4000)).astype(np.float32)
    for name, t in (("bfloat16", torch.bfloat16), ("float16", torch.float16)):
        assert np.array_equal(ow.to_type(v, name), torch.from_numpy(v).to(t).double().numpy())


def test_hand_groups():
    w = np.zeros((1, 64))
    w[0, :6] = [7, -7, 3.5, 0.5, -8, 1.5]          # s = 8 / 7 without zero points
    q, s, z = ow.quant(w, 32, False, "float16")
    assert s[0, 0] == float(np.float16(8 / 7)) and s[0, 1] == 0 and z[0, 0] == 8
    assert list(q[0, :6]) == [14, 2, 11, 8, 1, 9] and set(q[0, 6:]) == {8}
    w[0, :6] = [15, 0, 1, 0.5, 1.5, 14.5]          # s = 1, z = 0: ties go to even
    q, s, z = ow.quant(w, 32, True, "float16")
    assert s[0, 0] == 1 and z[0, 0] == 0 and list(q[0, :6]) == [15, 0, 1, 0, 2, 14]
    assert s[0, 1] == 0 and z[0, 1] == 0 and not q[0, 32:].any()
    w[0, :6] = [-15, 0, -1, -0.5, -1.5, -14.5]     # z = 15
    q, s, z = ow.quant(w, 32, True, "bfloat16")
    assert s[0, 0] == 1 and z[0, 0] == 15 and list(q[0, :6]) == [0, 15, 14, 15, 13, 1]
    assert np.array_equal(ow.unpack(ow.pack(q)), q)
    v = ow.values(ow.pack(q), s, z, 32)
    assert list(v[0, :6]) == [-15, 0, -1, 0, -2, -14]
