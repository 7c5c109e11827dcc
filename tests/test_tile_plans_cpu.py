"""The sizes that the tests of large tiles use do run on them: the plan's model,
compiled for the host.  And those tests' formulas against the oracle's."""
import os
import subprocess

import numpy as np
import pytest
import torch

import large_tiles as lt
from block_scaled_fp8_act_amd import build
from oracle import gated as og
from oracle import w4 as ow

PROGRAM = """
#include <stdio.h>
#include "tile16.h"
int main() {
  long long rows, cols, k;
  int w4;
  while (scanf("%lld %lld %lld %d", &rows, &cols, &k, &w4) == 4) {
    const auto c = fp8blk::t16::cut_of(rows, cols, k, w4);
    printf("%d %d %d\\n", c.plan.shape == fp8blk::t16::kLarge, c.plan.ranges, c.first < cols);
  }
}
"""


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    at = tmp_path_factory.mktemp("plans")
    (at / "plans.hip").write_text(PROGRAM)
    subprocess.run([build.hipcc(), "--cuda-host-only", "-std=c++17", "-O1", "-x", "hip", str(at / "plans.hip"),
                    "-I", build.CSRC, "-o", str(at / "plans")], check=True, capture_output=True, timeout=120)

    def of(rows, cols, k, w4=0):
        out = subprocess.run([str(at / "plans")], input=f"{rows} {cols} {k} {w4}\n", text=True, check=True,
                             capture_output=True, timeout=60).stdout
        large, ranges, cut = map(int, out.split())
        return "" if not large else "L+" if cut else "L" if ranges == 1 else f"L{ranges}"
    return of


@pytest.mark.parametrize("size,want", lt.GATED)
def test_gated_sizes_run_on_large_tiles(plans, size, want):
    up = lambda n: -(-n // 8) * 8  # noqa: E731
    M, I, K = size
    assert (plans(M, 2 * I, up(K)), plans(M, K, up(2 * I)), plans(2 * I, K, M)) == want


@pytest.mark.parametrize("size,want", lt.W4)
def test_w4_sizes_run_on_large_tiles(plans, size, want):
    assert plans(*size, 1) == want


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("saved", [False, True])
def test_formulas_on_the_device_are_the_oracles(name, saved):
    g = torch.Generator().manual_seed(1)
    x, w, d = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((9, 7), (12, 7), (9, 6)))
    h, e = lt.gated(*lt.project(x, w), name)
    got = (h, lt.rounded(h, e, "float16"), *lt.gated_backward(d, x, w, name, "float16", saved))
    n = [t.numpy() for t in (x, w, d)]
    want = (*og.forward(n[0], n[1], name, "float16"), *og.backward(n[2], n[0], n[1], name, "float16", saved))
    for a, b in zip(got, want):
        np.testing.assert_allclose(a.numpy(), b, rtol=1e-11, atol=1e-13)


@pytest.mark.parametrize("zeros", [False, True])
def test_w4_formula_on_the_device_is_the_oracles(zeros):
    g = np.random.default_rng(1)
    x, s = g.standard_normal((5, 128)), ow.to_type(g.random((6, 2)), "bfloat16")
    codes = g.integers(0, 256, (6, 64)).astype(np.uint8)
    z = g.integers(0, 16, (6, 2)).astype(np.uint8) if zeros else None
    t = torch.from_numpy
    got = lt.w4_product(t(x), t(codes), t(s), None if z is None else t(z), 64)
    for a, b in zip(got, ow.product(x, codes, s, z, 64)):
        np.testing.assert_allclose(a.numpy(), b, rtol=1e-12, atol=1e-13)
