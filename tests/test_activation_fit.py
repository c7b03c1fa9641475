"""The constants of erfc in the linear layers' epilogue, evaluated in 64 bits (CPU)."""
import math
import os
import re

import pytest

torch = pytest.importorskip("torch")

from tiled_matrix_multiply_gb300 import build  # noqa: E402


def constants():
    """{degree: (c / sqrt 2, coefficients, the highest first)} of normal_tail, as FP32 values."""
    with open(os.path.join(build.CSRC, "activation.cuh")) as f:
        text = f.read()
    few, more = (re.search(name + r"\[\d\] = \{([^}]*)\}", text).group(1) for name in ("few", "more"))
    c = re.search(r"fma2\(a, both\(FAST \? ([\d.]+)f : ([\d.]+)f\), both\(1\.0f\)\)", text).groups()
    f32 = [torch.tensor([float(v.strip().rstrip("f")) for v in t.split(",")]).double()
           for t in (few, more)]
    return {len(k) - 1: (float(torch.tensor(float(v))), k) for k, v in zip(f32, c)}


@pytest.mark.parametrize("degree,bound", [(7, 2.0 ** -23.2), (8, 2.0 ** -25.4)])
def test_the_fit_is_as_close_as_stated(degree, bound):
    c, k = constants()[degree]
    assert len(k) == degree + 1
    x = torch.linspace(0, 10, 40001, dtype=torch.float64)
    t = 1 / (1 + c * x * math.sqrt(2))
    q = torch.zeros_like(x)
    for v in k:
        q = q * t + v
    off = (t * q / (torch.special.erfcx(x) / 2) - 1).abs().max()
    assert float(off) <= bound, math.log2(float(off))
