"""Constants of the 8-bit cache's kernels against their definitions, in exact fractions."""
import os
import re
from fractions import Fraction

from conftest import ROOT


def inverse_tangent(n):
    """arctan(1 / n) to below 2^-120."""
    return sum(Fraction((-1) ** k, (2 * k + 1) * n ** (2 * k + 1)) for k in range(60))


PI = 4 * (4 * inverse_tangent(5) - inverse_tangent(239))


def test_turns():
    text = open(os.path.join(ROOT, "turboquant_compressed_kv_tq_gb300", "csrc", "kv8_device.cuh")).read()
    c = int(re.search(r"kC = 0x([0-9A-F]+)ull;", text).group(1), 16)
    assert abs(c - 2 ** 66 / (2 * PI)) <= Fraction(1, 2)   # rounded, as the comment there says
