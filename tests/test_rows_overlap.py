"""Whether rows of heads share memory, as the calls that take tq_rows tell it (host code, compiled for the test), against every pair of rows."""
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include <cstdio>
#include "rows.h"
// lines of: address and three strides of two sets, batch, heads of each, tokens, D -> whether the first meets itself, and the second
int main() {
    long long v[13];
    for (;;) {
        for (long long& x : v)
            if (std::scanf("%lld", &x) != 1) return 0;
        const tq_rows a{reinterpret_cast<void*>(v[0]), v[1], v[2], v[3]}, b{reinterpret_cast<void*>(v[4]), v[5], v[6], v[7]};
        const int D = static_cast<int>(v[12]);
        std::printf("%d %d\n", tq::Axes(&a, v[8], v[9], v[11]).meets_itself(D), tq::rows_meet(&a, v[9], &b, v[10], v[8], v[11], D, 2));
    }
}
"""


@pytest.fixture(scope="module")
def tell(tmp_path_factory):
    d = tmp_path_factory.mktemp("rows")
    (d / "tell.cpp").write_text(PROGRAM)
    exe = str(d / "tell")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "include"), "-I",
                           os.path.join(ROOT, "turboquant_compressed_kv_tq_gb300", "csrc"), str(d / "tell.cpp"), "-o", exe])

    def call(cases):
        text = "\n".join(" ".join(str(x) for x in c) for c in cases) + "\n"
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True, timeout=600).stdout.split()
        return [(out[2 * i] == "1", out[2 * i + 1] == "1") for i in range(len(cases))]
    return call


BASE = 1 << 40   # an address that is never looked at


def test_a_single_head_in_a_projection(tell):
    # [batch][tokens][8 queries, a key, a value][D], rotated in place: keys have no stride of heads
    D, n, nb, H = 64, 5, 3, 10
    q, k = (BASE, n * H * D, D, H * D), (BASE + 8 * D * 2, n * H * D, 0, H * D)
    over = (BASE + 7 * D * 2, n * H * D, 0, H * D)
    got = tell([q + k + (nb, 8, 1, n, D), k + q + (nb, 1, 8, n, D), q + over + (nb, 8, 1, n, D), over + q + (nb, 1, 8, n, D), k + over + (nb, 1, 1, n, D)])
    assert [m for _, m in got] == [False, False, True, True, False]
