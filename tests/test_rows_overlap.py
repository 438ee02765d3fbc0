"""Whether rows of heads share memory, as the calls that take tq_rows tell it (host code, compiled for the test), against every pair of rows."""
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include <cstdio>
#include "rows.h"
// "0" and lines of: address and three strides of two sets, batch, heads of each, tokens, D -> whether the first meets itself, and the second
// "1" and lines of: an array's address and bytes; rows' address, stride, number, stride, number, bytes -> whether they meet
int main() {
    long long v[13], kind;
    while (std::scanf("%lld", &kind) == 1) {
        if (kind == 1) {
            for (int i = 0; i < 8; ++i)
                if (std::scanf("%lld", v + i) != 1) return 1;
            std::printf("%d\n", tq::Span(reinterpret_cast<void*>(v[0]), v[1]).meets_rows(reinterpret_cast<void*>(v[2]), v[3], v[4], v[5], v[6], v[7]));
            continue;
        }
        for (long long& x : v)
            if (std::scanf("%lld", &x) != 1) return 1;
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

    def call(cases, kind=0):
        text = "\n".join(" ".join(str(x) for x in (kind, *c)) for c in cases) + "\n"
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True, timeout=600).stdout.split()
        if kind:
            return [x == "1" for x in out]
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


def starts(at, strides, n):
    sb, sh, st = (s if k > 1 else 0 for s, k in zip(strides, n))
    return [at + b * sb + h * sh + t * st for b in range(n[0]) for h in range(n[1]) for t in range(n[2])]


def meet_themselves(rows, D):
    rows = sorted(rows)
    return any(y - x < D for x, y in zip(rows, rows[1:]))


def test_any_strides(tell):
    # strides of which none need be as long as what the others span; rows shifted against each other
    rnd = random.Random(1)
    cases, want = [], []
    for _ in range(20000):
        D = rnd.choice([1, 2, 8])
        n = [rnd.randint(1, 5) for _ in range(3)]
        hb = rnd.choice([n[1], n[1], 1, rnd.randint(1, 5)])
        a = [rnd.randint(-12, 12) * rnd.choice([1, D]) for _ in range(3)]
        b = list(a)
        if n[1] == 1 or hb == 1:
            b[1] = rnd.randint(-40, 40)
        apart = rnd.randint(-60, 60)
        ra, rb = starts(0, a, n), starts(apart, b, [n[0], hb, n[2]])
        cases.append((BASE, *a, BASE + 2 * apart, *b, n[0], n[1], hb, n[2], D))
        want.append((meet_themselves(ra, D), any(abs(x - y) < D for x in ra for y in rb)))
    got = tell(cases)
    assert [m for m, _ in got] == [m for m, _ in want]
    assert [m for _, m in got] == [m for _, m in want]


def test_strides_that_share_multiples(tell):
    # heads 192 apart, tokens 128: the third head's first token is the first head's fourth
    D = 64
    alone = (BASE + (1 << 30), 1 << 20, 64, 512)
    got = tell([(BASE, 4096, 192, 128) + alone + (1, 3, 3, 4, D), (BASE, 4096, 192, 128) + alone + (1, 3, 3, 3, D),
                (BASE, 4096, 192, 128) + alone + (1, 2, 2, 64, D), (BASE, 4096, 64 * 101, 64 * 100) + alone + (1, 100, 100, 101, D),
                (BASE, 4096, 64 * 101, 64 * 100) + alone + (1, 100, 100, 102, D), (BASE, 4096, 64 * 101, 64 * 100) + alone + (1, 101, 101, 102, D)])
    assert [m for m, _ in got] == [True, False, False, False, False, True]


def test_layouts_that_take_too_long_to_tell(tell):
    # heads s + 1 apart, tokens s: apart as long as there are at most s of either; so many that it is not looked through are refused
    def call(s, n):
        return tell([(BASE, 0, s + 1, s, BASE + (1 << 60), 0, s + 1, s, 1, n, n, n, 1)])[0][0]
    assert [call(1000, 1000), call(1000, 1002), call(10 ** 7, 10 ** 7)] == [False, True, True]


def test_an_array_and_rows(tell):
    rnd = random.Random(2)
    cases, want = [], []
    for _ in range(20000):
        size, bytes_ = rnd.randint(0, 20), rnd.randint(1, 12)
        sb, nb, sr, nr = rnd.randint(-40, 40), rnd.randint(0, 5), rnd.randint(-15, 15), rnd.randint(0, 5)
        at = rnd.randint(-150, 150)
        cases.append((BASE + at, size, BASE, sb, nb, sr, nr, bytes_))
        want.append(size > 0 and any(at < b * sb + r * sr + bytes_ and b * sb + r * sr < at + size for b in range(nb) for r in range(nr)))
    assert tell(cases, 1) == want
