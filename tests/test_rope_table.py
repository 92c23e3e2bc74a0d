"""Rotary frequencies (host) against 60-digit arithmetic: every turn fraction to the nearest 2^-64, every
angle to 2^-31 turns at the farthest positions.  No GPU: the table's source is compiled by itself."""
import os
import shutil
import subprocess
from decimal import Decimal as D
from decimal import getcontext

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "compressed_sparse_attention_fp4_gb300", "csrc")
MAIN = r"""
#include <cstdio>
#include "rope_table.cuh"
int main() {
  csa2_rope r = {};
  r.mscale = 1.0f;
  while (std::scanf("%d %d %lf %lf %lf %lf %lf", &r.rot, &r.scaling, &r.theta, &r.factor, &r.orig_ctx, &r.turns_lo,
                    &r.turns_hi) == 7) {
    const csa2::RopeTable t = csa2::make_rope_table(r);
    for (int i = 0; i < t.pairs; ++i) std::printf("%llu ", (unsigned long long)t.turn[i]);
    std::printf("\n");
  }
}
"""
# rot, scaling (0 plain, 1 linear, 2 parts, 3 base), theta, factor, original context, turns
CASES = [(64, 0, 10000.0, 1.0, 0.0, 1.0, 32.0), (128, 0, 500000.0, 1.0, 0.0, 1.0, 32.0), (256, 0, 1e6, 1.0, 0.0, 1.0, 32.0),
         (2, 0, 10000.0, 1.0, 0.0, 1.0, 32.0), (26, 0, 1.0000001, 1.0, 0.0, 1.0, 32.0), (64, 0, 1e300, 1.0, 0.0, 1.0, 32.0),
         (64, 1, 10000.0, 8.0, 0.0, 1.0, 32.0), (64, 1, 10000.0, 3.7, 0.0, 1.0, 32.0), (8, 1, 160000.5, 1e30, 0.0, 1.0, 32.0),
         (64, 2, 10000.0, 16.0, 4096.0, 1.0, 32.0), (64, 2, 10000.0, 40.0, 65536.0, 1.0, 32.0),
         (128, 2, 10000.0, 2.5, 1e300, 0.0, 1e-300), (32, 2, 100.0, 4.0, 0.001, 1.0, 32.0), (96, 2, 1e5, 7.0, 8192.0, 0.1, 1000.3),
         (64, 3, 10000.0, 4.0, 0.0, 1.0, 32.0), (4, 3, 10000.0, 4.0, 0.0, 1.0, 32.0), (2, 3, 10000.0, 4.0, 0.0, 1.0, 32.0),
         (256, 3, 1e8, 1.1, 0.0, 1.0, 32.0), (64, 3, 1e300, 1e300, 0.0, 1.0, 32.0)]


def two_pi():
    def arctan_inverse(x):
        term = total = 1 / D(x)
        k = 1
        while abs(term) > D(10) ** -65:
            term = -term / (x * x)
            k += 2
            total += term / k
        return total
    return 8 * (4 * arctan_inverse(5) - arctan_inverse(239))


def exact(rot, scaling, theta, factor, orig, lo, hi, i, turn):
    theta, factor, orig, lo, hi = (D(v) for v in (theta, factor, orig, lo, hi))
    if scaling == 3 and rot > 2:
        theta = theta * factor ** (D(rot) / (rot - 2))
    f = theta ** (D(-2 * i) / rot)
    if scaling == 1:
        f = f / factor
    if scaling == 2:
        k = min(max((orig * f / turn - lo) / (hi - lo), D(0)), D(1))
        f = f * k + f / factor * (1 - k)
    return f / turn


@pytest.fixture(scope="module")
def tables(tmp_path_factory):
    cc = shutil.which("g++")
    if not cc:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("rope")
    (d / "main.cpp").write_text(MAIN)
    subprocess.run([cc, "-O2", "-std=c++17", "-I" + CSRC, str(d / "main.cpp"), "-o", str(d / "main")], check=True)
    text = "\n".join(" ".join(repr(v) for v in c) for c in CASES)
    out = subprocess.run([str(d / "main")], input=text, capture_output=True, text=True, check=True).stdout
    return [[int(v) for v in line.split()] for line in out.splitlines()]


@pytest.mark.parametrize("n", range(len(CASES)))
def test_fractions_and_angles(tables, n):
    getcontext().prec = 60
    getcontext().Emin = -10 ** 9
    turn = two_pi()
    case, got = CASES[n], tables[n]
    assert len(got) == case[0] // 2
    for i, g in enumerate(got):
        want = exact(*case, i, turn)
        # to the nearest, but for the pairs of doubles' own errors (below 2^-94 of a sixth of a turn: 2^-32 units)
        assert abs(D(g) - want * 2 ** 64) <= D("0.5") + D(2) ** -30, (case, i)
        for pos in (1, -1, 12345, 2 ** 20, 2 ** 31 - 1, -2 ** 31):
            angle = D(((pos % 2 ** 64) * g % 2 ** 64) >> 32) / 2 ** 32        # as the kernels take it
            off = abs((angle - pos * want) % 1)                               # in (-1, 1), of the dividend's sign
            assert min(off, 1 - off) <= D(2) ** -31, (case, i, pos)
