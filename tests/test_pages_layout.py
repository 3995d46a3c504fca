"""The page container's own C++ (csrc/kvp_pages.cuh), compiled for the host and
called: the fixed-point frequencies.  (No GPU needed: nothing is launched.)"""
import subprocess
from decimal import Decimal, getcontext
from fractions import Fraction

import numpy as np
import pytest

from agent_shared_compressed_gb300 import build as kvbuild

getcontext().prec = 150
INV_2PI = Fraction(1 / (2 * Decimal(
    "3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798214808651328230664709384460955")))

PROGRAM = r"""
#include <cstdio>
#include "kvp_pages.cuh"
using namespace kvp;
int main() {
    unsigned bits;
    while (std::scanf("%x", &bits) == 1) {
        float w;
        std::memcpy(&w, &bits, 4);
        std::printf("%016llx\n", (unsigned long long)turn_fraction(w));
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    at = tmp_path_factory.mktemp("layout")
    (at / "layout.cu").write_text(PROGRAM)
    cmd = [kvbuild.nvcc()] + kvbuild.ARCH + ["-std=c++17", "--expt-relaxed-constexpr", "-I", kvbuild.INCLUDE, "-I", kvbuild.CSRC,
                                             str(at / "layout.cu"), "-o", str(at / "layout")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return str(at / "layout")


def test_fixed_point_frequencies(program):
    """The 64-bit fraction of w / 2 pi is w / 2 pi mod 1 cut off, less 2^-64 at most
    for the end of 1 / 2 pi's 128 bits; with a position in 64-bit integers the turn
    is right to |position| 2^-64."""
    rng = np.random.default_rng(2)
    w = np.concatenate([
        np.array([0.0, 1.0, -1.0, 2.0 ** -149, 2.0 ** -126, 2.0 ** 59, -2.0 ** 59, 6.2831855, 0.5, 3.0], np.float32),
        np.array([500000.0 ** (-2.0 * i / 128) for i in range(64)], np.float32),
        np.array([10000.0 ** (-2.0 * i / 64) for i in range(32)], np.float32),
        (2.0 ** rng.uniform(-70, 60, 400) * rng.choice([-1, 1], 400)).astype(np.float32)])
    text = "\n".join("%08x" % b for b in w.view(np.uint32))
    got = [int(x, 16) for x in subprocess.run([program], input=text, capture_output=True, text=True, check=True).stdout.split()]
    assert len(got) == len(w)
    for x, f in zip(w, got):
        exact = Fraction(float(x)) * INV_2PI
        for pos in (1, 4095, 131071, (1 << 31) + 12345, -7):
            turn = Fraction((f * pos) % 2 ** 64, 2 ** 64)
            err = (turn - exact * pos) % 1
            assert min(err, 1 - err) <= Fraction(abs(pos), 2 ** 64), (x, pos)
