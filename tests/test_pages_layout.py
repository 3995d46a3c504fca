"""The page container's own C++ (csrc/kvp_pages.cuh), compiled for the host and
called: the fixed-point frequencies, and the places of a block's bytes.  (No GPU
needed: nothing is launched.)"""
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

// the block's constants, then the place of every byte of every key and value row
template <int D, int FMT>
static void places() {
    using B = Block<D, FMT>;
    std::printf("%d %d %u %u %u %u %u %u %u %u\n", D, FMT, B::KROW, B::VROW, B::SROW, B::VSROW, B::OFF_V, B::OFF_KS, B::OFF_VS,
                B::BYTES);
    for (uint32_t t = 0; t < 16; ++t)
        for (uint32_t x = 0; x < B::KROW; ++x) std::printf("%u ", B::key(t, x));
    std::printf("\n");
    for (uint32_t t = 0; t < 16; ++t)
        for (uint32_t x = 0; x < B::VROW; ++x) std::printf("%u ", B::value(t, x));
    std::printf("\n");
}

int main(int argc, char **) {
    if (argc > 1) {
        places<64, 0>(), places<64, 1>(), places<64, 2>(), places<128, 0>(), places<128, 1>(), places<128, 2>();
        return 0;
    }
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


@pytest.fixture(scope="module")
def blocks(program):
    """{(head_dim, format): (constants, place[t][x] of keys, of values)}"""
    lines = subprocess.run([program, "places"], capture_output=True, text=True, check=True).stdout.splitlines()
    out = {}
    for i in range(0, len(lines), 3):
        d, fmt, krow, vrow, *rest = (int(x) for x in lines[i].split())
        names = ("srow", "vsrow", "off_v", "off_ks", "off_vs", "bytes")
        c = dict(zip(names, rest), krow=krow, vrow=vrow)
        out[d, fmt] = (c, np.array(lines[i + 1].split(), int).reshape(16, krow), np.array(lines[i + 2].split(), int).reshape(16, vrow))
    return out


CASES = [(d, f) for d in (64, 128) for f in (0, 1, 2)]


@pytest.mark.parametrize("case", CASES)
def test_sections_of_a_block(blocks, case):
    """Keys, values, key scales, value scales, one after the other, each byte once; a
    16-byte chunk stays together and its 128-byte line holds the same bytes."""
    d, fmt = case
    c, key, value = blocks[case]
    assert (c["krow"], c["vrow"]) == {0: (2 * d, 2 * d), 1: (d, d), 2: (d, d // 2)}[fmt]
    scales = 0 if fmt == 0 else 16 * c["srow"]
    assert c["off_v"] == 16 * c["krow"] and c["off_ks"] == c["off_v"] + 16 * c["vrow"] and c["off_vs"] == c["off_ks"] + scales
    assert c["bytes"] == c["off_vs"] + (0 if fmt == 0 else 16 * c["vsrow"]) and c["bytes"] % 16 == 0
    assert sorted(key.ravel()) == list(range(c["off_v"])) and sorted(value.ravel()) == list(range(c["off_v"], c["off_ks"]))
    for place, row, base in ((key, c["krow"], 0), (value, c["vrow"], c["off_v"])):
        plain = base + np.arange(16 * row).reshape(16, row)
        assert np.array_equal(place % 16, plain % 16)
        assert np.array_equal(place // 128, plain // 128)


def _banks_once(addresses, size):
    """Every shared-memory pass of a warp's load (32 lanes at 4 bytes, 16 at 8, 8 at
    16) touches every bank once."""
    per_pass = 128 // size
    for first in range(0, 32, per_pass):
        banks = [(int(a) // 4 + i) % 32 for a in addresses[first:first + per_pass] for i in range(size // 4)]
        assert sorted(banks) == list(range(32))


@pytest.mark.parametrize("case", CASES)
def test_attention_reads_no_bank_twice(blocks, case):
    """The loads of attention, lane (g, tig): 8-bit keys 16 bytes of token g at
    tig d / 4 (and the 16 after them, placed by the same exclusive or); values of
    tokens 2 tig and 2 tig + 1, the granule at g vrow / 8; 16-bit keys and values by
    ldmatrix, rows of 16 bytes of eight tokens at one place of the row."""
    d, fmt = case
    c, key, value = blocks[case]
    lanes = [(lane >> 2, lane & 3) for lane in range(32)]
    for half in (0, 8):
        if fmt:
            at = [key[g, tig * d // 4] + half * c["krow"] for g, tig in lanes]
            assert at == [key[g + half, tig * d // 4] for g, tig in lanes]  # a constant offset serves the second half
            _banks_once(at, 16)
            if d == 128:
                assert [a ^ 16 for a in at] == [key[g + half, tig * 32 + 16] for g, tig in lanes]
                _banks_once([a ^ 16 for a in at], 16)
            for odd in (0, 1):
                at = [value[2 * tig + odd, g * c["vrow"] // 8] + half * c["vrow"] for g, tig in lanes]
                assert at == [value[2 * tig + odd + half, g * c["vrow"] // 8] for g, tig in lanes]
                _banks_once(at, c["vrow"] // 8)
        else:
            for place in (key, value):
                for x in range(0, 2 * d, 16):
                    banks = sorted((int(place[t + half, x]) // 4 + i) % 32 for t in range(8) for i in range(4))
                    assert banks == list(range(32))
                    for k in range(0, 2 * d, 32):  # k-steps are an exclusive or of the first one's address
                        if x < 32:
                            assert all(int(place[t + half, x]) ^ k == place[t + half, x + k] for t in range(8))


@pytest.mark.parametrize("case", CASES)
def test_lane_quads_own_their_bytes(blocks, case):
    """What a lane stores or loads of a row at once (16 bytes, or 8 of a 32-byte row)
    lies together and on its size's boundary."""
    d, fmt = case
    c, key, value = blocks[case]
    for place, row in ((key, c["krow"]), (value, c["vrow"])):
        size = min(16, row // 4)
        for t in range(16):
            for x in range(0, row, size):
                assert place[t, x] % size == 0 and np.array_equal(place[t, x:x + size], place[t, x] + np.arange(size))
