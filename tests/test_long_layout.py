"""4-bit keys in the page container's own C++ (csrc/kvp_pages.cuh), compiled for the
host and called, and the arithmetic that attention expands them by (no GPU needed)."""
import subprocess

import numpy as np
import pytest

from agent_shared_compressed_gb300 import build as kvbuild
from test_pages_layout import PROGRAM, _banks_once


@pytest.fixture(scope="module")
def blocks(tmp_path_factory):
    """{head_dim: (constants, place[t][x] of keys, of values)} of the 4-bit format."""
    at = tmp_path_factory.mktemp("layout4")
    (at / "layout.cu").write_text(PROGRAM.replace("places<64, 0>()", "places<64, 4>(), places<128, 4>(), places<64, 0>()"))
    cmd = [kvbuild.nvcc()] + kvbuild.ARCH + ["-std=c++17", "--expt-relaxed-constexpr", "-I", kvbuild.INCLUDE, "-I", kvbuild.CSRC,
                                             str(at / "layout.cu"), "-o", str(at / "layout")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    lines = subprocess.run([str(at / "layout"), "places"], capture_output=True, text=True, check=True).stdout.splitlines()
    out = {}
    for i in (0, 3):
        d, fmt, krow, vrow, *rest = (int(x) for x in lines[i].split())
        assert fmt == 4
        c = dict(zip(("srow", "vsrow", "off_v", "off_ks", "off_vs", "bytes"), rest), krow=krow, vrow=vrow)
        out[d] = (c, np.array(lines[i + 1].split(), int).reshape(16, krow), np.array(lines[i + 2].split(), int).reshape(16, vrow))
    return out


@pytest.mark.parametrize("d", [64, 128])
def test_sections_of_a_block(blocks, d):
    """Keys, values, key scales and zero points, value scales and zero points: each byte
    once, 16-byte chunks together and within their 128-byte line."""
    c, key, value = blocks[d]
    assert (c["krow"], c["vrow"], c["srow"], c["vsrow"]) == (d // 2, d // 2, d // 8, d // 8)
    assert c["off_v"] == 8 * d and c["off_ks"] == 16 * d and c["off_vs"] == 18 * d and c["bytes"] == 20 * d
    assert sorted(key.ravel()) == list(range(c["off_v"])) and sorted(value.ravel()) == list(range(c["off_v"], c["off_ks"]))
    for place, base in ((key, 0), (value, c["off_v"])):
        plain = base + np.arange(8 * d).reshape(16, d // 2)
        assert np.array_equal(place % 16, plain % 16) and np.array_equal(place // 128, plain // 128)


@pytest.mark.parametrize("d", [64, 128])
def test_attention_reads_no_bank_twice(blocks, d):
    """A lane's d / 8 bytes of a key row of tokens g and g + 8, and its value granules."""
    c, key, value = blocks[d]
    lanes = [(lane >> 2, lane & 3) for lane in range(32)]
    for half in (0, 8):
        at = [key[g, tig * d // 8] + half * c["krow"] for g, tig in lanes]
        assert at == [key[g + half, tig * d // 8] for g, tig in lanes]
        _banks_once(at, d // 8)
        for odd in (0, 1):
            at = [value[2 * tig + odd, g * c["vrow"] // 8] + half * c["vrow"] for g, tig in lanes]
            assert at == [value[2 * tig + odd + half, g * c["vrow"] // 8] for g, tig in lanes]
            _banks_once(at, c["vrow"] // 8)


def test_nibbles_as_fp16_subnormals():
    """Nibble j of both halves, masked where it lies after a shift by whole bytes, is the
    code times 2^-24 (j even) or 2^-20 (j odd) as fp16."""
    for j in range(4):
        for code in range(16):
            half = np.uint16(code << (4 * j) | (0xA5A5 & ~(15 << (4 * j))))
            kept = np.uint16((int(half) >> (8 * (j // 2))) & (0x00F0 if j % 2 else 0x000F))
            assert float(kept.view(np.float16)) == code * 2.0 ** (-20 if j % 2 else -24)


def test_query_sums_as_three_fp16():
    """A group's sum of 32 elements below 2^15, times 2^-6, is three fp16 to 2^-25, the
    least fp16's half step."""
    rng = np.random.default_rng(0)
    s = np.concatenate([rng.uniform(-2.0 ** 20, 2.0 ** 20, 4000), rng.standard_normal(4000) * 2.0 ** rng.integers(-20, 20, 4000),
                        [0.0, 2.0 ** 20, -(2.0 ** 20)]]).astype(np.float32) * np.float32(2.0 ** -6)
    left = s.copy()
    total = np.zeros(len(s))
    for _ in range(3):
        part = left.astype(np.float16)
        assert np.all(np.isfinite(part))
        total += part.astype(np.float64)
        left -= part.astype(np.float32)
    assert np.all(np.abs(total - s) <= 2.0 ** -25)
