"""Arithmetic and layout that the page kernels rely on, checked on the CPU over
every value they can see (no GPU needed): the in-register expansions of codes,
the rotation's fixed-point angles, the integer nearest to a group's zero, and
the byte order of a block."""
import struct
from decimal import Decimal, getcontext
from fractions import Fraction

import numpy as np
import pytest

getcontext().prec = 120
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798214808651")
INV_2PI = Fraction(1 / (2 * PI))


def _bf16(bits):
    return (np.asarray(bits, np.uint32) << 16).view(np.float32)


def test_byte_to_fp16_code():
    """0x6400 | u is 1024 + u in fp16; less 1152 it is u - 128 exactly."""
    u = np.arange(256, dtype=np.uint16)
    x = (u | np.uint16(0x6400)).view(np.float16)
    got = x - np.uint16(0x6480).view(np.float16)
    assert np.array_equal(got.astype(int), u.astype(int) - 128)


def test_byte_to_bf16_code():
    """(u & 0x7F) | 0x4300 plus (u & 0x80) ^ 0xC380, both bf16, is u - 128, which
    bf16 holds exactly."""
    u = np.arange(256, dtype=np.uint32)
    s = _bf16((u & 0x7F) | 0x4300).astype(np.float64) + _bf16((u & 0x80) ^ 0xC380)
    assert np.array_equal(s, u.astype(np.float64) - 128)
    assert np.all(s.astype(np.float32).view(np.uint32) & 0xFFFF == 0)


def test_nibble_to_bf16_code():
    """q | 0x4300 plus -(128 + c): q - c for every nibble and every c, with c's
    bias exact in bf16."""
    q, c = np.meshgrid(np.arange(16), np.arange(16))
    bias = np.float32(-128) - c.astype(np.float32)
    assert np.all(bias.view(np.uint32) & 0xFFFF == 0)
    s = _bf16(q.astype(np.uint32) | 0x4300).astype(np.float64) + bias
    assert np.array_equal(s, (q - c).astype(np.float64))


def test_zero_of_a_group_does_not_cancel():
    """With c the integer of [0, 15] nearest to -z / s, the code term (q - c) s is
    within 3 |v| wherever the remainder z + c s is not the whole value, for any
    fp16 scale and zero point, and one-sided groups add terms of one sign."""
    rng = np.random.default_rng(0)
    s = (2.0 ** rng.uniform(-20, 10, 20000)).astype(np.float16).astype(np.float64)
    z = (-s * rng.uniform(-40, 60, 20000)).astype(np.float16).astype(np.float64)
    q = np.arange(16)[:, None]
    c = np.clip(np.rint(-z / s), 0, 15)
    v, term, rest = q * s + z, (q - c) * s, z + c * s
    inside = (-z / s > 0) & (-z / s < 15)
    assert np.all(np.abs(rest[inside]) <= 0.5 * s[inside] * (1 + 1e-12))
    assert np.all((np.abs(term) <= 3 * np.abs(v) * (1 + 1e-9)) | (term == 0))
    outside = ~inside & (np.abs(rest) > 0.5 * s)
    assert np.all((term * rest)[:, outside] >= 0)


def test_fixed_point_angles():
    """position * W mod 2^64, W the 64-bit fraction of w / 2 pi from 128 bits of
    1 / 2 pi: the turn is right to position * 2^-63 at far positions."""
    hi_lo = int(INV_2PI * 2 ** 128)
    assert hi_lo == (0x28be60db9391054a << 64) | 0x7f09d5f47d4d3770
    rng = np.random.default_rng(1)
    for _ in range(300):
        w = np.float32(2.0 ** rng.uniform(-40, 3))
        bits = struct.unpack("<I", struct.pack("<f", w))[0]
        m, e = (bits & 0x7FFFFF) | 0x800000, (bits >> 23) - 150
        p, shift = m * hi_lo, 64 - e
        turn = (p >> shift if shift >= 0 else p << -shift) & (2 ** 64 - 1)
        for pos in (0, 1, 4095, 131071, int(rng.integers(1 << 31)), -7):
            got = Fraction((turn * pos) % 2 ** 64, 2 ** 64)
            want = (Fraction(float(w)) * INV_2PI * pos) % 1
            err = abs(got - want)
            assert min(err, 1 - err) <= Fraction(abs(pos) + 1, 2 ** 63)


def _value_offset(t, x, row):
    at = t * row + x
    if row == 32:
        return at ^ (((t >> 2) & 1) << 5)
    return at ^ (((t >> 1) & 3) << 5)


@pytest.mark.parametrize("row", [32, 64, 128])
def test_value_rows_fall_on_distinct_banks(row):
    """A lane's granule (row / 8 bytes) of tokens 2 tig + k: the lanes that one
    shared-memory pass serves (32 at 4 bytes, 16 at 8, 8 at 16) touch every bank
    once; and a block's bytes are a permutation."""
    gran = row // 8
    lanes = 128 // gran
    for k in (0, 1, 8, 9):
        for first in range(0, 32, lanes):
            banks = set()
            for lane in range(first, first + lanes):
                g, tig = lane >> 2, lane & 3
                at = _value_offset(2 * tig + k, g * gran, row)
                banks |= {(at // 4 + i) % 32 for i in range(gran // 4)}
            assert len(banks) == 32
    seen = {_value_offset(t, x, row) for t in range(16) for x in range(row)}
    assert seen == set(range(16 * row))


def test_key_rows_fall_on_distinct_banks():
    """8-bit keys at head_dim 128: 16 bytes of token g at 32 tig (and at 32 tig +
    16), eight lanes a pass."""
    for x in (0, 16):
        for first in range(0, 32, 8):
            banks = set()
            for lane in range(first, first + 8):
                g, tig = lane >> 2, lane & 3
                at = (g * 128 + tig * 32) ^ ((g & 1) << 4) ^ x
                banks |= {(at // 4 + i) % 32 for i in range(4)}
            assert len(banks) == 32
