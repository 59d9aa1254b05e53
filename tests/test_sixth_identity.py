"""The many-rows norm computes the block-scale quotient a_b / 6 of a bf16 block
maximum in three fp32 operations: q = RN(a c), r = a - 6 q (one fma), RN(q + r c)
(one fma) with c = RN(1/6).  It equals the IEEE fp32 quotient for every bf16 value
of at least 2^-100; checked here for all of them in rational arithmetic."""
from fractions import Fraction

import numpy as np


def _round32(v: Fraction) -> Fraction:
    """Nearest fp32 value (ties to even) of a rational in the normal range."""
    if v == 0:
        return v
    sign, v = (-1, -v) if v < 0 else (1, v)
    e = v.numerator.bit_length() - v.denominator.bit_length()
    if Fraction(2) ** e > v:
        e -= 1
    assert -126 <= e <= 127
    unit = Fraction(2) ** (e - 23)
    n, rest = divmod(v, unit)
    half = unit / 2
    n += rest > half or (rest == half and n % 2 == 1)
    return sign * n * unit


def _exact(f) -> Fraction:
    return Fraction(float(f))


def _values():
    bits = np.arange(27 << 7, 0x7F80, dtype=np.uint32)       # 2^-100 .. the largest finite one
    return (bits << 16).view(np.float32)


def _sixth(a: Fraction, c: Fraction) -> Fraction:
    q = _round32(a * c)
    r = _round32(a - 6 * q)
    return _round32(r * c + q)


def test_three_operations_equal_the_quotient_for_all_bf16():
    c = _exact(np.float32(1.0) / np.float32(6.0))
    values = _values()
    assert _exact(values[0]) == Fraction(1, 2 ** 100)
    want = values / np.float32(6.0)
    for a, w in zip(values, want):
        assert _sixth(_exact(a), c) == _exact(w), float(a)


def test_without_the_correction_it_does_not():
    """Negative control: q alone rounds many values differently."""
    values = _values()
    assert np.count_nonzero(values * (np.float32(1.0) / np.float32(6.0)) != values / np.float32(6.0)) > 1000
