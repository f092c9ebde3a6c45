"""The fixed-point turns of ``api.Rope`` against 400-bit integers: pi by Machin's
series, powers of the base by integer roots."""

import math
from fractions import Fraction

import pytest

from tree_verify_attention_gb300 import api

BITS = 400
ONE = 1 << BITS


def arctan_of_inverse(n):
    total = term = ONE // n
    k = 1
    while term:
        term //= n * n
        k += 2
        total += -(term // k) if k % 4 == 3 else term // k
    return total


TWO_PI = 8 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239))


def power(base, pairs, i):
    """base ** (-i / pairs), pairs a power of two from 8 on, in units of 2^-BITS."""
    f = Fraction(base)
    root = ONE * f.denominator // f.numerator
    while pairs > 1:
        root = math.isqrt(root * ONE)
        pairs //= 2
    out = ONE
    for _ in range(i):
        out = out * root // ONE
    return out


@pytest.mark.parametrize("base,rot", [(1e4, 64), (1e6, 256), (1e6, 64), (5e5, 128), (1e7, 256),
                                      (10000, 32), (500000.5, 16), (1.0, 16), (0.5, 32)])
def test_turns_of_a_base(base, rot):
    """To the nearest 2^-64 of a turn (the integers here are off by 2^-380)."""
    pairs = rot // 2
    got = api.Rope(256, rot, base=base, device="cpu").turns.tolist()
    assert len(got) == pairs
    for i, t in enumerate(got):
        want = power(base, pairs, i) * 2 ** 64 * 2 // TWO_PI      # in halves of 2^-64
        off = (2 * t - want + 2 ** 64) % 2 ** 65 - 2 ** 64
        assert -1 <= off <= 1, (i, off)


def test_bases_that_are_none():
    for base in (0.0, -1.0, -1e4, math.nan):
        with pytest.raises(api.DfvError, match="base"):
            api.Rope(64, base=base, device="cpu")
    assert api.Rope(64, 0, device="cpu").turns.numel() == 0
    # an infinite base turns the first pair alone
    t = api.Rope(64, base=math.inf, device="cpu").turns
    assert t[0] != 0 and not t[1:].any()


def test_turns_of_given_frequencies():
    """Doubles, divided as such: 2^-52 of a frequency, and the fraction's cut."""
    freq = [1e6 ** (-i / 128) for i in range(128)]
    got = api.Rope(256, inv_freq=freq, device="cpu").turns.tolist()
    for f, t in zip(freq, got):
        want = Fraction(f) * ONE / TWO_PI
        assert abs(Fraction(t, 1 << 64) - want) <= want / 2 ** 52 + Fraction(1, 1 << 64)
