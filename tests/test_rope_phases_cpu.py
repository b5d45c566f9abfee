"""Phases of rotary frequencies, to the last place."""

import math
import random
from fractions import Fraction

import pytest

import exact_attention_92_gb300 as fa
from oracle import rope as oracle


@pytest.fixture(scope="module", autouse=True)
def lib():
    from exact_attention_92_gb300 import build

    build.build()
    return fa.load()


def _frequencies():
    r = random.Random(0)
    out = [0.0, 1.0, -1.0, 7.25, 123456.789, -0.3, 2 * math.pi, math.pi, 1e-300, 5e-324, 2.0 ** 31, 2.0 ** 52 + 1, 1.8e19]
    out += [10000.0 ** (-2.0 * j / 128) for j in range(64)]
    out += [r.choice((-1, 1)) * math.ldexp(r.uniform(1, 2), r.randint(-80, 63)) for _ in range(2000)]
    return out


def test_phases_are_the_nearest():
    """f / (2 pi) modulo 1 in units of 2^-64, off by half a unit (and what five truncations at 2^-128 and three doubles of
    1 / (2 pi), off by 2^-164 of a frequency below 2^64, can add: 2^-95)."""
    freq = _frequencies()
    for f, p in zip(freq, fa.fa_rope_phases(freq)):
        assert 0 <= p < 1 << 64
        off = Fraction(f) * oracle._TURN - Fraction(p, 1 << 64)
        off -= round(off)
        assert abs(off) <= Fraction(1, 1 << 65) + Fraction(1, 1 << 95), f


def test_angles_at_far_positions():
    """The fraction of a turn at positions up to 2^32: off by |t| 2^-65, so 2^-33 at most where 2^-25 of a turn are promised
    in all (the kernel keeps 32 bits, 2^-32, as a float, 2^-26)."""
    freq = _frequencies()
    for f, p in zip(freq, fa.fa_rope_phases(freq)):
        for t in (1, 131071, -5, 2 ** 31 - 1, -2 ** 31, 2 ** 32 - 2):
            off = Fraction((p * t) % (1 << 64), 1 << 64) - t * Fraction(f) * oracle._TURN
            off -= round(off)
            assert abs(off) <= abs(t) * (Fraction(1, 1 << 65) + Fraction(1, 1 << 95)), (f, t)


def test_frequencies_of_any_size_are_taken():
    """Above 2^64 what is left of a turn means nothing; the call still answers."""
    for f in (1e30, 1.7e308, -1.7e308):
        assert 0 <= fa.fa_rope_phases([f])[0] < 1 << 64
