"""CPU pins of the 4-bit cache's scales in the oracle against rational arithmetic, where
a spread is no 64-bit number or code 15 stands next to the type's largest one."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import quantised as Q


def scale_of(low, high, dt):
    """The smallest number s of the type with 15 s >= high - low, or the one below it where
    15 s + low passes the type's largest."""
    def below(s):
        return s - float(Q.step(s * (1 - 2.0 ** -20), dt))
    span = Fraction(high) - Fraction(low)
    s = float(Q.rounded(float(span / 15), dt))
    while 15 * Fraction(s) < span:
        s += float(Q.step(s, dt))
    while s > 0 and 15 * Fraction(below(s)) >= span:
        s = below(s)
    return below(s) if 15 * Fraction(s) + Fraction(low) > Fraction(Q._MAX[dt]) else s


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_scales_are_those_of_rational_arithmetic(dt):
    rng = np.random.default_rng(0)
    big, smallest, largest = Q._MAX[dt], (-24 if dt == "f16" else -130), (14 if dt == "f16" else 119)
    highs = [15.0, 15.9375, 30.0, big, 255 * 2.0 ** (120 if dt == "bf16" else 8)]
    for _ in range(1500):
        high = float(Q.rounded(rng.choice(highs + [rng.random() * 100]), dt))
        low = float(Q.rounded(rng.choice([-1.0, 0.0, 1.0]) * 2.0 ** rng.integers(smallest, largest), dt))
        low, high = min(low, high), max(low, high)
        x = np.full(64, low)
        x[3] = high
        _, s, m = Q.quantise(x, dt)
        assert s == scale_of(low, high, dt) and m == low


@pytest.mark.parametrize("dt,least", [("f16", 2.0 ** -24), ("bf16", 2.0 ** -133)])
def test_groups_of_the_smallest_numbers(dt, least):
    """Spreads below 15 of the smallest number have the smallest scale, not none."""
    assert Q.step(0.0, dt) == least and Q.step(least, dt) == least
    for high, low in ((1, 0), (1, -1), (15, 0), (16, 0), (3, -3), (0, 0)):
        x = np.full(64, low * least)
        x[5] = high * least
        c, s, m = Q.quantise(x, dt)
        assert s == -(-(high - low) // 15) * least and m == low * least
        assert np.array_equal(Q.values(c[None], s[None], m[None])[0], x) or high - low > 15
