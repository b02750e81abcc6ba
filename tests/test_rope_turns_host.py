"""Frequencies as 64-bit fractions of a turn (no GPU), against exact rationals: round(2^64 f / 2 pi) mod 2^64 for the double f
as it is.  The host's two-part quotient is off by 2^-25 of a unit at most, so the two differ (by one) only that close to a tie."""
from fractions import Fraction

import numpy as np
import pytest

DIGITS = 10 ** 90


def two_pi() -> Fraction:
    """Machin's formula, in integers."""
    def atan_inverse(n):
        t = DIGITS // n
        total, k, sign = t, 3, -1
        while t:
            t //= n * n
            total += sign * (t // k)
            k, sign = k + 2, -sign
        return total
    return Fraction(8 * (4 * atan_inverse(5) - atan_inverse(239)), DIGITS)


TWO_PI = two_pi()


@pytest.fixture(scope="module")
def ops():
    from fp8_block_scaled_fp8blk_gb300 import build
    build.build()
    from fp8_block_scaled_fp8blk_gb300 import ops as o
    return o


def cases(ops):
    rng = np.random.default_rng(5)
    for rot in (2, 20, 64, 128, 1024):
        for base in (10000.0, 500000.0, 1.5):
            yield ops.rope_frequencies(rot, base)[0]
        yield ops.rope_frequencies(rot, 10000.0, "ramp", factor=16.0, original_len=4096.0)[0]
    yield np.array([0.0, 1.0, -1.0, 0.5, 2 * np.pi, -2 * np.pi, np.pi, 1e6, -1e6, 1e-12, -1e-12, 1e-19, 5e-324, -5e-324, 1e-300])
    yield rng.uniform(-10, 10, 512)
    yield rng.uniform(-1e6, 1e6, 512)
    yield 10.0 ** rng.uniform(-25, 6, 512) * rng.choice([-1, 1], 512)
    yield np.nextafter(np.arange(1, 400) * 2 * np.pi, 0.0)  # just below whole turns


def test_turns_are_rounded_once(ops):
    for freqs in cases(ops):
        turns = ops.rope_turns(freqs, "cpu").numpy().view(np.uint64)
        for f, t in zip(freqs, turns):
            exact = abs(Fraction(float(f))) / TWO_PI * 2 ** 64  # (ties and signs: half away from zero)
            want = int(exact + Fraction(1, 2))
            got = int(t) if f >= 0 else -int(t) % 2 ** 64
            if (got - want) % 2 ** 64:
                tie = abs(exact - int(exact) - Fraction(1, 2))
                assert tie < Fraction(1, 2 ** 25) and (got - want + 1) % 2 ** 64 in (0, 2), (f, got, want)


def test_a_negative_frequency_is_the_positive_ones_negative(ops):
    freqs = 10.0 ** np.random.default_rng(6).uniform(-12, 6, 500)
    a, b = (ops.rope_turns(s * freqs, "cpu").numpy().view(np.uint64) for s in (1.0, -1.0))
    assert not (a + b).any()
