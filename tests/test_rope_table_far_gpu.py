"""The table of cosines and sines at far positions: the wanted angle comes from the integer turns themselves, so no tolerance
grows with the position.  Both are within 2^-23 of the exact value before the scale, whose product rounds once more:
scale x (2^-23 + 2^-24); turns are within 2^-64 (half a unit, and 2^-25 of one) of the frequency, so that the last position's
phase is within 2^-33 of a turn, 7.4e-10 rad."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from _helpers import to_dev
from test_rope_gpu import ops  # noqa: F401
from test_rope_turns_host import TWO_PI

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
POSITIONS = np.array([0, 1, 2, 7, 4095, 131071, 2 ** 20 - 1, 2 ** 24 + 1, 10 ** 9 + 7, 2 ** 30, 2 ** 31 - 2, 2 ** 31 - 1], np.int32)


@pytest.mark.parametrize("rot", [2, 20, 128, 1024])
@pytest.mark.parametrize("base,scale", [(10000.0, 1.0), (500000.0, 1.2707), (1.5, 1.0)])
def test_far_positions(ops, rot, base, scale):  # noqa: F811
    freqs, _ = ops.rope_frequencies(rot, base)
    turns = ops.rope_turns(freqs, "cpu")
    got = ops.fp8blk_rope_table(to_dev(POSITIONS), turns.to(DEV), scale).cpu().numpy().astype(np.float64)
    phase = POSITIONS.astype(object)[:, None] * turns.numpy().view(np.uint64).astype(object)[None] % 2 ** 64
    signed = np.where(phase >= 2 ** 63, phase - 2 ** 64, phase).astype(np.float64)
    angle = signed * (2 * np.pi / 2.0 ** 64)  # within half a turn: 2^-51 of error
    want = np.stack([np.cos(angle), np.sin(angle)], 1) * float(np.float32(scale))
    assert (np.abs(got - want) <= scale * (2.0 ** -23 + 2.0 ** -24)).all(), np.abs(got - want).max()
    # ... and against the frequencies themselves, in exact rationals.
    for i in (0, len(freqs) // 3, len(freqs) - 1):
        exact = [Fraction(float(freqs[i])) * int(p) / TWO_PI % 1 for p in POSITIONS]
        off = [abs((Fraction(int(x), 2 ** 64) - e + Fraction(1, 2)) % 1 - Fraction(1, 2)) for x, e in zip(phase[:, i], exact)]
        assert max(off) <= Fraction(1, 2 ** 33)
