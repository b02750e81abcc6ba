"""Plain 64-bit restatements (numpy) of the rotary positions, for the tests.  Nothing here uses the package."""
import math

import numpy as np


def frequencies(rot, base=10000.0, scaling="plain", factor=1.0, original=0.0, low=1.0, high=32.0):
    """Radians a token, from the formulas of the header."""
    half = rot // 2
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    f = np.array([base ** (-2.0 * i / rot) for i in range(half)])
    if scaling in ("plain", "base"):
        return f, 1.0
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "ramp":
        at = [rot * math.log(original / (t * 2 * math.pi)) / (2 * math.log(base)) for t in (high, low)]
        a, b = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        r = np.clip((np.arange(half) - a) / max(b - a, 0.001), 0.0, 1.0)
        return f / factor * r + f * (1 - r), 0.1 * math.log(factor) + 1.0
    turns = original * f / (2 * math.pi)
    keep = np.clip((turns - low) / (high - low), 0.0, 1.0)
    return f / factor * (1 - keep) + f * keep, 1.0


def rotate(x, cos, sin, interleaved, start):
    """(rotated x, |a c| + |b s| of every value) for x [n, heads, dim], cos and sin [n, rot / 2], all in 64 bits."""
    half = cos.shape[1]
    i = np.arange(half)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    a, b = x[:, :, start + first], x[:, :, start + second]
    c, s = cos[:, None], sin[:, None]
    y, size = x.copy(), np.abs(x)
    y[:, :, start + first], y[:, :, start + second] = a * c - b * s, b * c + a * s
    size[:, :, start + first] = np.abs(a * c) + np.abs(b * s)
    size[:, :, start + second] = np.abs(b * c) + np.abs(a * s)
    return y, size
