"""First tiles of a unit that are seen whole, where a row has no maximum yet: scores around 2^19 and 2^20, where a score's own
rounding begins to show, and far beyond.  Tolerance: see test_kv_chunk_gpu."""
import numpy as np
import pytest
import torch

from test_kv_attn_gpu import Case
from test_kv_chunk_gpu import TYPES, check, ops  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("log", [12, 17, 18, 19, 20, 21, 23, 26, 40])
@pytest.mark.parametrize("lens,rows,heads,kv,dim,block", [([260], [3], 4, 1, 64, 16), ([300, 4000], [130, 2], 2, 1, 128, 128),
                                                          ([200], [40], 2, 2, 256, 64)])
def test_large_scores_in_a_first_tile(ops, lens, rows, heads, kv, dim, block, log, dtype):  # noqa: F811
    c = Case(lens, rows, heads, kv, dim, block, seed=log + dim)
    top = np.abs(c.q).max() * 3 * dim * c.scale * 1.4427  # about a row's largest score, in powers of two
    check(ops, c, dtype, scale=c.scale * 2.0 ** log / top)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_a_first_tile_of_one_sign(ops, sign, dtype):  # noqa: F811
    """All scores far above or below zero."""
    c = Case([400], [9], 4, 1, 128, 64, seed=31)
    c.q = np.abs(c.q) * sign
    c.kc[c.kc < 0x7F] &= 0x3F
    c.kc[(c.kc >= 0x80) & (c.kc < 0xFF)] &= 0x3F
    check(ops, c, dtype, scale=c.scale * 3000)
