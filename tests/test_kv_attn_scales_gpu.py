"""GPU tests of fp8blk_kv_attn where the value scales of one tile of 128 tokens lie far apart.

The bound is check's (test_kv_attn_gpu.py).  It is relative to sum_t p_t |v_t| of the row itself, so a block that the row
does not attend to may not cost it anything, whatever that block's scale."""
import math

import numpy as np
import pytest
import torch

import _step_ref as ref
from test_kv_attn_gpu import Case, check, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from fp8_block_scaled_fp8blk_gb300 import ops as o
    yield o
    assert o.fp8blk_device_status(clear=True) == 0


def quiet_block(e, block, heads, rows, dim, seed):
    """In each tile one block has value scales 2^-e of the others' and all of the rows' weight: its scores are the others'
    and a gap of e ln 2 + 12, so the others keep e^-12 of the output."""
    c = Case([300], [rows], heads, 1, dim, block, seed=seed, spread=0)
    rng = np.random.default_rng(seed)
    c.q = (0.5 + 0.1 * rng.standard_normal(c.q.shape)).astype(np.float32)
    gap = e * math.log(2.0) + 12.0
    for j, b in enumerate(c.table[0]):
        c.vs[b] = 1.0
        if j % (128 // block) == 1:
            c.vs[b] = 2.0 ** -e
            c.kc[b] = ref.e4m3_encode(64.0 * (1.0 + 0.1 * rng.standard_normal(c.kc[b].shape)))
            c.ks[b] = gap / (64.0 * 0.5 * dim * c.scale)
    return c


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("heads,rows,dim", [(4, 2, 64), (8, 2, 64), (8, 4, 64), (16, 4, 128), (4, 2, 256), (8, 2, 192)])
@pytest.mark.parametrize("block", [16, 32, 64])
@pytest.mark.parametrize("e", [4, 8, 12, 16, 20, 40, 100])
def test_weight_on_a_block_of_small_scale(ops, dtype, heads, rows, dim, block, e):
    check(ops, quiet_block(e, block, heads, rows, dim, seed=e + block + dim), dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("heads", [4, 16])
def test_every_sixteen_tokens_their_own_scale(ops, dtype, heads):
    """Rows that attend to different blocks of one tile, each of another scale."""
    c = Case([384], [8], heads, 2, 64, 16, seed=31, spread=0)
    rng = np.random.default_rng(32)
    c.vs[c.table[0]] = (2.0 ** rng.integers(-45, 45, (24, 2))).astype(np.float32)
    c.q *= 8.0
    check(ops, c, dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scale", [2.0 ** 30, 2.0 ** 100, 2.0 ** -60, 0.0])
def test_scale_of_a_block_that_rows_do_not_see(ops, dtype, scale):
    """Rows before a block are the same bits whatever its scale."""
    c = Case([114], [4], 8, 2, 64, 16, seed=33, spread=0)  # rows at 110 .. 113, the last block begins at 112
    c.vs[c.table[0]] = 1.0
    want, lse, _ = run(ops, c, dtype)
    c.vs[c.table[0, 7]] = scale
    out, lse2, _ = run(ops, c, dtype)
    assert torch.equal(out[:2], want[:2]) and torch.equal(lse2, lse)
    check(ops, c, dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("heads,block", [(4, 16), (16, 64), (16, 128)])
def test_scales_that_are_not_finite(ops, dtype, value, heads, block):
    """They count as NaN: the rows that see the block are NaN in that cache head, all others the same bits."""
    c = Case([258, 40], [4, 1], heads, 2, 64, block, seed=41)  # rows at 254 .. 257; a block begins at 256
    want, lse, _ = run(ops, c, dtype)
    page = 256 // block
    for scales in (c.ks, c.vs):
        for j, first in ((0, 0), (page, 2)):                    # a block that every row sees; one that two rows see
            b = c.table[0, j]
            kept = scales[b, 1]
            scales[b, 1] = value
            out, lse2, _ = run(ops, c, dtype)
            scales[b, 1] = kept
            bad = out[first:4, heads // 2:]
            assert torch.isnan(bad).all()
            bad.copy_(want[first:4, heads // 2:])
            assert torch.equal(out, want)
            if scales is c.ks:
                assert torch.isnan(lse2[first:4, heads // 2:]).all()
                lse2[first:4, heads // 2:] = lse[first:4, heads // 2:]
            assert torch.equal(lse2, lse)
    assert ops.fp8blk_device_status(clear=True) == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [1e3, 1e8, 1e14])
@pytest.mark.parametrize("e", [12, 30, 90])
@pytest.mark.parametrize("heads,block", [(4, 16), (16, 64)])
def test_huge_scores_on_a_block_of_small_scale(ops, dtype, size, e, heads, block):
    """Scores of up to 1e14: one token of a block of value scale 2^-e has all the weight, so the output is its value, to what
    a weight of one keeps (a power of two: both planes hold it, 2^-20 of the sums)."""
    c = Case([200], [2], heads, 1, 64, block, seed=61, spread=0)
    rng = np.random.default_rng(62)
    at = {0: 37, 1: 171}                                    # the token of each tile that can win; the second one does
    c.vs[c.table[0]] = 1.0
    for tile, t in at.items():
        b, r = c.table[0, t // block], t % block
        c.vs[b] = 2.0 ** -e
        c.kc[b, 0, r] = ref.e4m3_encode(np.full(64, 448.0 if tile else 352.0))
        c.ks[b] = c.ks[c.table[0]].max()
    for b in c.table[0]:                                    # all others: below a quarter of it
        keep = c.kc[b, 0].copy()
        low = ref.E4M3[keep] * 0.2
        for t in at.values():
            if b == c.table[0, t // block]:
                low[t % block] = ref.E4M3[keep[t % block]]
        c.kc[b, 0] = np.where(keep & 0x7F == 0x7F, keep, ref.e4m3_encode(low))
    c.ks[c.table[0]] = c.ks[c.table[0]].max()
    c.q[:] = size / (448.0 * c.ks[c.table[0, 0], 0] * 64 * c.scale) * (1.0 + 0.02 * rng.standard_normal(c.q.shape))
    out, lse, q = run(ops, c, dtype)
    b, r = c.table[0, 171 // block], 171 % block
    want = ref.E4M3[c.vc[b, 0, r]] * 2.0 ** -e
    got = out.float().cpu().numpy().astype(np.float64)
    bound = (2.0 ** -8 if dtype is torch.bfloat16 else 2.0 ** -16) * np.abs(want) + 2.0 ** -20 * 448.0 * 2.0 ** -e
    assert (np.abs(got - want) <= bound).all(), float((np.abs(got - want) / bound).max())
