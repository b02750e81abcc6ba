"""GPU tests of fp8blk_kv_append with tokens enough (9728 (token, head) pairs and more) for its prompt kernel: whole CTAs on
one run at a time, values staged in shared memory, chunks of 16 to 64 tokens.  Compared with plain loops bit for bit."""
import numpy as np
import pytest
import torch

import _step_ref as ref
from _helpers import to_dev
from test_kv_cache_gpu import random_pool, slots_for

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from fp8_block_scaled_fp8blk_gb300 import ops as o
    yield o
    assert o.fp8blk_device_status(clear=True) == 0


def check(ops, ctx, new, heads, dim, block, dtype, seed, poison=False, skip=False, pad=0):
    """K and V are slices of one projection (pad: further columns of it) in `dtype`."""
    rng = np.random.default_rng(seed)
    blocks = sum(-(-(c + f) // block) for c, f in zip(ctx, new)) + 2
    slots = slots_for(ctx, new, block, blocks, rng)
    n = len(slots)
    assert n * heads >= 9728
    both = rng.standard_normal((n, 2 * heads + pad, dim)).astype(np.float32)
    both *= (2.0 ** rng.integers(-8, 9, (n, 2 * heads + pad, 1))).astype(np.float32)
    if poison:  # rows with NaN and infinities, and rows of nothing else
        for t in rng.integers(0, n, n // 20):
            h, d = rng.integers(0, 2 * heads), rng.integers(0, dim)
            both[t, h, d] = rng.choice([np.nan, np.inf, -np.inf])
            both[t, h, :] = rng.choice([np.nan, np.inf]) if rng.random() < 0.2 else both[t, h, :]
        both[:block, 0] = np.nan  # a whole run, or a part of two
        both[: 2 * block, 1, 0] = 0.0
    if skip:  # whole runs, their first tokens or their last ones: what is left of a block's run is one run
        first = np.nonzero(np.append(True, (slots[1:] != slots[:-1] + 1) | (slots[1:] % block == 0)))[0]
        for a, b in zip(first, np.append(first[1:], n)):
            cut = rng.integers(a, b + 1)
            if rng.random() < 0.3:
                slots[a:cut] = -1
            elif rng.random() < 0.3:
                slots[cut:b] = -1
    x = to_dev(both).to(dtype)
    k, v = x[:, :heads], x[:, heads: 2 * heads]
    kc, ks = random_pool(rng, blocks, heads, block, dim)
    vc, vs = random_pool(rng, blocks, heads, block, dim)
    dev = [to_dev(a) for a in (kc, ks, vc, vs)]
    ops.fp8blk_kv_append(k, v, to_dev(slots), *dev)
    assert ops.fp8blk_device_status(clear=True) == 0
    for y, codes, scales, gc, gs in ((k, kc, ks, dev[0], dev[1]), (v, vc, vs, dev[2], dev[3])):
        wc, ws = ref.kv_append(y.float().cpu().numpy().astype(np.float64), slots, codes, scales, block)
        assert np.array_equal(gs.cpu().numpy().astype(np.float64), ws)
        assert ref.same_codes(gc.cpu().numpy(), wc)


DTYPES = [torch.float32, torch.bfloat16]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("ctx,new,heads,dim,block", [
    ([0], [1300], 8, 128, 64),                 # one prompt
    ([37], [1300], 8, 128, 64),                # ... behind a partly filled block
    ([0, 5], [700, 611], 8, 256, 128),         # f32: a run does not fit the staging buffer, its tail does
    ([100, 0, 63, 64], [900, 1100, 640, 3], 16, 64, 64),
    ([3], [5003], 8, 48, 32),                  # chunks of 64 tokens, runs of 32
    ([120, 0], [2600, 2501], 8, 32, 128),      # runs of two chunks
    ([9], [9999], 1, 80, 16),                  # one head, four runs a chunk
    ([0], [2432], 4, 16, 128),
    ([15], [620], 16, 192, 64),
])
def test_prompts(ops, dtype, ctx, new, heads, dim, block):
    check(ops, ctx, new, heads, dim, block, dtype, seed=sum(new) + dim)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,most,heads,dim,block", [(700, 3, 16, 32, 16), (1500, 1, 8, 64, 64), (400, 40, 4, 32, 16),
                                                    (150, 30, 16, 64, 32)])
def test_many_short_runs(ops, dtype, n, most, heads, dim, block):
    """Four leaders and more in a chunk (a warp a run) beside chunks of fewer."""
    rng = np.random.default_rng(n)
    new = rng.integers(1, most + 1, n)
    check(ops, rng.integers(0, 2 * block, n), new, heads, dim, block, dtype, seed=n, pad=1)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("ctx,new,heads,dim,block", [([0], [1300], 8, 128, 64), ([70, 9], [800, 700], 8, 256, 128),
                                                     ([3], [2500], 4, 64, 16), ([50] * 120, [21] * 120, 4, 32, 32)])
def test_values_that_are_not_finite_and_skipped_tokens(ops, dtype, ctx, new, heads, dim, block):
    check(ops, ctx, new, heads, dim, block, dtype, seed=7, poison=True, pad=2)
    check(ops, ctx, new, heads, dim, block, dtype, seed=8, poison=True, skip=True)


@pytest.mark.parametrize("dtype", DTYPES)
def test_few_tokens_that_are_not_finite(ops, dtype):
    """The decode kernel on the same: runs of one to forty tokens, bf16 as well."""
    rng = np.random.default_rng(11)
    ctx, new = [0, 5, 16, 31, 40], [1, 3, 40, 1, 17]
    blocks = 20
    slots = slots_for(ctx, new, 16, blocks, rng)
    x = rng.standard_normal((len(slots), 2, 64)).astype(np.float32) * np.float32(30.0)
    x[0, 0, 3], x[2, 1, 5], x[10, 0, 0], x[20, 1, 63], x[25, 0] = np.inf, np.nan, -np.inf, np.inf, np.nan
    x[43:46] = np.inf
    d = to_dev(x).to(dtype)
    kc, ks = random_pool(rng, blocks, 2, 16, 64)
    dev = [to_dev(a) for a in (kc, ks, kc, ks)]
    ops.fp8blk_kv_append(d, -d, to_dev(slots), *dev)
    for y, gc, gs in ((d, dev[0], dev[1]), (-d, dev[2], dev[3])):
        wc, ws = ref.kv_append(y.float().cpu().numpy().astype(np.float64), slots, kc, ks, 16)
        assert np.array_equal(gs.cpu().numpy().astype(np.float64), ws) and ref.same_codes(gc.cpu().numpy(), wc)


@pytest.mark.parametrize("n,heads,block,blocks", [(4, 1, 16, 3), (64, 8, 64, 70), (3000, 8, 16, 700), (3000, 1, 128, 20),
                                                  (200, 2, 16, 600000)])
def test_two_runs_in_one_block_are_flagged(ops, n, heads, block, blocks):
    """Rows out of order, tokens of two requests in turn, a token skipped inside a block, one slot twice; near and far apart,
    in the first and the last blocks of a pool.  The same tokens in order raise nothing."""
    shape = (blocks, heads, block, 16)
    dev = [torch.zeros(shape, dtype=torch.uint8, device="cuda:0"), torch.zeros(shape[:2], device="cuda:0")]
    dev += [torch.zeros_like(t) for t in dev]
    x = torch.ones((n, heads, 16), device="cuda:0")
    span = min(n, blocks * block)
    good = np.full(n, -1, np.int64)
    good[:span] = np.arange(span) + (blocks * block - span)  # the pool's last blocks
    swapped, turns, twice, hole = good.copy(), good.copy(), good.copy(), good.copy()
    at = next(t for t in range(span - 1) if good[t] % block == block - 3) if span >= block else 0
    swapped[[at, at + 1]] = swapped[[at + 1, at]]
    half = span // 2
    turns[0: 2 * half: 2], turns[1: 2 * half: 2] = good[:half], good[half: 2 * half]
    twice[span - 1] = twice[0]
    hole[at + 1] = -1
    for slots, bad in ((good, False), (swapped, True), (turns, True), (twice, True), (hole, True), (good, False)):
        ops.fp8blk_kv_append(x, x, to_dev(slots), *dev)
        assert ops.fp8blk_device_status(clear=True) == (ops.STATUS_BAD_KV if bad else 0)
