"""GPU tests of fp8blk_kv_append into blocks whose old scale is no power of two: e4m3(x / s) and e4m3(code * old / s) are
rounded once, also where the f32 quotient or product would lie on a tie between two codes.  Bit for bit against 64 bits
(whose quotients and products keep 2^-52, far below the 2^-25 that decides these cases)."""
import numpy as np
import pytest
import torch

import _step_ref as ref
from _helpers import to_dev

pytestmark = pytest.mark.gpu
TIES = (ref.E4M3[:126] + ref.E4M3[1:127]) / 2  # between neighbouring codes


@pytest.fixture(scope="module")
def ops():
    from fp8_block_scaled_fp8blk_gb300 import ops as o
    yield o
    assert o.fp8blk_device_status(clear=True) == 0


def check(ops, x, slots, codes, scales, block, dtype):
    """K and V alike; x [n, heads, dim]."""
    d = to_dev(x.astype(np.float32)).to(dtype)
    dev = [to_dev(a) for a in (codes, scales, codes, scales)]
    ops.fp8blk_kv_append(d, -d, to_dev(slots), *dev)
    for y, gc, gs in ((d, dev[0], dev[1]), (-d, dev[2], dev[3])):
        wc, ws = ref.kv_append(y.float().cpu().numpy().astype(np.float64), slots, codes, scales, block)
        assert np.array_equal(gs.cpu().numpy().astype(np.float64), ws)
        assert ref.same_codes(gc.cpu().numpy(), wc)


def odd_scales(rng, n, low, high):
    """Any f32 in [1, 2) times 2^low .. 2^high."""
    return (rng.uniform(1.0, 2.0, n) * 2.0 ** rng.integers(low, high + 1, n)).astype(np.float32)


# 9728 (token, head) pairs and more take the prompt kernel, fewer the decode kernel.
@pytest.mark.parametrize("blocks,tokens", [(60, 1), (60, 5), (700, 15)])
@pytest.mark.parametrize("low,high", [(-3, 3), (-126, -100), (80, 118)])
def test_quotients_next_to_ties(ops, blocks, tokens, low, high):
    rng = np.random.default_rng(abs(blocks + tokens + low))
    block, dim = 16, 128
    scales = odd_scales(rng, blocks, low, high)[:, None]
    codes = rng.integers(0, 126, (blocks, 1, block, dim)).astype(np.uint8)
    ties = TIES[TIES <= 200.0]  # with these the old scale stays the block's
    t = ties[rng.integers(0, len(ties), (blocks * tokens, 1, dim))] * rng.choice([-1.0, 1.0], (blocks * tokens, 1, dim))
    x = (t * np.repeat(scales.astype(np.float64), tokens, 0)[:, :, None]).astype(np.float32)
    slots = (np.arange(blocks)[:, None] * block + 1 + np.arange(tokens)).ravel().astype(np.int64)
    check(ops, x, slots, codes, scales, block, torch.float32)


@pytest.mark.parametrize("blocks", [90, 1400])
def test_quotients_of_bf16_next_to_ties(ops, blocks):
    """One tie a block: its scale is the value over the tie."""
    rng = np.random.default_rng(blocks)
    block, dim, tokens = 16, 64, 8
    t = TIES[40 + rng.integers(0, 50, blocks)]
    x = torch.from_numpy(rng.uniform(1.0, 2.0, blocks)).to(torch.bfloat16).double().numpy()
    scales = (x / t).astype(np.float32)[:, None]
    rows = np.repeat(x, tokens)[:, None, None] * rng.choice([-1.0, 1.0, 0.5, 0.25], (blocks * tokens, 1, dim))
    codes = rng.integers(0, 126, (blocks, 1, block, dim)).astype(np.uint8)
    slots = (np.arange(blocks)[:, None] * block + 2 + np.arange(tokens)).ravel().astype(np.int64)
    check(ops, rows, slots, codes, scales, block, torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("blocks,tokens", [(400, 1), (1000, 10)])
def test_products_next_to_ties(ops, dtype, blocks, tokens):
    """Codes that follow a larger scale: the old one brings one of them next to a tie."""
    rng = np.random.default_rng(blocks)
    block, dim = 16, 64
    code = rng.integers(40, 127, blocks)
    tie = TIES[np.array([rng.integers(20, c - 1) for c in code])]
    scales = (tie / ref.E4M3[code]).astype(np.float32)[:, None]  # below 1, which the new rows ask for
    codes = rng.integers(0, 126, (blocks, 1, block, dim)).astype(np.uint8)
    codes[:, 0, :5, ::3] = code[:, None, None]
    codes[:, 0, :5, ::6] |= 0x80
    x = rng.standard_normal((blocks * tokens, 1, dim))
    x[::tokens, 0, 0] = 448.0
    slots = (np.arange(blocks)[:, None] * block + 5 + np.arange(tokens)).ravel().astype(np.int64)
    check(ops, x, slots, codes, scales, block, dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_any_scale_and_any_value(ops, dtype):
    rng = np.random.default_rng(5)
    blocks, block, heads, dim = 40, 32, 3, 80
    scales = odd_scales(rng, blocks * heads, -9, 9).reshape(blocks, heads)
    codes = rng.integers(0, 126, (blocks, heads, block, dim)).astype(np.uint8)
    x = rng.standard_normal((blocks * 7, heads, dim)) * 2.0 ** rng.integers(-6, 14, (blocks * 7, heads, 1))
    slots = (np.arange(blocks)[:, None] * block + 3 + np.arange(7)).ravel().astype(np.int64)
    check(ops, x, slots, codes, scales, block, dtype)
