"""GPU tests of fp8blk_kv_map with block counts carried from step to step: verify steps whose last rows are rejected take
and lose no block.  Whole numbers, compared with plain loops."""
import numpy as np
import pytest
import torch

from _helpers import to_dev

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def ops():
    from fp8_block_scaled_fp8blk_gb300 import ops as o
    yield o
    assert o.fp8blk_device_status(clear=True) == 0


def ceil(a, b):
    return -(-a // b)


def loops(ctx, new, held, table, free, head, block, most):
    """(table, slots, positions, head, held_out, exhausted, bad): entries below max(held, ceil(ctx / block)) are kept."""
    n, width = table.shape
    table, slots, positions = table.copy(), np.full(most, -1, np.int64), np.full(most, -1, np.int32)
    held_out, at, exhausted, bad = np.zeros(n, np.int32), 0, False, False
    for r in range(n):
        c, f = max(int(ctx[r]), 0), max(int(new[r]), 0)
        bad |= held[r] < 0 or held[r] > width or ceil(c + f, block) > width
        h = max(min(ceil(c, block), width), min(int(held[r]), width))
        held_out[r] = h
        for b in range(h, min(ceil(c + f, block), width)):
            table[r, b] = free[head] if head < len(free) else -1
            held_out[r] += head < len(free)
            exhausted |= head >= len(free)
            head += 1
        for p in range(c, c + f):
            positions[at] = p
            if p // block < width and table[r, p // block] >= 0:
                slots[at] = int(table[r, p // block]) * block + p % block
            at += 1
    return table, slots, positions, min(head, len(free)), held_out, exhausted, bad


@pytest.mark.parametrize("n,block,start", [(1, 64, 60), (5, 16, 9), (64, 16, 30), (700, 32, 31)])
def test_verify_steps_with_rejections(ops, n, block, start):
    """Eight rows a request around a block's edge, one to eight of them accepted: after every step the ids of the tables and
    of the rest of the free list are all ids, each once, and the cached tokens' blocks have not moved."""
    rng = np.random.default_rng(n + block)
    steps, width = 12, ceil(start + 12 * 8 + 8, block)
    ids = rng.permutation(n * width + 3).astype(np.int32)
    table = torch.full((n, width), -1, dtype=torch.int32, device=DEV)
    free, head = to_dev(ids), torch.zeros(1, dtype=torch.int32, device=DEV)
    held, spare = torch.zeros(n, dtype=torch.int32, device=DEV), torch.empty(n, dtype=torch.int32, device=DEV)
    ctx, new = np.zeros(n, np.int32), np.full(n, start, np.int32)
    for step in range(steps):
        before, was = table.cpu().numpy(), held.cpu().numpy()
        most = int(new.sum())
        want = loops(ctx, new, was, before, ids, int(head), block, most)
        got = ops.fp8blk_kv_map(to_dev(ctx), to_dev(new), table, free, head, block, most, held=held, held_out=spare)
        head, held, spare = got.free_head, spare, held
        t, h = table.cpu().numpy(), held.cpu().numpy()
        assert np.array_equal(t, want[0]) and np.array_equal(h, want[4]) and int(head) == want[3]
        assert np.array_equal(got.slots.cpu().numpy(), want[1]) and np.array_equal(got.positions.cpu().numpy(), want[2])
        assert not want[5] and not want[6]
        for r in range(n):
            assert np.array_equal(t[r, : was[r]], before[r, : was[r]])
        owned = np.concatenate([t[r, : h[r]] for r in range(n)] + [ids[int(head):]])
        assert np.array_equal(np.sort(owned), np.arange(len(ids)))
        ctx = ctx + (new if step == 0 else rng.integers(1, 9, n)).astype(np.int32)  # some of the rows are accepted
        new = np.full(n, 8, np.int32)


def test_the_step_of_a_rejected_block(ops):
    """60 cached tokens, blocks of 64: eight rows take a block, two are accepted, and the next eight take none."""
    table = torch.tensor([[7, -1, -1]], dtype=torch.int32, device=DEV)
    free, head = to_dev(np.array([3, 4, 5], np.int32)), torch.zeros(1, dtype=torch.int32, device=DEV)
    held = torch.ones(1, dtype=torch.int32, device=DEV)
    out = torch.empty_like(held)
    eight = torch.full((1,), 8, dtype=torch.int32, device=DEV)
    a = ops.fp8blk_kv_map(torch.full_like(eight, 60), eight, table, free, head, 64, 8, held=held, held_out=out)
    assert table.tolist() == [[7, 3, -1]] and out.tolist() == [2] and int(a.free_head) == 1
    b = ops.fp8blk_kv_map(torch.full_like(eight, 62), eight, table, free, a.free_head, 64, 8, held=out, held_out=held)
    assert table.tolist() == [[7, 3, -1]] and held.tolist() == [2] and int(b.free_head) == 1
    assert b.slots.tolist() == [7 * 64 + 62, 7 * 64 + 63] + [3 * 64 + i for i in range(6)]


@pytest.mark.parametrize("n", [6, 40, 900])
def test_counts_without_blocks_and_bad_counts(ops, n):
    """When the list runs out, the counts leave out what it could not give; bad counts are bounded and flagged."""
    rng = np.random.default_rng(n)
    block, width = 16, 6
    for case in range(4):
        ctx, new = rng.integers(0, 50, n).astype(np.int32), rng.integers(0, 40, n).astype(np.int32)
        held = np.minimum(-(-ctx // block) + rng.integers(0, 3, n), width).astype(np.int32)
        if case == 1:
            held[n // 2] = -3
        if case == 2:
            held[n // 2] = width + 5
        table = rng.integers(0, 1000, (n, width)).astype(np.int32)
        ids = rng.permutation(3 * n if case != 3 else n // 2).astype(np.int32)
        most = max(1, int(new.sum()))
        want = loops(ctx, new, held, table, ids, 1, block, most)
        t, out = to_dev(table), torch.empty(n, dtype=torch.int32, device=DEV)
        got = ops.fp8blk_kv_map(to_dev(ctx), to_dev(new), t, to_dev(ids), to_dev(np.array([1], np.int32)), block, most,
                                held=to_dev(held), held_out=out)
        status = ops.fp8blk_device_status(clear=True)
        assert status == (want[5] and ops.STATUS_KV_EXHAUSTED or 0) | (want[6] and ops.STATUS_BAD_KV or 0)
        assert np.array_equal(t.cpu().numpy(), want[0]) and np.array_equal(out.cpu().numpy(), want[4])
        assert np.array_equal(got.slots.cpu().numpy(), want[1]) and int(got.free_head) == want[3]
        assert bool(want[5]) == (case == 3) and bool(want[6]) >= (case in (1, 2))


def test_counts_equal_the_plain_call_where_nothing_was_rejected(ops):
    rng = np.random.default_rng(3)
    ctx, new = rng.integers(0, 90, 30).astype(np.int32), rng.integers(0, 30, 30).astype(np.int32)
    table = rng.integers(0, 1000, (30, 8)).astype(np.int32)
    ids, head = to_dev(rng.permutation(200).astype(np.int32)), to_dev(np.array([4], np.int32))
    a, b = to_dev(table), to_dev(table)
    plain = ops.fp8blk_kv_map(to_dev(ctx), to_dev(new), a, ids, head, 16, 900)
    zero, out = torch.zeros(30, dtype=torch.int32, device=DEV), torch.empty(30, dtype=torch.int32, device=DEV)
    with_counts = ops.fp8blk_kv_map(to_dev(ctx), to_dev(new), b, ids, head, 16, 900, held=zero, held_out=out)
    assert torch.equal(a, b) and all(torch.equal(x, y) for x, y in zip(plain, with_counts))
    assert np.array_equal(out.cpu().numpy(), -(-(ctx + new) // 16))


def test_verify_loop_example(ops):
    """The example's loop: every block is in one table entry or free, step after step."""
    import importlib.util
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location("verify_step", os.path.join(root, "examples", "verify_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    cache, lens, accepted = m.loop(steps=6)
    h, t = cache.held.cpu().numpy(), cache.table.cpu().numpy()
    owned = np.concatenate([t[r, : h[r]] for r in range(len(h))] + [cache.free_blocks.cpu().numpy()[int(cache.free_head):]])
    assert np.array_equal(np.sort(owned), np.arange(len(owned))) and len(owned) == cache.k_codes.shape[0]
    assert (h >= ceil(lens.cpu().numpy(), cache.block_tokens)).all()
    assert accepted.min() >= 1 and accepted.sum() < 6 * 3 * 8


def test_an_empty_free_list(ops):
    """A step whose tokens all fit in blocks that the requests have; then one that needs a block."""
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    table = torch.tensor([[5, -1], [2, 9]], dtype=torch.int32, device=DEV)
    head = torch.zeros(1, dtype=torch.int32, device=DEV)
    one = torch.ones(2, dtype=torch.int32, device=DEV)
    got = ops.fp8blk_kv_map(to_dev(np.array([3, 20], np.int32)), one, table, none, head, 16, 4)
    assert ops.fp8blk_device_status(clear=True) == 0
    assert got.slots.tolist() == [5 * 16 + 3, 9 * 16 + 4, -1, -1] and int(got.free_head) == 0
    got = ops.fp8blk_kv_map(to_dev(np.array([16, 20], np.int32)), one, table, none, head, 16, 4)
    assert ops.fp8blk_device_status(clear=True) == ops.STATUS_KV_EXHAUSTED
    assert got.slots.tolist() == [-1, 9 * 16 + 4, -1, -1] and table.tolist() == [[5, -1], [2, 9]]
