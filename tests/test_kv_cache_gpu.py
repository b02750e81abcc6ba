"""GPU tests of the paged e4m3 cache: fp8blk_kv_map and fp8blk_kv_append,
against plain loops.  Every output is a whole number or an exactly defined
rounding, so everything is compared bit for bit."""
import numpy as np
import pytest
import torch

import _step_ref as ref
from _helpers import to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from fp8_block_scaled_fp8blk_gb300 import ops as o
    yield o
    assert o.fp8blk_device_status(clear=True) == 0


# ------------------------------------------------------------------- map
def check_map(ops, ctx, new, width, free, head, block, max_tokens, status=0, seed=0):
    rng = np.random.default_rng(seed)
    ctx, new = np.asarray(ctx, np.int32), np.asarray(new, np.int32)
    n = len(ctx)
    table = np.full((n, width), -1, np.int32)
    for r in range(n):
        held = min(-(-max(int(ctx[r]), 0) // block), width)
        table[r, :held] = rng.integers(0, 1000, held)
    free = np.asarray(free, np.int32)
    want = ref.kv_map(ctx, new, table, free, head, block, max_tokens)
    t = to_dev(table)
    got = ops.fp8blk_kv_map(to_dev(ctx), to_dev(new), t, to_dev(free), to_dev(np.array([head], np.int32)), block, max_tokens)
    assert ops.fp8blk_device_status(clear=True) == status
    for name, g, w in (("table", t, want[0]), ("seq_lens", got.seq_lens, want[1]), ("q_starts", got.q_starts, want[2]),
                       ("slots", got.slots, want[3]), ("positions", got.positions, want[4])):
        assert np.array_equal(g.cpu().numpy(), w), name
    assert int(got.free_head) == want[5]
    assert (want[6] and ops.STATUS_KV_EXHAUSTED or 0) | (want[7] and ops.STATUS_BAD_KV or 0) == status


@pytest.mark.parametrize("n,most_ctx,most_new,block", [(1, 0, 1, 16), (1, 15, 1, 16), (1, 16, 1, 16), (7, 300, 9, 32),
                                                       (64, 500, 1, 64), (513, 200, 8, 16), (1025, 40, 3, 128),
                                                       (2000, 33, 5, 16), (5, 1000, 3001, 64)])
def test_map_matches_loops(ops, n, most_ctx, most_new, block):
    rng = np.random.default_rng(n * 7 + block)
    ctx, new = rng.integers(0, most_ctx + 1, n), rng.integers(0, most_new + 1, n)
    new[0] = most_new
    width = int(max(-(-(ctx + new) // block))) + 1
    need = int(sum(-(-(ctx + new) // block) - -(-ctx // block)))
    for pad in (0, 5):
        check_map(ops, ctx, new, width, rng.permutation(need + 20), 3, block, int(new.sum()) + pad)


def test_map_nothing_new(ops):
    check_map(ops, [0, 5, 16], [0, 0, 0], 3, [9, 8], 1, 16, 8)


def test_map_runs_out_of_blocks(ops):
    check_map(ops, [0, 30, 0], [40, 10, 5], 4, [7, 3, 5], 0, 16, 60, status=8)
    check_map(ops, [0], [40], 4, np.zeros(1), 1, 16, 40, status=8)


def test_map_flags_bad_lengths(ops):
    check_map(ops, [-3, 10], [4, -2], 2, np.arange(8), 0, 16, 16, status=4)    # negative lengths count as zero
    check_map(ops, [10, 40], [40, 3], 2, np.arange(8), 0, 16, 64, status=4)    # past the table's width
    check_map(ops, [0, 0], [10, 10], 2, np.arange(8), 0, 16, 13, status=4)     # more tokens than the step has room for


def test_map_step_by_step_equals_once(ops):
    """Ten steps of one token each take the same blocks per request as their order says, and the head moves along."""
    n, block, width = 5, 16, 4
    ctx = torch.tensor([0, 15, 16, 31, 7], dtype=torch.int32, device="cuda:0")
    free = torch.arange(100, 160, dtype=torch.int32, device="cuda:0")
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda:0")
    start = ops.fp8blk_kv_map(torch.zeros_like(ctx), ctx, table, free, torch.zeros(1, dtype=torch.int32, device="cuda:0"),
                              block, 80)
    head, lens = start.free_head, start.seq_lens
    one = torch.ones_like(ctx)
    for step in range(10):
        m = ops.fp8blk_kv_map(lens, one, table, free, head, block, n)
        slots = m.slots.cpu().numpy()
        for r in range(n):
            p = int(ctx[r]) + step
            assert slots[r] == int(table[r, p // block]) * block + p % block
        head, lens = m.free_head, m.seq_lens
    used = table[table >= 0].cpu().numpy()
    assert sorted(used) == list(range(100, 100 + int(head)))


def test_map_on_another_stream_and_in_a_graph(ops):
    ctx = torch.tensor([3, 20], dtype=torch.int32, device="cuda:0")
    new = torch.tensor([2, 15], dtype=torch.int32, device="cuda:0")
    free = torch.arange(10, dtype=torch.int32, device="cuda:0")
    head = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    table = torch.zeros((2, 4), dtype=torch.int32, device="cuda:0")
    want = ops.fp8blk_kv_map(ctx, new, table, free, head, 16, 32)
    torch.cuda.synchronize()
    out = ops.kv_map_buffers(2, 32, "cuda:0")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        ops.fp8blk_kv_map(ctx, new, table, free, head, 16, 32, out=out)
    side.synchronize()
    assert torch.equal(out.slots, want.slots)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.fp8blk_kv_map(ctx, new, table, free, head, 16, 32, out=out)
    new.copy_(torch.tensor([1, 30], dtype=torch.int32))
    g.replay()
    w = ref.kv_map([3, 20], [1, 30], table.cpu().numpy(), np.arange(10), 0, 16, 32)
    torch.cuda.synchronize()
    assert np.array_equal(out.slots.cpu().numpy(), w[3]) and np.array_equal(out.q_starts.cpu().numpy(), w[2])


# ---------------------------------------------------------------- append
def slots_for(ctx, new, block, blocks, rng):
    """Slots of requests' new tokens over shuffled pages."""
    order, at, out = rng.permutation(blocks), 0, []
    for c, f in zip(ctx, new):
        pages = -(-(c + f) // block)
        ids = order[at: at + pages]
        at += pages
        out += [int(ids[p // block]) * block + p % block for p in range(c, c + f)]
    return np.array(out, np.int64)


def random_pool(rng, blocks, heads, block, dim):
    codes = rng.integers(0, 254, (blocks, heads, block, dim)).astype(np.uint8)
    codes = np.where(codes >= 127, codes + 1, codes).astype(np.uint8)
    return codes, (2.0 ** rng.integers(-12, 3, (blocks, heads))).astype(np.float32)


def run_append(ops, k, v, slots, kc, ks, vc, vs, dtype):
    dev = [to_dev(a) for a in (kc, ks, vc, vs)]
    kd, vd = (to_dev(a.astype(np.float32)).to(dtype) for a in (k, v))
    ops.fp8blk_kv_append(kd, vd, to_dev(slots), *dev)
    for x, codes, scales, gc, gs in ((kd, kc, ks, dev[0], dev[1]), (vd, vc, vs, dev[2], dev[3])):
        wc, ws = ref.kv_append(x.float().cpu().numpy().astype(np.float64), slots, codes, scales, codes.shape[2])
        assert np.array_equal(gs.cpu().numpy().astype(np.float64), ws)
        assert ref.same_codes(gc.cpu().numpy(), wc)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("ctx,new,heads,dim,block", [
    ([0], [1], 1, 16, 16), ([5], [1], 1, 128, 64), ([15], [2], 3, 80, 16), ([0, 63, 64, 65], [1, 1, 1, 1], 8, 128, 64),
    ([3, 0, 17, 100], [1, 8, 5, 3], 2, 256, 32), ([0, 7], [300, 129], 2, 48, 128), ([1], [127], 1, 64, 128),
    ([0, 31, 2], [64, 33, 700], 4, 192, 32)])
def test_append_matches_loops(ops, dtype, ctx, new, heads, dim, block):
    rng = np.random.default_rng(sum(new) * 31 + dim + block)
    blocks = sum(-(-(c + f) // block) for c, f in zip(ctx, new)) + 2
    slots = slots_for(ctx, new, block, blocks, rng)
    shape = (len(slots), heads, dim)
    mag = 2.0 ** rng.integers(-8, 9, (len(slots), heads, 1))
    k, v = rng.standard_normal(shape) * mag, rng.standard_normal(shape)
    run_append(ops, k, v, slots, *random_pool(rng, blocks, heads, block, dim), *random_pool(rng, blocks, heads, block, dim), dtype)


def test_append_extremes(ops):
    """Zeros, the largest and smallest values, exact maxima (448 s, and just past it), NaN and infinities."""
    rng = np.random.default_rng(5)
    rows = np.zeros((9, 1, 32))
    rows[1, 0, :2] = 3.4e38, -1.0
    rows[2, 0, :2] = 1e-44, -1e-45
    rows[3, 0, :3] = 448.0, 0.25, -2.0 ** -10
    rows[4, 0, :3] = 448.0 + 2.0 ** -14, 1.0, 3.0
    rows[5, 0, :3] = np.inf, 5.0, -0.0
    rows[6, 0, :3] = np.nan, -np.inf, 0.1
    rows[7, 0, :] = np.nan
    rows[8, 0, :2] = 2.0 ** -126 * 448, 2.0 ** -130
    for off in (0, 3):
        slots = np.array([16 * i + off for i in range(9)], np.int64)
        pool, pool2 = random_pool(rng, 9, 1, 16, 32), random_pool(rng, 9, 1, 16, 32)
        run_append(ops, rows, rows[::-1].copy(), slots, *pool, *pool2, torch.float32)


def test_append_skips_and_flags(ops):
    rng = np.random.default_rng(6)
    kc, ks = random_pool(rng, 3, 2, 16, 32)
    x = rng.standard_normal((5, 2, 32))
    slots = np.array([-1, 4, 5, -1, 48], np.int64)  # 48 is past the pool
    kd = [to_dev(a) for a in (kc, ks, kc, ks)]
    ops.fp8blk_kv_append(to_dev(x.astype(np.float32)), to_dev(x.astype(np.float32)), to_dev(slots), *kd)
    assert ops.fp8blk_device_status(clear=True) == ops.STATUS_BAD_KV
    wc, ws = ref.kv_append(x.astype(np.float32).astype(np.float64)[:3], slots[:3], kc, ks, 16)
    assert np.array_equal(kd[0].cpu().numpy(), wc) and np.array_equal(kd[1].cpu().numpy(), ws)


def test_append_strided_rows(ops):
    """Keys and values as slices of one fused projection, on a stream of their own."""
    rng = np.random.default_rng(7)
    kc, ks = random_pool(rng, 4, 2, 32, 64)
    vc, vs = random_pool(rng, 4, 2, 32, 64)
    qkv = to_dev(rng.standard_normal((50, 9, 64)).astype(np.float32))
    k, v = qkv[:, 5:7], qkv[:, 7:9]
    slots = np.arange(20, 70, dtype=np.int64)
    dev = [to_dev(a) for a in (kc, ks, vc, vs)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        ops.fp8blk_kv_append(k, v, to_dev(slots), *dev)
    side.synchronize()
    wc, ws = ref.kv_append(v.cpu().numpy().astype(np.float64), slots, vc, vs, 32)
    assert np.array_equal(dev[2].cpu().numpy(), wc) and np.array_equal(dev[3].cpu().numpy(), ws)
    wc, ws = ref.kv_append(k.cpu().numpy().astype(np.float64), slots, kc, ks, 32)
    assert np.array_equal(dev[0].cpu().numpy(), wc)


def test_append_row_by_row(ops):
    """A block filled one token a call: each call's rounding on what the last one left, and a roll back in between."""
    rng = np.random.default_rng(8)
    kc, ks = random_pool(rng, 2, 1, 16, 32)
    dev = [to_dev(a) for a in (kc, ks, kc, ks)]
    for step, row in enumerate([0, 1, 2, 3, 2, 3, 4, 0, 1]):
        x = rng.standard_normal((1, 1, 32)).astype(np.float32) * np.float32(2.0 ** (step % 5))
        slots = np.array([16 + row], np.int64)
        ops.fp8blk_kv_append(to_dev(x), to_dev(x), to_dev(slots), *dev)
        kc, ks = ref.kv_append(x.astype(np.float64), slots, kc, ks, 16)
        assert np.array_equal(dev[0].cpu().numpy(), kc) and np.array_equal(dev[1].cpu().numpy(), ks)


def test_append_far_into_a_long_pool(ops):
    """Blocks whose byte offset is past 2^31 (and past 2^32 in the pair of pools)."""
    blocks, heads, block, dim = 70000, 2, 128, 128  # 2.3 GB a pool
    kc = torch.zeros((blocks, heads, block, dim), dtype=torch.uint8, device="cuda:0")
    ks = torch.zeros((blocks, heads), dtype=torch.float32, device="cuda:0")
    vc, vs = torch.zeros_like(kc), torch.zeros_like(ks)
    rng = np.random.default_rng(9)
    x = rng.standard_normal((3, heads, dim)).astype(np.float32)
    slots = np.arange(3, dtype=np.int64) + (blocks - 1) * block
    ops.fp8blk_kv_append(to_dev(x), to_dev(-x), to_dev(slots), kc, ks, vc, vs)
    wc, ws = ref.kv_append(x.astype(np.float64), np.arange(3), np.zeros((1, heads, block, dim), np.uint8),
                           np.zeros((1, heads), np.float32), block)
    assert np.array_equal(kc[-1].cpu().numpy(), wc[0]) and np.array_equal(ks[-1].cpu().numpy(), ws[0])
    assert int(kc[:-1].max()) == 0 and int(vc[:-1].max()) == 0 and float(vs[:-1].max()) == 0
