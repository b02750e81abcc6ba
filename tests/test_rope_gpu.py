"""GPU tests of the rotary positions: table, rotation, and the append that rotates, against plain 64-bit restatements.

Tolerances, from the arithmetic.  A cosine or sine is within 2^-23 (the angle's roundings, the series' sums and the final
rounding) before its scale, which rounds once more: scale x (2^-23 + 2^-24).  A rotated f32 value rounds one product and
one sum: 2^-24 (|b s| + |y|) <= 2^-23 (|a c| + |b s|); bf16 adds 2^-8 |y|."""
import numpy as np
import pytest
import torch

import _rope_ref as rref
import _step_ref as ref
from _helpers import to_dev

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def ops():
    from fp8_block_scaled_fp8blk_gb300 import ops as o
    o.fp8blk_device_status(clear=True)
    yield o
    assert o.fp8blk_device_status(clear=True) == 0


# ---------------------------------------------------------------- table
@pytest.mark.parametrize("rot", [2, 6, 20, 64, 128, 1024])
@pytest.mark.parametrize("scaling,kw", [("plain", {}), ("ramp", dict(factor=32.0, original_len=4096.0))])
def test_table(ops, rot, scaling, kw):
    rng = np.random.default_rng(rot)
    pos = np.concatenate([[0, 1, 2, -1, -(2 ** 31), 131071, 2 ** 31 - 1], rng.integers(0, 2 ** 20, 50)]).astype(np.int32)
    freqs, scale = ops.rope_frequencies(rot, 10000.0, scaling, **kw)
    got = ops.fp8blk_rope_table(to_dev(pos), ops.rope_turns(freqs, DEV), scale).cpu().numpy().astype(np.float64)
    want_f, want_scale = rref.frequencies(rot, 10000.0, scaling, kw.get("factor", 1.0), kw.get("original_len", 0.0))
    # (numpy's 64-bit angle of the farthest position is good to 2^31 x 2^-52, that of the frequency's own bits to as much)
    angle = pos[:, None].astype(np.float64) * want_f
    want = np.stack([np.cos(angle), np.sin(angle)], 1) * want_scale
    want[pos < 0, 0], want[pos < 0, 1] = 1.0, 0.0
    tol = want_scale * (2.0 ** -23 + 2.0 ** -24) + np.abs(angle)[:, None] * 2.0 ** -50
    assert got.shape == want.shape and (np.abs(got - want) <= tol).all(), np.abs(got - want).max()
    assert np.array_equal(got[pos < 0], want[pos < 0])


def test_a_negative_frequency_turns_back(ops):
    pos = torch.arange(0, 5000, 7, dtype=torch.int32, device=DEV)
    freqs, _ = ops.rope_frequencies(64)
    there, back = (ops.fp8blk_rope_table(pos, ops.rope_turns(s * freqs, DEV)) for s in (1.0, -1.0))
    # The two turns are each other's negative up to their roundings (2^-53 of a turn a token).
    assert (there[:, 0] - back[:, 0]).abs().max() <= 2.0 ** -22 and (there[:, 1] + back[:, 1]).abs().max() <= 2.0 ** -22


# ---------------------------------------------------------------- rotation
def table(n, rot, seed):
    a = np.random.default_rng(seed).uniform(0, 2 * np.pi, (n, rot // 2))
    return np.stack([1.3 * np.cos(a), 1.3 * np.sin(a)], 1).astype(np.float32)


SHAPES = [  # rows, heads, dim, rot, start
    (1, 1, 2, 2, 0), (3, 2, 16, 16, 0), (1, 5, 64, 64, 0), (67, 8, 128, 128, 0), (130, 3, 80, 32, 0), (33, 5, 80, 20, 0),
    (9, 7, 192, 64, 128), (5, 2, 576, 64, 512), (11, 3, 96, 24, 8), (4, 9, 64, 32, 5), (6, 4, 10, 6, 3), (2, 1, 1024, 1024, 0),
    (40, 13, 256, 256, 0),
]


def close(got, want, size, dtype):
    tol = 2.0 ** -23 * size + (2.0 ** -8 * np.abs(want) if dtype is torch.bfloat16 else 0.0) + 1e-40
    g = got.float().cpu().numpy().astype(np.float64)
    assert (np.abs(g - want) <= tol).all(), (np.abs(g - want) / tol).max()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,heads,dim,rot,start", SHAPES)
def test_rope(ops, n, heads, dim, rot, start, interleaved, dtype):
    gen = torch.Generator(device=DEV).manual_seed(n * dim + rot)
    wide = torch.randn((n, heads + 3, dim), device=DEV, generator=gen).to(dtype)
    x, cs = wide[:, 1: 1 + heads], table(n, rot, 3)
    want, size = rref.rotate(x.float().cpu().numpy().astype(np.float64), cs[:, 0].astype(np.float64), cs[:, 1].astype(np.float64),
                             interleaved, start)
    before = wide.clone()
    got = ops.fp8blk_rope(x, to_dev(cs), interleaved, start)
    assert torch.equal(wide, before) and got.is_contiguous()
    close(got, want, size, dtype)
    outside = [d for d in range(dim) if d < start or d >= start + rot]
    assert torch.equal(got[:, :, outside], x[:, :, outside])
    # In place, rows strided, what lies beside them left alone.
    assert ops.fp8blk_rope(x, to_dev(cs), interleaved, start, out=x).data_ptr() == x.data_ptr()
    assert torch.equal(x, got)
    assert torch.equal(wide[:, 0], before[:, 0]) and torch.equal(wide[:, 1 + heads:], before[:, 1 + heads:])


def test_rope_unaligned_rows(ops):
    """Rows that start off a 16-byte boundary take the pairs one by one, with the same result."""
    gen = torch.Generator(device=DEV).manual_seed(5)
    flat = torch.randn(7 * 4 * 64 + 1, device=DEV, generator=gen).to(torch.bfloat16)
    cs = to_dev(table(7, 64, 1))
    off = flat[1:].view(7, 4, 64)
    assert off.data_ptr() % 16 == 2
    for pairs in (False, True):
        assert torch.equal(ops.fp8blk_rope(off, cs, pairs), ops.fp8blk_rope(off.clone(), cs, pairs))


def test_rope_takes_what_is_not_finite(ops):
    """A NaN or infinity spoils its pair and nothing else."""
    x = torch.ones((2, 1, 64), device=DEV)
    x[0, 0, 3], x[1, 0, 40] = float("nan"), float("inf")
    y = ops.fp8blk_rope(x, to_dev(table(2, 64, 2)))
    bad = ~torch.isfinite(y)
    assert bad.nonzero().tolist() == [[0, 0, 3], [0, 0, 35], [1, 0, 8], [1, 0, 40]]


def test_rope_empty(ops):
    assert ops.fp8blk_rope(torch.zeros((0, 4, 64), device=DEV), torch.zeros((0, 2, 32), device=DEV)).shape == (0, 4, 64)
    assert ops.fp8blk_rope_table(torch.zeros(0, dtype=torch.int32, device=DEV), ops.rope_turns([0.5], DEV)).shape == (0, 2, 1)


# ---------------------------------------------------------------- the append that rotates
class Cache:
    def __init__(self, blocks, kv, block, dim, seed):
        rng = np.random.default_rng(seed)
        self.kc, self.vc = (rng.integers(0, 127, (blocks, kv, block, dim)).astype(np.uint8) for _ in range(2))
        self.ks, self.vs = (np.exp2(rng.integers(-9, -3, (blocks, kv))).astype(np.float32) for _ in range(2))

    def dev(self):
        return [to_dev(a) for a in (self.kc, self.ks, self.vc, self.vs)]


def slots_for(ctx, new, block, blocks, seed, skip=False):
    """Slots of requests with `ctx` tokens each and `new` more, over shuffled blocks."""
    order, at, out = np.random.default_rng(seed).permutation(blocks), 0, []
    for c, f in zip(ctx, new):
        pages = order[at: at + -(-(c + f) // block)]
        at += len(pages)
        out += [int(pages[p // block]) * block + p % block for p in range(c, c + f)]
        if skip and f > 1:
            out[-1] = -1
    return np.array(out, np.int64)


APPENDS = [  # ctx, new, kv, q heads, dim, block, rot, start
    ([5], [1], 1, 1, 16, 16, 16, 0),
    ([0, 17, 63, 200], [1, 1, 1, 1], 8, 32, 128, 64, 128, 0),
    ([3, 0, 40], [8, 2, 5], 3, 15, 80, 16, 20, 0),
    ([3, 0, 40], [8, 2, 5], 3, 6, 80, 16, 32, 48),
    ([0, 30], [100, 77], 2, 4, 96, 32, 24, 9),
    ([100, 0, 5], [600, 900, 33], 8, 16, 128, 64, 128, 0),       # whole runs by a CTA
    ([1], [1300], 8, 8, 64, 16, 64, 0),
    ([7], [1500], 8, 8, 256, 128, 128, 64),                      # runs that shared memory does not hold
    ([7, 64], [900, 900], 8, 8, 80, 64, 20, 30),                 # pairs one by one
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("ctx,new,kv,heads,dim,block,rot,start", APPENDS)
def test_append_rope(ops, ctx, new, kv, heads, dim, block, rot, start, interleaved, dtype):
    """The cache is what fp8blk_kv_append makes of the keys rotated in f32, code by code, and against the 64-bit definition
    each key is within its code's rounding; the queries are fp8blk_rope's."""
    blocks = sum(-(-(c + f) // block) for c, f in zip(ctx, new)) + 2
    slots, cache = slots_for(ctx, new, block, blocks, 1), Cache(blocks, kv, block, dim, 2)
    n = len(slots)
    gen = torch.Generator(device=DEV).manual_seed(n + dim)
    qkv = torch.randn((n, heads + 2 * kv, dim), device=DEV, generator=gen).to(dtype)
    q, k, v = qkv[:, :heads], qkv[:, heads: heads + kv], qkv[:, heads + kv:]
    cs = table(n, rot, 4)
    t, s, before = to_dev(cs), to_dev(slots), qkv.clone()
    got, want = cache.dev(), cache.dev()
    q_out = ops.fp8blk_kv_append_rope(k, v, s, t, *got, interleaved=interleaved, start=start, q=q)
    assert torch.equal(qkv, before) and torch.equal(q_out, ops.fp8blk_rope(q, t, interleaved, start))
    turned = ops.fp8blk_rope(k.float(), t, interleaved, start)
    ops.fp8blk_kv_append(turned, v.float(), s, *want)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    exact, size = rref.rotate(k.float().cpu().numpy().astype(np.float64), cs[:, 0].astype(np.float64), cs[:, 1].astype(np.float64),
                              interleaved, start)
    codes, scales = got[0].cpu().numpy(), got[1].cpu().numpy().astype(np.float64)
    sc = scales[slots // block][:, :, None]
    back = ref.E4M3[codes[slots // block, :, slots % block]] * sc
    tol = 2.0 ** -4 * np.abs(exact) + 2.0 ** -10 * sc + 2.0 ** -22 * size
    assert (np.abs(back - exact) <= tol).all()
    # Without queries, and with queries in place.
    again = cache.dev()
    assert ops.fp8blk_kv_append_rope(k, v, s, t, *again, interleaved=interleaved, start=start) is None
    assert all(torch.equal(a, b) for a, b in zip(again, got))
    again = cache.dev()
    ops.fp8blk_kv_append_rope(k, v, s, t, *again, interleaved=interleaved, start=start, q=q, q_out=q)
    assert torch.equal(q, q_out) and all(torch.equal(a, b) for a, b in zip(again, got))


@pytest.mark.parametrize("old", [0.011, 2.0 ** -3])
def test_append_rope_under_an_old_scale(ops, old):
    """A larger scale that is there stays, power of two or not; skipped tokens leave their rows alone."""
    ctx, new, block = [5, 20], [7, 9], 32
    slots = slots_for(ctx, new, block, 4, 3, skip=True)
    gen = torch.Generator(device=DEV).manual_seed(8)
    k, v = (torch.randn((16, 2, 64), device=DEV, generator=gen) for _ in range(2))
    t, s = to_dev(table(16, 64, 5)), to_dev(slots)
    got, want = Cache(4, 2, block, 64, 6).dev(), Cache(4, 2, block, 64, 6).dev()
    for c in (got, want):
        c[1].fill_(old)
    ops.fp8blk_kv_append_rope(k, v, s, t, *got)
    ops.fp8blk_kv_append(ops.fp8blk_rope(k, t), v, s, *want)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_append_rope_flags_bad_slots(ops):
    k = torch.ones((2, 1, 64), device=DEV)
    cache = Cache(2, 1, 16, 64, 7).dev()
    q_out = ops.fp8blk_kv_append_rope(k, k, torch.tensor([3, 32], device=DEV), to_dev(table(2, 64, 6)), *cache, q=k)
    assert ops.fp8blk_device_status(clear=True) == ops.STATUS_BAD_KV
    assert torch.isfinite(q_out).all()
    ops.fp8blk_kv_append_rope(k, k, torch.tensor([16, 18], device=DEV), to_dev(table(2, 64, 6)), *cache)  # two runs in one block
    assert ops.fp8blk_device_status(clear=True) == ops.STATUS_BAD_KV


def test_captured_and_on_another_stream(ops):
    """Table, rotation and append in one graph, replayed on new positions and values, and the calls on a side stream."""
    n, kv, heads, dim, block = 6, 2, 4, 64, 16
    turns = ops.rope_turns(ops.rope_frequencies(dim)[0], DEV)
    gen = torch.Generator(device=DEV).manual_seed(11)
    pos, slots = torch.zeros(n, dtype=torch.int32, device=DEV), torch.arange(n, device=DEV) * block  # (a block each)
    qkv = torch.zeros((n, heads + 2 * kv, dim), device=DEV)
    cs, q_out = torch.empty((n, 2, dim // 2), device=DEV), torch.empty((n, heads, dim), device=DEV)
    cache = [torch.zeros((n, kv, block, dim), dtype=torch.uint8, device=DEV), torch.zeros((n, kv), device=DEV)]
    cache += [c.clone() for c in cache]

    def step():
        ops.fp8blk_rope_table(pos, turns, out=cs)
        ops.fp8blk_kv_append_rope(qkv[:, heads: heads + kv], qkv[:, heads + kv:], slots, cs, *cache, q=qkv[:, :heads], q_out=q_out)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        pos.copy_(torch.randint(0, 100000, (n,), device=DEV, generator=gen))
        slots.copy_(torch.randperm(n, device=DEV, generator=gen) * block)
        qkv.normal_(generator=gen)
        graph.replay()
        got = [t.clone() for t in (*cache, q_out)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for c in cache:
                c.zero_()
            step()
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got[-1], q_out)
        page = slots // block
        assert all(torch.equal(a[page], b[page]) for a, b in zip(got[:4], cache))
