"""GPU tests of fp8blk_kv_attn against a plain 64-bit restatement.

Tolerance, from the arithmetic.  Let A be the largest scale * sum_d |q_d k_td|
over the row's tokens.  A score is off by at most u A: u = 2^-16 (f32 queries,
carried to 2^-16 of each element; bf16 queries are exact) + (dim + 16) 2^-24
(f32 sums).  A weight is off by that, by 2^-20 (exponential, scale products) and
by w = 2^-16 (f32) or 2^-8 (bf16), to which it is carried into the second
product; sums add 2^-20.  So
  |out - exact| <= (2 u A + w + 2^-19) * sum_t p_t |v_t|   (+ 2^-8 |exact| + tiny, the rounding to bf16)
  |lse - exact| <= u A + 2^-19 + 2^-21 |lse|."""
import numpy as np
import pytest
import torch

import _step_ref as ref
from _helpers import to_dev

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def ops():
    from fp8_block_scaled_fp8blk_gb300 import ops as o
    yield o
    assert o.fp8blk_device_status(clear=True) == 0


class Case:
    """A random cache over shuffled pages; unused rows and blocks hold NaN codes and NaN scales."""

    def __init__(self, lens, rows, heads, kv, dim, block, seed=0, spread=3, q_std=1.5, extra=3):
        rng = np.random.default_rng(seed)
        self.lens, self.rows = np.asarray(lens, np.int32), np.asarray(rows, np.int32)
        n = len(lens)
        self.block, self.dim, self.heads, self.kv = block, dim, heads, kv
        pages = [-(-int(t) // block) for t in lens]
        blocks = sum(pages) + extra
        order = rng.permutation(blocks)
        width = max(1, max(pages))
        self.table = np.full((n, width), -1, np.int32)
        self.kc = np.full((blocks, kv, block, dim), 0x7F, np.uint8)
        self.vc = np.full((blocks, kv, block, dim), 0xFF, np.uint8)
        self.ks, self.vs = np.full((blocks, kv), np.nan, np.float32), np.full((blocks, kv), np.nan, np.float32)
        at = 0
        for s in range(n):
            ids = order[at: at + pages[s]]
            at += pages[s]
            self.table[s, : pages[s]] = ids
            for j, b in enumerate(ids):
                used = min(block, int(lens[s]) - j * block)
                for codes, scales in ((self.kc, self.ks), (self.vc, self.vs)):
                    x = rng.standard_normal((kv, used, dim))
                    mag = 2.0 ** rng.integers(-spread, 1, kv)
                    for h in range(kv):
                        sc = ref.pow2_scale(np.abs(x[h] * mag[h]).max())
                        codes[b, h, :used] = ref.e4m3_encode(x[h] * mag[h] / sc)
                        scales[b, h] = sc
        self.starts = np.concatenate([[0], np.cumsum(self.rows)]).astype(np.int32)
        self.q = (q_std * rng.standard_normal((int(self.starts[-1]), heads, dim))).astype(np.float32)
        self.scale = 1.0 / np.sqrt(dim)

    def dev(self):
        return [to_dev(a) for a in (self.kc, self.ks, self.vc, self.vs, self.table, self.lens, self.starts)]


def run(ops, c, dtype, q=None, max_m=None, dev=None):
    kc, ks, vc, vs, table, lens, starts = dev or c.dev()
    q = to_dev(c.q).to(dtype) if q is None else q
    max_m = max_m or max(1, int(c.rows.max()))
    ws = ops.kv_attn_workspace(len(c.lens), max_m, c.heads, c.kv, c.dim, DEV)
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=DEV)
    out = ops.fp8blk_kv_attn(q, kc, ks, vc, vs, table, lens, starts, max_m, c.scale, ws, lse=lse)
    return out, lse, q


def check(ops, c, dtype, **kw):
    out, lse, q = run(ops, c, dtype, **kw)
    assert ops.fp8blk_device_status(clear=True) == 0
    want, wlse, peak, spread = ref.kv_attn(q.float().cpu().numpy().astype(np.float64), c.kc, c.ks, c.vc, c.vs, c.table, c.lens,
                                           c.starts, c.scale)
    f32 = dtype is torch.float32
    u = (2.0 ** -16 if f32 else 0.0) + (c.dim + 16) * 2.0 ** -24
    w = 2.0 ** -16 if f32 else 2.0 ** -8
    tol = (2 * u * peak[:, :, None] + w + 2.0 ** -19) * spread
    if not f32:
        tol = tol + 2.0 ** -8 * np.abs(want) + 1e-38
    g = out.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(g).all()
    assert (np.abs(g - want) <= tol).all(), float((np.abs(g - want) / np.maximum(tol, 1e-300)).max())
    gl = lse.cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isneginf(gl), np.isneginf(wlse))
    fin = np.isfinite(wlse)
    tl = u * peak + 2.0 ** -19 + 2.0 ** -21 * np.abs(np.where(fin, wlse, 0))
    assert (np.abs(gl - wlse)[fin] <= tl[fin]).all()


SHAPES = [  # lens, rows, heads, kv, dim, block
    ([1], [1], 1, 1, 16, 16),
    ([2], [2], 2, 1, 32, 16),
    ([127, 128, 129], [1, 1, 1], 4, 2, 128, 64),
    ([300], [1], 8, 1, 128, 128),
    ([1000, 5, 64], [1, 1, 1], 8, 8, 64, 32),
    ([513, 40], [8, 3], 8, 2, 128, 16),
    ([260, 131], [8, 8], 16, 2, 128, 64),
    ([200], [8], 16, 1, 128, 128),       # 128 query rows per cache head
    ([150, 33], [5, 2], 15, 3, 80, 16),
    ([140], [4], 6, 2, 96, 32),
    ([200, 7], [2, 1], 4, 2, 256, 32),
    ([129], [7], 10, 2, 192, 128),
    ([390], [8], 8, 1, 144, 16),
    ([64] * 40, [1] * 40, 4, 2, 64, 64),
    ([300, 77], [8, 5], 4, 2, 64, 32),   # sixteen query rows per cache head, and ten
    ([600, 129], [4, 8], 4, 1, 112, 16),
    ([257], [8], 4, 2, 208, 64),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lens,rows,heads,kv,dim,block", SHAPES)
def test_matches_plain(ops, dtype, lens, rows, heads, kv, dim, block):
    check(ops, Case(lens, rows, heads, kv, dim, block, seed=sum(lens) + dim), dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_more_requests_than_threads(ops, dtype):
    """Lists that each thread scans several requests of, with idle requests and empty caches among them."""
    rng = np.random.default_rng(21)
    lens, rows = rng.integers(0, 40, 1500), rng.integers(0, 3, 1500)
    lens[7], rows[7] = 900, 2
    check(ops, Case(lens, rows, 2, 1, 32, 16, seed=22), dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_one_long_request(ops, dtype):
    check(ops, Case([20011], [3], 4, 1, 64, 64, seed=2), dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lens,rows,heads,kv,dim,block", [
    ([20001], [1], 2, 1, 64, 128),       # one unit in as many parts as there are CTAs
    ([9000, 12000, 7], [8, 5, 1], 4, 1, 128, 64),
    ([3500, 3600, 3700, 3800], [2] * 4, 6, 1, 256, 32),
    ([6000] * 3, [8] * 3, 8, 1, 64, 128),  # two row groups, parts of 32 rows
])
def test_units_in_many_parts(ops, dtype, lens, rows, heads, kv, dim, block):
    """Joined in two steps; the counters are back at zero for the next call."""
    c = Case(lens, rows, heads, kv, dim, block, seed=21)
    check(ops, c, dtype)
    dev, q = c.dev(), to_dev(c.q).to(dtype)
    ws = ops.kv_attn_workspace(len(lens), max(rows), heads, kv, dim, DEV)
    first = ops.fp8blk_kv_attn(q, *dev, max(rows), c.scale, ws)
    head = ws[:2048].clone()
    again = ops.fp8blk_kv_attn(q, *dev, max(rows), c.scale, ws)
    assert torch.equal(first, again) and int(head.count_nonzero()) == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_that_see_nothing(ops, dtype):
    """Requests with fewer tokens than rows, with none, and with no row at all."""
    check(ops, Case([3, 0, 200, 0, 1, 17], [5, 2, 0, 0, 1, 8], 6, 3, 48, 16, seed=4), dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_peaked_and_flat_scores(ops, dtype):
    check(ops, Case([700], [2], 2, 1, 128, 64, seed=5, q_std=20.0), dtype)   # scores of tens: one token takes all
    c = Case([700], [2], 2, 1, 128, 64, seed=6)
    c.q[:] = 0.0                                                             # all tokens alike
    check(ops, c, dtype)


def test_scores_that_rise_along_the_cache(ops):
    """The running maximum moves in every tile, by more than any weight's range."""
    c = Case([1500], [1], 2, 1, 64, 64, seed=7)
    for j, b in enumerate(c.table[0]):
        c.kc[b] = ref.e4m3_encode(np.ones((1, 64, 64)) * 64)
        c.ks[b] = 2.0 ** (j // 2 - 8)
    c.q[:] = 0.5
    check(ops, c, torch.float32)
    c.ks[c.table[0]] = c.ks[c.table[0]][::-1]
    check(ops, c, torch.float32)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_scales_of_any_size(ops, dtype):
    """Value scales from 2^-60 to 2^40 from block to block, and scales that are no powers of two."""
    c = Case([400, 100], [2, 1], 4, 2, 64, 16, seed=8)
    rng = np.random.default_rng(9)
    used = c.table[c.table >= 0]
    c.vs[used] = (2.0 ** rng.integers(-60, 41, (len(used), 2))).astype(np.float32)
    check(ops, c, dtype)
    c.vs[used] = rng.uniform(0.1, 3.0, (len(used), 2)).astype(np.float32)
    c.ks[used] *= rng.uniform(0.5, 2.0, (len(used), 2)).astype(np.float32)
    c.vs[used[0]] = 0.0
    check(ops, c, dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("length,block", [(130, 16), (129, 64), (64, 16), (131, 128)])
def test_what_a_row_does_not_see(ops, dtype, length, block):
    """NaN codes and scales of later positions leave earlier rows untouched, and reach the rows that see them."""
    rows = 4
    c = Case([length, 90], [rows, 1], 4, 2, 64, block, seed=length)
    clean = run(ops, c, dtype)[0]
    for back in range(1, rows):      # poison the position `back` from the end
        p = length - back
        d = Case([length, 90], [rows, 1], 4, 2, 64, block, seed=length)
        b, r = d.table[0, p // block], p % block
        d.vc[b, 1, r, 5] = 0x7F
        d.vc[b, 1, r, 63] = 0xFF
        d.kc[b, 0, r, 2] = 0x7F
        out = run(ops, d, dtype)[0]
        first = rows - back          # the first row that sees p
        assert torch.equal(out[:first], clean[:first]) and torch.equal(out[rows:], clean[rows:])
        assert torch.isnan(out[first:rows, :2]).all()                  # heads 0, 1 read cache head 0: a NaN score
        assert torch.isnan(out[first:rows, 2:, [5, 63]]).all()
        keep = [i for i in range(64) if i not in (5, 63)]
        assert torch.equal(out[first:rows, 2:][:, :, keep], clean[first:rows, 2:][:, :, keep])
    # A block of later positions alone, with NaN scales: the rows before it do not see it.
    first_of_block = (length - 1) // block * block
    hidden = length - first_of_block
    if hidden < rows:
        d = Case([length, 90], [rows, 1], 4, 2, 64, block, seed=length)
        d.vs[d.table[0, first_of_block // block]] = np.nan
        out = run(ops, d, dtype)[0]
        assert torch.equal(out[: rows - hidden], clean[: rows - hidden])
        assert torch.isnan(out[rows - hidden: rows]).all()
    assert ops.fp8blk_device_status(clear=True) == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_queries_that_are_not_finite(ops, dtype):
    c = Case([70], [3], 4, 2, 64, 16, seed=12)
    clean = run(ops, c, dtype)[0]
    c.q[1, 2, 5] = np.nan
    c.q[2, 0, 9] = np.inf
    out = run(ops, c, dtype)[0]
    assert torch.isnan(out[1, 2]).all() and torch.isnan(out[2, 0]).all()
    out[1, 2], out[2, 0] = clean[1, 2], clean[2, 0]
    assert torch.equal(out, clean)


def test_bad_ids_and_lengths_are_flagged(ops):
    c = Case([70, 40], [2, 2], 2, 1, 64, 16, seed=13)
    clean = run(ops, c, torch.float32)[0]
    for bad in (-1, c.kc.shape[0], 2 ** 31 - 1):
        d = Case([70, 40], [2, 2], 2, 1, 64, 16, seed=13)
        d.table[0, 1] = bad
        out = run(ops, d, torch.float32)[0]
        assert ops.fp8blk_device_status(clear=True) == ops.STATUS_BAD_KV
        assert torch.isnan(out[:2]).all() and torch.equal(out[2:], clean[2:])
    d = Case([70, 40], [2, 2], 2, 1, 64, 16, seed=13)
    d.lens[0] = 16 * d.table.shape[1] + 5
    out = run(ops, d, torch.float32)[0]
    assert ops.fp8blk_device_status(clear=True) == ops.STATUS_BAD_KV
    assert torch.isnan(out[:2]).all() and torch.equal(out[2:], clean[2:])
    d.lens[0] = -4
    out = run(ops, d, torch.float32)[0]
    assert ops.fp8blk_device_status(clear=True) == ops.STATUS_BAD_KV
    assert (out[:2] == 0).all() and torch.equal(out[2:], clean[2:])


@pytest.mark.parametrize("heads,kv,rows", [(32, 4, 4), (8, 8, 1)])
@pytest.mark.parametrize("n", [20, 50])
def test_lengths_far_past_the_table(ops, n, heads, kv, rows):
    """They make their own rows NaN, whatever their sum, and take no longer than the table is wide."""
    c = Case([40 + 7 * s for s in range(n)], [rows] * n, heads, kv, 64, 16, seed=15)
    want, _, peak, spread = ref.kv_attn(c.q.astype(np.float64), c.kc, c.ks, c.vc, c.vs, c.table, c.lens, c.starts, c.scale)
    u = 2.0 ** -16 + (c.dim + 16) * 2.0 ** -24  # check's bound for f32
    tol = (2 * u * peak[:, :, None] + 2.0 ** -16 + 2.0 ** -19) * spread
    c.lens[::2] = 2 ** 31 - 1
    c.lens[0] = 16 * c.table.shape[1] + 129 + 128
    out = run(ops, c, torch.float32)[0]
    assert ops.fp8blk_device_status(clear=True) == ops.STATUS_BAD_KV
    assert torch.isnan(out.view(n, -1)[::2]).all()
    near = np.abs(out.cpu().numpy().astype(np.float64) - want) <= tol
    assert near.reshape(n, -1)[1::2].all()


def test_bad_row_starts_are_flagged(ops):
    c = Case([70, 40, 30], [2, 2, 2], 2, 1, 64, 16, seed=14)
    clean = run(ops, c, torch.float32)[0]
    for starts in ([0, 2, 4, 7], [0, 6, 4, 6], [-1, 2, 4, 6]):
        d = Case([70, 40, 30], [2, 2, 2], 2, 1, 64, 16, seed=14)
        d.starts[:] = starts
        q = to_dev(d.q)
        ws = ops.kv_attn_workspace(3, 2, 2, 1, 64, DEV)
        out = torch.full_like(q, 7.0)
        dev = d.dev()
        ops.fp8blk_kv_attn(q, *dev, 2, d.scale, ws, out=out)
        assert ops.fp8blk_device_status(clear=True) == ops.STATUS_BAD_KV
        for s in range(3):
            if 0 <= starts[s] and 0 <= starts[s + 1] - starts[s] <= 2 and starts[s + 1] <= 6:
                assert torch.equal(out[starts[s]: starts[s + 1]], clean[starts[s]: starts[s + 1]])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strided_queries_side_stream_and_no_lse(ops, dtype):
    c = Case([150, 33], [4, 4], 8, 2, 64, 32, seed=15)
    want, _, q = run(ops, c, dtype)
    fused = torch.zeros((8, 20, 64), dtype=dtype, device=DEV)
    fused[:, 3:11] = q
    dev = c.dev()
    ws = ops.kv_attn_workspace(2, 4, 8, 2, 64, DEV)
    big = torch.full((8, 10, 64), 5.0, dtype=dtype, device=DEV)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        ops.fp8blk_kv_attn(fused[:, 3:11], *dev, 4, c.scale, ws, out=big[:, 1:9])
    side.synchronize()
    assert torch.equal(big[:, 1:9], want)
    assert (big[:, 0] == 5).all() and (big[:, 9] == 5).all()


def test_repeats_bit_for_bit_and_in_a_graph(ops):
    c = Case([900, 33, 257], [8, 1, 5], 8, 2, 128, 64, seed=16)
    dev = c.dev()
    q = to_dev(c.q)
    ws = ops.kv_attn_workspace(3, 8, 8, 2, 128, DEV)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
    ops.fp8blk_kv_attn(q, *dev, 8, c.scale, ws, out=out, lse=lse)
    first = out.clone()
    for _ in range(20):
        ops.fp8blk_kv_attn(q, *dev, 8, c.scale, ws, out=out)
        assert torch.equal(out, first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.fp8blk_kv_attn(q, *dev, 8, c.scale, ws, out=out)
    dev[5].copy_(torch.tensor([500, 20, 100], dtype=torch.int32))  # other lengths, the same graph
    c.lens[:] = [500, 20, 100]
    g.replay()
    torch.cuda.synchronize()
    want = ref.kv_attn(c.q.astype(np.float64), c.kc, c.ks, c.vc, c.vs, c.table, c.lens, c.starts, c.scale)[0]
    assert np.abs(out.cpu().numpy() - want).max() < 1e-3
    assert ops.fp8blk_device_status(clear=True) == 0


def test_far_into_a_long_pool(ops):
    """Blocks whose byte offset is past 2^31."""
    blocks, kv, block, dim = 70000, 2, 128, 128
    c = Case([300], [2], 4, kv, dim, block, seed=17)
    used = c.table[0]
    far = np.array([blocks - 1, 3, blocks - 2], np.int32)
    dev = c.dev()
    pools = []
    for a in dev[:4]:
        p = torch.zeros((blocks, *a.shape[1:]), dtype=a.dtype, device=DEV)
        p[torch.from_numpy(far.astype(np.int64)).to(DEV)] = a[torch.from_numpy(used.astype(np.int64)).to(DEV)]
        pools.append(p)
    want = run(ops, c, torch.bfloat16)[0]
    c.table = far[None].copy()
    got = run(ops, c, torch.bfloat16, dev=pools + [to_dev(c.table), dev[5], dev[6]])[0]
    assert torch.equal(got, want)


def test_workspace_is_left_ready_for_other_shapes(ops):
    """One workspace, sized for the largest, serves smaller calls in between."""
    big = Case([900, 700], [8, 8], 8, 2, 64, 64, seed=18)
    small = Case([130], [1], 4, 2, 64, 64, seed=19)
    ws = ops.kv_attn_workspace(2, 8, 8, 2, 64, DEV)
    want = [run(ops, big, torch.float32)[0], run(ops, small, torch.float32)[0]]
    db, ds = big.dev(), small.dev()
    for _ in range(3):
        a = ops.fp8blk_kv_attn(to_dev(big.q), *db, 8, big.scale, ws)
        b = ops.fp8blk_kv_attn(to_dev(small.q), *ds, 1, small.scale, ws)
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])
