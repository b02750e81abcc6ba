"""GPU tests of fp8blk_kv_attn_chunk against a plain 64-bit restatement.

Tolerance, from the arithmetic.  Let A be the largest scale * sum_d |q_d k_td| over the row's tokens.  A score is off by at
most u A, u = (dim + 24) 2^-24: f32 sums over dim, q to 2^-22 of each element, the scale and the exponent's own rounding.  A
weight is off by that, by 2^-21 (exponential, and the denominator's share of it), and by w, to which it is carried into the
second product: f16 has 11 significant bits, so a rounding is off by half of 2^-10 of the value at most, w = 2^-11 for bf16
(one f16), and 2^-22 for f32 (a second one rounds what the first leaves, 2^-11 of it).  (With tokens (v, -v) of weights
1/2 each both roundings show in full.)  Or it is off by 2^-30 of the row's largest p |s_v| where f16 ends, times a code of
at most 448, for each token.  Sums over n tokens go through n / 16 + 32 additions of f32 accuracy (2^-23: the tensor
cores may cut).  So
  |out - exact| <= (2 u A + w + 2^-20 + (n / 16 + 32) 2^-23) sum_t p_t |v_t| + 2^-30 448 n max_t p_t |s_v(t)|
                   (+ 2^-8 |exact|, the rounding to bf16)
  |lse - exact| <= u A + 2^-20 + (n / 16 + 32) 2^-23 + 2^-23 |lse|."""
import numpy as np
import pytest
import torch

import _chunk_ref as cref
from _helpers import to_dev
from test_kv_attn_gpu import Case

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.float32, torch.bfloat16]


@pytest.fixture(scope="module")
def ops():
    from fp8_block_scaled_fp8blk_gb300 import ops as o
    o.fp8blk_device_status(clear=True)
    yield o
    assert o.fp8blk_device_status(clear=True) == 0


def run(ops, c, dtype, q=None, out=None, dev=None, scale=None):
    dev = dev or c.dev()
    q = to_dev(c.q).to(dtype) if q is None else q
    ws = ops.kv_attn_chunk_workspace(c.heads, c.kv, c.dim, DEV)
    ws.fill_(0xFF)  # whatever it holds: nothing is read that the call has not written
    lse = torch.full(q.shape[:2], 7.0, dtype=torch.float32, device=DEV)
    out = ops.fp8blk_kv_attn_chunk(q, *dev, c.scale if scale is None else scale, ws, out=out, lse=lse)
    return out, lse, q


def compare(c, out, lse, q, dtype, scale=None):
    host = (c.kc, c.ks, c.vc, c.vs, c.table, c.lens, c.starts)
    want, wlse, peak, spread, seen, top = cref.attn(q.float().cpu().numpy().astype(np.float64), *host, c.scale if scale is None else scale)
    tol, tl = cref.tolerances(want, wlse, peak, spread, seen, top, c.dim, dtype is torch.bfloat16)
    g, gl = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    assert np.isfinite(g).all()
    ratio = np.abs(g - want) / np.maximum(tol, 1e-300)
    assert (np.abs(g - want) <= tol).all(), (float(ratio.max()), np.unravel_index(ratio.argmax(), ratio.shape))
    assert np.array_equal(np.isneginf(gl), np.isneginf(wlse))
    fin = np.isfinite(wlse)
    assert (np.abs(gl - wlse)[fin] <= tl[fin]).all(), float((np.abs(gl - wlse)[fin] / tl[fin]).max())


def check(ops, c, dtype, **kw):
    out, lse, q = run(ops, c, dtype, **kw)
    assert ops.fp8blk_device_status(clear=True) == 0
    compare(c, out, lse, q, dtype, kw.get("scale"))
    return out, lse, q


SHAPES = [  # lens, rows, heads, kv, dim, block
    ([1], [1], 1, 1, 16, 16),
    ([40], [40], 1, 1, 64, 16),
    ([128], [128], 1, 1, 128, 128),
    ([129, 127], [129, 127], 1, 1, 128, 64),
    ([300], [300], 2, 2, 128, 32),
    ([257], [33], 8, 1, 128, 64),
    ([600, 5, 64], [70, 5, 1], 8, 2, 128, 64),
    ([513, 40, 900], [100, 3, 250], 15, 3, 80, 16),
    ([260, 131], [9, 131], 16, 2, 96, 64),
    ([200], [200], 4, 2, 256, 32),
    ([129, 500], [70, 90], 10, 2, 192, 128),
    ([400], [17], 32, 1, 48, 16),          # 32 query heads on one cache head
    ([70], [3], 300, 1, 32, 16),           # more query heads a cache head than a tile has rows
    ([90, 33], [40, 33], 3, 3, 208, 16),
    ([1000], [1000], 2, 1, 112, 128),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens,rows,heads,kv,dim,block", SHAPES)
def test_shapes(ops, lens, rows, heads, kv, dim, block, dtype):
    check(ops, Case(lens, rows, heads, kv, dim, block, seed=sum(lens) + dim), dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens,rows,heads,kv,dim,block", [
    ([6000], [5], 8, 1, 128, 64),            # one unit in many parts
    ([5000, 17, 3000], [40, 17, 2], 4, 2, 64, 16),
    ([9000], [10], 2, 1, 256, 128),
    ([2500, 2500], [600, 300], 4, 1, 128, 32),
])
def test_units_in_parts(ops, lens, rows, heads, kv, dim, block, dtype):
    check(ops, Case(lens, rows, heads, kv, dim, block, seed=sum(lens)), dtype)


@pytest.mark.parametrize("dtype", TYPES)
def test_many_requests(ops, dtype):
    """More requests than the kernel has threads, some without rows, some without tokens."""
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 40, 1300)
    rows = np.minimum(rng.integers(0, 9, 1300), lens + 1)
    check(ops, Case(lens, rows, 2, 1, 32, 16, seed=4), dtype)


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_that_see_nothing(ops, dtype):
    """More rows than tokens (the first ones sit before position 0), an empty cache, no rows at all."""
    out, lse, _ = check(ops, Case([3, 0, 20, 0, 200], [10, 150, 0, 1, 300], 4, 2, 64, 16, seed=5), dtype)
    assert (out[:7] == 0).all() and torch.isneginf(lse[:7]).all() and torch.isfinite(lse[7:10]).all()
    assert (out[10:161] == 0).all() and torch.isneginf(lse[10:161]).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scale", [-0.3, 0.0, 3.0, 1e-6])
def test_softmax_scales(ops, dtype, scale):
    check(ops, Case([300], [60], 4, 1, 64, 32, seed=6), dtype, scale=scale)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 256])
def test_any_cache_scale(ops, dtype, dim):
    """Scales that are no powers of two, negative, zero, far apart, and smaller than 2^-126."""
    c = Case([700, 90], [200, 90], 4, 2, dim, 16, seed=7)
    rng = np.random.default_rng(8)
    for s, low in ((c.ks, -9), (c.vs, -60)):
        used = np.isfinite(s)
        x = rng.uniform(1, 2, s.shape) * np.exp2(rng.integers(low, 1, s.shape)) * rng.choice([-1, 1], s.shape)
        x = np.where(rng.random(s.shape) < 0.1, 0.0, x)
        s[used] = x[used].astype(np.float32)
    c.ks[c.ks != 0] *= 2.0 ** -6
    c.vs[c.table[1, 2], 0] = 2.0 ** -140
    check(ops, c, dtype)


@pytest.mark.parametrize("dtype", TYPES)
def test_a_row_keeps_values_far_below_others(ops, dtype):
    """The largest value scale belongs to blocks that a row gives no weight: its own small values keep their bits."""
    c = Case([256], [128], 1, 1, 64, 16, seed=9, spread=0)
    c.q *= 30.0
    c.vs[c.table[0]] = np.exp2(np.random.default_rng(10).integers(-70, 30, (16, 1))).astype(np.float32)
    check(ops, c, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("grow", [1.0, -1.0])
def test_maxima_that_rise_and_fall(ops, dtype, grow):
    """Scores that grow (or fall) by thousands along the cache: the reference moves at every tile, or never again."""
    c = Case([1500], [300], 2, 1, 128, 64, seed=11, spread=0)
    c.ks[c.table[0]] = (2.0 ** -6 * np.exp(grow * np.linspace(-3, 3, 24)[:, None])).astype(np.float32)
    c.q = np.abs(c.q) * 3
    check(ops, c, dtype)


@pytest.mark.parametrize("dtype", TYPES)
def test_queries_of_any_size(ops, dtype):
    """Rows of zeros, of the type's smallest and largest values, with one element far above the rest."""
    c = Case([300], [80], 2, 1, 64, 64, seed=12)
    c.q[0], c.q[1], c.q[2] = 0.0, 1e-38, 1e-41
    c.q[3] *= 1e30
    c.q[4, :, 5] = 3e4
    c.scale = 1e-6
    check(ops, c, dtype)
    # A row that is not finite is NaN, and no other is.
    q = to_dev(c.q).to(dtype)
    q[10, 1, 3], q[11, 0, 0] = float("nan"), float("inf")
    out, lse, _ = run(ops, c, dtype, q=q)
    bad = torch.isnan(lse)
    assert bad.nonzero().tolist() == [[10, 1], [11, 0]] and torch.equal(torch.isnan(out).all(2), bad) and torch.equal(torch.isnan(out).any(2), bad)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [128, 256])
@pytest.mark.parametrize("rows", [200, 4])
def test_nan_codes_and_scales(ops, dtype, dim, rows):
    """NaN codes, scales that are not finite and blocks outside the pool reach the rows that see them, and nothing else."""
    c = Case([2300], [rows], 2, 1, dim, 64, seed=13)
    first = 2300 - rows
    clean, clean_lse, q = run(ops, c, dtype)
    assert ops.fp8blk_device_status(clear=True) == 0
    at = first + rows // 2                       # a position that the later half of the rows sees
    page, off = c.table[0, at // 64], at % 64

    def affected(kc=None, vc=None, ks=None, vs=None, table=None):
        dev = [to_dev(x if y is None else y) for x, y in ((c.kc, kc), (c.ks, ks), (c.vc, vc), (c.vs, vs), (c.table, table), (c.lens, None),
                                                         (c.starts, None))]
        out, lse, _ = run(ops, c, dtype, q=q, dev=dev)
        return out, lse

    late = torch.arange(rows, device=DEV) >= rows // 2
    kc = c.kc.copy()
    kc[page, 0, off, 3] = 0xFF
    out, lse = affected(kc=kc)
    assert torch.equal(torch.isnan(lse).all(1), late) and torch.equal(torch.isnan(out).all(2).all(1), late)
    assert torch.equal(out[~late], clean[~late]) and torch.equal(lse[~late], clean_lse[~late])
    vc = c.vc.copy()
    vc[page, 0, off, 5] = 0x7F
    out, lse = affected(vc=vc)
    assert torch.equal(torch.isnan(out[:, 0, 5]), late) and not torch.isnan(lse).any()
    others = [d for d in range(dim) if d != 5]
    assert not torch.isnan(out[:, :, others]).any() and torch.equal(out[~late], clean[~late])
    # A whole block: from its first token on.
    head = int(at // 64 * 64 - first)            # the first row that sees any of it
    sees = torch.arange(rows, device=DEV) >= head
    for value in (float("inf"), float("nan")):
        ks, vs = c.ks.copy(), c.vs.copy()
        ks[page, 0], vs[page, 0] = value, value
        for kw in (dict(ks=ks), dict(vs=vs)):
            out, lse = affected(**kw)
            assert torch.equal(torch.isnan(out).all(2).all(1), sees) and torch.equal(torch.isnan(out).any(2).any(1), sees)
            assert torch.equal(out[~sees], clean[~sees])
    assert ops.fp8blk_device_status(clear=True) == 0
    for bad in (-1, len(c.kc), 2 ** 31 - 1):
        table = c.table.copy()
        table[0, at // 64] = bad
        out, lse = affected(table=table)
        assert ops.fp8blk_device_status(clear=True) == ops.STATUS_BAD_KV
        assert torch.equal(torch.isnan(out).all(2).all(1), sees) and torch.equal(out[~sees], clean[~sees])


def test_lengths_and_starts_out_of_range(ops):
    c = Case([100, 64, 90], [20, 10, 30], 2, 1, 64, 16, seed=14)
    kc, ks, vc, vs, table, lens, starts = c.dev()
    want, want_lse, q = run(ops, c, torch.float32)
    cases = []
    long = lens.clone()
    long[1] = 2 ** 31 - 1                        # past the table: its rows are NaN
    cases.append((long, starts, slice(20, 30), True))
    negative = lens.clone()
    negative[1] = -5                             # counts as 0
    cases.append((negative, starts, slice(20, 30), False))
    for at, value in ((1, -3), (3, 61)):         # rows outside: those requests are skipped, their rows left alone
        s = starts.clone()
        s[at] = value
        cases.append((lens, s, None, False))
    for l, s, rows, nan in cases:
        out = torch.full_like(q, 5.0)
        got, lse, _ = run(ops, c, torch.float32, q=q, out=out, dev=(kc, ks, vc, vs, table, l, s))
        assert ops.fp8blk_device_status(clear=True) == ops.STATUS_BAD_KV
        if rows is not None:
            assert torch.isnan(got[rows]).all() if nan else (got[rows] == 0).all()
            keep = torch.ones(len(q), dtype=torch.bool, device=DEV)
            keep[rows] = False
            assert torch.equal(got[keep], want[keep])
        elif int(s[3]) == 61:
            assert torch.equal(got[:30], want[:30]) and (got[30:] == 5).all() and (lse[30:] == 7).all()
        else:
            assert torch.equal(got[30:], want[30:]) and (got[:20] == 5).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_more_rows_in_the_requests_than_there_are(ops, dtype):
    """Starts that go back give several requests the same rows: nothing is written."""
    c = Case([100, 64, 90], [20, 10, 30], 2, 1, 64, 16, seed=17)
    kc, ks, vc, vs, table, lens, _ = c.dev()
    starts = torch.tensor([0, 60, 0, 60], dtype=torch.int32, device=DEV)
    q = to_dev(c.q).to(dtype)
    out, lse, _ = run(ops, c, dtype, q=q, out=torch.full_like(q, 5.0), dev=(kc, ks, vc, vs, table, lens, starts))
    assert ops.fp8blk_device_status(clear=True) == ops.STATUS_BAD_KV
    assert (out == 5).all() and (lse == 7).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_strides_and_rows_behind_the_last(ops, dtype):
    """Queries inside a fused projection, outputs inside a wider buffer; rows behind the last request stay as they are."""
    c = Case([300, 77], [130, 20], 4, 2, 80, 32, seed=15)
    want, want_lse, q = run(ops, c, dtype)
    wide = torch.full((160, 9, 80), 3.0, dtype=dtype, device=DEV)
    wide[:150, 2:6] = q
    big = torch.full((160, 6, 80), 9.0, dtype=dtype, device=DEV)
    ws = ops.kv_attn_chunk_workspace(4, 2, 80, DEV)
    lse = torch.full((160, 4), 9.0, device=DEV)
    ops.fp8blk_kv_attn_chunk(wide[:, 2:6], *c.dev(), c.scale, ws, out=big[:, 1:5], lse=lse)
    assert torch.equal(big[:150, 1:5], want) and torch.equal(lse[:150], want_lse)
    assert (big[150:] == 9).all() and (lse[150:] == 9).all() and (big[:, 0] == 9).all() and (big[:, 5] == 9).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_as_kv_attn_for_few_rows(ops, dtype):
    """The same rows through fp8blk_kv_attn: within the sum of both calls' bounds."""
    c = Case([700, 33, 5], [8, 3, 5], 8, 2, 128, 64, seed=16)
    out, lse, q = check(ops, c, dtype)
    ws = ops.kv_attn_workspace(3, 8, 8, 2, 128, DEV)
    lse2 = torch.empty_like(lse)
    out2 = ops.fp8blk_kv_attn(q, *c.dev(), 8, c.scale, ws, lse=lse2)
    assert (out.float() - out2.float()).abs().max() <= (2e-2 if dtype is torch.bfloat16 else 2e-4)
    assert (lse - lse2).abs().max() <= 2e-3


def test_same_result_every_time_captured_and_on_two_streams(ops):
    """Bit for bit, call by call; replayed from a graph on new inputs; two calls at once on two streams, each its workspace."""
    a, b = Case([1500, 40], [300, 40], 8, 2, 128, 64, seed=17), Case([900], [77], 4, 1, 256, 32, seed=18)
    da, db = a.dev(), b.dev()
    qa, qb = to_dev(a.q).to(torch.bfloat16), to_dev(b.q)
    wa, wb = ops.kv_attn_chunk_workspace(8, 2, 128, DEV), ops.kv_attn_chunk_workspace(4, 1, 256, DEV)
    want_a, want_b = ops.fp8blk_kv_attn_chunk(qa, *da, a.scale, wa), ops.fp8blk_kv_attn_chunk(qb, *db, b.scale, wb)
    for _ in range(5):
        assert torch.equal(ops.fp8blk_kv_attn_chunk(qa, *da, a.scale, wa), want_a)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        with torch.cuda.stream(s1):
            x = ops.fp8blk_kv_attn_chunk(qa, *da, a.scale, wa)
        with torch.cuda.stream(s2):
            y = ops.fp8blk_kv_attn_chunk(qb, *db, b.scale, wb)
        torch.cuda.synchronize()
        assert torch.equal(x, want_a) and torch.equal(y, want_b)
    out = torch.zeros_like(qa)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.fp8blk_kv_attn_chunk(qa, *da, a.scale, wa, out=out)
    graph.replay()
    assert torch.equal(out, want_a)
    qa.copy_(torch.roll(qa, 1, 0))
    da[5].copy_(torch.tensor([700, 20], dtype=torch.int32))
    da[6].copy_(torch.tensor([0, 300, 320], dtype=torch.int32))
    graph.replay()
    assert torch.equal(out[:320], ops.fp8blk_kv_attn_chunk(qa, *da, a.scale, wa)[:320])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens,rows,heads,kv,dim,block", [([300], [40], 8, 8, 256, 128), ([129, 500], [70, 90], 10, 2, 192, 128),
                                                          ([513, 40, 900], [100, 3, 250], 15, 3, 80, 16), ([40] * 200, [8] * 200, 2, 1, 32, 16)])
def test_a_hundred_calls_in_a_row(ops, lens, rows, heads, kv, dim, block, dtype):
    """The same bits from calls back to back, with warm and with cold caches."""
    c = Case(lens, rows, heads, kv, dim, block, seed=20)
    dev, q = c.dev(), to_dev(c.q).to(dtype)
    ws, junk = ops.kv_attn_chunk_workspace(heads, kv, dim, DEV), torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    outs = []
    for i in range(100):
        if i % 3 == 0:
            junk.fill_(i)
        outs.append(ops.fp8blk_kv_attn_chunk(q, *dev, c.scale, ws))
    assert all(torch.equal(o, outs[0]) for o in outs)


def test_offsets_past_32_bits(ops):
    """A pool of more than 2^32 bytes, its last blocks in use."""
    kv, block, dim, blocks = 8, 128, 256, 16500
    c = Case([300], [40], 8, 8, 256, 128, seed=19)
    codes = torch.zeros((2, blocks, kv, block, dim), dtype=torch.uint8, device=DEV)
    assert codes[0].numel() > 2 ** 32
    scales = torch.zeros((2, blocks, kv), device=DEV)
    kc, ks, vc, vs, table, lens, starts = c.dev()
    n = len(c.kc)
    for i, (x, s) in enumerate(((kc, ks), (vc, vs))):
        codes[i, -n:], scales[i, -n:] = x, s
    want, _, q = run(ops, c, torch.bfloat16)
    moved = torch.where(table >= 0, table + (blocks - n), table)
    got, _, _ = run(ops, c, torch.bfloat16, q=q, dev=(codes[0], scales[0], codes[1], scales[1], moved, lens, starts))
    assert torch.equal(got, want)
