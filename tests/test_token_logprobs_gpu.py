"""GPU tests of fp8blk_token_logprobs against a plain 64-bit restatement.

Tolerance, from the arithmetic: x - max is one f32 rounding of numbers up to
R = max|x| (2^-24 R each way); the f32 sums of n positive terms, each within
2^-21 of itself (exponential) and summed in a tree, are within 2^-19 relative;
logs and the final differences add a few roundings of numbers up to the result's
size.  So |err| <= 2^-18 (1 + R) for log probabilities and for the entropy, whose
weighted mean of x - max has terms up to 2 R + log n.  Ranks and ids are exact."""
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


def check(ops, logits, targets, top):
    """`logits` a device tensor [n, vocab] (any row stride)."""
    x = logits.float().cpu().numpy().astype(np.float64)
    targets = np.asarray(targets, np.int32)
    got = ops.fp8blk_token_logprobs(logits, to_dev(targets), top)
    logprob, rank, entropy, ids, tops = ref.token_logprobs(x, targets, top)
    assert np.array_equal(got.rank.cpu().numpy(), rank)
    assert np.array_equal(got.top_ids.cpu().numpy(), ids)
    fin = np.where(np.isfinite(x), np.abs(x), 0.0).max(1)
    tol = 2.0 ** -18 * (1.0 + fin)
    for g, w, t in ((got.logprob, logprob, tol), (got.entropy, entropy, tol * 3), (got.top_logprobs, tops, tol[:, None])):
        g = g.cpu().numpy().astype(np.float64)
        assert np.array_equal(np.isnan(g), np.isnan(w))
        ok = (g == w) | (np.abs(g - w) <= t) | np.isnan(w)
        assert ok.all(), float(np.nanmax(np.abs(g - w) / t))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,vocab,top", [(1, 1, 1), (1, 2, 0), (3, 7, 7), (2, 33, 32), (5, 1000, 5), (1, 4097, 20), (160, 777, 3),
                                         (2, 32768, 1), (3, 32769, 32), (8, 131072, 5), (2, 100003, 10), (1, 262144, 32),
                                         (200, 5003, 0)])
def test_matches_plain(ops, dtype, n, vocab, top):
    rng = np.random.default_rng(n + vocab + top)
    x = to_dev((2.5 * rng.standard_normal((n, vocab))).astype(np.float32)).to(dtype)
    check(ops, x, rng.integers(0, vocab, n), top)


def test_ties_take_the_lowest_index(ops):
    rng = np.random.default_rng(1)
    x = rng.integers(-2, 3, (4, 5000)).astype(np.float32)
    x[1] = 0.0
    x[1, ::3] = -0.0
    x[2] = 7.5
    x[3, 100:] = x[3, 99]
    check(ops, to_dev(x), [4999, 3, 4000, 100], 32)


@pytest.mark.parametrize("vocab", [100, 9000, 70001])
def test_masked_infinite_and_nan_rows(ops, vocab):
    rng = np.random.default_rng(vocab)
    x = (2 * rng.standard_normal((9, vocab))).astype(np.float32)
    x[0, 5:] = -np.inf                # few tokens allowed
    x[1] = -np.inf                    # none
    x[2] = -np.inf
    x[2, vocab - 1] = -1e30           # exactly one
    x[3, vocab // 2] = np.nan
    x[4, vocab // 3] = np.inf
    x[5] = np.finfo(np.float32).min   # masks of the type's lowest value
    x[5, 7] = 1.0
    x[6] = np.finfo(np.float32).min
    x[7] = 3e38
    x[8, ::2] = -np.inf
    check(ops, to_dev(x), [2, 0, vocab - 1, vocab // 2, vocab // 3, 7, 50, 99, 1], 8)


def test_sorted_rows_and_large_logits(ops):
    """All of the top in one thread's reach, or spread over the ends; logits of hundreds."""
    v = np.linspace(-300, 300, 40000).astype(np.float32)
    x = np.stack([v, v[::-1], np.where(np.arange(40000) < 64, 300, -300) + np.arange(40000) % 7])
    check(ops, to_dev(np.ascontiguousarray(x, dtype=np.float32)), [39999, 5, 63], 32)


def test_targets_outside(ops):
    x = to_dev(np.random.default_rng(3).standard_normal((3, 50)).astype(np.float32))
    check(ops, x, [-1, 4, -1], 2)
    got = ops.fp8blk_token_logprobs(x, to_dev(np.array([50, 4, -2], np.int32)), 2)
    assert ops.fp8blk_device_status(clear=True) == ops.STATUS_BAD_TARGET
    assert torch.isnan(got.logprob[[0, 2]]).all() and got.rank.tolist()[0] == -1 and got.rank.tolist()[2] == -1
    assert torch.isfinite(got.entropy).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_with_a_stride_and_an_odd_start(ops, dtype):
    rng = np.random.default_rng(4)
    buf = to_dev(rng.standard_normal((6, 2003)).astype(np.float32)).to(dtype)
    check(ops, buf[:, 1:1990], rng.integers(0, 1989, 6), 9)
    check(ops, buf[1:, 7:1000], rng.integers(0, 993, 5), 4)
    check(ops, buf[2:3, 3:], [5], 4)


def test_agrees_with_the_fused_argmax(ops):
    """top_ids[:, 0] is the head GEMV's token on its own logits."""
    from fp8_block_scaled_fp8blk_gb300 import synth
    c = synth.fp8blk_case(5000, 512, 4, seed=11)
    w, s, x = to_dev(c.codes), to_dev(ops.fp8blk_scales_from_e8m0(c.scale_e8m0)), to_dev(c.x)
    ws = ops.argmax_workspace(4, 5000, 512, "cuda:0")
    logits = torch.empty((4, 5000), dtype=torch.float32, device="cuda:0")
    tok = ops.fp8blk_gemv_argmax(w, s, x, ws, logits=logits)
    got = ops.fp8blk_token_logprobs(logits, tok, 3)
    assert torch.equal(got.top_ids[:, 0], tok) and got.rank.tolist() == [0, 0, 0, 0]
    assert torch.equal(got.top_logprobs[:, 0], got.logprob)


def test_repeats_bit_for_bit_and_in_a_graph(ops):
    x = torch.randn((5, 70000), device="cuda:0")
    t = torch.arange(5, dtype=torch.int32, device="cuda:0")
    a = ops.fp8blk_token_logprobs(x, t, 20)
    torch.cuda.synchronize()
    out = ops.token_logprobs_buffers(5, 20, "cuda:0")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.fp8blk_token_logprobs(x, t, 20, out=out)
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(a, out))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab,start,top", [(1, 0, 1), (31, 1, 20), (1003, 3, 32), (70001, 1, 20), (262144, 0, 32)])
@pytest.mark.parametrize("n", [310, 461])
def test_many_rows_one_cta_each(ops, dtype, n, vocab, start, top):
    """Rows enough that each is one CTA's, wide or narrow: every kind of row at many places, the same everywhere."""
    rng = np.random.default_rng(vocab + n)
    kinds = (2.5 * rng.standard_normal((9, vocab))).astype(np.float32)
    kinds[1] = np.sort(kinds[1])
    kinds[2] = np.sort(kinds[2])[::-1]
    kinds[3] = rng.integers(-1, 2, vocab)      # ties
    kinds[4] = 0.0                             # nothing but ties
    kinds[5, vocab // 2:] = -np.inf
    kinds[6] = -np.inf
    kinds[7, vocab // 2] = np.nan
    kinds[8, : vocab // 2] = np.finfo(np.float32).min / 2
    buf = torch.zeros((9, start + vocab), dtype=dtype, device="cuda:0")
    buf[:, start:] = to_dev(kinds).to(dtype)
    targets = rng.integers(0, vocab, 9).astype(np.int32)
    top = min(top, vocab)
    check(ops, buf[:, start:], targets, top)
    which = torch.arange(n, device="cuda:0") % 9
    got = ops.fp8blk_token_logprobs(buf[which][:, start:], to_dev(targets)[which], top)
    x = buf[:, start:].float().cpu().numpy().astype(np.float64)
    logprob, rank, entropy, ids, tops = ref.token_logprobs(x, targets, top)
    k = which.cpu().numpy()
    assert np.array_equal(got.rank.cpu().numpy(), rank[k]) and np.array_equal(got.top_ids.cpu().numpy(), ids[k])
    fin = np.where(np.isfinite(x), np.abs(x), 0.0).max(1)
    tol = 2.0 ** -18 * (1.0 + fin)
    for g, w, t in ((got.logprob, logprob, tol), (got.entropy, entropy, tol * 3), (got.top_logprobs, tops, tol[:, None])):
        g = g.cpu().numpy().astype(np.float64)
        ok = (g == w[k]) | (np.abs(g - w[k]) <= t[k]) | (np.isnan(w[k]) & np.isnan(g))
        assert ok.all()


def test_many_rows_far_offsets(ops):
    """Rows whose byte offset is past 2^32."""
    n, vocab = 9000, 131072
    x = torch.zeros((n, vocab), dtype=torch.float32, device="cuda:0")
    x[-1] = torch.randn(vocab, device="cuda:0")
    t = torch.full((n,), 9, dtype=torch.int32, device="cuda:0")
    got = ops.fp8blk_token_logprobs(x, t, 2)
    want = ref.token_logprobs(x[-1:].cpu().numpy().astype(np.float64), np.array([9]), 2)
    assert int(got.rank[-1]) == want[1][0] and np.array_equal(got.top_ids[-1].cpu().numpy(), want[3][0])
    assert abs(float(got.logprob[-1]) - want[0][0]) < 1e-4
    assert torch.equal(got.rank[:-1], torch.full_like(got.rank[:-1], 9))
