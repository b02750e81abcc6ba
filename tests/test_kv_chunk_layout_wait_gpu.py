"""fp8blk_kv_attn_chunk where the layout of a CTA's units gives up: it waits for the place of the unit four before, so with a
wait limit of zero and many units a CTA it stops early, without hanging anything.  What it has not laid out is NaN all the
same, and nothing outside the batch is touched, whatever an earlier batch has left in the workspace."""
import pytest
import torch

from _helpers import to_dev
from test_kv_attn_gpu import Case
from test_kv_chunk_wait_gpu import ops  # noqa: F401

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
GUARD = 300  # rows before and behind the batch's own


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lens,rows,heads,kv,dim", [
    ([20] * 1500, [1] * 1500, 8, 4, 32),                    # some forty whole units a CTA
    ([300, 0, 90] * 150, [40, 2, 90] * 150, 8, 2, 128),     # empty caches among them
    ([5000] * 12, [700] * 12, 6, 2, 64),                    # units in parts at a range's ends
    ([130] * 200, [70] * 200, 4, 2, 256),
])
def test_a_layout_that_gives_up(ops, dtype, lens, rows, heads, kv, dim):  # noqa: F811
    c = Case(lens, rows, heads, kv, dim, 16, seed=61)
    dev, q = c.dev(), to_dev(c.q).to(dtype)
    n = q.shape[0]
    ws = ops.kv_attn_chunk_workspace(heads, kv, dim, DEV)
    wide, wide_lse = torch.empty((n + 2 * GUARD, heads, dim), dtype=dtype, device=DEV), torch.empty((n + 2 * GUARD, heads), device=DEV)
    out, lse = wide[GUARD: GUARD + n], wide_lse[GUARD: GUARD + n]

    def call():
        wide.fill_(3.0)
        wide_lse.fill_(7.0)
        ops.fp8blk_kv_attn_chunk(q, *dev, c.scale, ws, out=out, lse=lse)
        torch.cuda.synchronize()
        for t, x in ((wide, 3.0), (wide_lse, 7.0)):
            assert (t[:GUARD] == x).all() and (t[GUARD + n:] == x).all(), "rows outside the batch were written"
        return out.clone(), lse.clone(), ops.fp8blk_device_status(clear=True)

    # A larger batch of long units first: what it leaves of its cut units must not reach this one.
    b = Case([4000] * 3, [1500] * 3, heads, kv, dim, 128, seed=62)
    ops.fp8blk_kv_attn_chunk(to_dev(b.q).to(dtype), *b.dev(), b.scale, ws)
    want, want_lse, status = call()
    assert status == 0 and torch.isfinite(want).all()
    ops.set_wait_limit(0)
    gave_up = lost_rows = 0
    try:
        for _ in range(10):
            got, got_lse, status = call()
            assert status & ~ops.STATUS_WAIT_TIMEOUT == 0
            gave_up += status != 0
            lost = torch.isnan(got_lse)
            lost_rows += int(lost.sum())
            assert torch.isnan(got[lost]).all() and (status != 0 or not lost.any())
            assert torch.equal(got[~lost], want[~lost]) and torch.equal(got_lse[~lost], want_lse[~lost])
    finally:
        ops.set_wait_limit()
    assert gave_up > 0 and lost_rows > 0, "no wait ran out with a zero limit"
    got, got_lse, status = call()
    assert status == 0 and torch.equal(got, want) and torch.equal(got_lse, want_lse)
