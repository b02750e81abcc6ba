"""fp8blk_kv_attn's give-up path, exercised without hanging anything: with a wait limit of zero the first role that finds
its operand not there gives up, the kernel lets its copies and products land (with the fixed bound) and returns."""
import pytest
import torch

from _helpers import to_dev
from test_kv_attn_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from fp8_block_scaled_fp8blk_gb300 import ops as o
    o.fp8blk_device_status(clear=True)
    yield o
    o.set_wait_limit()
    assert o.fp8blk_device_status(clear=True) == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lens,rows,heads,kv,dim", [([4000], [8], 8, 1, 64), ([2000, 300, 0, 900], [8, 1, 2, 5], 8, 2, 128),
                                                    ([700] * 60, [1] * 60, 4, 2, 256)])
def test_a_wait_that_runs_out(ops, dtype, lens, rows, heads, kv, dim):
    """The status word says so, each row and head is right or NaN in both outputs, and the next call is right again."""
    c = Case(lens, rows, heads, kv, dim, 64, seed=51)
    dev, q = c.dev(), to_dev(c.q).to(dtype)
    ws = ops.kv_attn_workspace(len(lens), max(rows), heads, kv, dim, "cuda:0")
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float32, device="cuda:0")

    def call():
        ops.fp8blk_kv_attn(q, *dev, max(rows), c.scale, ws, out=out, lse=lse)
        return out.clone(), lse.clone(), ops.fp8blk_device_status(clear=True)

    want, want_lse, status = call()
    assert status == 0
    gave_up = 0
    ops.set_wait_limit(0)
    try:
        for _ in range(10):
            got, got_lse, status = call()
            assert status & ~ops.STATUS_WAIT_TIMEOUT == 0
            gave_up += status != 0
            lost = torch.isnan(got_lse)
            assert torch.isnan(got[lost]).all() and (status != 0 or not lost.any())
            assert torch.equal(got[~lost], want[~lost]) and torch.equal(got_lse[~lost], want_lse[~lost])
    finally:
        ops.set_wait_limit()
    assert gave_up > 0, "no wait ran out with a zero limit"
    got, got_lse, status = call()
    assert status == 0 and torch.equal(got, want) and torch.equal(got_lse, want_lse)
