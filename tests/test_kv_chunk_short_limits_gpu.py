"""fp8blk_kv_attn_chunk with wait limits of some microseconds, so that single roles give up in the middle of a CTA's many units
while others go on: rows are right, bit by bit, or NaN in both outputs.  (A unit of 128 rows or fewer is shared by two products,
and is written out from both; so are most of these.)"""
import numpy as np
import pytest
import torch

from _helpers import to_dev
from test_kv_attn_gpu import Case
from test_kv_chunk_wait_gpu import ops  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,kv,dim,longest,dtype", [(4, 1, 128, 200, torch.bfloat16), (16, 2, 128, 200, torch.bfloat16),
                                                        (4, 4, 128, 500, torch.bfloat16), (4, 2, 64, 300, torch.float32),
                                                        (4, 2, 256, 300, torch.bfloat16), (4, 2, 256, 300, torch.float32)])
def test_right_or_nan(ops, heads, kv, dim, longest, dtype):  # noqa: F811
    rng = np.random.default_rng(1)
    lens = rng.integers(1, longest + 1, 600)
    c = Case(lens, np.minimum(lens, rng.integers(1, 41, 600)), heads, kv, dim, 64, seed=3)
    c.vc[c.table[::7, 0], :, 0, dim - 1] = 0x7F  # a NaN that every row of some requests sees, and the other elements do not
    dev, q = c.dev(), to_dev(c.q).to(dtype)
    ws = ops.kv_attn_chunk_workspace(heads, kv, dim, "cuda:0")
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float32, device="cuda:0")

    def call():
        out.fill_(3.0)
        lse.fill_(7.0)
        ops.fp8blk_kv_attn_chunk(q, *dev, c.scale, ws, out=out, lse=lse)
        return out.clone(), lse.clone(), ops.fp8blk_device_status(clear=True)

    want, want_lse, status = call()
    assert status == 0 and torch.isnan(want[..., -1]).any() and not torch.isnan(want[..., :-1]).any()
    gave_up = 0
    try:
        for limit in (0, 1000, 4000, 8000, 12000, 15000, 20000):
            ops.set_wait_limit(limit)
            for _ in range(60):
                got, got_lse, status = call()
                gave_up += status != 0
                assert status & ~ops.STATUS_WAIT_TIMEOUT == 0
                lost = torch.isnan(got_lse)
                assert torch.isnan(got[lost]).all() and (status != 0 or not lost.any())
                same = (got == want) | (torch.isnan(got) & torch.isnan(want))
                assert same[~lost].all() and torch.equal(got_lse[~lost], want_lse[~lost]), limit
    finally:
        ops.set_wait_limit()
    assert gave_up > 0, "no wait ran out"
    got, got_lse, status = call()
    assert status == 0 and torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got_lse, want_lse)
