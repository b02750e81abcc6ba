"""fp8blk_kv_attn_chunk with out = q: the bits of a call with an output of its own."""
import pytest
import torch

from _helpers import to_dev
from test_kv_attn_gpu import Case
from test_kv_chunk_gpu import DEV, TYPES, ops, run  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens,rows,heads,kv,dim", [([6000], [5], 8, 1, 128), ([300, 40, 900], [300, 3, 250], 15, 3, 80),
                                                    ([700, 0], [500, 2], 4, 2, 256), ([60] * 400, [9] * 400, 8, 4, 64)])
def test_in_place(ops, dtype, lens, rows, heads, kv, dim):  # noqa: F811
    c = Case(lens, rows, heads, kv, dim, 32, seed=71)
    want, want_lse, q = run(ops, c, dtype)
    for _ in range(5):
        x = q.clone()
        out, lse, _ = run(ops, c, dtype, q=x, out=x)
        assert out.data_ptr() == x.data_ptr() and torch.equal(x, want) and torch.equal(lse, want_lse)
    # Between k and v in one fused tensor, which stay as they are.
    fused = torch.full((q.shape[0], heads + 2 * kv, dim), 7.0, dtype=dtype, device=DEV)
    mine = fused[:, kv: kv + heads]
    mine.copy_(to_dev(c.q))
    run(ops, c, dtype, q=mine, out=mine)
    assert torch.equal(mine, want) and (fused[:, :kv] == 7).all() and (fused[:, kv + heads:] == 7).all()
