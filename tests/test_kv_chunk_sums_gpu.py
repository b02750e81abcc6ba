"""f32's sums of fp8blk_kv_attn_chunk, which each tile loads from tensor memory and stores back: narrow heads, where a tile's
turn is shortest, over many tiles."""
import pytest
import torch

from test_kv_attn_gpu import Case
from test_kv_chunk_gpu import check, ops, run  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [16, 32, 64])
@pytest.mark.parametrize("lens,rows,heads,kv,block", [([6000], [6], 1, 1, 128), ([3000, 2900, 17], [130, 9, 17], 4, 1, 16)])
def test_narrow_heads_over_many_tiles(ops, lens, rows, heads, kv, block, dim):  # noqa: F811
    """Within tolerance of 64 bits (see test_kv_chunk_gpu), and the same bits in every call."""
    c = Case(lens, rows, heads, kv, dim, block, seed=dim + len(lens))
    out, lse, q = check(ops, c, torch.float32)
    for _ in range(20):
        again, lse2, _ = run(ops, c, torch.float32, q=q)
        assert torch.equal(again, out) and torch.equal(lse2, lse)
