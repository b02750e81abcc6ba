"""Host-side refusals of fp8blk_kv_map_held (no GPU)."""
import pytest
import torch

A16, A8, A4, A1 = 0x10000, 0x10008, 0x10004, 0x10001  # fake, never-dereferenced addresses


@pytest.fixture(scope="module")
def ops():
    from fp8_block_scaled_fp8blk_gb300 import build
    build.build()
    from fp8_block_scaled_fp8blk_gb300 import ops as o
    return o


def test_refusals(ops):
    lib = ops.raw_library()

    def call(ctx=A4, new=A8, held=0x20000, table=A4, free=A4, head=A4, lens=A16, starts=A4, slots=A16, pos=A16, out=A8,
             held_out=0x20010, n=4, width=8, n_free=10, block=16, most=64):
        return lib.fp8blk_kv_map_held(ctx, new, held, table, free, head, lens, starts, slots, pos, out, held_out, n, width,
                                      n_free, block, most, None)

    for kw, code in ((dict(held=None), ops.EINVAL), (dict(held_out=None), ops.EINVAL), (dict(held_out=0x20000), ops.EINVAL),
                     (dict(held_out=A4), ops.EINVAL), (dict(held_out=A8), ops.EINVAL), (dict(held=A1), ops.EALIGN),
                     (dict(held_out=A1), ops.EALIGN), (dict(table=None), ops.EINVAL), (dict(block=24), ops.EINVAL),
                     (dict(n=65537), ops.ERANGE)):
        assert call(**kw) == code, kw


def test_binding(ops):
    lens, table = torch.zeros(1, dtype=torch.int32), torch.zeros((1, 2), dtype=torch.int32)
    for kw in (dict(held=lens), dict(held_out=lens), dict(held=lens, held_out=torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(ValueError):
            ops.fp8blk_kv_map(lens, lens, table, lens, lens, 16, 8, **kw)
    with pytest.raises(TypeError):
        ops.fp8blk_kv_map(lens, lens, table, lens, lens, 16, 8, held=lens.long(), held_out=lens)


def test_an_empty_free_list_may_be_null(ops):
    """Refused for another reason only (a launch would need a GPU)."""
    lib = ops.raw_library()

    def call(free, n_free, most=64):
        return lib.fp8blk_kv_map(A4, A8, A4, free, A4, A16, A4, A16, A16, A8, 4, 8, n_free, 16, most, None)

    assert call(None, 10) == ops.EINVAL
    assert call(None, 0, most=1 << 31) == ops.ERANGE
