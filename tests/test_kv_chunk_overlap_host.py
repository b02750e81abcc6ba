"""fp8blk_kv_attn_chunk refuses an out that shares memory with q and is not q itself (no GPU)."""
import pytest

A = 0x100000  # a fake, never-dereferenced address


@pytest.fixture(scope="module")
def ops():
    from fp8_block_scaled_fp8blk_gb300 import build
    build.build()
    from fp8_block_scaled_fp8blk_gb300 import ops as o
    return o


@pytest.mark.parametrize("dtype,es", [(0, 4), (1, 2)])
def test_a_shifted_output_is_refused(ops, dtype, es):
    need = ops.fp8blk_kv_attn_chunk_ws_bytes(8, 2, 128)

    def call(out, q_stride=1024, out_stride=1024, rows=30):
        return ops.raw_library().fp8blk_kv_attn_chunk(A, dtype, A * 8, A * 9, A * 10, A * 11, A * 12, A * 13, A * 14, out, None, A * 16,
                                                      need, 2, rows, 8, 2, 128, 64, 100, 9, q_stride, out_stride, 0.1, None)

    for out in (A + 16, A - 16, A + 1024 * es, A - 1024 * es, A + 29 * 1024 * es, A - 29 * 1024 * es, A + 128 * es):
        assert call(out) == ops.EINVAL, out - A
    assert call(A, out_stride=1032) == ops.EINVAL and call(A + 1024 * es, q_stride=2048, out_stride=1024) == ops.EINVAL
    assert call(A + 1024 * es - 16, q_stride=2048, out_stride=2048) == ops.EINVAL
