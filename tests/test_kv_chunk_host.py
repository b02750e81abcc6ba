"""Host-side refusals of fp8blk_kv_attn_chunk (no GPU)."""
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
    need = ops.fp8blk_kv_attn_chunk_ws_bytes(8, 2, 128)
    assert need > 0 and need % 16 == 0
    for bad in ((0, 1, 128), (8, 0, 128), (7, 2, 128), (1, 2, 128), (8, 2, 120), (8, 2, 288), (8, 2, 0), (65536, 1, 128)):
        assert ops.fp8blk_kv_attn_chunk_ws_bytes(*bad) == 0, bad
        if bad[1]:
            with pytest.raises(ops.Fp8BlkError):
                ops.kv_attn_chunk_workspace(*bad, "cpu")

    def call(q=A16, dtype=0, kc=A16, ks=A4, vc=A16, vs=A4, table=A4, lens=A4, starts=A4, out=A16, lse=None, ws=A16, ws_bytes=need,
             n=4, rows=300, qh=8, kv=2, dim=128, block=64, blocks=100, width=9, q_stride=1024, out_stride=1024):
        return lib.fp8blk_kv_attn_chunk(q, dtype, kc, ks, vc, vs, table, lens, starts, out, lse, ws, ws_bytes, n, rows, qh, kv, dim,
                                        block, blocks, width, q_stride, out_stride, 0.1, None)

    cases = [({k: None}, ops.EINVAL) for k in ("q", "kc", "ks", "vc", "vs", "table", "lens", "starts", "out")]
    cases += [(dict(dtype=-1), ops.EINVAL), (dict(n=0), ops.EINVAL), (dict(rows=0), ops.EINVAL), (dict(qh=9), ops.EINVAL),
              (dict(kv=3), ops.EINVAL), (dict(dim=100), ops.EINVAL), (dict(width=0), ops.EINVAL), (dict(block=100), ops.EINVAL),
              (dict(q_stride=1023), ops.EINVAL), (dict(out_stride=1026), ops.EINVAL), (dict(n=65537), ops.ERANGE),
              (dict(rows=1 << 31), ops.ERANGE), (dict(rows=1 << 29), ops.ERANGE), (dict(blocks=1 << 27), ops.ERANGE),
              (dict(width=1 << 26), ops.ERANGE), (dict(rows=1 << 24, width=1 << 14), ops.ERANGE), (dict(q=A8), ops.EALIGN),
              (dict(out=A8), ops.EALIGN), (dict(lse=A1), ops.EALIGN), (dict(table=A1), ops.EALIGN), (dict(ws=None), ops.EWS),
              (dict(ws_bytes=need - 16), ops.EWS), (dict(ws=A8), ops.EALIGN)]
    for kw, code in cases:
        assert call(**kw) == code, kw


def test_binding_refuses_wrong_tensors(ops):
    kc, ks = torch.zeros((4, 2, 16, 32), dtype=torch.uint8), torch.zeros((4, 2))
    x = torch.zeros((3, 2, 32))
    table, lens, starts = torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    ws = torch.zeros(64, dtype=torch.uint8)
    for args, kw, error in (((x[:, :, :16], kc, ks, kc, ks, table, lens, starts), {}, ValueError),
                            ((x, kc, ks, kc, ks, table, lens, starts[:1]), {}, ValueError),
                            ((x, kc, ks, kc, ks, table, lens, starts), dict(out=x.bfloat16()), ValueError),
                            ((x, kc, ks, kc, ks, table, lens, starts), dict(lse=torch.zeros((3, 1))), ValueError),
                            ((x.half(), kc, ks, kc, ks, table, lens, starts), {}, TypeError),
                            ((x, kc, ks, kc, ks, table.long(), lens, starts), {}, TypeError),
                            ((x, kc.float(), ks, kc, ks, table, lens, starts), {}, TypeError)):
        with pytest.raises(error):
            ops.fp8blk_kv_attn_chunk(*args, 1.0, ws, **kw)
