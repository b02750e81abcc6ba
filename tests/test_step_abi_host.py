"""Host-side refusals of the cache, attention and scoring calls (no GPU): every
argument the host can judge is judged before CUDA is touched."""
import numpy as np
import pytest
import torch

A16, A8, A4, A1 = 0x10000, 0x10008, 0x10004, 0x10001  # fake, never-dereferenced addresses


@pytest.fixture(scope="module")
def ops():
    from fp8_block_scaled_fp8blk_gb300 import build
    build.build()
    from fp8_block_scaled_fp8blk_gb300 import ops as o
    return o


def refuses(call, cases):
    for kw, code in cases:
        assert call(**kw) == code, kw


def test_kv_map(ops):
    lib = ops.raw_library()

    def call(ctx=A4, new=A8, table=A4, free=A4, head=A4, lens=A16, starts=A4, slots=A16, pos=A16, out=A8, n=4, width=8,
             n_free=10, block=16, most=64):
        return lib.fp8blk_kv_map(ctx, new, table, free, head, lens, starts, slots, pos, out, n, width, n_free, block, most, None)

    refuses(call, [({k: None}, ops.EINVAL) for k in ("ctx", "new", "table", "free", "head", "lens", "starts", "slots", "pos", "out")])
    refuses(call, [(dict(n=0), ops.EINVAL), (dict(width=0), ops.EINVAL), (dict(n_free=-1), ops.EINVAL), (dict(most=0), ops.EINVAL),
                   (dict(block=24), ops.EINVAL), (dict(block=8), ops.EINVAL), (dict(block=256), ops.EINVAL),
                   (dict(head=A8, out=A8), ops.EINVAL), (dict(lens=A4, ctx=A4), ops.EINVAL),
                   (dict(n=65537), ops.ERANGE), (dict(most=1 << 31), ops.ERANGE),
                   (dict(slots=A8), ops.EALIGN), (dict(pos=A8), ops.EALIGN), (dict(ctx=A1), ops.EALIGN), (dict(table=A1), ops.EALIGN)])


def test_kv_append(ops):
    lib = ops.raw_library()

    def call(k=A16, v=A16, dtype=0, slots=A8, kc=A16, ks=A4, vc=A16, vs=A4, n=4, k_stride=256, v_stride=256, blocks=10, heads=2,
             block=16, dim=128):
        return lib.fp8blk_kv_append(k, v, dtype, slots, kc, ks, vc, vs, n, k_stride, v_stride, blocks, heads, block, dim, None)

    refuses(call, [({k: None}, ops.EINVAL) for k in ("k", "v", "slots", "kc", "ks", "vc", "vs")])
    refuses(call, [(dict(dtype=2), ops.EINVAL), (dict(n=0), ops.EINVAL), (dict(blocks=0), ops.EINVAL), (dict(heads=0), ops.EINVAL),
                   (dict(block=48), ops.EINVAL), (dict(dim=8), ops.EINVAL), (dict(dim=24), ops.EINVAL), (dict(dim=272), ops.EINVAL),
                   (dict(k_stride=255), ops.EINVAL), (dict(v_stride=240), ops.EINVAL), (dict(k_stride=258), ops.EINVAL),
                   (dict(dtype=1, v_stride=260), ops.EINVAL), (dict(blocks=1 << 31), ops.ERANGE),
                   (dict(blocks=1 << 27), ops.ERANGE), (dict(n=1 << 31), ops.ERANGE), (dict(k_stride=1 << 40), ops.ERANGE),
                   (dict(k=A8), ops.EALIGN), (dict(kc=A8), ops.EALIGN), (dict(vs=A1), ops.EALIGN), (dict(slots=A4), ops.EALIGN)])


def test_kv_attn(ops):
    lib = ops.raw_library()
    need = ops.fp8blk_kv_attn_ws_bytes(4, 8, 8, 2, 128)
    assert need > 0 and need % 16 == 0
    for bad in ((0, 1, 8, 2, 128), (4, 0, 8, 2, 128), (4, 9, 8, 2, 128), (4, 1, 7, 2, 128), (4, 1, 1, 2, 128), (4, 1, 8, 2, 120),
                (4, 1, 8, 2, 288), (1 << 20, 1, 8, 2, 128)):
        assert ops.fp8blk_kv_attn_ws_bytes(*bad) == 0, bad

    def call(q=A16, dtype=0, kc=A16, ks=A4, vc=A16, vs=A4, table=A4, lens=A4, starts=A4, out=A16, lse=None, ws=A16, ws_bytes=need,
             n=4, m=8, rows=32, qh=8, kv=2, dim=128, block=64, blocks=100, width=9, q_stride=1024, out_stride=1024):
        return lib.fp8blk_kv_attn(q, dtype, kc, ks, vc, vs, table, lens, starts, out, lse, ws, ws_bytes, n, m, rows, qh, kv, dim,
                                  block, blocks, width, q_stride, out_stride, 0.1, None)

    refuses(call, [({k: None}, ops.EINVAL) for k in ("q", "kc", "ks", "vc", "vs", "table", "lens", "starts", "out")])
    refuses(call, [(dict(dtype=-1), ops.EINVAL), (dict(m=0), ops.EINVAL), (dict(m=9), ops.EINVAL), (dict(n=0), ops.EINVAL),
                   (dict(rows=0), ops.EINVAL), (dict(qh=9), ops.EINVAL), (dict(kv=3), ops.EINVAL), (dict(dim=100), ops.EINVAL),
                   (dict(width=0), ops.EINVAL), (dict(block=100), ops.EINVAL), (dict(q_stride=1023), ops.EINVAL),
                   (dict(out_stride=1026), ops.EINVAL), (dict(n=65537), ops.ERANGE), (dict(rows=1 << 31), ops.ERANGE),
                   (dict(blocks=1 << 27), ops.ERANGE), (dict(q=A8), ops.EALIGN), (dict(out=A8), ops.EALIGN), (dict(lse=A1), ops.EALIGN),
                   (dict(table=A1), ops.EALIGN), (dict(ws=None), ops.EWS), (dict(ws_bytes=need - 16), ops.EWS), (dict(ws=A8), ops.EALIGN)])


def test_token_logprobs(ops):
    lib = ops.raw_library()

    def call(x=A16, dtype=0, t=A4, lp=A4, rank=A4, ent=A4, ids=A4, top_lp=A4, n=4, vocab=1000, stride=1000, top=5):
        return lib.fp8blk_token_logprobs(x, dtype, t, lp, rank, ent, ids, top_lp, n, vocab, stride, top, None)

    refuses(call, [({k: None}, ops.EINVAL) for k in ("x", "t", "lp", "rank", "ent", "ids", "top_lp")])
    refuses(call, [(dict(dtype=3), ops.EINVAL), (dict(n=0), ops.EINVAL), (dict(vocab=0), ops.EINVAL), (dict(stride=999), ops.EINVAL),
                   (dict(top=-1), ops.EINVAL), (dict(top=33), ops.EINVAL), (dict(vocab=4, stride=4), ops.EINVAL),
                   (dict(vocab=ops.MAX_VOCAB + 1, stride=1 << 20), ops.ERANGE), (dict(n=1 << 31), ops.ERANGE),
                   (dict(stride=1 << 33), ops.ERANGE), (dict(x=A1), ops.EALIGN), (dict(dtype=1, x=A1), ops.EALIGN),
                   (dict(ids=A1), ops.EALIGN)])


def test_binding_refuses_wrong_tensors(ops):
    """Types, shapes and layouts that raw pointers could not show; judged before the device is asked for a stream."""
    kc, ks = torch.zeros((4, 2, 16, 32), dtype=torch.uint8), torch.zeros((4, 2))
    slots = torch.zeros(3, dtype=torch.int64)
    x = torch.zeros((3, 2, 32))
    for bad in (x.half(), x.double()):
        with pytest.raises(TypeError):
            ops.fp8blk_kv_append(bad, bad, slots, kc, ks, kc, ks)
    with pytest.raises(TypeError):
        ops.fp8blk_kv_append(x, x, slots.int(), kc, ks, kc, ks)
    with pytest.raises(TypeError):
        ops.fp8blk_kv_append(x, x.bfloat16(), slots, kc, ks, kc, ks)
    with pytest.raises(TypeError):
        ops.fp8blk_kv_append(x, x, slots, kc, ks.double(), kc, ks)
    for shape in ((2, 2, 32), (3, 1, 32), (3, 2, 16)):
        with pytest.raises(ValueError):
            ops.fp8blk_kv_append(torch.zeros(shape), torch.zeros(shape), slots, kc, ks, kc, ks)
    with pytest.raises(ValueError):
        ops.fp8blk_kv_append(torch.zeros((3, 32, 2)).transpose(1, 2), x, slots, kc, ks, kc, ks)
    with pytest.raises(ValueError):
        ops.fp8blk_kv_append(x, x, slots, kc, ks, kc[:, :, :8], ks)
    table, lens, starts = torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    ws = torch.zeros(64, dtype=torch.uint8)
    with pytest.raises(ValueError):
        ops.fp8blk_kv_attn(torch.zeros((3, 2, 16)), kc, ks, kc, ks, table, lens, starts, 3, 1.0, ws)
    with pytest.raises(ValueError):
        ops.fp8blk_kv_attn(x, kc, ks, kc, ks, table, lens, starts[:1], 3, 1.0, ws)
    with pytest.raises(ValueError):
        ops.fp8blk_kv_attn(x, kc, ks, kc, ks, table, lens, starts, 3, 1.0, ws, out=x.bfloat16())
    with pytest.raises(TypeError):
        ops.fp8blk_kv_attn(x, kc, ks, kc, ks, table.long(), lens, starts, 3, 1.0, ws)
    with pytest.raises(ValueError):
        ops.fp8blk_token_logprobs(torch.zeros((2, 10)).t(), torch.zeros(10, dtype=torch.int32))
    with pytest.raises(TypeError):
        ops.fp8blk_token_logprobs(torch.zeros((2, 10)), torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        ops.fp8blk_token_logprobs(torch.zeros((2, 10)), torch.zeros(2, dtype=torch.int32), 3,
                                  out=ops.token_logprobs_buffers(2, 4, "cpu"))
    with pytest.raises(ValueError):
        ops.fp8blk_kv_map(lens, lens, table, lens, lens, 16, 8, out=ops.kv_map_buffers(1, 9, "cpu"))


def test_the_plain_restatement_of_e4m3():
    import _step_ref as ref
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(np.nan_to_num(t, nan=1e9), np.nan_to_num(ref.E4M3, nan=1e9))
    rng = np.random.default_rng(0)
    x = (rng.standard_normal(20000) * 2.0 ** rng.integers(-14, 10, 20000)).astype(np.float32)
    x = np.clip(x, -448, 448)
    x[:254] = ref.E4M3[[b for b in range(256) if b & 127 != 127]]
    x[300:426] = (ref.E4M3[:126] + ref.E4M3[1:127]) / 2   # halves
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.e4m3_encode(x), want)
    for a in (448.0, 448.0000305, 1.75, 1.7500001, 3.4e38, 0.0, 1e-40):
        s = ref.pow2_scale(a)
        assert a <= 448 * s and (s == 2.0 ** -126 or a > 448 * s / 2)
