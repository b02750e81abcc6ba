"""Rotary positions on the host (no GPU): frequencies and turns against the formulas, and every refusal."""
import math

import numpy as np
import pytest
import torch

import _rope_ref as ref

A16, A8, A4, A2, A1 = 0x10000, 0x10008, 0x10004, 0x10002, 0x10001  # fake, never-dereferenced addresses


@pytest.fixture(scope="module")
def ops():
    from fp8_block_scaled_fp8blk_gb300 import build
    build.build()
    from fp8_block_scaled_fp8blk_gb300 import ops as o
    return o


@pytest.mark.parametrize("rot", [2, 4, 20, 64, 128, 1024])
@pytest.mark.parametrize("scaling,kw", [("plain", {}), ("linear", dict(factor=4.0)), ("base", dict(factor=8.0)),
                                        ("ramp", dict(factor=16.0, original_len=4096.0)), ("ramp", dict(factor=1.0, original_len=100.0)),
                                        ("bands", dict(factor=8.0, original_len=8192.0, low=1.0, high=4.0))])
def test_frequencies(ops, rot, scaling, kw):
    """The host's pow and log are good to a few ulp: 1e-13 of the value."""
    if scaling == "base" and rot == 2:
        with pytest.raises(ops.Fp8BlkError):
            ops.rope_frequencies(rot, 10000.0, scaling, **kw)
        return
    got, scale = ops.rope_frequencies(rot, 10000.0, scaling, **kw)
    want, want_scale = ref.frequencies(rot, 10000.0, scaling, kw.get("factor", 1.0), kw.get("original_len", 0.0), kw.get("low", 1.0),
                                       kw.get("high", 32.0))
    assert got.shape == (rot // 2,) and np.abs(got / want - 1).max() < 1e-13
    assert abs(scale - want_scale) <= 2.0 ** -24 * want_scale


def test_turns(ops):
    """round(2^64 (f / 2 pi)) mod 2^64: the division in doubles is good to 2^-53 of the quotient, the rounding to half a unit."""
    freqs = np.array([1.0, 1e-9, 0.5, -0.5, 0.0, 2 * math.pi, 100.0, -1e-12, 1e6])
    turns = ops.rope_turns(freqs, "cpu").numpy().view(np.uint64)
    for f, t in zip(freqs, turns):
        got = int(t) / 2.0 ** 64
        want = f / (2 * math.pi)
        off = abs((got - want + 0.5) % 1.0 - 0.5)
        assert off <= 2.0 ** -52 * max(abs(want), 2.0 ** -11) + 2.0 ** -64, (f, off)
    assert int(turns[4]) == 0
    a, b = ops.rope_turns([0.25], "cpu").item(), ops.rope_turns([-0.25], "cpu").item()
    assert abs((a + b) % 2 ** 64) <= 2 ** 12 or abs((a + b) % 2 ** 64) >= 2 ** 64 - 2 ** 12  # one turns back what the other turns
    for bad in ([math.nan], [math.inf], [2e6], [], [0.1] * 513):
        with pytest.raises(ops.Fp8BlkError):
            ops.rope_turns(bad, "cpu")
    with pytest.raises(ValueError):
        ops.rope_turns([[0.1]], "cpu")


def test_frequency_refusals(ops):
    for kw in (dict(rot_dim=0), dict(rot_dim=3), dict(rot_dim=1026), dict(rot_dim=64, base=1.0), dict(rot_dim=64, base=math.nan),
               dict(rot_dim=64, base=math.inf), dict(rot_dim=64, scaling="linear", factor=0.5),
               dict(rot_dim=64, scaling="linear", factor=math.nan), dict(rot_dim=64, scaling="ramp", factor=2.0),
               dict(rot_dim=64, scaling="ramp", factor=2.0, original_len=100.0, low=4.0, high=4.0),
               dict(rot_dim=64, scaling="bands", factor=2.0, original_len=100.0, low=0.0, high=4.0)):
        with pytest.raises(ops.Fp8BlkError):
            ops.rope_frequencies(**kw)
    with pytest.raises(ValueError):
        ops.rope_frequencies(64, scaling="other")
    lib = ops.raw_library()
    out = np.zeros(32)
    assert lib.fp8blk_rope_frequencies(5, 64, 1e4, 1.0, 1.0, 1.0, 2.0, out.ctypes.data, None) == ops.EINVAL
    assert lib.fp8blk_rope_frequencies(0, 64, 1e4, 1.0, 1.0, 1.0, 2.0, None, None) == ops.EINVAL
    assert lib.fp8blk_rope_frequencies(0, 64, 1e4, 1.0, 1.0, 1.0, 2.0, out.ctypes.data, None) == ops.OK


def refuses(call, cases):
    for kw, code in cases:
        assert call(**kw) == code, kw


def test_table(ops):
    lib = ops.raw_library()

    def call(pos=A4, turns=A8, out=A16, n=4, rot=64):
        return lib.fp8blk_rope_table(pos, turns, 1.0, out, n, rot, None)

    refuses(call, [({k: None}, ops.EINVAL) for k in ("pos", "turns", "out")])
    refuses(call, [(dict(n=0), ops.EINVAL), (dict(rot=0), ops.EINVAL), (dict(rot=63), ops.EINVAL), (dict(rot=1026), ops.ERANGE),
                   (dict(n=1 << 26), ops.ERANGE), (dict(pos=A1), ops.EALIGN), (dict(turns=A4), ops.EALIGN), (dict(out=A8), ops.EALIGN)])


def test_rope(ops):
    lib = ops.raw_library()

    def call(x=A16, dtype=0, table=A16, out=A16 * 2, n=4, heads=2, dim=64, rot=64, start=0, pairs=0, xs=128, os=128):
        return lib.fp8blk_rope(x, dtype, table, out, n, heads, dim, rot, start, pairs, xs, os, None)

    refuses(call, [({k: None}, ops.EINVAL) for k in ("x", "table", "out")])
    refuses(call, [(dict(dtype=2), ops.EINVAL), (dict(n=0), ops.EINVAL), (dict(heads=0), ops.EINVAL), (dict(rot=0), ops.EINVAL),
                   (dict(rot=31), ops.EINVAL), (dict(rot=66), ops.EINVAL), (dict(start=-1), ops.EINVAL), (dict(start=2), ops.EINVAL),
                   (dict(rot=32, start=33), ops.EINVAL), (dict(pairs=2), ops.EINVAL), (dict(xs=127), ops.EINVAL), (dict(os=127), ops.EINVAL),
                   (dict(out=A16, os=136), ops.EINVAL), (dict(dim=1, rot=2), ops.EINVAL), (dict(dim=1026, xs=1 << 12, os=1 << 12), ops.ERANGE),
                   (dict(heads=65536, xs=1 << 23, os=1 << 23), ops.ERANGE), (dict(n=1 << 31), ops.ERANGE), (dict(xs=1 << 31), ops.ERANGE),
                   (dict(n=1 << 30), ops.ERANGE), (dict(x=A2), ops.EALIGN), (dict(x=A1, dtype=1), ops.EALIGN), (dict(out=A2), ops.EALIGN),
                   (dict(table=A8), ops.EALIGN)])


def test_append_rope(ops):
    lib = ops.raw_library()

    def call(k=A16, v=A16, dtype=0, slots=A8, table=A16, kc=A16, ks=A4, vc=A16, vs=A4, q=A16, qo=A16 * 2, n=4, k_stride=256, v_stride=256,
             q_stride=512, qo_stride=512, blocks=10, heads=2, qh=4, block=16, dim=128, rot=128, start=0, pairs=0):
        return lib.fp8blk_kv_append_rope(k, v, dtype, slots, table, kc, ks, vc, vs, q, qo, n, k_stride, v_stride, q_stride, qo_stride, blocks,
                                         heads, qh, block, dim, rot, start, pairs, None)

    refuses(call, [({k: None}, ops.EINVAL) for k in ("k", "v", "slots", "table", "kc", "ks", "vc", "vs", "q", "qo")])
    refuses(call, [(dict(dtype=2), ops.EINVAL), (dict(n=0), ops.EINVAL), (dict(rot=130), ops.EINVAL), (dict(rot=3), ops.EINVAL),
                   (dict(start=16), ops.EINVAL), (dict(pairs=-1), ops.EINVAL), (dict(qh=0), ops.EINVAL), (dict(q_stride=511), ops.EINVAL),
                   (dict(qo=A16, qo_stride=516), ops.EINVAL), (dict(block=48), ops.EINVAL), (dict(dim=8), ops.EINVAL), (dict(k_stride=258), ops.EINVAL),
                   (dict(table=A8), ops.EALIGN), (dict(q=A2), ops.EALIGN), (dict(k=A8), ops.EALIGN), (dict(blocks=1 << 31), ops.ERANGE)])


def test_binding_refuses_wrong_tensors(ops):
    x, t = torch.zeros((3, 2, 32)), torch.zeros((3, 2, 16))
    for bad in (torch.zeros((3, 16)), torch.zeros((2, 2, 16)), torch.zeros((3, 1, 16))):
        with pytest.raises(ValueError):
            ops.fp8blk_rope(x, bad)
    with pytest.raises(TypeError):
        ops.fp8blk_rope(x, t.double())
    with pytest.raises(ValueError):
        ops.fp8blk_rope(x, t, out=x.bfloat16())
    with pytest.raises(ValueError):
        ops.fp8blk_rope(x.transpose(1, 2), t)
    with pytest.raises(TypeError):
        ops.fp8blk_rope_table(torch.zeros(3, dtype=torch.int64), torch.zeros(16, dtype=torch.int64))
    with pytest.raises(TypeError):
        ops.fp8blk_rope_table(torch.zeros(3, dtype=torch.int32), torch.zeros(16))
    with pytest.raises(ValueError):
        ops.fp8blk_rope_table(torch.zeros(3, dtype=torch.int32), torch.zeros(16, dtype=torch.int64), out=torch.zeros((3, 2, 15)))
    kc, ks, slots = torch.zeros((4, 2, 16, 32), dtype=torch.uint8), torch.zeros((4, 2)), torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError):
        ops.fp8blk_kv_append_rope(x, x, slots, t[:2], kc, ks, kc, ks)
    with pytest.raises(ValueError):
        ops.fp8blk_kv_append_rope(x, x, slots, t, kc, ks, kc, ks, q_out=x)
    with pytest.raises(ValueError):
        ops.fp8blk_kv_append_rope(x, x, slots, t, kc, ks, kc, ks, q=x[:, :, :16])
    with pytest.raises(ValueError):
        ops.fp8blk_kv_append_rope(x, x, slots, t, kc, ks, kc, ks, q=x.bfloat16())
    with pytest.raises(ValueError):
        ops.fp8blk_kv_append_rope(x, x, slots, t, kc, ks, kc, ks, q=x, q_out=x[:2])
