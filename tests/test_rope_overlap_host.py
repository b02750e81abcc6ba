"""Outputs that share memory with what the same call reads are refused (no GPU): the rule byte by byte, and each call's use of
it.  Slices of one fused projection, and rotation in place, are no overlap."""
import ctypes
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x100000  # a fake, never-dereferenced address


@pytest.fixture(scope="module")
def ops():
    from fp8_block_scaled_fp8blk_gb300 import build
    build.build()
    from fp8_block_scaled_fp8blk_gb300 import ops as o
    return o


def test_rows_overlap(tmp_path):
    src, lib = tmp_path / "o.cpp", tmp_path / "o.so"
    src.write_text('#include "overlap.h"\nextern "C" int overlap(uint64_t a, int64_t as, int64_t aw, uint64_t b, int64_t bs, int64_t bw, '
                   'int64_t n) {\n    return fp8blk::rows_overlap(reinterpret_cast<void *>(a), as, aw, reinterpret_cast<void *>(b), bs, bw, n);\n}\n')
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", os.path.join(ROOT, "fp8_block_scaled_fp8blk_gb300", "csrc"),
                    "-o", str(lib), str(src)], check=True)
    f = ctypes.CDLL(str(lib)).overlap
    f.argtypes = [ctypes.c_uint64] + [ctypes.c_int64] * 2 + [ctypes.c_uint64] + [ctypes.c_int64] * 3
    rng = random.Random(3)
    hits = 0
    for _ in range(20000):
        n, aw, bw = rng.randint(1, 7), rng.randint(1, 6), rng.randint(1, 6)
        sa = aw + rng.choice([0, 0, rng.randint(0, 20)])
        sb = max(bw, sa) if rng.random() < 0.5 else bw + rng.randint(0, 20)
        a, b = 1000, 1000 + rng.randint(-120, 120)
        x = {a + i * sa + k for i in range(n) for k in range(aw)}
        y = {b + i * sb + k for i in range(n) for k in range(bw)}
        assert bool(f(a, sa, aw, b, sb, bw, n)) == bool(x & y), (a, sa, aw, b, sb, bw, n)
        hits += bool(x & y)
    assert 2000 < hits < 18000
    big = 2 ** 31 - 1
    assert f(A, 4 * big, 64, A + 64, 4 * big, 64, big) == 0 and f(A, 4 * big, 64, A + 63, 4 * big, 64, big) == 1
    assert f(A, 4 * big, 4 * big, A - 1, 64, 64, big) == 1 and f(A, 64, 64, A + 64 * big, 64, 64, big) == 0


def test_rope_refuses_a_shifted_output(ops):
    def call(x, out, dtype=0, n=4, heads=2, dim=64, xs=128, os=128):
        return ops.raw_library().fp8blk_rope(x, dtype, A * 16, out, n, heads, dim, 64, 0, 0, xs, os, None)

    for dtype, es in ((0, 4), (1, 2)):
        for out in (A + es, A - es, A + 16, A + 64 * es, A - 64 * es, A + 128 * es, A - 128 * es, A + 3 * 128 * es, A + 4 * 128 * es - es):
            assert call(A, out, dtype) == ops.EINVAL, (dtype, out - A)
        # Between the rows of a wider tensor, half a head too near; and with another stride.
        assert call(A, A + 127 * es, dtype, xs=256, os=256) == ops.EINVAL
        assert call(A, A + 256 * es - 16, dtype, xs=256, os=256) == ops.EINVAL
        assert call(A, A + 128 * es, dtype, xs=256, os=136) == ops.EINVAL
        assert call(A, A - 16, dtype, n=1) == ops.EINVAL


def test_append_rope_refuses_queries_over_keys_and_values(ops):
    def call(k, v, q, qo, stride=768, qo_stride=768, n=5):
        return ops.raw_library().fp8blk_kv_append_rope(k, v, 0, A * 16, A * 16, A * 32, A * 33, A * 34, A * 35, q, qo, n, stride, stride,
                                                       stride, qo_stride, 10, 1, 4, 16, 128, 128, 0, 0, None)

    k, v, q = A + 4 * 512, A + 4 * 640, A  # one fused row: 4 query heads, a key head, a value head of 128
    for qo in (k, v, k - 16, A + 16, v - 4 * 512, A + 4 * 768 * 3 + 16, k + 4 * 768 * 4):
        assert call(k, v, q, qo) == ops.EINVAL, qo - A
    assert call(k, v, q, A + 4 * 768, qo_stride=512) == ops.EINVAL  # another stride, over all of them
    assert call(q, v, q, q) == ops.EINVAL  # keys that are the queries' own rows, turned in place
