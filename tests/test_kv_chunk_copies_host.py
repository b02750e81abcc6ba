"""CPU check of the codes that fp8blk_kv_attn_chunk's converting threads copy: csrc/kv_chunk_copy.h, compiled for the host
and walked thread by thread and tile by tile as the kernel does.  Every copy that is not empty lies inside its own (block,
head), empty ones have an address inside the pool too, and each code of the request's tokens is copied once."""
import ctypes
import itertools
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CONVERTERS = 256  # threads

WALK = r"""
#include "kv_chunk_copy.h"
#include <cstring>
using namespace fp8blk;
// Tiles [j0, j1) of one request (pages: its row of the table); seen: a count for each 16 codes of the pool.  Returns the
// number of copies outside their own (block, head); *stray: of empty ones with an address outside the pool.
extern "C" int walk(int tile, int each, int threads, int head_dim, int block, int kv_heads, int head, int n_blocks, int len, int j0,
                    int j1, const int *pages, int width, unsigned char *seen, int *stray) {
    const int G = tile / 16, window_tiles = 32 / G, per = head_dim / 16;
    const int64_t id_bytes = static_cast<int64_t>(kv_heads) * block * head_dim, pool = id_bytes * n_blocks;
    const int64_t at_head = static_cast<int64_t>(head) * block * head_dim;
    int bad = 0, ids[32], ahead = j0;
    *stray = 0;
    auto window = [&](int j) {  // a lane's block id, as the kernel looks it up
        for (int lane = 0; lane < 32; ++lane) {
            const int64_t t = static_cast<int64_t>(j + lane / G) * tile + 16 * (lane % G), page = t / block;
            ids[lane] = j + lane / G >= j1 || t >= len ? -2 : page < width ? pages[page] : -1;
        }
    };
    window(j0);
    for (int j = j0; j < j1 + 6; ++j) {  // (copies run ahead of the unit's last tile)
        if (j == ahead + window_tiles) window(ahead = j);
        const int left = ch_tile_left(len, j, tile), codes = ch_tile_from(j, tile, block, head_dim);
        for (int tid = 0; tid < threads; ++tid)
            for (int i = 0; i < each; ++i) {
                const ChunkGroup x = ch_group(tid + i * threads, tile, per);
                const int id = ids[((j - ahead) * G + (x.token >> 4)) & 31];
                const bool there = ch_group_copied(x.token, left, static_cast<uint32_t>(id), static_cast<uint32_t>(n_blocks));
                const int64_t from = at_head + codes + (there ? id : 0) * id_bytes + ch_group_from(x, tile, block, head_dim);
                if (!there) {
                    *stray += from < 0 || from + 16 > pool;
                    continue;
                }
                const int64_t t = static_cast<int64_t>(j) * tile + x.token;
                const int64_t own = static_cast<int64_t>(pages[t / block < width ? t / block : 0]) * id_bytes + at_head;
                const bool right = x.token < tile && t < len && from == own + (t % block) * head_dim + 16 * x.part;
                bad += !right;
                if (right && seen[from / 16] < 255) ++seen[from / 16];
            }
    }
    return bad;
}
"""


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    d = tmp_path_factory.mktemp("copies")
    src, lib = d / "walk.cpp", d / "walk.so"
    src.write_text(WALK)
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", os.path.join(ROOT, "fp8_block_scaled_fp8blk_gb300", "csrc"),
                    "-o", str(lib), str(src)], check=True)
    f = ctypes.CDLL(str(lib)).walk
    f.restype = ctypes.c_int
    return f


# (tokens of a tile, columns a thread's groups cover): bf16, f32 or a wide bf16 head, wide heads of either type.
SHAPES = ((128, 128), (64, 128), (64, 256))


@pytest.mark.parametrize("tile,columns", SHAPES)
@pytest.mark.parametrize("block", (16, 32, 64, 128))
def test_every_copy_lies_in_its_own_block_and_head(walk, tile, columns, block):
    each = tile * columns // 16 // CONVERTERS
    dims = range(16, 129, 16) if columns == 128 else range(144, 257, 16)
    for dim, heads, len_ in itertools.product(dims, (1, 3), (1, 15, 63, 64, 65, 127, 128, 129, 191, 200, 256, 300, 384, 500)):
        width = -(-len_ // block)
        pages = list(range(width))  # the request's last page is the pool's last block ...
        if heads == 3:
            pages = pages[::-1]     # ... or its first page is
        tiles = -(-len_ // tile)
        row = (ctypes.c_int * width)(*pages)
        for head in range(heads):
            for j0 in {0, tiles // 2, tiles - 1}:
                seen = (ctypes.c_ubyte * (width * heads * block * dim // 16))()
                stray = ctypes.c_int(-1)
                bad = walk(tile, each, CONVERTERS, dim, block, heads, head, width, len_, j0, tiles, row, width, seen, ctypes.byref(stray))
                what = (tile, dim, block, heads, head, len_, j0)
                assert (bad, stray.value) == (0, 0), what
                for t in range(0, len_, 7):
                    at = ((pages[t // block] * heads + head) * block + t % block) * dim // 16
                    assert list(seen[at: at + dim // 16]) == [int(t >= j0 * tile)] * (dim // 16), (what, t)


def test_a_table_that_ends_and_blocks_outside_the_pool(walk):
    """Copies stay inside their blocks where the table is too short, or names blocks that the pool has not."""
    for tile, columns in SHAPES:
        for pages in ([0, 7, -3, 1], [1, 0], [1 << 30, 1, -1]):
            for block in (16, 64, 128):
                dim, stray = columns - 48, ctypes.c_int(-1)
                row = (ctypes.c_int * len(pages))(*pages)
                seen = (ctypes.c_ubyte * (2 * block * dim // 16))()
                bad = walk(tile, tile * columns // 16 // CONVERTERS, CONVERTERS, dim, block, 1, 0, 2, 900, 0, -(-900 // tile), row,
                           len(pages), seen, ctypes.byref(stray))
                assert (bad, stray.value) == (0, 0), (tile, pages, block)
