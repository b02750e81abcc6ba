// kv_chunk_copy.h -- which codes the converting threads of kv_chunk.cuh copy.
// Plain C++ beside the kernel, so that a host test can go through every address.
//
// A thread has a few groups of sixteen codes of each tile, numbered g = thread +
// i x threads; a tile of T tokens of head_dim values has T x per of them,
// per = head_dim / 16.  Where head_dim is no 128 (256), some numbers are past the
// last one: those groups belong to token T, which no tile has.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define FP8BLK_HD __host__ __device__ __forceinline__
#else
#define FP8BLK_HD inline
#endif

namespace fp8blk {

struct ChunkGroup {
    int token, part;  // its token in the tile, and which sixteen of the token's codes
};
// (Where a token has a multiple of four groups, four of them and the same of the next token go to eight lanes: their
// stores then meet no bank twice.)
FP8BLK_HD ChunkGroup ch_group(int g, int tile, int per) {
    if (g >= tile * per) return {tile, 0};
    const int four = per & 3 ? 0 : per >> 2;
    if (four) return {(g / (2 * per) << 1) + (g >> 2 & 1), (g & 3) + (g / 8 % four << 2)};
    return {g / per, g - g / per * per};
}

// Bytes from the first code of the head in the block that the group's token lies in, in a request's first tile; and what
// a later tile adds (a block of 128 tokens may be two tiles).
FP8BLK_HD int ch_group_from(ChunkGroup x, int tile, int block, int head_dim) {
    return x.token < tile ? (x.token & (block - 1)) * head_dim + 16 * x.part : 0;
}
FP8BLK_HD int ch_tile_from(int j, int tile, int block, int head_dim) { return (j * tile & (block - 1)) * head_dim; }

// Tokens of tile j that a request of `len` tokens has, never more than a tile holds (so a group of no token is copied
// nowhere), and whether a group of `token` is copied out of block `id`.
FP8BLK_HD int ch_tile_left(int len, int j, int tile) { return len - j * tile < tile ? len - j * tile : tile; }
FP8BLK_HD bool ch_group_copied(int token, int left, uint32_t id, uint32_t n_blocks) { return id < n_blocks && token < left; }

}  // namespace fp8blk
