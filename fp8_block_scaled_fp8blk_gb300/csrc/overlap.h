// overlap.h -- whether two tensors of n rows each share memory.  Plain C++, host
// only, so that a host test can hold it against every byte.
#pragma once

#include <cstdint>

namespace fp8blk {

// Rows of `aw` bytes from a on, `as` bytes apart, and of `bw` bytes from b on, `bs` bytes apart (rows of one tensor do not
// overlap: as >= aw > 0).  Slices of one wider tensor lie between each other's rows and share nothing.
inline bool rows_overlap(const void *a, int64_t as, int64_t aw, const void *b, int64_t bs, int64_t bw, int64_t n) {
    using Wide = __int128;  // (a stride times a row may pass 64 bits)
    const Wide d = static_cast<Wide>(reinterpret_cast<uintptr_t>(b)) - static_cast<Wide>(reinterpret_cast<uintptr_t>(a));
    const Wide a_end = static_cast<Wide>(n - 1) * as + aw, b_end = d + static_cast<Wide>(n - 1) * bs + bw;
    if (d >= a_end || b_end <= 0) return false;
    auto below = [](Wide x, Wide y) { return x >= 0 ? x / y : -((y - 1 - x) / y); };  // floor(x / y)
    if (as == bs) {  // rows m apart: -bw < d + m as < aw for an m of -(n - 1) .. n - 1
        Wide m = below(-bw - d, as) + 1;
        if (m < 1 - n) m = 1 - n;
        return m < n && d + m * as < aw;
    }
    for (int64_t i = 0; i < n; ++i) {  // row i of a: the first row of b that ends behind its start
        const Wide at = static_cast<Wide>(i) * as;
        Wide j = below(at - bw - d, bs) + 1;
        if (j < 0) j = 0;
        if (j >= n) return false;  // (all later rows of a lie behind b too)
        if (d + j * bs < at + aw) return true;
    }
    return false;
}

}  // namespace fp8blk
