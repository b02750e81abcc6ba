// rope.cuh -- rotation of heads by a step's cosines and sines: what
// fp8blk_rope and fp8blk_kv_append_rope share.
//
// A pair (a, b) of the rotated part [start, start + rot) of a head becomes
//   a' = a c - b s,   b' = b c + a s,
// in f32 and rounded once to the tensor's type.  Pair i is (i, i + rot / 2) of
// the part (half layout) or (2 i, 2 i + 1) (interleaved).  c and s come from the
// row's table [2][rot / 2], cosines first.
#pragma once

#include "device_common.cuh"

namespace fp8blk {

struct RopeArgs {
    const void *x;          // [n, heads, dim], rows x_stride elements apart
    void *out;              // the same, rows out_stride apart; may be x
    const float *cos_sin;   // [n, 2, rot / 2]
    int64_t n, x_stride, out_stride;
    int heads, dim, rot, start;
    int interleaved;
    int fast;               // whole 16-byte words everywhere: units of eight pairs
    int units, chunks;      // threads of a chunk of heads (units of pairs, then groups to copy), chunks of heads a row
};

// Heads a thread takes: their loads are in flight together, the row's cosines are
// read once.  With 1, 2, 4 and 8 of them 16384 bf16 rows of 64 heads took 87, 90, 119
// and 194 us (the registers of more leave too few threads), and 1001 f32 rows of 24
// heads, a third of each rotated, 8.2, 7.4, 8.7 and 9.9 us.
template <typename T>
constexpr int kRopeHeads = sizeof(T) == 2 ? 1 : 2;

// Eight values as f32, from and to memory (16-byte aligned).
__device__ __forceinline__ void rope_load8(const float *p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void rope_load8(const __nv_bfloat16 *p, float (&v)[8]) {
    const uint4 w = *reinterpret_cast<const uint4 *>(p);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = bf16x2_to_f32(u[i]);
        v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ void rope_store8(float *p, const float (&v)[8]) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void rope_store8(__nv_bfloat16 *p, const float (&v)[8]) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                               pack_bf16x2(v[6], v[7]));
}

// One pair.
__device__ __forceinline__ void rope_pair(float &a, float &b, float c, float s) {
    const float x = a, y = b;
    a = fmaf(x, c, -(y * s));
    b = fmaf(y, c, x * s);
}

// Eight pairs: in the half layout (a[i], b[i]), else neighbours in a and in b.
__device__ __forceinline__ void rope_unit(float (&a)[8], float (&b)[8], const float (&c)[8], const float (&s)[8], int interleaved) {
    if (!interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) rope_pair(a[i], b[i], c[i], s[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            rope_pair(a[2 * i], a[2 * i + 1], c[i], s[i]);
            rope_pair(b[2 * i], b[2 * i + 1], c[4 + i], s[4 + i]);
        }
    }
}

// Where unit u of eight pairs lies in a head: its two groups of eight.
__device__ __forceinline__ int rope_first(const RopeArgs &r, int u) { return r.start + (r.interleaved ? 16 * u : 8 * u); }
__device__ __forceinline__ int rope_second(const RopeArgs &r, int u) {
    return r.start + (r.interleaved ? 16 * u + 8 : r.rot / 2 + 8 * u);
}

// Item `item` of a tensor: unit (fastest), chunk of HEADS heads, row.  (Below 2^31 items: the host sees to it.)
template <typename T, int HEADS>
__device__ __forceinline__ void rope_item(const RopeArgs &r, uint32_t item) {
    const uint32_t rest = item / static_cast<uint32_t>(r.units);
    const int u = static_cast<int>(item - rest * r.units);
    const uint32_t row = rest / static_cast<uint32_t>(r.chunks);
    const int h0 = static_cast<int>(rest - row * r.chunks) * HEADS, half = r.rot / 2;
    const T *x = static_cast<const T *>(r.x) + row * r.x_stride + static_cast<int64_t>(h0) * r.dim;
    T *out = static_cast<T *>(r.out) + row * r.out_stride + static_cast<int64_t>(h0) * r.dim;
    if (r.fast) {
        if (u < half / 8) {
            const float *t = r.cos_sin + static_cast<int64_t>(row) * r.rot + 8 * u;
            const int at = rope_first(r, u), bt = rope_second(r, u);
            float a[HEADS][8], b[HEADS][8], c[8], s[8];
#pragma unroll
            for (int h = 0; h < HEADS; ++h)
                if (h0 + h < r.heads) {
                    rope_load8(x + h * r.dim + at, a[h]);
                    rope_load8(x + h * r.dim + bt, b[h]);
                }
            rope_load8(t, c);
            rope_load8(t + half, s);
#pragma unroll
            for (int h = 0; h < HEADS; ++h)
                if (h0 + h < r.heads) {
                    rope_unit(a[h], b[h], c, s, r.interleaved);
                    rope_store8(out + h * r.dim + at, a[h]);
                    rope_store8(out + h * r.dim + bt, b[h]);
                }
        } else {  // a group outside the rotated part
            int d = 8 * (u - half / 8);
            d = d < r.start ? d : d + r.rot;
            float v[HEADS][8];
#pragma unroll
            for (int h = 0; h < HEADS; ++h)
                if (h0 + h < r.heads) rope_load8(x + h * r.dim + d, v[h]);
#pragma unroll
            for (int h = 0; h < HEADS; ++h)
                if (h0 + h < r.heads) rope_store8(out + h * r.dim + d, v[h]);
        }
        return;
    }
    // Any start, part and alignment: a pair, or a value outside the part.  (Bound by its narrow loads and stores: 16384 bf16
    // rows of 64 heads of 80, 40 of each rotated, 342 us, 15% of the copy rate, and 74 us with 48, by the units above; 24 of
    // 96 444 us, 13%; f32, 32 heads of 80, 40 of each, 228 us, 22%.)
    for (int h = 0; h < HEADS && h0 + h < r.heads; ++h, x += r.dim, out += r.dim) {
        if (u < half) {
            const int at = r.start + (r.interleaved ? 2 * u : u), bt = r.interleaved ? at + 1 : at + half;
            const float *t = r.cos_sin + static_cast<int64_t>(row) * r.rot + u;
            float a = static_cast<float>(x[at]), b = static_cast<float>(x[bt]);
            rope_pair(a, b, t[0], t[half]);
            out[at] = static_cast<T>(a);
            out[bt] = static_cast<T>(b);
        } else {
            int d = u - half;
            d = d < r.start ? d : d + r.rot;
            out[d] = x[d];
        }
    }
}

// The eight rotated values of group d0 (a multiple of eight) of one head at x,
// with the row's table t; the pairs' other values are read from where they lie.
template <typename T>
__device__ __forceinline__ void rope_eight(const RopeArgs &r, const T *x, const float *t, int d0, float (&v)[8]) {
    const int half = r.rot / 2, j0 = d0 - r.start;
    rope_load8(x + d0, v);
    if (j0 + 8 <= 0 || j0 >= r.rot) return;
    if (r.fast) {
        float c[8], s[8], w[8];
        if (!r.interleaved) {
            const bool second = j0 >= half;
            const int i = second ? j0 - half : j0;
            rope_load8(x + (second ? d0 - half : d0 + half), w);
            rope_load8(t + i, c);
            rope_load8(t + half + i, s);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (second) rope_pair(w[k], v[k], c[k], s[k]);
                else rope_pair(v[k], w[k], c[k], s[k]);
            }
        } else {
            const float4 c4 = *reinterpret_cast<const float4 *>(t + j0 / 2), s4 = *reinterpret_cast<const float4 *>(t + half + j0 / 2);
            rope_pair(v[0], v[1], c4.x, s4.x);
            rope_pair(v[2], v[3], c4.y, s4.y);
            rope_pair(v[4], v[5], c4.z, s4.z);
            rope_pair(v[6], v[7], c4.w, s4.w);
        }
        return;
    }
#pragma unroll 1
    for (int k = 0; k < 8; ++k) {
        const int j = j0 + k;
        if (j < 0 || j >= r.rot) continue;
        const bool second = r.interleaved ? (j & 1) != 0 : j >= half;
        const int i = r.interleaved ? j >> 1 : (second ? j - half : j), step = r.interleaved ? 1 : half;
        float a = static_cast<float>(x[d0 + k]), b = static_cast<float>(x[second ? d0 + k - step : d0 + k + step]);
        if (second) rope_pair(b, a, t[i], t[half + i]);
        else rope_pair(a, b, t[i], t[half + i]);
#pragma unroll
        for (int m = 0; m < 8; ++m)
            if (m == k) v[m] = a;  // (no indexed registers)
    }
}

}  // namespace fp8blk
