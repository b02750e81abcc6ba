// kv_cache.cu -- the paged e4m3 cache of a decode / verify step: block tables
// and slots from request lengths (fp8blk_kv_map), and keys and values written
// with one power-of-two scale per (block of tokens, head) (fp8blk_kv_append),
// the keys rotated on their way there (fp8blk_kv_append_rope).
//
// A pool holds uint8 e4m3 codes [n_blocks, kv_heads, block_tokens, head_dim]
// and f32 scales [n_blocks, kv_heads].  Head-major inside a block: what one
// head reads of one block is a single run of block_tokens x head_dim bytes
// under one scale.
#include "overlap.h"
#include "rope.cuh"
#include "step.h"

#include <algorithm>
#include <type_traits>

namespace fp8blk {

// ------------------------------------------------------------------ kv_map
struct MapArgs {
    const int32_t *ctx_lens, *new_lens;  // [n]
    const int32_t *held_blocks;          // [n] or null: blocks that a request has beside those of its context
    int32_t *held_out;                   // [n], with held_blocks
    int32_t *table;                      // [n, width]
    const int32_t *free_blocks;          // [n_free]
    const int32_t *free_head;            // [1]
    int32_t *seq_lens, *q_starts;        // [n], [n + 1]
    int64_t *slots;                      // [max_tokens]
    int32_t *positions;                  // [max_tokens]
    int32_t *free_head_out;              // [1]
    unsigned int *status;
    int n, width, n_free, block_log2;
    int64_t max_tokens;
};

constexpr int kMapThreads = 512;
constexpr int kMapPerThread = 4;  // consecutive tokens of one thread: 32-byte slot and 16-byte position stores

// One request's lengths, bounded: negative lengths count as zero, a sum past
// 2^31 - 1 stops there.  `held` and `wanted` are its blocks before and after,
// never more than the table is wide.  A request whose last rows were rejected
// holds more blocks than its context needs.
struct MapRequest {
    int32_t ctx, fresh, held, wanted;
    bool bad;
};

__device__ __forceinline__ MapRequest map_request(const MapArgs &a, int r) {
    MapRequest q;
    const int32_t c = a.ctx_lens[r], f = a.new_lens[r];
    q.ctx = max(c, 0);
    const int64_t len = min(static_cast<int64_t>(q.ctx) + max(f, 0), static_cast<int64_t>(0x7FFFFFFF));
    q.fresh = static_cast<int32_t>(len - q.ctx);
    const int64_t up = (1 << a.block_log2) - 1;
    const int32_t need = static_cast<int32_t>((len + up) >> a.block_log2);
    q.held = min(static_cast<int32_t>((q.ctx + up) >> a.block_log2), a.width);
    q.bad = c < 0 || f < 0 || need > a.width;
    if (a.held_blocks) {
        const int32_t h = a.held_blocks[r];
        q.held = max(q.held, min(h, a.width));
        q.bad |= h < 0 || h > a.width;
    }
    q.wanted = max(min(need, a.width), q.held);
    return q;
}

// Every CTA scans all n lengths by itself (n x 8 bytes out of L2, cheaper than
// a second launch or a grid-wide wait) and then writes its share of the
// outputs: tokens and fresh table entries, each found by a search in the scan.
// Thread i scans requests [i q, (i + 1) q), q = ceil(n / 512).
//   Bound: latency (the scan, then a search of nine dependent steps).  Measured
// in a graph: 64 requests of one token 5.1 us; 512 requests with 2.1 M new
// tokens 12.7 us, 3.9 of them what the bytes take.
__global__ void __launch_bounds__(kMapThreads) kv_map_kernel(const MapArgs a) {
    __shared__ int64_t s_tok[kMapThreads + 1], s_blk[kMapThreads + 1];  // exclusive prefixes per thread
    __shared__ int64_t w_tok[kMapThreads / 32], w_blk[kMapThreads / 32];
    __shared__ MapRequest s_req[kMapThreads];  // the requests themselves, when each thread scans at most one
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dependency_wait();
    grid_launch_dependents();
    const int q = (a.n + kMapThreads - 1) / kMapThreads;
    const int r0 = min(tid * q, a.n), r1 = min(r0 + q, a.n);
    int64_t tok = 0, blk = 0;
    bool bad = false;
    for (int r = r0; r < r1; ++r) {
        const MapRequest m = map_request(a, r);
        s_req[tid] = m;
        tok += m.fresh;
        blk += m.wanted - m.held;
        bad |= m.bad;
    }
    int64_t pt = tok, pb = blk;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t ut = __shfl_up_sync(0xFFFFFFFFu, pt, d), ub = __shfl_up_sync(0xFFFFFFFFu, pb, d);
        if (lane >= d) {
            pt += ut;
            pb += ub;
        }
    }
    if (lane == 31) {
        w_tok[warp] = pt;
        w_blk[warp] = pb;
    }
    __syncthreads();
    int64_t bt = 0, bb = 0;
    for (int w = 0; w < warp; ++w) {
        bt += w_tok[w];
        bb += w_blk[w];
    }
    s_tok[tid] = bt + pt - tok;
    s_blk[tid] = bb + pb - blk;
    if (tid == kMapThreads - 1) {
        s_tok[kMapThreads] = bt + pt;
        s_blk[kMapThreads] = bb + pb;
    }
    __syncthreads();
    const int64_t total = s_tok[kMapThreads], taken = s_blk[kMapThreads];
    const int32_t head_in = *a.free_head;
    const int64_t head = max(head_in, 0);

    if (blockIdx.x == 0) {  // per-request outputs, the new head and the status
        int64_t at = s_tok[tid], left = a.n_free - head - s_blk[tid];  // ids left for the request
        for (int r = r0; r < r1; ++r) {
            const MapRequest m = map_request(a, r);
            a.seq_lens[r] = m.ctx + m.fresh;
            a.q_starts[r] = static_cast<int32_t>(min(at, a.max_tokens));
            at += m.fresh;
            const int32_t need = m.wanted - m.held;
            if (a.held_out) a.held_out[r] = m.held + static_cast<int32_t>(min(max(left, int64_t(0)), static_cast<int64_t>(need)));
            left -= need;
        }
        if (tid == 0) {
            a.q_starts[a.n] = static_cast<int32_t>(min(total, a.max_tokens));
            *a.free_head_out = static_cast<int32_t>(min(head + taken, max(head, static_cast<int64_t>(a.n_free))));
            bad |= head_in < 0 || total > a.max_tokens;
            if (head + taken > a.n_free) atomicOr(a.status, FP8BLK_STATUS_KV_EXHAUSTED);
        }
        if (bad) atomicOr(a.status, FP8BLK_STATUS_BAD_KV);
    }

    auto request = [&](int r) { return q == 1 ? s_req[r] : map_request(a, r); };
    // The thread whose prefix range holds `at` (< the last entry): the last
    // one with prefix <= at, so threads without a share are passed over.
    auto find = [&](const int64_t *s, int64_t at) {
        int lo = 0, hi = kMapThreads - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s[mid] <= at) lo = mid;
            else hi = mid - 1;
        }
        return lo;
    };
    auto fresh_block = [&](int64_t index) -> int32_t {  // index into the free list
        return index < a.n_free ? a.free_blocks[index] : -1;
    };
    const int64_t step = static_cast<int64_t>(gridDim.x) * kMapThreads;

    // Fresh table entries.
    for (int64_t e = static_cast<int64_t>(blockIdx.x) * kMapThreads + tid; e < taken; e += step) {
        const int t = find(s_blk, e);
        int64_t at = s_blk[t];
        for (int r = t * q; r < a.n; ++r) {
            const MapRequest m = request(r);
            const int32_t need = m.wanted - m.held;
            if (e < at + need) {
                a.table[static_cast<int64_t>(r) * a.width + m.held + (e - at)] = fresh_block(head + e);
                break;
            }
            at += need;
        }
    }

    // Slots and positions; past the last token both are -1.
    const int64_t live = min(total, a.max_tokens);
    for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kMapThreads + tid) * kMapPerThread; t0 < a.max_tokens;
         t0 += step * kMapPerThread) {
        int r = -1;
        int64_t start = 0, end = 0, first = 0;  // the request's tokens [start, end), its first fresh block
        MapRequest m = {};
        int64_t slot[kMapPerThread];
        int32_t pos[kMapPerThread];
#pragma unroll
        for (int j = 0; j < kMapPerThread; ++j) {
            const int64_t t = t0 + j;
            slot[j] = -1;
            pos[j] = -1;
            if (t >= live) continue;
            if (r < 0) {
                const int i = find(s_tok, t);
                r = i * q;
                m = request(r);
                start = s_tok[i];
                end = start + m.fresh;
                first = s_blk[i];
            }
            while (t >= end) {
                first += m.wanted - m.held;
                start = end;
                m = request(++r);
                end = start + m.fresh;
            }
            pos[j] = static_cast<int32_t>(m.ctx + (t - start));
            const int32_t b = pos[j] >> a.block_log2;
            int32_t id = -1;
            if (b < m.held) id = a.table[static_cast<int64_t>(r) * a.width + b];
            else if (b < m.wanted) id = fresh_block(head + first + (b - m.held));
            if (id >= 0) slot[j] = (static_cast<int64_t>(id) << a.block_log2) + (pos[j] & ((1 << a.block_log2) - 1));
        }
        if (t0 + kMapPerThread <= a.max_tokens) {
            longlong2 *sp = reinterpret_cast<longlong2 *>(a.slots + t0);
            sp[0] = make_longlong2(slot[0], slot[1]);
            sp[1] = make_longlong2(slot[2], slot[3]);
            *reinterpret_cast<int4 *>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        } else {
#pragma unroll
            for (int j = 0; j < kMapPerThread; ++j)
                if (t0 + j < a.max_tokens) {
                    a.slots[t0 + j] = slot[j];
                    a.positions[t0 + j] = pos[j];
                }
        }
    }
}

// --------------------------------------------------------------- kv_append
struct AppendArgs {
    const void *k, *v;       // [n_tokens, kv_heads, head_dim], token strides below
    const int64_t *slots;    // [n_tokens]
    uint8_t *k_codes, *v_codes;
    float *k_scales, *v_scales;
    unsigned int *status;
    int64_t n_tokens, k_stride, v_stride;  // strides in elements
    int64_t n_slots;                       // n_blocks * block_tokens
    int kv_heads, head_dim, block_log2;
    int chunk;                             // tokens a CTA looks after
    int checks, check_words;               // CTAs that look for blocks with two runs, words of their bitmaps
    int staged;                            // values of one run that shared memory holds (0: none)
    uint32_t per_inverse;                  // ceil(2^32 / (head_dim / 8)): divides group numbers below 2^16
};
// Query heads a thread takes beside the cache's CTAs: with 1, 2 and 4 the 16.7 k tokens below took 96, 91 and 98 us (f32: 152 and 142).
constexpr int kAppendQueryHeads = 2;
// ... with keys that are rotated first, and queries that are rotated beside them.
struct AppendRopeArgs : AppendArgs {
    RopeArgs rope;       // the keys' (x, out and strides unused)
    RopeArgs q;          // the queries'
    uint32_t q_items;    // 0: no queries
    int q_first;         // from this blockIdx.x on CTAs take the queries' items, kAppendThreads each
};

// |v| for a block's maximum: what is not finite does not count.
__device__ __forceinline__ uint32_t finite_abs_bits(float v) {
    const uint32_t u = __float_as_uint(v) & 0x7FFFFFFFu;
    return u < 0x7F800000u ? u : 0u;
}

// Biased exponent of the smallest power of two s >= 2^-126 with amax <= 448 s
// (amax as f32 bits): 448 = 1.75 x 2^8, so amax = 1.f x 2^x needs x - 8, and
// one more when 1.f > 1.75.  amax < 2^128 gives at most 2^120.
__device__ __forceinline__ int scale_exponent(uint32_t amax_bits) {
    const int e = static_cast<int>(amax_bits >> 23) - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u);
    return e < 1 ? 1 : e;
}

// Two f32 -> two e4m3 codes (nearest even; NaN and, by the caller, infinities
// become the NaN code).
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// Scales written here are powers of two, and products and quotients by them exact; one that was there may be any number.
// q, the f32 next to a result, and the sign of what it leaves of it: rounded to odd instead, so that rounding q to e4m3
// rounds the result once.
__device__ __forceinline__ float round_to_odd(float q, float left) {
    const uint32_t u = __float_as_uint(q);
    if (left == 0.f || q == 0.f || (u & 1u)) return q;
    return __uint_as_float((left > 0.f) == (q > 0.f) ? u + 1u : u - 1u);
}
__device__ __forceinline__ float times_to_odd(float a, float b) {
    const float p = a * b;
    return round_to_odd(p, fmaf(a, b, -p));
}
// x / s from inv = 1 / s and one correction of the quotient by its remainder (Markstein); all brought up where a
// remainder would be too small for an f32.
__device__ __forceinline__ float over_to_odd(float x, float s, float inv) {
    const bool small = s < 0x1p-60f;
    x = small ? x * 0x1p60f : x;
    s = small ? s * 0x1p60f : s;
    inv = small ? inv * 0x1p-60f : inv;
    float q = x * inv;
    q = fmaf(fmaf(-q, s, x), inv, q);
    return round_to_odd(q, fmaf(-q, s, x));
}
__device__ __forceinline__ bool power_of_two(float s) { return (__float_as_uint(s) & 0x7FFFFFu) == 0; }
__device__ __forceinline__ float poison_inf(float v) { return isfinite(v) ? v : __int_as_float(0x7FC00000); }

// Eight consecutive values as they lie in memory: two or one 16-byte words.
template <typename T>
struct Eight;
template <>
struct Eight<float> {
    float4 a, b;
    __device__ __forceinline__ void set(const float (&v)[8]) {
        a = make_float4(v[0], v[1], v[2], v[3]);
        b = make_float4(v[4], v[5], v[6], v[7]);
    }
    __device__ __forceinline__ void load(const float *p) {
        a = *reinterpret_cast<const float4 *>(p);
        b = *reinterpret_cast<const float4 *>(p + 4);
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
    // The largest magnitude, NaN left out.
    __device__ __forceinline__ float peak(float m) const {
        float x[8];
        get(x);
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
        return m;
    }
};
template <>
struct Eight<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { a = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = bf16x2_to_f32(w[i]);
            x[2 * i] = f.x, x[2 * i + 1] = f.y;
        }
    }
    __device__ __forceinline__ float peak(float m) const {
        const __nv_bfloat162 *w = reinterpret_cast<const __nv_bfloat162 *>(&a);
        const __nv_bfloat162 h = __hmax2(__hmax2(__habs2(w[0]), __habs2(w[1])), __hmax2(__habs2(w[2]), __habs2(w[3])));
        return fmaxf(m, fmaxf(__low2float(h), __high2float(h)));
    }
};

constexpr int kAppendThreads = 256;
constexpr int kAppendWarps = kAppendThreads / 32;
constexpr int kAppendHeld = 4;       // groups of eight values a thread keeps between its two passes
constexpr int kAppendMaxChunk = 64;  // tokens a CTA looks after
constexpr int kCheckWords = 1024;    // words of a bitmap of blocks, at most (more would take L1 from the CTAs that write)
constexpr int kCheckAhead = 8;       // slots of a thread in flight

// The token of group i of a run (i < 128 x 32): i / (head_dim / 8) by its inverse,
// exact (the excess, i x (head_dim / 8) / 2^32, is below one group).
__device__ __forceinline__ int append_row(const AppendArgs &a, int i) {
    return static_cast<int>(__umulhi(static_cast<uint32_t>(i), a.per_inverse));
}

// One run for one head of K or V: maximum, scale, codes.  THREADS threads (a
// warp, or the CTA) take the run's groups of eight in turn.  A warp keeps its
// first kAppendHeld groups in registers between the two passes (1024 values; the
// rest comes from L1 again); the CTA takes them from shared memory, where they
// were copied for K and V at once, so that V's are on their way while K's are
// encoded.  staged: null if the run does not fit there.  red: a word per warp.
// ROPE: keys, rotated in f32 as they are read (staged ones have been); the scale
// and the codes go by the rotated values, unrounded.
template <typename T, int THREADS, int kHeld, bool ROPE, typename A>
__device__ __forceinline__ void append_run(const A &a, int64_t t, int64_t slot, int run, int h, bool is_v, int tid,
                                           const std::conditional_t<ROPE, float, T> *staged, uint32_t *red) {
    using Group = Eight<std::conditional_t<ROPE, float, T>>;
    const int D = a.head_dim, block = 1 << a.block_log2, off = static_cast<int>(slot & (block - 1));
    const int64_t stride = is_v ? a.v_stride : a.k_stride;
    const T *x = static_cast<const T *>(is_v ? a.v : a.k) + t * stride + static_cast<int64_t>(h) * D;
    const int64_t bh = (slot >> a.block_log2) * a.kv_heads + h;
    uint8_t *codes = (is_v ? a.v_codes : a.k_codes) + bh * block * D;
    float *scale = (is_v ? a.v_scales : a.k_scales) + bh;
    const int per = D / 8, total = run * per;
    auto at = [&](int i) {
        const int row = append_row(a, i);
        return x + row * stride + 8 * (i - row * per);
    };
    auto fetch = [&](Group &e, int i) {
        if constexpr (ROPE) {
            const int row = append_row(a, i);
            float f[8];
            rope_eight(a.rope, x + row * stride, a.rope.cos_sin + (t + row) * a.rope.rot, 8 * (i - row * per), f);
            e.set(f);
        } else {
            e.load(at(i));
        }
    };
    Group held[kHeld + 1];
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
        if (tid + k * THREADS < total) fetch(held[k], tid + k * THREADS);
    const float old = off > 0 ? *scale : 0.f;
    // Over all the run's groups, and over the threads.  (Magnitudes are not negative: their bits order as they do.)
    auto over_run = [&](auto f) {
#pragma unroll
        for (int k = 0; k < kHeld; ++k)
            if (tid + k * THREADS < total) f(held[k], tid + k * THREADS);
        if (THREADS > 32 && staged) {
#pragma unroll 4
            for (int i = tid; i < total; i += THREADS) {
                Group e;
                e.load(staged + 8 * i);
                f(e, i);
            }
        } else {
#pragma unroll 1
            for (int i = tid + kHeld * THREADS; i < total; i += THREADS) {
                Group e;
                fetch(e, i);
                f(e, i);
            }
        }
    };
    auto over_threads = [&](uint32_t m) {
        m = __reduce_max_sync(0xFFFFFFFFu, m);
        if constexpr (THREADS > 32) {
            if ((tid & 31) == 0) red[tid >> 5] = m;
            __syncthreads();
            m = __reduce_max_sync(0xFFFFFFFFu, red[tid & (THREADS / 32 - 1)]);
        }
        return m;
    };
    float peak = 0.f;
    over_run([&](const Group &e, int) { peak = e.peak(peak); });
    uint32_t amax = over_threads(__float_as_uint(peak));
    const bool infinite = amax >= 0x7F800000u;
    if (infinite) {  // not often: once more, infinities left out (NaN already are)
        if constexpr (THREADS > 32) __syncthreads();
        uint32_t m = 0;
        over_run([&](const Group &e, int) {
            float f[8];
            e.get(f);
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max(m, finite_abs_bits(f[j]));
        });
        amax = over_threads(m);
    }
    float s = __uint_as_float(static_cast<uint32_t>(scale_exponent(amax)) << 23);
    if (off > 0) {
        if (old < s) {  // the codes that were there follow the larger scale
            const float ratio = old / s;
            uint32_t *w = reinterpret_cast<uint32_t *>(codes);
#pragma unroll 1
            for (int i = tid; i < off * per * 2; i += THREADS) {
                float2 lo, hi;
                e4m3x4_to_f32(w[i], lo, hi);
                w[i] = to_e4m3x2(times_to_odd(lo.x, ratio), times_to_odd(lo.y, ratio)) |
                       (to_e4m3x2(times_to_odd(hi.x, ratio), times_to_odd(hi.y, ratio)) << 16);
            }
        } else {
            s = old;
        }
    }
    const float inv = 1.0f / s;
    uint2 *w = reinterpret_cast<uint2 *>(codes + static_cast<int64_t>(off) * D);
    auto encode = [&](const float (&f)[8], int i) {
        w[i] = make_uint2(to_e4m3x2(f[0], f[1]) | (to_e4m3x2(f[2], f[3]) << 16), to_e4m3x2(f[4], f[5]) | (to_e4m3x2(f[6], f[7]) << 16));
    };
    if (power_of_two(s)) {
        over_run([&](const Group &e, int i) {
            float f[8];
            e.get(f);
            if (infinite) {
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = poison_inf(f[j]);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] *= inv;
            encode(f, i);
        });
    } else {  // (a loop of its own: as a branch in the other one it cost prompts 4%)
#pragma unroll 1
        for (int i = tid; i < total; i += THREADS) {
            Group e;
            float f[8];
            fetch(e, i);
            e.get(f);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = over_to_odd(poison_inf(f[j]), s, inv);
            encode(f, i);
        }
    }
    if constexpr (THREADS > 32) __syncthreads();  // red, the staged values and the old scale have been read
    else __syncwarp();
    if (tid == 0) *scale = s;
}

// Two runs in one block would be written by two CTAs at once.  CTA c of the first
// few marks the blocks of its range in a bitmap, run by run, and flags what is
// marked twice: one pass over the slots beside the CTAs that write (no time of its
// own with 64 tokens, 16.7 k or 131 k of 8 heads; 131 k of one head in a pool of
// two million blocks wait for it, 80 us instead of 32).
__device__ __noinline__ void append_check(const int64_t *slots, int64_t n_tokens, int64_t n_slots, int block_log2,
                                          int check_words, unsigned int *status, uint32_t *bitmap, int c) {
    const int tid = threadIdx.x, lane = tid & 31, block = 1 << block_log2;
    const int64_t base = static_cast<int64_t>(c) * check_words * 32;
    for (int i = tid; i < check_words; i += kAppendThreads) bitmap[i] = 0;
    __syncthreads();
    bool twice = false;
    // A warp takes 32 x kCheckAhead consecutive slots at a time.
    for (int64_t t0 = (tid >> 5) * 32 * kCheckAhead; t0 < n_tokens; t0 += kAppendThreads * kCheckAhead) {
        int64_t mine[kCheckAhead], before = t0 > 0 ? slots[t0 - 1] : -1;
#pragma unroll
        for (int j = 0; j < kCheckAhead; ++j) mine[j] = t0 + 32 * j + lane < n_tokens ? slots[t0 + 32 * j + lane] : -1;
#pragma unroll
        for (int j = 0; j < kCheckAhead; ++j) {
            const int64_t left = __shfl_up_sync(0xFFFFFFFFu, mine[j], 1), b = (mine[j] >> block_log2) - base;
            if (lane > 0) before = left;
            if (mine[j] >= 0 && mine[j] < n_slots && ((mine[j] & (block - 1)) == 0 || before != mine[j] - 1) && b >= 0 &&
                b < static_cast<int64_t>(check_words) * 32) {
                const uint32_t bit = 1u << (b & 31);
                twice |= (atomicOr(bitmap + (b >> 5), bit) & bit) != 0;
            }
            before = __shfl_sync(0xFFFFFFFFu, mine[j], 31);
        }
    }
    if (twice) atomicOr(status, FP8BLK_STATUS_BAD_KV);
}

// A run is a maximal group of consecutive tokens with consecutive slots of one
// block; its first token leads it, and the CTA whose chunk holds that token
// writes it.  Chunks with few leaders (prompts) take one run at a time with the
// whole CTA, chunks with many (decode) a warp per run.
//   Bound: HBM for prompts (es bytes in, 1 out per value), latency for decode.
// Measured in a graph: 16.7 k bf16 tokens of 16 prompts, 8 heads of 128, 24.2 us
// (64% of the copy rate; ncu: 81% of the issue slots busy while an SM has work,
// 35% of DRAM's throughput, and 2104 CTAs of 912 at a time leave the last wave a
// third full); 64 tokens of f32, one a request, 2.8 us.
//   With rotated keys (A = AppendRopeArgs) the CTA stages K as rotated f32, and
// CTAs behind the cache's rotate the queries of the same rows.  The 16.7 k tokens
// with 32 query heads: 91 us, 62% of the copy rate, about half for the queries (whose
// CTAs have the staging's share of an SM: four at a time) and half for the cache,
// where 64 registers and 48 KiB leave four CTAs waiting on loads one after the other.
// Measured and not kept: the queries by a kernel of their own (96 us) or spread among
// the cache's CTAs (90), both halves of a head by one thread (no gain).  The same of
// f32: 138 us, 78% of the copy rate.  64 tokens of f32: 19 us a call from the host,
// 4.4 in a graph, 8.6 alone on the device with cold caches.
template <typename T, bool WHOLE, typename A>
__global__ void __launch_bounds__(kAppendThreads, !WHOLE ? 2 : std::is_same_v<A, AppendArgs> ? 6 : 4) kv_append_kernel(const A a) {
    constexpr bool ROPE = std::is_same_v<A, AppendRopeArgs>;
    extern __shared__ __align__(16) uint8_t append_smem[];  // a run's values, K's and V's
    __shared__ uint32_t s_starts[kAppendWarps], s_leads[kAppendWarps];  // a bit per token from the chunk's first on
    __shared__ uint32_t red[kAppendWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = blockIdx.y;
    const int64_t t0 = (static_cast<int64_t>(blockIdx.x) - a.checks) * a.chunk;
    const int block = 1 << a.block_log2;
    grid_dependency_wait();
    grid_launch_dependents();
    if constexpr (ROPE) {
        if (static_cast<int>(blockIdx.x) >= a.q_first) {
            const uint32_t cta = ((blockIdx.x - a.q_first) * gridDim.y + blockIdx.y) * gridDim.z + blockIdx.z;
            const uint32_t item = cta * kAppendThreads + tid;
            if (item < a.q_items) rope_item<T, kAppendQueryHeads>(a.q, item);
            return;
        }
    }
    if (t0 < 0) {
        if (h == 0 && blockIdx.z == 0)
            append_check(a.slots, a.n_tokens, a.n_slots, a.block_log2, a.check_words, a.status,
                         reinterpret_cast<uint32_t *>(append_smem), static_cast<int>(blockIdx.x));
        return;
    }
    // Where runs start, in the chunk and as far past it as its last run can reach (chunk + block <= 192 tokens).
    const int64_t mine = t0 + tid < a.n_tokens ? a.slots[t0 + tid] : -1;
    const int64_t before = t0 + tid > 0 && t0 + tid < a.n_tokens ? a.slots[t0 + tid - 1] : -1;
    const bool good = mine >= 0 && mine < a.n_slots, here = tid < a.chunk;
    const bool starts = !good || (mine & (block - 1)) == 0 || before != mine - 1;
    if (here && mine >= a.n_slots) atomicOr(a.status, FP8BLK_STATUS_BAD_KV);
    const uint32_t sb = __ballot_sync(0xFFFFFFFFu, starts), lb = __ballot_sync(0xFFFFFFFFu, starts && good && here);
    if (lane == 0) {
        s_starts[warp] = sb;
        s_leads[warp] = lb;
    }
    __syncthreads();
    uint64_t leads = s_leads[0] | (static_cast<uint64_t>(s_leads[1]) << 32);
    const bool whole = WHOLE && __popcll(leads) < kAppendWarps / 2;  // the CTA on one run at a time
    for (int n = 0; leads != 0; ++n) {
        const int i = __ffsll(static_cast<long long>(leads)) - 1;
        leads &= leads - 1;
        if (!whole && n % kAppendWarps != warp) continue;
        int end = i + 1;  // the next start
        while ((s_starts[end >> 5] >> (end & 31)) == 0) end = (end | 31) + 1;
        end += __ffs(s_starts[end >> 5] >> (end & 31)) - 1;
        const int64_t slot = a.slots[t0 + i];
        if constexpr (WHOLE) if (whole) {
            const int per = a.head_dim / 8, total = (end - i) * per;
            const bool fits = total * 8 <= a.staged;
            // K's values (rotated ones as f32), then V's.
            using Key = std::conditional_t<ROPE, float, T>;
            Key *k_staged = reinterpret_cast<Key *>(append_smem);
            T *v_staged = reinterpret_cast<T *>(k_staged + a.staged);
            if (fits) {
                auto copy = [&](const void *from, int64_t stride, T *to) {
                    const T *x = static_cast<const T *>(from) + (t0 + i) * stride + static_cast<int64_t>(h) * a.head_dim;
                    for (int g = tid; g < total; g += kAppendThreads) {
                        const int row = append_row(a, g);
                        const T *src = x + row * stride + 8 * (g - row * per);
                        const uint32_t dst = smem_addr(to + 8 * g);
#pragma unroll
                        for (int y = 0; y < static_cast<int>(sizeof(T)) / 2; ++y)
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + 16 * y),
                                         "l"(reinterpret_cast<const char *>(src) + 16 * y)
                                         : "memory");
                    }
                    asm volatile("cp.async.commit_group;" ::: "memory");
                };
                if constexpr (ROPE) {
                    copy(a.v, a.v_stride, v_staged);
                    const T *x = static_cast<const T *>(a.k) + (t0 + i) * a.k_stride + static_cast<int64_t>(h) * a.head_dim;
#pragma unroll 2
                    for (int g = tid; g < total; g += kAppendThreads) {
                        const int row = append_row(a, g);
                        float f[8];
                        rope_eight(a.rope, x + row * a.k_stride, a.rope.cos_sin + (t0 + i + row) * a.rope.rot, 8 * (g - row * per), f);
                        rope_store8(k_staged + 8 * g, f);
                    }
                } else {
#pragma unroll 1
                    for (int v = 0; v < 2; ++v)
                        copy(v ? a.v : a.k, v ? a.v_stride : a.k_stride, v ? v_staged : reinterpret_cast<T *>(k_staged));
                }
            }
            if constexpr (ROPE) {
                __syncthreads();
                append_run<T, kAppendThreads, 0, true>(a, t0 + i, slot, end - i, h, false, tid, fits ? k_staged : nullptr, red);
                asm volatile("cp.async.wait_group 0;" ::: "memory");
                __syncthreads();
                append_run<T, kAppendThreads, 0, false>(a, t0 + i, slot, end - i, h, true, tid, fits ? v_staged : nullptr, red);
            } else {
#pragma unroll 1
                for (int v = 0; v < 2; ++v) {
                    if (v == 0) asm volatile("cp.async.wait_group 1;" ::: "memory");
                    else asm volatile("cp.async.wait_group 0;" ::: "memory");
                    __syncthreads();
                    append_run<T, kAppendThreads, 0, false>(a, t0 + i, slot, end - i, h, v != 0, tid,
                                                            fits ? (v ? v_staged : reinterpret_cast<T *>(k_staged)) : nullptr, red);
                }
            }
        }
        if (!whole) {
#pragma unroll 1
            for (int v = blockIdx.z; v < 2; v += gridDim.z) {
                if (ROPE && v == 0) append_run<T, 32, WHOLE ? 0 : kAppendHeld, ROPE>(a, t0 + i, slot, end - i, h, false, lane, nullptr, nullptr);
                else append_run<T, 32, WHOLE ? 0 : kAppendHeld, false>(a, t0 + i, slot, end - i, h, v != 0, lane, nullptr, nullptr);
            }
        }
    }
}

}  // namespace fp8blk

using namespace fp8blk;

extern "C" int fp8blk_kv_map_held(const int32_t *ctx_lens, const int32_t *new_lens, const int32_t *held_blocks,
                                  int32_t *block_table, const int32_t *free_blocks, const int32_t *free_head,
                                  int32_t *seq_lens, int32_t *q_starts, int64_t *slots, int32_t *positions,
                                  int32_t *free_head_out, int32_t *held_out, int n_seqs, int max_blocks, int n_free,
                                  int block_tokens, int64_t max_tokens, void *stream) {
    if (!ctx_lens || !new_lens || !block_table || (!free_blocks && n_free != 0) || !free_head || !seq_lens || !q_starts ||
        !slots || !positions || !free_head_out || !held_blocks != !held_out)
        return FP8BLK_EINVAL;
    if (n_seqs < 1 || max_blocks < 1 || n_free < 0 || !step_block_ok(block_tokens) || max_tokens < 1) return FP8BLK_EINVAL;
    if (n_seqs > 65536 || max_tokens > kStepMaxIndex) return FP8BLK_ERANGE;
    if (!step_aligned(ctx_lens, 4) || !step_aligned(new_lens, 4) || !step_aligned(block_table, 4) ||
        !step_aligned(free_blocks, 4) || !step_aligned(free_head, 4) || !step_aligned(seq_lens, 4) ||
        !step_aligned(q_starts, 4) || !step_aligned(free_head_out, 4) || !step_aligned(held_blocks, 4) ||
        !step_aligned(held_out, 4) || !step_aligned(slots, 16) || !step_aligned(positions, 16))
        return FP8BLK_EALIGN;
    if (free_head == free_head_out || seq_lens == ctx_lens || seq_lens == new_lens ||
        (held_out && (held_out == held_blocks || held_out == ctx_lens || held_out == new_lens)))
        return FP8BLK_EINVAL;
    DeviceInfo dev;
    if (current_device_info(&dev) != cudaSuccess) return step_from_cuda(cudaErrorUnknown);
    MapArgs a = {ctx_lens, new_lens, held_blocks, held_out, block_table, free_blocks, free_head, seq_lens, q_starts, slots,
                 positions, free_head_out, dev.status, n_seqs, max_blocks, n_free, step_log2(block_tokens), max_tokens};
    int64_t grid = (max_tokens + kMapThreads * kMapPerThread - 1) / (kMapThreads * kMapPerThread);
    if (grid > 3 * dev.sms) grid = 3 * dev.sms;
    return step_from_cuda(step_launch(kv_map_kernel, dim3(static_cast<unsigned>(grid)), kMapThreads, 0,
                                      static_cast<cudaStream_t>(stream), a));
}

extern "C" int fp8blk_kv_map(const int32_t *ctx_lens, const int32_t *new_lens, int32_t *block_table,
                             const int32_t *free_blocks, const int32_t *free_head, int32_t *seq_lens, int32_t *q_starts,
                             int64_t *slots, int32_t *positions, int32_t *free_head_out, int n_seqs, int max_blocks,
                             int n_free, int block_tokens, int64_t max_tokens, void *stream) {
    return fp8blk_kv_map_held(ctx_lens, new_lens, nullptr, block_table, free_blocks, free_head, seq_lens, q_starts, slots,
                              positions, free_head_out, nullptr, n_seqs, max_blocks, n_free, block_tokens, max_tokens, stream);
}

static int append_check_args(const void *k, const void *v, int dtype, const int64_t *slots, const uint8_t *k_codes, const float *k_scales,
                             const uint8_t *v_codes, const float *v_scales, int64_t n_tokens, int64_t k_stride, int64_t v_stride,
                             int64_t n_blocks, int kv_heads, int block_tokens, int head_dim) {
    if (!k || !v || !slots || (dtype != FP8BLK_F32 && dtype != FP8BLK_BF16) || n_tokens < 1) return FP8BLK_EINVAL;
    const int rc = step_check_cache(k_codes, k_scales, v_codes, v_scales, n_blocks, kv_heads, block_tokens, head_dim);
    if (rc != FP8BLK_OK) return rc;
    const int64_t row = static_cast<int64_t>(kv_heads) * head_dim;
    const int es = dtype == FP8BLK_F32 ? 4 : 2;
    if (k_stride < row || v_stride < row || k_stride * es % 16 != 0 || v_stride * es % 16 != 0) return FP8BLK_EINVAL;
    if (n_tokens > kStepMaxIndex || k_stride > kStepMaxIndex || v_stride > kStepMaxIndex) return FP8BLK_ERANGE;
    if (!step_aligned(k, 16) || !step_aligned(v, 16) || !step_aligned(slots, 8)) return FP8BLK_EALIGN;
    return FP8BLK_OK;
}

template <typename A>
static int append_launch(A a, int dtype, int64_t n_blocks, int block_tokens, const DeviceInfo &dev, cudaStream_t s) {
    constexpr bool kRope = std::is_same_v<A, AppendRopeArgs>;
    const int es = dtype == FP8BLK_F32 ? 4 : 2;
    // Tokens per CTA: four, for a decode step, and twice as many again while that leaves eight chunks an SM.  From 16 on
    // (9728 (token, head) pairs on 152 SMs) a CTA takes whole runs.  The rule goes by the total: one prompt of 1000 tokens
    // and 8 heads is below it, and a warp writes each of its runs (15.5 us).
    while (a.chunk < kAppendMaxChunk && a.n_tokens * a.kv_heads * 2 / (2 * a.chunk) >= 8 * dev.sms) a.chunk *= 2;
    // K and V by the same CTA where it takes whole runs, by CTAs of their own where a warp does.  Runs are staged in
    // shared memory up to 32 KiB (three CTAs per SM or more); rotated keys take four bytes a value.
    const bool whole = a.chunk > 8;
    if (whole) a.staged = std::min(block_tokens * a.head_dim, 32768 / es);
    a.check_words = static_cast<int>(std::min<int64_t>((n_blocks + 31) / 32, kCheckWords));
    a.checks = static_cast<int>((n_blocks + a.check_words * 32ll - 1) / (a.check_words * 32ll));
    dim3 grid(static_cast<unsigned>(a.checks + (a.n_tokens + a.chunk - 1) / a.chunk), static_cast<unsigned>(a.kv_heads), whole ? 1 : 2);
    if constexpr (kRope) {
        a.q_first = static_cast<int>(grid.x);
        const int64_t slice = static_cast<int64_t>(kAppendThreads) * grid.y * grid.z;
        grid.x += static_cast<unsigned>((a.q_items + slice - 1) / slice);
    }
    const size_t smem = std::max(static_cast<size_t>(a.staged) * ((kRope ? 4 : es) + es), a.check_words * sizeof(uint32_t));
    auto launch = [&](auto kernel) {
        int per_sm = 0;
        const cudaError_t err = kernel_occupancy(reinterpret_cast<const void *>(kernel), kAppendThreads, smem, &per_sm);
        if (err != cudaSuccess) return err;
        if (per_sm < 1) return cudaErrorInvalidConfiguration;
        return step_launch(kernel, grid, kAppendThreads, smem, s, a);
    };
    if (dtype == FP8BLK_F32) return step_from_cuda(whole ? launch(kv_append_kernel<float, true, A>) : launch(kv_append_kernel<float, false, A>));
    return step_from_cuda(whole ? launch(kv_append_kernel<__nv_bfloat16, true, A>) : launch(kv_append_kernel<__nv_bfloat16, false, A>));
}

extern "C" int fp8blk_kv_append(const void *k, const void *v, int dtype, const int64_t *slots, uint8_t *k_codes,
                                float *k_scales, uint8_t *v_codes, float *v_scales, int64_t n_tokens, int64_t k_stride,
                                int64_t v_stride, int64_t n_blocks, int kv_heads, int block_tokens, int head_dim,
                                void *stream) {
    const int rc = append_check_args(k, v, dtype, slots, k_codes, k_scales, v_codes, v_scales, n_tokens, k_stride, v_stride,
                                     n_blocks, kv_heads, block_tokens, head_dim);
    if (rc != FP8BLK_OK) return rc;
    DeviceInfo dev;
    if (current_device_info(&dev) != cudaSuccess) return step_from_cuda(cudaErrorUnknown);
    const AppendArgs a = {k, v, slots, k_codes, v_codes, k_scales, v_scales, dev.status, n_tokens, k_stride, v_stride,
                          n_blocks * block_tokens, kv_heads, head_dim, step_log2(block_tokens), 4, 0, 0, 0,
                          static_cast<uint32_t>(((uint64_t(1) << 32) + head_dim / 8 - 1) / (head_dim / 8))};
    return append_launch(a, dtype, n_blocks, block_tokens, dev, static_cast<cudaStream_t>(stream));
}

extern "C" int fp8blk_kv_append_rope(const void *k, const void *v, int dtype, const int64_t *slots, const float *cos_sin,
                                     uint8_t *k_codes, float *k_scales, uint8_t *v_codes, float *v_scales, const void *q, void *q_out,
                                     int64_t n_tokens, int64_t k_stride, int64_t v_stride, int64_t q_stride, int64_t q_out_stride,
                                     int64_t n_blocks, int kv_heads, int q_heads, int block_tokens, int head_dim, int rot_dim,
                                     int rot_start, int interleaved, void *stream) {
    const int rc = append_check_args(k, v, dtype, slots, k_codes, k_scales, v_codes, v_scales, n_tokens, k_stride, v_stride,
                                     n_blocks, kv_heads, block_tokens, head_dim);
    if (rc != FP8BLK_OK) return rc;
    if (!q != !q_out) return FP8BLK_EINVAL;
    AppendRopeArgs a = {};
    uint32_t items = 0;
    // (The keys' rotation has no output of its own: the checks and the layout are those of one in place.)
    int plan = rope_plan(k, const_cast<void *>(k), cos_sin, dtype, n_tokens, kv_heads, head_dim, rot_dim, rot_start, interleaved,
                         k_stride, k_stride, &a.rope, &items);
    if (plan != FP8BLK_OK) return plan;
    if (q) {
        plan = rope_plan(q, q_out, cos_sin, dtype, n_tokens, q_heads, head_dim, rot_dim, rot_start, interleaved, q_stride, q_out_stride,
                         &a.q, &a.q_items);
        if (plan != FP8BLK_OK) return plan;
        // Some CTAs turn the queries while others read keys and values.
        const int64_t es = dtype == FP8BLK_F32 ? 4 : 2, row = es * kv_heads * head_dim, q_row = es * q_heads * head_dim;
        if (rows_overlap(q_out, q_out_stride * es, q_row, k, k_stride * es, row, n_tokens) ||
            rows_overlap(q_out, q_out_stride * es, q_row, v, v_stride * es, row, n_tokens))
            return FP8BLK_EINVAL;
        a.q.chunks = (q_heads + kAppendQueryHeads - 1) / kAppendQueryHeads;
        a.q_items = static_cast<uint32_t>(n_tokens * a.q.units * a.q.chunks);
    }
    DeviceInfo dev;
    if (current_device_info(&dev) != cudaSuccess) return step_from_cuda(cudaErrorUnknown);
    static_cast<AppendArgs &>(a) = {k, v, slots, k_codes, v_codes, k_scales, v_scales, dev.status, n_tokens, k_stride, v_stride,
                                    n_blocks * block_tokens, kv_heads, head_dim, step_log2(block_tokens), 4, 0, 0, 0,
                                    static_cast<uint32_t>(((uint64_t(1) << 32) + head_dim / 8 - 1) / (head_dim / 8))};
    return append_launch(a, dtype, n_blocks, block_tokens, dev, static_cast<cudaStream_t>(stream));
}
