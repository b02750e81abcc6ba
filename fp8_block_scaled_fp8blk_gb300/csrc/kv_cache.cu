// kv_cache.cu -- the paged e4m3 cache of a decode / verify step: block tables
// and slots from request lengths (fp8blk_kv_map), and keys and values written
// with one power-of-two scale per (block of tokens, head) (fp8blk_kv_append).
//
// A pool holds uint8 e4m3 codes [n_blocks, kv_heads, block_tokens, head_dim]
// and f32 scales [n_blocks, kv_heads].  Head-major inside a block: what one
// head reads of one block is a single run of block_tokens x head_dim bytes
// under one scale.
#include "step.h"

namespace fp8blk {

// ------------------------------------------------------------------ kv_map
struct MapArgs {
    const int32_t *ctx_lens, *new_lens;  // [n]
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
// never more than the table is wide.
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
    q.wanted = min(need, a.width);
    q.bad = c < 0 || f < 0 || need > a.width;
    return q;
}

// Every CTA scans all n lengths by itself (n x 8 bytes out of L2, cheaper than
// a second launch or a grid-wide wait) and then writes its share of the
// outputs: tokens and fresh table entries, each found by a search in the scan.
// Thread i scans requests [i q, (i + 1) q), q = ceil(n / 512).
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
        int64_t at = s_tok[tid];
        for (int r = r0; r < r1; ++r) {
            const MapRequest m = map_request(a, r);
            a.seq_lens[r] = m.ctx + m.fresh;
            a.q_starts[r] = static_cast<int32_t>(min(at, a.max_tokens));
            at += m.fresh;
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
__device__ __forceinline__ float poison_inf(float v) { return isfinite(v) ? v : __int_as_float(0x7FC00000); }

// Eight consecutive values as they lie in memory: two or one 16-byte words.
template <typename T>
struct Eight;
template <>
struct Eight<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = *reinterpret_cast<const float4 *>(p);
        b = *reinterpret_cast<const float4 *>(p + 4);
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
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
};

constexpr int kAppendThreads = 256;
constexpr int kAppendWarps = kAppendThreads / 32;
constexpr int kAppendHeld = 4;       // groups of eight values a thread keeps between its two passes
constexpr int kAppendMaxChunk = 64;  // tokens a CTA looks after

// One run for one head of K or V: maximum, scale, codes.  THREADS threads (a
// warp, or the CTA) take the run's groups of eight in turn; the first
// kAppendHeld groups of a thread stay in registers, so that runs of up to 8192
// values (a CTA) or 1024 (a warp) are read once, and the rest comes from L1.
// red: a word per warp (CTA only).
template <typename T, int THREADS>
__device__ __forceinline__ void append_run(const AppendArgs &a, int64_t t, int64_t slot, int run, int h, bool is_v, int tid,
                                           uint32_t *red) {
    const int D = a.head_dim, block = 1 << a.block_log2, off = static_cast<int>(slot & (block - 1));
    const int64_t stride = is_v ? a.v_stride : a.k_stride;
    const T *x = static_cast<const T *>(is_v ? a.v : a.k) + t * stride + static_cast<int64_t>(h) * D;
    const int64_t bh = (slot >> a.block_log2) * a.kv_heads + h;
    uint8_t *codes = (is_v ? a.v_codes : a.k_codes) + bh * block * D;
    float *scale = (is_v ? a.v_scales : a.k_scales) + bh;
    const int per = D / 8, total = run * per;
    auto at = [&](int i) {
        const int row = i / per;
        return x + row * stride + 8 * (i - row * per);
    };
    Eight<T> held[kAppendHeld];
#pragma unroll
    for (int k = 0; k < kAppendHeld; ++k)
        if (tid + k * THREADS < total) held[k].load(at(tid + k * THREADS));
    const float old = off > 0 ? *scale : 0.f;
    uint32_t amax = 0;
    auto peak = [&](const Eight<T> &e) {
        float f[8];
        e.get(f);
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = max(amax, finite_abs_bits(f[j]));
    };
#pragma unroll
    for (int k = 0; k < kAppendHeld; ++k)
        if (tid + k * THREADS < total) peak(held[k]);
    for (int i = tid + kAppendHeld * THREADS; i < total; i += THREADS) {
        Eight<T> e;
        e.load(at(i));
        peak(e);
    }
    amax = __reduce_max_sync(0xFFFFFFFFu, amax);
    if constexpr (THREADS > 32) {
        if ((tid & 31) == 0) red[tid >> 5] = amax;
        __syncthreads();
        amax = __reduce_max_sync(0xFFFFFFFFu, red[tid & (THREADS / 32 - 1)]);
    }
    float s = __uint_as_float(static_cast<uint32_t>(scale_exponent(amax)) << 23);
    if (off > 0) {
        if (old < s) {  // the codes that were there follow the larger scale: a product by a power of two, rounded once
            const float ratio = old / s;
            uint32_t *w = reinterpret_cast<uint32_t *>(codes);
            for (int i = tid; i < off * per * 2; i += THREADS) {
                float2 lo, hi;
                e4m3x4_to_f32(w[i], lo, hi);
                w[i] = to_e4m3x2(lo.x * ratio, lo.y * ratio) | (to_e4m3x2(hi.x * ratio, hi.y * ratio) << 16);
            }
        } else {
            s = old;
        }
    }
    const float inv = 1.0f / s;
    uint2 *w = reinterpret_cast<uint2 *>(codes + static_cast<int64_t>(off) * D);
    auto encode = [&](const Eight<T> &e, int i) {
        float f[8];
        e.get(f);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = poison_inf(f[j]) * inv;
        w[i] = make_uint2(to_e4m3x2(f[0], f[1]) | (to_e4m3x2(f[2], f[3]) << 16), to_e4m3x2(f[4], f[5]) | (to_e4m3x2(f[6], f[7]) << 16));
    };
#pragma unroll
    for (int k = 0; k < kAppendHeld; ++k)
        if (tid + k * THREADS < total) encode(held[k], tid + k * THREADS);
    for (int i = tid + kAppendHeld * THREADS; i < total; i += THREADS) {
        Eight<T> e;
        e.load(at(i));
        encode(e, i);
    }
    if constexpr (THREADS > 32) __syncthreads();  // red and the old scale have been read
    else __syncwarp();
    if (tid == 0) *scale = s;
}

// A run is a maximal group of consecutive tokens with consecutive slots of one
// block; its first token leads it, and the CTA whose chunk holds that token
// writes it.  Chunks with few leaders (prompts) take one run at a time with the
// whole CTA, chunks with many (decode) a warp per run.
//   Bound: HBM for prompts (es bytes in, 1 out per value), latency for decode.
template <typename T>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const AppendArgs a) {
    __shared__ int s_lead[kAppendMaxChunk], s_leads, s_run;
    __shared__ uint32_t red[kAppendWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = blockIdx.y;
    const bool is_v = blockIdx.z != 0;
    const int block = 1 << a.block_log2;
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.chunk;
    const int here = static_cast<int>(min(static_cast<int64_t>(a.chunk), a.n_tokens - t0));
    if (tid == 0) {
        s_leads = 0;
        s_run = block;
    }
    __syncthreads();
    if (tid < here) {
        const int64_t slot = a.slots[t0 + tid], before = t0 + tid > 0 ? a.slots[t0 + tid - 1] : -1;
        if (slot >= a.n_slots) atomicOr(a.status, FP8BLK_STATUS_BAD_KV);
        else if (slot >= 0 && ((slot & (block - 1)) == 0 || before != slot - 1)) s_lead[atomicAdd(&s_leads, 1)] = tid;
    }
    __syncthreads();
    const int leads = s_leads;
    if (leads >= kAppendWarps / 2 || (here <= 32 && leads * 8 >= here)) {
        for (int i = warp; i < leads; i += kAppendWarps) {
            const int64_t t = t0 + s_lead[i], slot = a.slots[t];
            const int most = block - static_cast<int>(slot & (block - 1));
            int run = 1;
            for (int base = 1; base < most; base += 32) {
                const int j = base + lane;
                const bool follows = j < most && t + j < a.n_tokens && a.slots[t + j] == slot + j;
                const unsigned stop = __ballot_sync(0xFFFFFFFFu, !follows);
                if (stop) {
                    run += __ffs(stop) - 1;
                    break;
                }
                run += 32;
            }
            append_run<T, 32>(a, t, slot, run, h, is_v, lane, nullptr);
        }
    } else {
        for (int i = 0; i < leads; ++i) {
            const int64_t t = t0 + s_lead[i], slot = a.slots[t];
            const int most = block - static_cast<int>(slot & (block - 1));
            if (tid > 0 && tid < most && !(t + tid < a.n_tokens && a.slots[t + tid] == slot + tid)) atomicMin(&s_run, tid);
            __syncthreads();
            const int run = min(s_run, most);
            append_run<T, kAppendThreads>(a, t, slot, run, h, is_v, tid, red);
            if (tid == 0) s_run = block;
            __syncthreads();
        }
    }
}

}  // namespace fp8blk

using namespace fp8blk;

extern "C" int fp8blk_kv_map(const int32_t *ctx_lens, const int32_t *new_lens, int32_t *block_table,
                             const int32_t *free_blocks, const int32_t *free_head, int32_t *seq_lens, int32_t *q_starts,
                             int64_t *slots, int32_t *positions, int32_t *free_head_out, int n_seqs, int max_blocks,
                             int n_free, int block_tokens, int64_t max_tokens, void *stream) {
    if (!ctx_lens || !new_lens || !block_table || !free_blocks || !free_head || !seq_lens || !q_starts || !slots ||
        !positions || !free_head_out)
        return FP8BLK_EINVAL;
    if (n_seqs < 1 || max_blocks < 1 || n_free < 0 || !step_block_ok(block_tokens) || max_tokens < 1) return FP8BLK_EINVAL;
    if (n_seqs > 65536 || max_tokens > kStepMaxIndex) return FP8BLK_ERANGE;
    if (!step_aligned(ctx_lens, 4) || !step_aligned(new_lens, 4) || !step_aligned(block_table, 4) ||
        !step_aligned(free_blocks, 4) || !step_aligned(free_head, 4) || !step_aligned(seq_lens, 4) ||
        !step_aligned(q_starts, 4) || !step_aligned(free_head_out, 4) || !step_aligned(slots, 16) ||
        !step_aligned(positions, 16))
        return FP8BLK_EALIGN;
    if (free_head == free_head_out || seq_lens == ctx_lens || seq_lens == new_lens) return FP8BLK_EINVAL;
    DeviceInfo dev;
    if (current_device_info(&dev) != cudaSuccess) return step_from_cuda(cudaErrorUnknown);
    MapArgs a = {ctx_lens, new_lens, block_table, free_blocks, free_head, seq_lens, q_starts, slots, positions,
                 free_head_out, dev.status, n_seqs, max_blocks, n_free, step_log2(block_tokens), max_tokens};
    int64_t grid = (max_tokens + kMapThreads * kMapPerThread - 1) / (kMapThreads * kMapPerThread);
    if (grid > 3 * dev.sms) grid = 3 * dev.sms;
    return step_from_cuda(step_launch(kv_map_kernel, dim3(static_cast<unsigned>(grid)), kMapThreads, 0,
                                      static_cast<cudaStream_t>(stream), a));
}

extern "C" int fp8blk_kv_append(const void *k, const void *v, int dtype, const int64_t *slots, uint8_t *k_codes,
                                float *k_scales, uint8_t *v_codes, float *v_scales, int64_t n_tokens, int64_t k_stride,
                                int64_t v_stride, int64_t n_blocks, int kv_heads, int block_tokens, int head_dim,
                                void *stream) {
    if (!k || !v || !slots || (dtype != FP8BLK_F32 && dtype != FP8BLK_BF16) || n_tokens < 1) return FP8BLK_EINVAL;
    const int rc = step_check_cache(k_codes, k_scales, v_codes, v_scales, n_blocks, kv_heads, block_tokens, head_dim);
    if (rc != FP8BLK_OK) return rc;
    const int64_t row = static_cast<int64_t>(kv_heads) * head_dim;
    const int es = dtype == FP8BLK_F32 ? 4 : 2;
    if (k_stride < row || v_stride < row || k_stride * es % 16 != 0 || v_stride * es % 16 != 0) return FP8BLK_EINVAL;
    if (n_tokens > kStepMaxIndex || k_stride > kStepMaxIndex || v_stride > kStepMaxIndex) return FP8BLK_ERANGE;
    if (!step_aligned(k, 16) || !step_aligned(v, 16) || !step_aligned(slots, 8)) return FP8BLK_EALIGN;
    DeviceInfo dev;
    if (current_device_info(&dev) != cudaSuccess) return step_from_cuda(cudaErrorUnknown);
    AppendArgs a = {k, v, slots, k_codes, v_codes, k_scales, v_scales, dev.status, n_tokens, k_stride, v_stride,
                    n_blocks * block_tokens, kv_heads, head_dim, step_log2(block_tokens), 4};
    // Tokens per CTA: about one run of a prompt when there are tokens enough to fill the SMs, down to a few tokens (a
    // warp each) for a decode step.
    while (a.chunk < kAppendMaxChunk && n_tokens * kv_heads * 2 / (2 * a.chunk) >= 8 * dev.sms) a.chunk *= 2;
    const dim3 grid(static_cast<unsigned>((n_tokens + a.chunk - 1) / a.chunk), static_cast<unsigned>(kv_heads), 2);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return step_from_cuda(dtype == FP8BLK_F32
                              ? step_launch(kv_append_kernel<float>, grid, kAppendThreads, 0, s, a)
                              : step_launch(kv_append_kernel<__nv_bfloat16>, grid, kAppendThreads, 0, s, a));
}
