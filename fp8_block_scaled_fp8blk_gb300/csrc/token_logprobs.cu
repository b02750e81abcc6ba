// token_logprobs.cu -- log probability, rank and entropy of given tokens, with
// the top alternatives, from rows of logits (fp8blk_token_logprobs).
#include <cooperative_groups.h>

#include <algorithm>

#include "step.h"

namespace cg = cooperative_groups;

namespace fp8blk {

struct LogprobArgs {
    const void *logits;      // [n, vocab], row stride in elements
    const int32_t *targets;  // [n]
    float *logprob, *entropy;
    int32_t *rank;
    int32_t *top_ids;     // [n, top]
    float *top_logprobs;  // [n, top]
    unsigned int *status;
    int64_t stride;
    int vocab, top;
    int cluster;  // CTAs of a row
    int words;    // 16-byte words of a row's slice
    int shift;    // a segment is kLpUnroll << shift words of a thread
};

constexpr int kLpWide = 512, kLpNarrow = 256;            // threads of a CTA: of several a row, of one a row
constexpr int kLpResident = 1024;                        // threads of an SM
constexpr int kLpGroups = 128;                           // thread groups whose maxima bound the k-th largest
constexpr int kLpMaxTop = FP8BLK_MAX_TOP;  // a lane's each in the last merge
constexpr int kLpCandidates = 1024;                      // room for what reaches the bound; more takes the slow selection
constexpr int kLpMaxCluster = 8;
constexpr int kLpUnrollLog2 = 2, kLpUnroll = 1 << kLpUnrollLog2;  // words of a thread in flight
constexpr int kLpSegments = 16;                          // parts of a thread's words whose maxima are kept
constexpr float kLpLog2e = 1.4426950408889634f;
constexpr float kLpFloor = -3.402823466e38f;             // reference of a thread that has seen nothing finite

// f32 values as ordered integers: -0 and +0 alike, NaN (0) below everything.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    return v != v ? 0u : ((u & 0x80000000u) ? ~u : (u | 0x80000000u));
}
constexpr uint32_t kLpKeyInf = 0x007FFFFFu;  // of -inf
// A key's value; 0's is NaN.
__device__ __forceinline__ float key_value(uint32_t k) {
    return k == 0 ? __int_as_float(0x7FC00000) : __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
// Unique order of (value, index): larger values first, the lowest index first among equal ones.
__device__ __forceinline__ uint64_t full_key(float v, uint32_t index) {
    return (static_cast<uint64_t>(order_key(v)) << 32) | (0xFFFFFFFFu - index);
}
// The next f32 above v (NaN above +inf and for NaN).
__device__ __forceinline__ float next_up(float v) {
    const int u = __float_as_int(v + 0.0f);
    return __int_as_float(u >= 0 ? u + 1 : u - 1);
}

// 16 bytes of logits as f32.
template <typename T>
struct LpVec;
template <>
struct LpVec<float> {
    static constexpr int kN = 4;
    static __device__ __forceinline__ void unpack(const uint4 &w, float (&x)[4]) {
        x[0] = __uint_as_float(w.x);
        x[1] = __uint_as_float(w.y);
        x[2] = __uint_as_float(w.z);
        x[3] = __uint_as_float(w.w);
    }
    // The largest, NaN left out (-inf or NaN if there is nothing else).
    static __device__ __forceinline__ float peak(const uint4 &w) {
        return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)), fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
    }
};
template <>
struct LpVec<__nv_bfloat16> {
    static constexpr int kN = 8;
    static __device__ __forceinline__ void unpack(const uint4 &w, float (&x)[8]) {
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = bf16x2_to_f32(v[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
    static __device__ __forceinline__ float peak(const uint4 &w) {
        const __nv_bfloat162 *p = reinterpret_cast<const __nv_bfloat162 *>(&w);
        const __nv_bfloat162 m = __hmax2(__hmax2(p[0], p[1]), __hmax2(p[2], p[3]));
        return fmaxf(__low2float(m), __high2float(m));
    }
};

// What a CTA of the cluster tells the first.
struct LpShare {
    float max;            // largest value, NaN left out
    float sum, weighted;  // of 2^y and of y 2^y, y = (x - max) log2 e; NaN if there is a NaN or +inf
    int rank;
    int n_top;
    uint64_t top[kLpMaxTop];
};

// A whole word of a row, issued where it stands.
__device__ __forceinline__ uint4 lp_load(const uint4 *p) {
    uint4 v;
    asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ float lp_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A CTA's slice of one row, as 16-byte words: word w holds the elements
// [w V - off, w V - off + V) of the row, of which the row's first and last word
// may hold fewer.  Words [w0, w1) are the slice's, [g0, g1) the whole ones.
template <typename T, int TH>
struct LpSlice {
    static constexpr int V = LpVec<T>::kN;
    const T *x;
    const uint4 *words;
    int off, w0, w1, g0, g1;
    __device__ __forceinline__ LpSlice(const LogprobArgs &a, int64_t row, int c) {
        x = static_cast<const T *>(a.logits) + row * a.stride;
        off = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
        words = reinterpret_cast<const uint4 *>(x - off);
        w0 = c * a.words;
        w1 = min(w0 + a.words, (a.vocab + off + V - 1) / V);
        g0 = off == 0 ? w0 : max(w0, 1);
        g1 = min(w1, (a.vocab + off) / V);
    }
    // Elements of word w: [first, last).
    __device__ __forceinline__ int first(int w) const { return max(0, w * V - off); }
    __device__ __forceinline__ int last(int w, int vocab) const { return min(vocab, w * V - off + V); }
    // A thread's first whole word; the row's first word, if partial, is thread 0's before that.
    __device__ __forceinline__ int start(int tid) const { return w0 + tid + (w0 + tid < g0 ? TH : 0); }
};

// One cluster per row, one slice of the row per CTA, one pass over memory:
// thread t takes the slice's 16-byte words t, t + TH, ... and keeps its own
// maximum, sum, weighted sum and rank count; what is joined, is joined at the
// end.  The sums are relative to the maximum of the words so far (four at a
// time), so the terms that matter have exponents near 0, where they are exact;
// a reference that lags by up to 20 saves a few instructions and costs 1e-6.
//   The top: the k-th largest of 128 group maxima bounds the k-th largest of the
// slice from below.  Only segments (a thread's four words, or more in a long
// row) whose own maximum reaches it hold candidates: some 20 segments are read
// again, out of L2, and the few candidates are ranked by counting.  Rows where
// too many values tie with the bound are selected one by one, a pass over the slice
// each: rows of -inf with 5 or 100 other values take 71 us instead of 7.7 (8 rows),
// 7.5 ms instead of 0.18 (2048).
//   Bound: HBM (4 or 2 bytes a logit) for many rows of f32, at about 9
// instructions a logit; instructions for bf16; the chain of joins for few rows.
// Measured, top 20 and 131072 logits: 2048 rows of f32 187 us (86% of the copy
// rate; without the top about 100%), of bf16 148 us (54%); top 5, 8 rows of f32
// 7.4 us.
// (A resident grid that asks for the next row's words before it joins a row,
// clusters of 16, and words staged by asynchronous copies, twice as many in
// flight, each measured slower.)
template <typename T, int TH>
__global__ void __launch_bounds__(TH, kLpResident / TH) token_logprobs_kernel(const LogprobArgs a) {
    constexpr int V = LpVec<T>::kN, UN = kLpUnroll, kLpWarps = TH / 32, kLpGroupSize = TH / kLpGroups;
    __shared__ LpShare s_all[kLpMaxCluster];  // of every CTA, in the cluster's first
    __shared__ uint64_t s_top[kLpMaxTop];
    __shared__ float w_max[kLpWarps], w_sum[kLpWarps], w_wgt[kLpWarps];
    __shared__ int w_rank[kLpWarps];
    __shared__ __align__(16) uint32_t s_group[kLpGroups];
    __shared__ float s_bound;
    __shared__ float s_seg[kLpSegments][TH];  // maxima of the threads' segments
    __shared__ int s_hot[TH], s_hots, s_count;
    __shared__ uint64_t s_cand[kLpCandidates], w_best[kLpWarps];
    cg::cluster_group cluster = cg::this_cluster();
    const int nc = a.cluster, c = nc > 1 ? static_cast<int>(cluster.block_rank()) : 0;
    // The first CTA's shared memory is written to below: it has to have started.
    if (nc > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t row = blockIdx.x / nc;
    const LpSlice<T, TH> r(a, row, c);
    const int w0 = r.w0, w1 = r.w1, g0 = r.g0, g1 = r.g1, off = r.off;
    const T *x = r.x;
    // The first words are on their way before the target's logit is asked for.
    uint4 next[UN];
    auto fetch = [&](int at) {
#pragma unroll
        for (int u = 0; u < UN; ++u)
            if (at + u * TH < g1) next[u] = lp_load(r.words + at + u * TH);
    };
    fetch(r.start(tid));
    const int target = a.targets[row];
    const bool has_target = target >= 0 && target < a.vocab;
    const float t = has_target ? static_cast<float>(x[target]) : __int_as_float(0x7FC00000);

    float ref = kLpFloor, top = -INFINITY, sum = 0.f, weighted = 0.f;
    int rank = 0;
    auto raise = [&](float m) {  // a new reference; m > ref
        const float d = (ref - m) * kLpLog2e, f = lp_exp2(d);
        weighted = f == 0.f ? 0.f : f * fmaf(sum, d, weighted);
        sum *= f;
        ref = m;
    };
    auto add = [&](float v) {
        const float y = (v - ref) * kLpLog2e, e = lp_exp2(y);
        sum += e;
        weighted = fmaf(e, fmaxf(y, kLpFloor), weighted);
    };
    auto word = [&](int w, const uint4 &bits, float m) {  // a whole word, its maximum m
        float v[V];
        LpVec<T>::unpack(bits, v);
#pragma unroll
        for (int i = 0; i < V; ++i) add(v[i]);
        if (m >= t) {  // some may come before the target
            const int e0 = w * V - off;
            const float bar = e0 + V <= target ? t : next_up(t);
#pragma unroll
            for (int i = 0; i < V; ++i) rank += v[i] >= bar;
            if (e0 <= target && target < e0 + V) {
#pragma unroll
                for (int i = 0; i < V; ++i) rank += e0 + i < target && v[i] == t;
            }
        }
    };
    auto element = [&](int i, float v) {  // one of a partial word
        if (v > ref) raise(v);
        top = fmaxf(top, v);
        add(v);
        rank += v > t || (v == t && i < target);
    };
    auto partial = [&](int w) {
        for (int i = r.first(w); i < r.last(w, a.vocab); ++i) element(i, static_cast<float>(x[i]));
    };
    const int w_first = r.start(tid);
    const bool leads = w0 + tid < g0 && w0 + tid < w1;                         // thread 0's: the row's first word, partial
    const bool trails = g1 < w1 && g1 >= g0 && (g1 - w0) % TH == tid;  // the row's last word, partial
    if (leads) partial(w0 + tid);
    int turn = 0;
    float most = -INFINITY;  // of the segment
    for (int w = w_first; w < g1; w += UN * TH, ++turn) {
        uint4 bits[UN];
#pragma unroll
        for (int u = 0; u < UN; ++u) bits[u] = next[u];
        fetch(w + UN * TH);
        float m[UN];
        if ((turn & ((1 << a.shift) - 1)) == 0) most = -INFINITY;
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            m[u] = w + u * TH < g1 ? LpVec<T>::peak(bits[u]) : -INFINITY;
            most = fmaxf(most, m[u]);
        }
        if (most > ref) raise(most);
        top = fmaxf(top, most);
        s_seg[turn >> a.shift][tid] = most;
#pragma unroll
        for (int u = 0; u < UN; ++u)
            if (w + u * TH < g1) word(w + u * TH, bits[u], m[u]);
    }
    if (trails) partial(g1);
    if (has_target && t != t) {  // a NaN target: every number comes before it, and the NaNs of lower index
        rank = 0;
        for (int w = w0 + tid; w < w1; w += TH)
            for (int i = r.first(w); i < r.last(w, a.vocab); ++i) {
                const float v = static_cast<float>(x[i]);
                rank += v == v || i < target;
            }
    }

    // ---- the slice's maximum and the bound on its k-th largest
    float m = top;
#pragma unroll
    for (int d = 1; d < kLpGroupSize; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    // The groups' maxima as keys that no two share: the last 7 bits give way to the group's number.
    const uint32_t mine = (order_key(m) & ~(kLpGroups - 1u)) | (tid / kLpGroupSize);
    if ((tid & (kLpGroupSize - 1)) == 0) s_group[tid / kLpGroupSize] = mine;
#pragma unroll
    for (int d = kLpGroupSize; d < 32; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    if (lane == 0) w_max[warp] = m;
    if (tid == 0) {
        s_hots = 0;
        s_count = 0;
    }
    __syncthreads();
    m = w_max[lane & (kLpWarps - 1)];
#pragma unroll
    for (int d = 1; d < kLpWarps; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    const float slice_max = m, base = fmaxf(m, kLpFloor);
    if (a.top > 0) {  // a group's four lanes count the keys above its own
        int above = 0;
#pragma unroll
        for (int g = 0; g < kLpGroups / 4 / kLpGroupSize; ++g) {
            const uint4 o = *reinterpret_cast<const uint4 *>(s_group + (g * kLpGroupSize + (tid & (kLpGroupSize - 1))) * 4);
            above += (o.x > mine) + (o.y > mine) + (o.z > mine) + (o.w > mine);
        }
#pragma unroll
        for (int d = 1; d < kLpGroupSize; d <<= 1) above += __shfl_xor_sync(0xFFFFFFFFu, above, d);
        // Not above the k-th largest group maximum, by the bits left out.
        if (above == a.top - 1) s_bound = key_value(max(mine & ~(kLpGroups - 1u), kLpKeyInf));
    }
    // ---- the slice's sums, at its own maximum
    {
        const float d = (ref - base) * kLpLog2e, f = lp_exp2(d);
        float ws = f == 0.f && sum == sum ? 0.f : f * fmaf(sum, d, weighted), ss = sum * f;
        int rr = rank;
#pragma unroll
        for (int k = 16; k; k >>= 1) {
            ss += __shfl_xor_sync(0xFFFFFFFFu, ss, k);
            ws += __shfl_xor_sync(0xFFFFFFFFu, ws, k);
            rr += __shfl_xor_sync(0xFFFFFFFFu, rr, k);
        }
        if (lane == 0) {
            w_sum[warp] = ss;
            w_wgt[warp] = ws;
            w_rank[warp] = rr;
        }
    }
    __syncthreads();
    if (warp == 0) {
        float ss = lane < kLpWarps ? w_sum[lane] : 0.f, ws = lane < kLpWarps ? w_wgt[lane] : 0.f;
        int rr = lane < kLpWarps ? w_rank[lane] : 0;
#pragma unroll
        for (int k = kLpWarps / 2; k; k >>= 1) {
            ss += __shfl_xor_sync(0xFFFFFFFFu, ss, k);
            ws += __shfl_xor_sync(0xFFFFFFFFu, ws, k);
            rr += __shfl_xor_sync(0xFFFFFFFFu, rr, k);
        }
        __syncwarp();
        if (lane == 0) {
            w_sum[0] = ss;
            w_wgt[0] = ws;
            w_rank[0] = rr;
        }
    }

    // ---- the slice's top: candidates out of the hot threads' words, ranked by counting
    const int elements = max(0, min(a.vocab, w1 * V - off) - max(0, w0 * V - off));
    const int want = min(a.top, elements);
    if (want > 0) {
        const float bound = s_bound;
        auto consider = [&](float v, int i) {
            if (v < bound || (v != v && bound != -INFINITY)) return;
            const int at = atomicAdd(&s_count, 1);
            if (at < kLpCandidates) s_cand[at] = full_key(v, i);
        };
        auto consider_word = [&](int w) {
            if (w >= g0 && w < g1) {
                float v[V];
                LpVec<T>::unpack(lp_load(r.words + w), v);
#pragma unroll
                for (int i = 0; i < V; ++i) consider(v[i], w * V - off + i);
            } else {
                for (int i = r.first(w); i < r.last(w, a.vocab); ++i) consider(static_cast<float>(x[i]), i);
            }
        };
        const int lg = kLpUnrollLog2 + a.shift, span = 1 << lg;  // words of a segment
        const bool hot = !(top < bound);
        if (hot)
            for (int g = 0; w_first + g * span * TH < g1; ++g)
                if (!(s_seg[g][tid] < bound)) {
                    const int at = atomicAdd(&s_hots, 1);
                    if (at < TH) s_hot[at] = g * TH + tid;
                }
        if (leads && hot) consider_word(w0 + tid);
        if (trails && hot) consider_word(g1);
        __syncthreads();
        const int hots = s_hots;
        if (hots <= TH) {  // their words, all at once
            for (int i = tid; i < hots * span; i += TH) {
                const int h = s_hot[i >> lg], w = r.start(h & (TH - 1)) + ((h / TH << lg) + (i & (span - 1))) * TH;
                if (w < g1) consider_word(w);
            }
        } else {
            for (int w = w_first; w < g1; w += TH) consider_word(w);
        }
        __syncthreads();
        const int n = s_count;
        if (n <= kLpCandidates) {
            constexpr int kShare = 16;  // threads of a candidate
            for (int i = tid / kShare; i - tid / kShare < n; i += TH / kShare) {
                const uint64_t k = i < n ? s_cand[i] : 0;
                int above = 0;
                for (int j = tid % kShare; j < n; j += kShare) above += s_cand[j] > k;
#pragma unroll
                for (int d = 1; d < kShare; d <<= 1) above += __shfl_xor_sync(0xFFFFFFFFu, above, d);
                if (i < n && above < want) s_top[above] = k;
            }
        } else {  // too many at the bound: the next largest key, `want` times
            uint64_t last = ~0ull;
            for (int k = 0; k < want; ++k) {
                uint64_t best = 0;
                for (int w = w0 + tid; w < w1; w += TH)
                    for (int i = r.first(w); i < r.last(w, a.vocab); ++i) {
                        const uint64_t key = full_key(static_cast<float>(x[i]), i);
                        if (key < last && key > best) best = key;
                    }
#pragma unroll
                for (int d = 16; d; d >>= 1) {
                    const uint64_t o = __shfl_xor_sync(0xFFFFFFFFu, best, d);
                    best = o > best ? o : best;
                }
                if (lane == 0) w_best[warp] = best;
                __syncthreads();
                for (int w = 0; w < kLpWarps; ++w) best = w_best[w] > best ? w_best[w] : best;
                last = best;
                if (tid == 0) s_top[k] = best;
                __syncthreads();
            }
        }
    }
    __syncthreads();

    // ---- into the first CTA's shared memory (no CTA waits for it but the first), and the row
    {
        if (nc > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        LpShare *to = nc > 1 ? cluster.map_shared_rank(&s_all[c], 0) : &s_all[0];
        if (tid < want) to->top[tid] = s_top[tid];
        if (tid == 0) {
            to->max = slice_max;
            to->sum = w_sum[0];
            to->weighted = w_wgt[0];
            to->rank = w_rank[0];
            to->n_top = want;
        }
        if (nc > 1) {
            asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
            if (c != 0) return;
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        } else {
            __syncthreads();
        }
    }
    {
        // Lane q of every eight has slice q.
        const int q = lane & (kLpMaxCluster - 1);
        const LpShare &o = s_all[q < nc ? q : 0];
        float peak = o.max;
#pragma unroll
        for (int d = 1; d < kLpMaxCluster; d <<= 1) peak = fmaxf(peak, __shfl_xor_sync(0xFFFFFFFFu, peak, d));
        const float ground = fmaxf(peak, kLpFloor);
        float total = 0.f, wsum = 0.f;
        int before = 0;
        if (q < nc) {
            const float d = (fmaxf(o.max, kLpFloor) - ground) * kLpLog2e, f = lp_exp2(d), s = o.sum;
            total = s * f;
            if (f != 0.f || s != s) wsum = f * fmaf(s, d, o.weighted);
            before = o.rank;
        }
#pragma unroll
        for (int d = 1; d < kLpMaxCluster; d <<= 1) {
            total += __shfl_xor_sync(0xFFFFFFFFu, total, d);
            wsum += __shfl_xor_sync(0xFFFFFFFFu, wsum, d);
            before += __shfl_xor_sync(0xFFFFFFFFu, before, d);
        }
        const float nanf = __int_as_float(0x7FC00000);
        const float logz = peak == -INFINITY ? nanf : logf(total);
        if (tid == 0) {
            a.logprob[row] = has_target ? (t - ground) - logz : nanf;
            a.rank[row] = has_target ? before : -1;
            a.entropy[row] = logz - wsum / total * 0.6931471805599453f;
            if (!has_target && target != -1) atomicOr(a.status, FP8BLK_STATUS_BAD_TARGET);
        }
        // Merge the slices' sorted lists: a key's place is the sum of its places in all.
        if (warp < nc && lane < s_all[warp].n_top) {
            const uint64_t k = s_all[warp].top[lane];
            int place[kLpMaxCluster], room[kLpMaxCluster];
#pragma unroll
            for (int y = 0; y < kLpMaxCluster; ++y) {
                place[y] = y == warp ? lane : 0;
                room[y] = y < nc && y != warp ? s_all[y].n_top : 0;
            }
            for (int step = kLpMaxTop; step; step >>= 1) {
#pragma unroll
                for (int y = 0; y < kLpMaxCluster; ++y) {
                    const int to = place[y] + step;
                    if (to <= room[y] && s_all[y].top[to - 1] > k) place[y] = to;
                }
            }
            int at = 0;
#pragma unroll
            for (int y = 0; y < kLpMaxCluster; ++y) at += place[y];
            if (at < a.top) {
                const uint32_t id = 0xFFFFFFFFu - static_cast<uint32_t>(k);
                a.top_ids[row * a.top + at] = static_cast<int32_t>(id);
                a.top_logprobs[row * a.top + at] = (key_value(static_cast<uint32_t>(k >> 32)) - ground) - logz;
            }
        }
    }
}

}  // namespace fp8blk

using namespace fp8blk;

extern "C" int fp8blk_token_logprobs(const void *logits, int dtype, const int32_t *targets, float *logprob, int32_t *rank,
                                     float *entropy, int32_t *top_ids, float *top_logprobs, int64_t n_rows, int64_t vocab,
                                     int64_t stride, int top, void *stream) {
    if (!logits || !targets || !logprob || !rank || !entropy || (dtype != FP8BLK_F32 && dtype != FP8BLK_BF16))
        return FP8BLK_EINVAL;
    if (n_rows < 1 || vocab < 1 || stride < vocab || top < 0 || top > FP8BLK_MAX_TOP || top > vocab) return FP8BLK_EINVAL;
    if (top > 0 && (!top_ids || !top_logprobs)) return FP8BLK_EINVAL;
    const int es = dtype == FP8BLK_F32 ? 4 : 2;
    if (n_rows > kStepMaxIndex / 16 || vocab > FP8BLK_MAX_VOCAB || stride > kStepMaxIndex) return FP8BLK_ERANGE;
    if (!step_aligned(logits, es) || !step_aligned(targets, 4) || !step_aligned(logprob, 4) || !step_aligned(rank, 4) ||
        !step_aligned(entropy, 4) || (top > 0 && (!step_aligned(top_ids, 4) || !step_aligned(top_logprobs, 4))))
        return FP8BLK_EALIGN;
    DeviceInfo dev;
    if (current_device_info(&dev) != cudaSuccess) return step_from_cuda(cudaErrorUnknown);
    // From three rows per SM on, a narrow CTA per row, four of them resident: they take turns at the end of a row, when
    // nothing streams (4000 x 32000 f32: 112 us, with wide CTAs 139; 2048 x 131072: 4% less).  With fewer rows, wide
    // CTAs and as many a row as fit at once, with slices of 8 KiB at least (380 x 131072 f32: 46 us, narrow 55).
    const int64_t bytes = vocab * es, slots = kLpResident / kLpWide * static_cast<int64_t>(dev.sms);
    const bool narrow = n_rows >= 3 * static_cast<int64_t>(dev.sms);
    const int threads = narrow ? kLpNarrow : kLpWide;
    const int nc = static_cast<int>(std::max<int64_t>(std::min<int64_t>({slots / n_rows, kLpMaxCluster, bytes / 8192}), 1));
    const int64_t words = (bytes + 15) / 16 + 1;  // a row that starts inside a word reaches into one more
    LogprobArgs a = {logits, targets, logprob, entropy, rank, top_ids, top_logprobs, dev.status, stride,
                     static_cast<int>(vocab), top, nc, static_cast<int>((words + nc - 1) / nc), 0};
    const int64_t whole = std::min<int64_t>(a.words, bytes / 16);  // words of a slice, at most
    while (static_cast<int64_t>(kLpSegments << a.shift) * kLpUnroll * threads < whole) ++a.shift;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(n_rows * nc));
    cfg.blockDim = dim3(threads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(nc);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = tuning().use_pdl ? 2 : 1;
    auto kernel = dtype == FP8BLK_F32
                      ? (narrow ? token_logprobs_kernel<float, kLpNarrow> : token_logprobs_kernel<float, kLpWide>)
                      : (narrow ? token_logprobs_kernel<__nv_bfloat16, kLpNarrow> : token_logprobs_kernel<__nv_bfloat16, kLpWide>);
    return step_from_cuda(cudaLaunchKernelEx(&cfg, kernel, a));
}
