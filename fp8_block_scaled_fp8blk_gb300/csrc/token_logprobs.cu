// token_logprobs.cu -- log probability, rank and entropy of given tokens, with
// the top alternatives, from rows of logits (fp8blk_token_logprobs).
#include <cooperative_groups.h>

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
    int slice;  // elements per CTA of a row's cluster (a multiple of 16)
};

constexpr int kLpThreads = 512;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpGroups = 128;             // thread groups whose maxima bound the k-th largest
constexpr int kLpGroupSize = kLpThreads / kLpGroups;
constexpr int kLpMaxTop = FP8BLK_MAX_TOP;

// Order key of a logit: larger value first, -0 and +0 alike, NaN below all;
// 0 is no logit's key but NaN's.
__device__ __forceinline__ uint32_t value_key(float v) {
    if (v != v) return 0u;
    const uint32_t u = __float_as_uint(v + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
// Unique order of (value, index): the lowest index first among equal values.
__device__ __forceinline__ uint64_t full_key(float v, uint32_t index) {
    return (static_cast<uint64_t>(value_key(v)) << 32) | (0xFFFFFFFFu - index);
}

template <typename T>
__device__ __forceinline__ float logit(const T *p) { return static_cast<float>(*p); }

// What a CTA of the cluster tells the others.
struct LpShare {
    float max;
    float sum, weighted;  // sum of e, sum of e * (x - max)
    int rank;
    int n_top;
    uint64_t top[kLpMaxTop];
};

// One cluster per row, one slice of the row per CTA, held in shared memory as
// f32: the row is read from global memory once, and the maximum, the sums and
// the candidates each take a sweep of shared memory.
template <typename T>
__global__ void __launch_bounds__(kLpThreads) token_logprobs_kernel(const LogprobArgs a) {
    extern __shared__ __align__(16) float s_x[];
    __shared__ LpShare share;
    __shared__ float w_f[kLpWarps], w_g[kLpWarps];
    __shared__ int w_i[kLpWarps];
    __shared__ uint64_t s_group[kLpGroups];
    __shared__ uint64_t s_tau;
    __shared__ int s_count;
    cg::cluster_group cluster = cg::this_cluster();
    const int c = static_cast<int>(cluster.block_rank()), nc = static_cast<int>(cluster.num_blocks());
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x / nc;
    grid_dependency_wait();
    grid_launch_dependents();
    const int base = c * a.slice;
    const int count = max(0, min(a.slice, a.vocab - base));
    const T *x = static_cast<const T *>(a.logits) + row * a.stride + base;
    uint64_t *cand = reinterpret_cast<uint64_t *>(s_x + a.slice);

    // Sweep 1: the slice into shared memory, its maximum, and each thread's best key.
    float mx = -INFINITY;
    bool nan = false;
    uint64_t best = 0;
    for (int i = tid; i < count; i += kLpThreads) {
        const float v = logit(x + i);
        s_x[i] = v;
        mx = fmaxf(mx, v);
        nan |= v != v;
        if (a.top > 0) {
            const uint64_t k = full_key(v, base + i);
            best = k > best ? k : best;
        }
    }
    mx = nan ? __int_as_float(0x7FC00000) : mx;
    // Maximum over the CTA; a NaN anywhere wins.
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        const float o = __shfl_xor_sync(0xFFFFFFFFu, mx, d);
        mx = (mx != mx || o != o) ? __int_as_float(0x7FC00000) : fmaxf(mx, o);
    }
    if (lane == 0) w_f[warp] = mx;
#pragma unroll
    for (int d = 1; d < kLpGroupSize; d <<= 1) {
        const uint64_t o = __shfl_xor_sync(0xFFFFFFFFu, best, d);
        best = o > best ? o : best;
    }
    if (tid % kLpGroupSize == 0) s_group[tid / kLpGroupSize] = best;
    if (tid == 0) {
        s_count = 0;
        s_tau = 0;
    }
    __syncthreads();
    if (tid == 0) {
        float m = w_f[0];
        for (int w = 1; w < kLpWarps; ++w) m = (m != m || w_f[w] != w_f[w]) ? __int_as_float(0x7FC00000) : fmaxf(m, w_f[w]);
        share.max = m;
    }
    // tau = the k-th largest group maximum: at least k elements reach it, and
    // only elements of k groups can.
    if (a.top > 0 && tid < kLpGroups) {
        const uint64_t mine = s_group[tid];
        int above = 0;
        for (int g = 0; g < kLpGroups; ++g) above += s_group[g] > mine;
        if (above == a.top - 1) s_tau = mine;
    }
    cluster.sync();
    float m = -INFINITY;
    for (int r = 0; r < nc; ++r) {
        const float o = cluster.map_shared_rank(&share, r)->max;
        m = (m != m || o != o) ? __int_as_float(0x7FC00000) : fmaxf(m, o);
    }
    const float ref = m == -INFINITY ? 0.f : m;

    // Sweep 2: sums, rank and candidates.
    const int target = a.targets[row];
    const bool has_target = target >= 0 && target < a.vocab;
    const uint64_t tkey = has_target ? full_key(logit(static_cast<const T *>(a.logits) + row * a.stride + target), target) : ~0ull;
    const uint64_t tau = s_tau;
    float sum = 0.f, weighted = 0.f;
    int rank = 0;
    for (int i = tid; i < count; i += kLpThreads) {
        const float v = s_x[i];
        const float d = v - ref, e = __expf(d);
        sum += e;
        if (e > 0.f) weighted = fmaf(e, d, weighted);
        const uint64_t k = full_key(v, base + i);
        rank += k > tkey;
        if (a.top > 0 && k >= tau) cand[atomicAdd(&s_count, 1)] = k;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        weighted += __shfl_xor_sync(0xFFFFFFFFu, weighted, d);
        rank += __shfl_xor_sync(0xFFFFFFFFu, rank, d);
    }
    if (lane == 0) {
        w_f[warp] = sum;
        w_g[warp] = weighted;
        w_i[warp] = rank;
    }
    __syncthreads();
    if (tid == 0) {
        float fs = 0.f, gs = 0.f;
        int is = 0;
        for (int w = 0; w < kLpWarps; ++w) {
            fs += w_f[w];
            gs += w_g[w];
            is += w_i[w];
        }
        share.sum = fs;
        share.weighted = gs;
        share.rank = is;
        share.n_top = min(s_count, a.top);
    }
    // The slice's top: each candidate's place is the number of larger ones.
    if (a.top > 0) {
        const int n = s_count;
        for (int i = tid; i < n; i += kLpThreads) {
            const uint64_t k = cand[i];
            int above = 0;
            for (int j = 0; j < n; ++j) above += cand[j] > k;
            if (above < a.top) share.top[above] = k;
        }
    }
    cluster.sync();
    if (c == 0) {
        float total = 0.f, wsum = 0.f;
        int rk = 0;
        for (int r = 0; r < nc; ++r) {
            const LpShare *o = cluster.map_shared_rank(&share, r);
            total += o->sum;
            wsum += o->weighted;
            rk += o->rank;
        }
        const float logz = logf(total);
        if (tid == 0) {
            const float nanf = __int_as_float(0x7FC00000);
            if (has_target) {
                const float t = logit(static_cast<const T *>(a.logits) + row * a.stride + target);
                a.logprob[row] = m == -INFINITY ? nanf : (t - m) - logz;
                a.rank[row] = rk;
            } else {
                a.logprob[row] = nanf;
                a.rank[row] = -1;
                if (target != -1) atomicOr(a.status, FP8BLK_STATUS_BAD_TARGET);
            }
            a.entropy[row] = m == -INFINITY ? nanf : logz - wsum / total;
        }
        // Merge the slices' sorted lists: a key's place is the sum of its places.
        for (int i = tid; i < nc * a.top; i += kLpThreads) {
            const int r = i / a.top, j = i - r * a.top;
            const LpShare *o = cluster.map_shared_rank(&share, r);
            if (j >= o->n_top) continue;
            const uint64_t k = o->top[j];
            int place = j;
            for (int s = 0; s < nc && place < a.top; ++s) {
                if (s == r) continue;
                const LpShare *p = cluster.map_shared_rank(&share, s);
                for (int y = 0; y < p->n_top && p->top[y] > k; ++y) ++place;
            }
            if (place < a.top) {
                const uint32_t id = 0xFFFFFFFFu - static_cast<uint32_t>(k);
                const float t = logit(static_cast<const T *>(a.logits) + row * a.stride + id);
                a.top_ids[row * a.top + place] = static_cast<int32_t>(id);
                a.top_logprobs[row * a.top + place] = m == -INFINITY ? __int_as_float(0x7FC00000) : (t - m) - logz;
            }
        }
    }
    cluster.sync();  // the others' shared memory is read above
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
    LogprobArgs a = {logits, targets, logprob, entropy, rank, top_ids, top_logprobs, dev.status, stride,
                     static_cast<int>(vocab), top, 0};
    // Slices of at most 32768 elements; more CTAs per row while there are fewer than one per SM.
    int nc = 1;
    while (nc < 8 && ((vocab + nc - 1) / nc > 32768 || (n_rows * nc < dev.sms && vocab / nc > 4096))) nc *= 2;
    a.slice = static_cast<int>(((vocab + nc - 1) / nc + 15) / 16 * 16);
    const size_t cand = top > 0 ? static_cast<size_t>(top) * kLpGroupSize * ((a.slice + kLpThreads - 1) / kLpThreads) * 8 : 0;
    const size_t smem = static_cast<size_t>(a.slice) * 4 + cand;
    const void *kernel = dtype == FP8BLK_F32 ? reinterpret_cast<const void *>(token_logprobs_kernel<float>)
                                             : reinterpret_cast<const void *>(token_logprobs_kernel<__nv_bfloat16>);
    int per_sm = 0;
    cudaError_t err = kernel_occupancy(kernel, kLpThreads, smem, &per_sm);
    if (err != cudaSuccess || per_sm < 1) return step_from_cuda(err != cudaSuccess ? err : cudaErrorInvalidConfiguration);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(n_rows * nc));
    cfg.blockDim = dim3(kLpThreads);
    cfg.dynamicSmemBytes = smem;
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
    return step_from_cuda(dtype == FP8BLK_F32 ? cudaLaunchKernelEx(&cfg, token_logprobs_kernel<float>, a)
                                              : cudaLaunchKernelEx(&cfg, token_logprobs_kernel<__nv_bfloat16>, a));
}
