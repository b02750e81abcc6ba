// kv_attn.cu -- attention of 1..8 new rows per request over the paged e4m3
// cache (fp8blk_kv_attn): entry point and launch.
#include "step.h"

namespace fp8blk {

struct AttnArgs {
    const void *q;
    void *out;
    float *lse;
    const uint8_t *k_codes, *v_codes;
    const float *k_scales, *v_scales;
    const int32_t *table, *seq_lens, *q_starts;
    unsigned int *status;
    int64_t q_stride, out_stride, n_blocks;
    int n_seqs, max_m, total_rows, q_heads, kv_heads, head_dim, block_log2, width;
    float scale_log2;
};

template <typename T>
__device__ __forceinline__ float attn_load(const T *p) { return static_cast<float>(*p); }

// One CTA per (row, head); each warp takes every fourth token, online softmax
// per warp, the four joined at the end.
template <typename T>
__global__ void __launch_bounds__(128) kv_attn_simple_kernel(const AttnArgs a) {
    __shared__ float s_o[4][FP8BLK_MAX_HEAD_DIM], s_m[4], s_l[4];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int s = blockIdx.x / a.max_m, i = blockIdx.x - s * a.max_m, h = blockIdx.y;
    grid_dependency_wait();
    grid_launch_dependents();
    const int first = a.q_starts[s];
    const int64_t rows64 = static_cast<int64_t>(a.q_starts[s + 1]) - first;
    const int len = max(a.seq_lens[s], 0);
    const bool bad = first < 0 || rows64 < 0 || rows64 > a.max_m || first + rows64 > a.total_rows;
    if (i == 0 && h == 0 && threadIdx.x == 0 && (bad || a.seq_lens[s] < 0)) atomicOr(a.status, FP8BLK_STATUS_BAD_KV);
    if (bad || i >= rows64) return;
    const int rows = static_cast<int>(rows64), row = first + i;
    const int last = len - rows + i;
    const int kvh = h / (a.q_heads / a.kv_heads), D = a.head_dim, block = 1 << a.block_log2;
    const T *q = static_cast<const T *>(a.q) + row * a.q_stride + static_cast<int64_t>(h) * D;
    float qv[8], o[8], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        qv[j] = lane + 32 * j < D ? attn_load(q + lane + 32 * j) * a.scale_log2 : 0.f;
        o[j] = 0.f;
    }
    for (int t = warp; t <= last; t += 4) {
        const int page = t >> a.block_log2;
        const int id = page < a.width ? a.table[static_cast<int64_t>(s) * a.width + page] : -1;
        const bool ok = id >= 0 && id < a.n_blocks;
        if (!ok && lane == 0) atomicOr(a.status, FP8BLK_STATUS_BAD_KV);
        const int64_t bh = static_cast<int64_t>(ok ? id : 0) * a.kv_heads + kvh;
        const int64_t at = (bh * block + (t & (block - 1))) * D;
        float d = 0.f, vv[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = lane + 32 * j;
            vv[j] = 0.f;
            if (c < D) {
                d = fmaf(qv[j], e4m3x2_to_f32(a.k_codes[at + c]).x, d);
                vv[j] = e4m3x2_to_f32(a.v_codes[at + c]).x;
            }
        }
#pragma unroll
        for (int x = 16; x; x >>= 1) d += __shfl_xor_sync(0xFFFFFFFFu, d, x);
        d *= ok ? a.k_scales[bh] : __int_as_float(0x7FC00000);
        const float nm = fmaxf(m, d), c = exp2f(m - nm), p = exp2f(d - nm);
        l = l * c + p;
        const float pv = p * a.v_scales[bh];
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = fmaf(o[j], c, pv * vv[j]);
        m = nm;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (lane + 32 * j < D) s_o[warp][lane + 32 * j] = o[j];
    if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
    }
    __syncthreads();
    const float mm = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
    float w[4], tl = 0.f;
    for (int i = 0; i < 4; ++i) {
        w[i] = s_m[i] == -INFINITY ? 0.f : exp2f(s_m[i] - mm);
        tl += w[i] * s_l[i];
    }
    const float inv = last >= 0 ? 1.f / tl : 0.f;
    T *out = static_cast<T *>(a.out) + row * a.out_stride + static_cast<int64_t>(h) * D;
    for (int c = threadIdx.x; c < D; c += 128) {
        float v = 0.f;
        for (int i = 0; i < 4; ++i) v += s_m[i] == -INFINITY ? 0.f : w[i] * s_o[i][c];
        out[c] = static_cast<T>(v * inv);
    }
    if (a.lse && threadIdx.x == 0)
        a.lse[static_cast<int64_t>(row) * a.q_heads + h] = last >= 0 ? (mm + log2f(tl)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace fp8blk

using namespace fp8blk;

static bool attn_shape_ok(int n_seqs, int max_m, int q_heads, int kv_heads, int head_dim) {
    return n_seqs >= 1 && n_seqs <= 65536 && max_m >= 1 && max_m <= FP8BLK_MAX_M && kv_heads >= 1 && q_heads >= kv_heads &&
           q_heads <= 65535 && q_heads % kv_heads == 0 && head_dim >= 16 && head_dim <= FP8BLK_MAX_HEAD_DIM &&
           head_dim % 16 == 0;
}

extern "C" size_t fp8blk_kv_attn_ws_bytes(int n_seqs, int max_m, int q_heads, int kv_heads, int head_dim) {
    if (!attn_shape_ok(n_seqs, max_m, q_heads, kv_heads, head_dim)) return 0;
    return 16;
}

extern "C" int fp8blk_kv_attn(const void *q, int dtype, const uint8_t *k_codes, const float *k_scales,
                              const uint8_t *v_codes, const float *v_scales, const int32_t *block_table,
                              const int32_t *seq_lens, const int32_t *q_starts, void *out, float *lse, void *ws,
                              size_t ws_bytes, int n_seqs, int max_m, int64_t total_rows, int q_heads, int kv_heads,
                              int head_dim, int block_tokens, int64_t n_blocks, int max_blocks, int64_t q_stride,
                              int64_t out_stride, float sm_scale, void *stream) {
    if (!q || !block_table || !seq_lens || !q_starts || !out || (dtype != FP8BLK_F32 && dtype != FP8BLK_BF16))
        return FP8BLK_EINVAL;
    if (total_rows < 1 || max_blocks < 1) return FP8BLK_EINVAL;
    if (n_seqs > 65536 || q_heads > 65535 || total_rows > kStepMaxIndex) return FP8BLK_ERANGE;
    if (!attn_shape_ok(n_seqs, max_m, q_heads, kv_heads, head_dim)) return FP8BLK_EINVAL;
    const int rc = step_check_cache(k_codes, k_scales, v_codes, v_scales, n_blocks, kv_heads, block_tokens, head_dim);
    if (rc != FP8BLK_OK) return rc;
    const int64_t row = static_cast<int64_t>(q_heads) * head_dim;
    const int es = dtype == FP8BLK_F32 ? 4 : 2;
    if (q_stride < row || out_stride < row || q_stride * es % 16 != 0 || out_stride * es % 16 != 0) return FP8BLK_EINVAL;
    if (q_stride > kStepMaxIndex || out_stride > kStepMaxIndex) return FP8BLK_ERANGE;
    if (!step_aligned(q, 16) || !step_aligned(out, 16) || !step_aligned(block_table, 4) || !step_aligned(seq_lens, 4) ||
        !step_aligned(q_starts, 4) || (lse && !step_aligned(lse, 4)))
        return FP8BLK_EALIGN;
    if (!ws || ws_bytes < fp8blk_kv_attn_ws_bytes(n_seqs, max_m, q_heads, kv_heads, head_dim)) return FP8BLK_EWS;
    if (!step_aligned(ws, 16)) return FP8BLK_EALIGN;
    DeviceInfo dev;
    if (current_device_info(&dev) != cudaSuccess) return step_from_cuda(cudaErrorUnknown);
    AttnArgs a = {};
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.k_codes = k_codes;
    a.v_codes = v_codes;
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.table = block_table;
    a.seq_lens = seq_lens;
    a.q_starts = q_starts;
    a.status = dev.status;
    a.q_stride = q_stride;
    a.out_stride = out_stride;
    a.n_blocks = n_blocks;
    a.n_seqs = n_seqs;
    a.max_m = max_m;
    a.total_rows = static_cast<int>(total_rows);
    a.q_heads = q_heads;
    a.kv_heads = kv_heads;
    a.head_dim = head_dim;
    a.block_log2 = step_log2(block_tokens);
    a.width = max_blocks;
    a.scale_log2 = sm_scale * 1.4426950408889634f;
    const dim3 grid(static_cast<unsigned>(n_seqs) * max_m, static_cast<unsigned>(q_heads));
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return step_from_cuda(dtype == FP8BLK_F32 ? step_launch(kv_attn_simple_kernel<float>, grid, 128, 0, s, a)
                                              : step_launch(kv_attn_simple_kernel<__nv_bfloat16>, grid, 128, 0, s, a));
}
