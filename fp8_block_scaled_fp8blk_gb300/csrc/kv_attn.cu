// kv_attn.cu -- attention of 1..8 new rows per request over the paged e4m3
// cache (fp8blk_kv_attn): entry point, choice of the row group, launch.
#include "kv_attn.cuh"
#include "step.h"

#include <algorithm>

namespace fp8blk {

// Rows of one MMA group: the smallest of 8, 16, 32 that holds all query rows of
// a request and cache head, as far as tensor memory and registers go; more rows
// take more groups, which read the cache again (out of L2).
static int attn_rows(int rows, int halves) {
    const int most = halves == 2 ? 16 : 32;
    int r = 8;
    while (r < rows && r < most) r *= 2;
    return r;
}

// Partial sums are sized for the largest row group of either type.
static size_t attn_ws_bytes(int rows, int head_dim) {
    const int halves = head_dim > 128 ? 2 : 1;
    const size_t r = static_cast<size_t>(attn_rows(rows, halves));
    return kAtHeaderBytes + static_cast<size_t>(kAtMaxGrid) * 2 * (r * halves * 128 + 2 * r) * sizeof(float);
}

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                 const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Tensor map of a pool of codes as [rows, head_dim]: boxes of box_rows rows x 128 codes.  Encoded anew by each call (bit
// packing on the host): nothing is kept by a pool's address.
static cudaError_t pool_map(const uint8_t *codes, int64_t rows, int head_dim, int box_rows, CUtensorMap *out) {
    static const EncodeTiled encode = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q);
        return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<EncodeTiled>(f) : nullptr;
    }();
    if (!encode) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(head_dim), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(head_dim)};
    const cuuint32_t box[2] = {128u, static_cast<cuuint32_t>(box_rows)}, steps[2] = {1u, 1u};
    const CUresult r = encode(out, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(codes), dims, strides, box, steps,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <typename T, int PL, int R, int ND>
static cudaError_t launch_attn(const AttnArgs &a, const CUtensorMap &kmap, const CUtensorMap &vmap, int64_t grid,
                               cudaStream_t stream) {
    const size_t smem = AttnShape<PL, R, ND>::kSmem;
    const auto kernel = kv_attn_kernel<T, PL, R, ND>;
    int per_sm = 0;
    cudaError_t err = kernel_occupancy(reinterpret_cast<const void *>(kernel), kAtThreads, smem, &per_sm);
    if (err != cudaSuccess) return err;
    if (per_sm < 1) return cudaErrorInvalidConfiguration;
    return step_launch(kernel, dim3(static_cast<unsigned>(grid)), kAtThreads, smem, stream, kmap, vmap, a);
}

template <typename T, int PL>
static cudaError_t launch_attn_rows(const AttnArgs &a, int rows, const CUtensorMap &kmap, const CUtensorMap &vmap,
                                    int64_t grid, cudaStream_t s) {
    if (a.head_dim > 128) {
        return rows == 8 ? launch_attn<T, PL, 8, 2>(a, kmap, vmap, grid, s) : launch_attn<T, PL, 16, 2>(a, kmap, vmap, grid, s);
    }
    switch (rows) {
        case 8: return launch_attn<T, PL, 8, 1>(a, kmap, vmap, grid, s);
        case 16: return launch_attn<T, PL, 16, 1>(a, kmap, vmap, grid, s);
        default: return launch_attn<T, PL, 32, 1>(a, kmap, vmap, grid, s);
    }
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
    return attn_ws_bytes(max_m * (q_heads / kv_heads), head_dim);
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
    const int halves = head_dim > 128 ? 2 : 1, group = q_heads / kv_heads;
    const int rows = attn_rows(max_m * group, halves);
    AttnArgs a = {};
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.table = block_table;
    a.seq_lens = seq_lens;
    a.q_starts = q_starts;
    a.counters = static_cast<uint32_t *>(ws);
    a.partials = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + kAtHeaderBytes);
    a.status = dev.status;
    a.wait_limit_ns = tuning().wait_limit_ns;
    a.q_stride = q_stride;
    a.out_stride = out_stride;
    a.n_blocks = n_blocks;
    a.n_seqs = n_seqs;
    a.max_m = max_m;
    a.total_rows = static_cast<int>(total_rows);
    a.kv_heads = kv_heads;
    a.group = group;
    a.head_dim = head_dim;
    a.block_log2 = step_log2(block_tokens);
    a.width = max_blocks;
    a.scale_log2 = sm_scale * 1.4426950408889634f;
    // The pools as [(block, head, token), head_dim]: a box is one head's tokens of one block, 128 elements wide (zeros
    // past head_dim).
    CUtensorMap kmap, vmap;
    const int64_t pool_rows = n_blocks * kv_heads * block_tokens;
    cudaError_t err = pool_map(k_codes, pool_rows, head_dim, block_tokens, &kmap);
    if (err == cudaSuccess) err = pool_map(v_codes, pool_rows, head_dim, block_tokens, &vmap);
    if (err != cudaSuccess) return step_from_cuda(err);
    // One CTA per SM, and no more than the longest possible list has entries (a unit: its set-up, its tiles, and one for a
    // length past the table).
    const int64_t tiles = std::max<int64_t>(1, (static_cast<int64_t>(max_blocks) * block_tokens + kAtTile - 1) / kAtTile);
    const int64_t entries = static_cast<int64_t>(n_seqs) * kv_heads * ((max_m * group + rows - 1) / rows) * (tiles + 2);
    if (entries > kStepMaxIndex / at_max_weight(rows)) return FP8BLK_ERANGE;  // the kernel counts them in 32 bits
    a.max_tiles = static_cast<int>(tiles + 1);
    const int64_t grid = std::min<int64_t>(std::min(dev.sms, kAtMaxGrid), entries);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return step_from_cuda(dtype == FP8BLK_F32 ? launch_attn_rows<float, 4>(a, rows, kmap, vmap, grid, s)
                                              : launch_attn_rows<__nv_bfloat16, 2>(a, rows, kmap, vmap, grid, s));
}
