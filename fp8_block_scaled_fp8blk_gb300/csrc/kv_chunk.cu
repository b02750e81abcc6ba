// kv_chunk.cu -- attention of any number of new rows per request over the paged
// e4m3 cache (fp8blk_kv_attn_chunk): entry point and launch.
#include "kv_chunk.cuh"
#include "overlap.h"
#include "step.h"

#include <algorithm>

namespace fp8blk {

template <typename T, int PL, bool WIDE>
static cudaError_t launch_chunk(const ChunkArgs &a, int grid, cudaStream_t stream) {
    using Sh = ChunkShape<PL, WIDE>;
    const auto kernel = kv_chunk_kernel<T, PL, WIDE>;
    int per_sm = 0;
    cudaError_t err = kernel_occupancy(reinterpret_cast<const void *>(kernel), kChThreads, Sh::kSmem, &per_sm);
    if (err != cudaSuccess) return err;
    if (per_sm < 1) return cudaErrorInvalidConfiguration;
    err = step_launch(kernel, dim3(static_cast<unsigned>(grid)), kChThreads, Sh::kSmem, stream, a);
    if (err != cudaSuccess) return err;
    return step_launch(kv_chunk_join_kernel<T, Sh::U>, dim3(static_cast<unsigned>(grid), kChJoinCtas), 256, 0, stream,
                       a, grid);
}

}  // namespace fp8blk

using namespace fp8blk;

static bool chunk_shape_ok(int q_heads, int kv_heads, int head_dim) {
    return kv_heads >= 1 && q_heads >= kv_heads && q_heads <= 65535 && q_heads % kv_heads == 0 && head_dim >= 16 &&
           head_dim <= FP8BLK_MAX_HEAD_DIM && head_dim % 16 == 0;
}

extern "C" size_t fp8blk_kv_attn_chunk_ws_bytes(int q_heads, int kv_heads, int head_dim) {
    if (!chunk_shape_ok(q_heads, kv_heads, head_dim)) return 0;
    const size_t rows = head_dim > 128 ? ChunkShape<1, true>::U : ChunkShape<1, false>::U;  // of bf16, f32 has no more
    return kChHeaderBytes + static_cast<size_t>(kChMaxGrid) * 2 * rows * (head_dim + 2) * sizeof(float);
}

extern "C" int fp8blk_kv_attn_chunk(const void *q, int dtype, const uint8_t *k_codes, const float *k_scales, const uint8_t *v_codes,
                                    const float *v_scales, const int32_t *block_table, const int32_t *seq_lens, const int32_t *q_starts,
                                    void *out, float *lse, void *ws, size_t ws_bytes, int n_seqs, int64_t total_rows, int q_heads,
                                    int kv_heads, int head_dim, int block_tokens, int64_t n_blocks, int max_blocks, int64_t q_stride,
                                    int64_t out_stride, float sm_scale, void *stream) {
    if (!q || !block_table || !seq_lens || !q_starts || !out || (dtype != FP8BLK_F32 && dtype != FP8BLK_BF16)) return FP8BLK_EINVAL;
    if (n_seqs < 1 || total_rows < 1 || max_blocks < 1) return FP8BLK_EINVAL;
    if (n_seqs > 65536 || q_heads > 65535 || total_rows > kStepMaxIndex) return FP8BLK_ERANGE;
    if (!chunk_shape_ok(q_heads, kv_heads, head_dim)) return FP8BLK_EINVAL;
    const int rc = step_check_cache(k_codes, k_scales, v_codes, v_scales, n_blocks, kv_heads, block_tokens, head_dim);
    if (rc != FP8BLK_OK) return rc;
    const int64_t row = static_cast<int64_t>(q_heads) * head_dim;
    const int es = dtype == FP8BLK_F32 ? 4 : 2;
    if (q_stride < row || out_stride < row || q_stride * es % 16 != 0 || out_stride * es % 16 != 0) return FP8BLK_EINVAL;
    if (q_stride > kStepMaxIndex || out_stride > kStepMaxIndex) return FP8BLK_ERANGE;
    if (!step_aligned(q, 16) || !step_aligned(out, 16) || !step_aligned(block_table, 4) || !step_aligned(seq_lens, 4) ||
        !step_aligned(q_starts, 4) || (lse && !step_aligned(lse, 4)))
        return FP8BLK_EALIGN;
    if (!ws || ws_bytes < fp8blk_kv_attn_chunk_ws_bytes(q_heads, kv_heads, head_dim)) return FP8BLK_EWS;
    if (!step_aligned(ws, 16)) return FP8BLK_EALIGN;
    const bool wide = head_dim > 128;
    const int rows = wide || dtype == FP8BLK_F32 ? 128 : 256, tile = rows / 2, group = q_heads / kv_heads;
    static_assert(ChunkShape<1, false>::U == 256 && ChunkShape<1, true>::U == 128 && ChunkShape<2, false>::U == 128 &&
                      ChunkShape<2, true>::U == 128 && ChunkShape<1, false>::T == 128 && ChunkShape<2, false>::T == 64,
                  "row tiles and tiles");
    // What the kernel counts in 32 bits: rows times heads of a group, row tiles and tiles on one line, list entries.
    const int64_t tiles = (static_cast<int64_t>(max_blocks) * block_tokens + tile - 1) / tile + 1;
    const int64_t flat = total_rows * group, units = (flat + rows - 1) / rows + n_seqs;
    if (flat > kStepMaxIndex || tiles > kStepMaxIndex / 256 || tiles * group + 2 * units > kStepMaxIndex / 2) return FP8BLK_ERANGE;
    const int64_t slots = tiles + kChSetUp;
    if (units * kv_heads > kStepMaxIndex / (rows / 128) / slots) return FP8BLK_ERANGE;
    const int64_t entries = units * kv_heads * (rows / 128) * slots;
    // A row of a head is read by the units that write it, before they do (a unit in parts: before the join), so out may be q.
    if (q != out || q_stride != out_stride) {
        if (rows_overlap(q, q_stride * es, row * es, out, out_stride * es, row * es, total_rows)) return FP8BLK_EINVAL;
    }
    DeviceInfo dev;
    if (current_device_info(&dev) != cudaSuccess) return step_from_cuda(cudaErrorUnknown);
    const double c = static_cast<double>(sm_scale) * 1.4426950408889634073599246810019;
    ChunkArgs a = {};
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
    a.heads = static_cast<int4 *>(ws);
    a.partials = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + kChHeaderBytes);
    a.status = dev.status;
    a.wait_limit_ns = tuning().wait_limit_ns;
    a.q_stride = q_stride;
    a.out_stride = out_stride;
    a.n_blocks = n_blocks;
    a.n_seqs = n_seqs;
    a.total_rows = static_cast<int>(total_rows);
    a.kv_heads = kv_heads;
    a.group = group;
    a.head_dim = head_dim;
    a.block_log2 = step_log2(block_tokens);
    a.width = max_blocks;
    a.max_tiles = static_cast<int>(tiles);
    a.group_inverse = 0xFFFFFFFFu / static_cast<uint32_t>(group);
    a.c = static_cast<float>(c);
    a.c_low = static_cast<float>(c - static_cast<double>(a.c));
    const int grid = static_cast<int>(std::min<int64_t>(std::min(dev.sms, kChMaxGrid), entries));
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == FP8BLK_F32)
        return step_from_cuda(wide ? launch_chunk<float, 2, true>(a, grid, s) : launch_chunk<float, 2, false>(a, grid, s));
    return step_from_cuda(wide ? launch_chunk<__nv_bfloat16, 1, true>(a, grid, s) : launch_chunk<__nv_bfloat16, 1, false>(a, grid, s));
}
