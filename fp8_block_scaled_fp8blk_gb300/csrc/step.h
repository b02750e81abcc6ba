// step.h -- host-side pieces shared by the entry points of the cache,
// attention and scoring calls (kv_cache.cu, kv_attn.cu, token_logprobs.cu).
#pragma once

#include "fp8blk.h"
#include "launch.h"

namespace fp8blk {

constexpr int64_t kStepMaxIndex = (int64_t(1) << 31) - 1;

inline bool step_aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int step_from_cuda(cudaError_t e) {
    if (e == cudaSuccess) return FP8BLK_OK;
    (void)cudaGetLastError();  // do not leave a non-sticky launch error behind
    return FP8BLK_ECUDA;
}

// Tokens per block: a power of two from 16 to 128.
inline bool step_block_ok(int b) { return b == 16 || b == 32 || b == 64 || b == 128; }

inline int step_log2(int v) {
    int l = 0;
    while ((1 << l) < v) ++l;
    return l;
}

// Common checks of a paged cache: both pools, their scales and their shape.
inline int step_check_cache(const uint8_t *k_codes, const float *k_scales, const uint8_t *v_codes, const float *v_scales,
                            int64_t n_blocks, int kv_heads, int block_tokens, int head_dim) {
    if (!k_codes || !k_scales || !v_codes || !v_scales) return FP8BLK_EINVAL;
    if (n_blocks < 1 || kv_heads < 1 || !step_block_ok(block_tokens)) return FP8BLK_EINVAL;
    if (head_dim < 16 || head_dim > FP8BLK_MAX_HEAD_DIM || head_dim % 16 != 0) return FP8BLK_EINVAL;
    // Rows of a pool ((block, head, token) triples) are TMA coordinates: 31 bits.
    if (n_blocks > kStepMaxIndex || kv_heads > 65535 || n_blocks * kv_heads > kStepMaxIndex / block_tokens)
        return FP8BLK_ERANGE;
    if (!step_aligned(k_codes, 16) || !step_aligned(v_codes, 16) || !step_aligned(k_scales, 4) || !step_aligned(v_scales, 4))
        return FP8BLK_EALIGN;
    return FP8BLK_OK;
}

// Launch with programmatic dependent launch: every kernel of these files
// waits on the grid dependency before it touches global memory.
template <typename Kernel, typename... Args>
cudaError_t step_launch(Kernel kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream, const Args &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = tuning().use_pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace fp8blk
