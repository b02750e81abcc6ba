/*
 * fp8blk.h -- C ABI of libfp8blk: the GB300 (sm_103a) FP8 block-scaled decode
 * GEMV, its fused greedy argmax, and the NVFP4 routed-expert dequant + GEMV.
 *
 * Conventions for every entry point
 *   - Plain C types only.  `stream` is a cudaStream_t passed as void*
 *     (NULL = the legacy default stream).
 *   - Device pointers are CUDA device (or managed) memory owned by the caller.
 *     The library allocates nothing, frees nothing and never synchronizes:
 *     every GPU entry point only enqueues kernels on `stream` and returns.
 *     Buffers must stay alive until that work has run.
 *   - Arguments are checked on the host before anything is enqueued; on any
 *     error nothing is launched and the return value says why.
 *   - Matrices are row-major and dense (row stride = number of columns).
 *   - Integer sizes are int64_t; the product rows * cols may exceed 2^31.
 *   - Launch contract for e4m3 weight codes (fp8blk_gemv, fp8blk_gemv_argmax,
 *     fp8blk_gemv_argmax_noalloc): kernels are launched with programmatic
 *     dependent launch and start copying the weight codes as soon as they are
 *     resident, which can be before the kernel launched just before them on
 *     the same stream has finished; x, scales and outputs are touched only
 *     after that kernel has completed.  So the codes must not be written by
 *     that immediately preceding kernel (nor by a kernel it lets run
 *     concurrently by triggering its dependents before waiting on its own
 *     predecessors; the library's kernels never do).  Codes written by a copy,
 *     a memset, or any earlier kernel are safe -- weights loaded once at start
 *     up, as the pages' engine keeps them ("Module dsv4_gpu" page, struct
 *     Fp8Dense), always are.  fp8blk_set_launch_tuning(.., use_pdl = 0, ..)
 *     turns the early start off.  bf16 and FP4 weights are read only after
 *     the preceding kernel has completed (the bf16 GEMV's weights can be the
 *     dequant kernel's output).
 *
 * Return codes (int): FP8BLK_OK on success, otherwise one of the codes below;
 * fp8blk_strerror() names them.
 */
#ifndef FP8BLK_H
#define FP8BLK_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define FP8BLK_OK 0
#define FP8BLK_EINVAL 1  /* null pointer, size <= 0, m outside [1, 8], column count not a
                            multiple of the format's granule, bad or repeated expert id */
#define FP8BLK_EALIGN 2  /* a pointer is not aligned as documented */
#define FP8BLK_ESCALE 3  /* e8m0 code 0xFF, or an NVFP4 global scale that is not a finite
                            nonzero power of two (the bf16 dequant would not be exact) */
#define FP8BLK_EWS 4     /* workspace missing or smaller than the *_ws_bytes() answer */
#define FP8BLK_ECUDA 5   /* the CUDA runtime refused a launch or attribute call */
#define FP8BLK_ERANGE 6  /* a size is beyond what the kernels index (rows >= 2^31, ...) */

#define FP8BLK_MAX_M 8      /* activation rows per call: 1 (decode) .. 8 (batched verify) */
#define FP8BLK_BLOCK 128    /* side of a square scale block */
#define FP8BLK_MAX_HEAD_DIM 256  /* widest attention head of the paged cache */
#define FP8BLK_MAX_TOP 32        /* most alternatives per row of fp8blk_token_logprobs */
#define FP8BLK_MAX_VOCAB 262144  /* most logits per row of fp8blk_token_logprobs */

/* Element types of activations and logits (the `dtype` arguments). */
#define FP8BLK_F32 0
#define FP8BLK_BF16 1

/* Bits of the device status word (see fp8blk_device_status). */
#define FP8BLK_STATUS_WAIT_TIMEOUT 1u /* a kernel gave up waiting for a weight tile (bounded
                                         wait, about one second); its outputs are invalid */
#define FP8BLK_STATUS_BAD_EXPERT 2u   /* an expert GEMV met a device-side expert id outside
                                         [0, n_experts) or a global scale that is not a power
                                         of two in [2^-100, 2^100]; that slot's outputs are NaN */
#define FP8BLK_STATUS_BAD_KV 4u          /* a cache call met a negative or too long length, a block id or
                                            slot outside the pool, or row starts outside the rows */
#define FP8BLK_STATUS_KV_EXHAUSTED 8u    /* fp8blk_kv_map ran out of free blocks */
#define FP8BLK_STATUS_BAD_TARGET 16u     /* fp8blk_token_logprobs met a target outside [-1, vocab) */

/* Version of this ABI; bumped on any incompatible change. */
int fp8blk_abi_version(void);

/* Human-readable name of a return code (static storage). */
const char *fp8blk_strerror(int code);

/*
 * fp8blk_scales_from_e8m0 -- HOST function: decode an e8m0 block-scale grid
 * to f32, out[k] = 2^(codes[k] - 127).  Source: "Module dsv4_gpu" page,
 * struct Fp8Dense (the 128x128 block-scale grid is decoded to f32 on the host;
 * every e8m0 code is a power of two; 0xFF is refused at load).
 *   codes      host, n bytes
 *   out        host, n floats (code 0 decodes to the f32 subnormal 2^-127)
 *   bad_index  host, optional: on FP8BLK_ESCALE receives the first 0xFF index
 * Returns FP8BLK_ESCALE on any 0xFF code (out is then unspecified), EINVAL on
 * null codes/out with n > 0.
 */
int fp8blk_scales_from_e8m0(const uint8_t *codes, size_t n, float *out, size_t *bad_index);

/*
 * fp8blk_gemv -- y[i][r] = sum_c e4m3(W[r][c]) * S[r/128][c/128] * x[i][c]
 * for i < m, r < rows.  Source: "Module dsv4_gpu" page, struct Fp8Dense (the
 * device GEMV decodes e4m3(code) * scale in-register) and "Struct Dsv4Gpu"
 * page, field dense_fp8 (decode and verify read the FP8-blk linears as stored)
 * and method verify_batch_dev (m = T = k+1 verify rows).
 *   w_codes  device, uint8 e4m3 codes [rows, cols], 16-byte aligned.  NaN codes
 *            (0x7F, 0xFF) are not refused; they make the affected outputs NaN.
 *   scales   device, f32 grid [ceil(rows/128), ceil(cols/128)], 4-byte aligned
 *            (normally the output of fp8blk_scales_from_e8m0).
 *   x        device, f32 activations [m, cols], 16-byte aligned; used as f32.
 *   y        device, f32 outputs [m, rows], 4-byte aligned; fully overwritten.
 *            Must not overlap any input.
 *   m        1..8;  rows >= 1;  cols >= 16 and a multiple of 16.
 * Accumulation is f32 in a fixed order (results are deterministic run to
 * run); each product is formed as e4m3 * (x * S), exact unless x * S leaves
 * the f32 range.  Error bound versus the exact sum: |err| <= 1e-5 * sum|w x|
 * + 1e-6 per output.
 * Errors: EINVAL, EALIGN, ERANGE (rows or cols >= 2^31), ECUDA.
 */
int fp8blk_gemv(const uint8_t *w_codes, const float *scales, const float *x, float *y, int m,
                int64_t rows, int64_t cols, void *stream);

/*
 * fp8blk_gemv_argmax_ws_bytes -- workspace size (bytes) that
 * fp8blk_gemv_argmax needs for this shape.  Returns 0 for invalid shapes.
 */
size_t fp8blk_gemv_argmax_ws_bytes(int m, int64_t rows, int64_t cols);

/*
 * fp8blk_gemv_argmax -- the same GEMV fused with a greedy argmax per
 * activation row: tokens[i] = min{ r : y[i][r] = max_r' y[i][r'] }.
 * Source: "Struct Dsv4Gpu" page, method decode_step_greedy (the argmax runs on
 * the device and only 4 bytes cross back) and method verify_batch_dev (a
 * per-position argmax [T]); "dflash.rs source" page, fn dflash2_walk_greedy
 * (ascending scan with a strict '>': the lowest index wins ties).
 * NaN never wins; -0 and +0 tie; a row with nothing above -inf gives token 0.
 * The token is the argmax of the f32 logits this call computes (the same
 * values written to `logits` when it is given).
 *   logits   device, optional (NULL = not written): f32 [m, rows], 4-aligned
 *   tokens   device, uint32 [m], 4-byte aligned; the caller copies it back
 *   ws       device workspace of at least fp8blk_gemv_argmax_ws_bytes(m, rows,
 *            cols) bytes, 16-byte aligned.  It must be zero-filled once
 *            before its first use; every call leaves it ready for the next.
 *            Calls that share a workspace must be ordered (same stream).
 *   others   as fp8blk_gemv.
 * Errors: as fp8blk_gemv, plus EWS.
 */
int fp8blk_gemv_argmax(const uint8_t *w_codes, const float *scales, const float *x,
                       float *logits, uint32_t *tokens, void *ws, size_t ws_bytes, int m,
                       int64_t rows, int64_t cols, void *stream);

/*
 * fp8blk_gemv_argmax_noalloc -- fp8blk_gemv_argmax for callers that cannot
 * allocate device memory.  No counterpart in the paper: the pages' engine
 * preallocates its own arenas.  This entry point serves callers that cannot
 * hand the library a workspace: code running while a CUDA graph is being
 * captured (no cudaMalloc then), serving loops that must not call
 * cudaMalloc/cudaFree because those synchronize the device, and plain C hosts
 * or plugins that own no allocator.  It computes exactly what
 * fp8blk_gemv_argmax computes, with the workspace placed in a fixed array of
 * fp8blk_noalloc_scratch_bytes() bytes (64.25 KiB) in the library's own device
 * memory; every GPU that loads the library holds that array until the process
 * exits.  It allocates nothing, and calls no cudaMalloc or cudaFree.
 *   Arguments as fp8blk_gemv_argmax, without ws / ws_bytes.
 *   Size limit: the workspace fp8blk_gemv_argmax_ws_bytes(m, rows, cols) must
 *   fit in the array -- any m <= 8 with cols <= 4096; wider rows only for
 *   tiny rows x m.  Larger shapes return FP8BLK_ERANGE.
 *   Set-up: the first call on each device looks up the array's device address
 *   (cudaGetSymbolAddress) with that device current; make that first call
 *   before any stream capture.
 *   Sharing: every call uses the same array, which keeps the last call's
 *   contents; each call clears the part that must start at zero with a
 *   stream-ordered memset.  Calls whose GPU work overlaps (different streams,
 *   or different host threads) race on the array: serialize them.
 * Errors: as fp8blk_gemv_argmax, with ERANGE in place of EWS.
 */
int fp8blk_gemv_argmax_noalloc(const uint8_t *w_codes, const float *scales, const float *x,
                               float *logits, uint32_t *tokens, int m, int64_t rows, int64_t cols,
                               void *stream);

/* Size in bytes of the fixed device array fp8blk_gemv_argmax_noalloc uses. */
size_t fp8blk_noalloc_scratch_bytes(void);

/*
 * fp8blk_bf16_gemv -- y[i][r] = sum_c bf16(B[r][c]) * x[i][c], f32
 * accumulation.  The GEMV that follows the per-expert dequant.  Source:
 * "Module dsv4_gpu" page, module header (bf16 GEMMs with f32 accumulation)
 * and enum ExpertArm (Bf16Dequant).  x stays f32.
 *   w_bf16   device, bf16 bit patterns [rows, cols], 16-byte aligned
 *   x, y, m  as fp8blk_gemv;  cols >= 16 and a multiple of 16.
 * Errors: EINVAL, EALIGN, ERANGE, ECUDA.
 */
int fp8blk_bf16_gemv(const uint16_t *w_bf16, const float *x, float *y, int m, int64_t rows,
                     int64_t cols, void *stream);

/*
 * nvfp4_expert_dequant -- dequantise one NVFP4 expert to bf16:
 *   out[r][c] = bf16( e2m1(q[r][c]) * e4m3(s[r][c/16]) * g[e] ),
 * exact in bf16 (the host refuses global scales for which it would not be).
 * Source: "Module dsv4_gpu" page, module header and enum ExpertArm (routed
 * experts stay NVFP4 as stored and each activated expert is dequantised into a
 * reused bf16 scratch, exact in bf16) and enum ExpertKind (trunk = NVFP4).
 *   codes        device, uint8 [n_experts, rows, cols/2], two e2m1 codes per
 *                byte, column 2j in the LOW nibble; 16-byte aligned
 *   scales       device, uint8 e4m3 [n_experts, rows, cols/16], 2-byte aligned
 *   gscale_host  HOST, f32 [n_experts]: per-expert global scale, each a finite
 *                nonzero power of two (else ESCALE)
 *   expert_id    0 <= expert_id < n_experts
 *   out          device, uint16 bf16 bits [rows, cols], 16-byte aligned
 *   cols         a multiple of 32.
 * Errors: EINVAL, EALIGN, ESCALE, ERANGE, ECUDA.
 */
int nvfp4_expert_dequant(const uint8_t *codes, const uint8_t *scales, const float *gscale_host,
                         int n_experts, int expert_id, uint16_t *out, int64_t rows, int64_t cols,
                         void *stream);

/*
 * nvfp4_expert_dequant_gemv -- for k < n_active: dequantise expert
 * ids_host[k] into the reused bf16 scratch, then y[k] = scratch x.
 * Same sources as nvfp4_expert_dequant.  The scratch is reused in stream
 * order; when the call's work has run it holds the LAST active expert.
 *   ids_host     HOST, int32 [n_active], distinct, each in [0, n_experts)
 *   n_active     >= 1
 *   x            device, f32 [cols], 16-byte aligned
 *   y            device, f32 [n_active, rows], 4-byte aligned
 *   bf16_scratch device, uint16 [rows, cols], 16-byte aligned
 *   others       as nvfp4_expert_dequant.
 * Errors: as nvfp4_expert_dequant.
 */
int nvfp4_expert_dequant_gemv(const uint8_t *codes, const uint8_t *scales,
                              const float *gscale_host, int n_experts, const int32_t *ids_host,
                              int n_active, const float *x, float *y, uint16_t *bf16_scratch,
                              int64_t rows, int64_t cols, void *stream);

/*
 * nvfp4_expert_gemv -- y[k] = W(ids[k]) x for k < n_active in ONE launch,
 * with no bf16 scratch:
 *   y[k][r] = sum_c bf16(e2m1(q[e][r][c]) * e4m3(s[e][r][c/16]) * g[e]) * x[c],
 *   e = ids[k]; every product is exact, so the weights take the same values
 *   as nvfp4_expert_dequant writes; the sum is in f32.  Two kernels
 *   (fp8blk_set_fp4_kernel; by shape, the tensor cores from 12288 active rows
 *   on): the CUDA cores decode the weights in registers; the tensor cores take
 *   the codes as stored, x as five e4m3 planes per 16-column block (2^-20 of
 *   each element), and apply the block scales to the f32 block sums.  Both
 *   meet the GEMV error bound and are bit-identical run to run.
 * Source: "Module dsv4_gpu" page, module header (routed experts stay NVFP4 as
 * stored; one-launch-per-projection indirect expert dispatch) and enum
 * ExpertArm.  The router's output stays on the device: ids and global scales
 * are read by the kernel, so the host checks neither.
 *   codes, scales as nvfp4_expert_dequant, but scales 16-byte aligned
 *   gscale       DEVICE, f32 [n_experts], 4-byte aligned: per-expert global
 *                scale, a power of two in [2^-100, 2^100]
 *   ids          DEVICE, int32 [n_active], 4-byte aligned; repeats allowed
 *   n_active     1 .. 65536
 *   x            device, f32 [cols], 16-byte aligned
 *   y            device, f32 [n_active, rows], 4-byte aligned
 *   cols         a multiple of 256 (so every scale row starts on 16 bytes).
 * An id outside [0, n_experts) or an unusable global scale sets
 * FP8BLK_STATUS_BAD_EXPERT in the device status word and makes y[k] NaN.
 * An inf or NaN in x: the CUDA cores give the IEEE result, the tensor cores
 * NaN in every output.
 * Errors: EINVAL, EALIGN, ERANGE, ECUDA.
 */
int nvfp4_expert_gemv(const uint8_t *codes, const uint8_t *scales, const float *gscale, int n_experts,
                      const int32_t *ids, int n_active, const float *x, float *y, int64_t rows, int64_t cols,
                      void *stream);

/*
 * mxfp4_expert_gemv -- as nvfp4_expert_gemv, for OCP MXFP4 experts (the MTP
 * block's routed experts, "Module dsv4_gpu" page, enum ExpertKind):
 *   y[k][r] = sum_c e2m1(q[e][r][c]) * 2^(s[e][r][c/32] - 127) * x[c], e = ids[k].
 * Same two kernels and routing as nvfp4_expert_gemv (fp8blk_set_fp4_kernel);
 * on the tensor cores x is split into five e4m3 planes per 32-column block and
 * each 32-column block sum is scaled by its e8m0 factor.
 * The page names the format only; the layout is read from the OCP MX format:
 *   codes        device, uint8 [n_experts, rows, cols/2], two e2m1 codes per
 *                byte, column 2j in the LOW nibble; 16-byte aligned
 *   scales       device, uint8 e8m0 [n_experts, rows, cols/32], 16-byte
 *                aligned; code 0xFF is the MX NaN (its block's weights are NaN)
 *   ids          DEVICE, int32 [n_active]; repeats allowed
 *   cols         a multiple of 512 (so every scale row starts on 16 bytes).
 * No global scale.  An id outside [0, n_experts) sets
 * FP8BLK_STATUS_BAD_EXPERT and makes y[k] NaN.  An inf or NaN in x: the
 * CUDA cores give the IEEE result, the tensor cores NaN in every output.
 * Errors: EINVAL, EALIGN, ERANGE, ECUDA.
 */
int mxfp4_expert_gemv(const uint8_t *codes, const uint8_t *scales, int n_experts, const int32_t *ids,
                      int n_active, const float *x, float *y, int64_t rows, int64_t cols, void *stream);

/*
 * The paged e4m3 cache (fp8blk_kv_map, fp8blk_kv_append, fp8blk_kv_attn).
 * Keys and values of past tokens are kept in blocks of block_tokens tokens
 * (16, 32, 64 or 128) out of two pools, with one scale for each (block, head):
 *   k_codes, v_codes    device, uint8 e4m3 [n_blocks, kv_heads, block_tokens,
 *                       head_dim], 16-byte aligned
 *   k_scales, v_scales  device, f32 [n_blocks, kv_heads]; value = e4m3(code) *
 *                       scale.  fp8blk_kv_append writes powers of two;
 *                       fp8blk_kv_attn takes any f32; one that is not finite
 *                       counts as NaN.
 *   block_table         device, int32 [n_seqs, max_blocks]: token p of request
 *                       s is row p % block_tokens of block
 *                       block_table[s][p / block_tokens].
 *   q_starts            device, int32 [n_seqs + 1]: the rows of this step that
 *                       belong to request s are q_starts[s] .. q_starts[s+1].
 * A block belongs to one request.  n_blocks * kv_heads * block_tokens < 2^31;
 * head_dim a multiple of 16 up to FP8BLK_MAX_HEAD_DIM.  Lengths, tables and
 * slots stay on the device, so the host checks none of them: the kernels check
 * each before use, skip what is out of range, and set FP8BLK_STATUS_BAD_KV.
 * No counterpart on the pages (their engine keeps its caches elsewhere); these
 * calls serve the same decode step and verify batch, m = 1..8 rows a request
 * ("Struct Dsv4Gpu" page, decode_step_greedy and verify_batch_dev).
 */

/*
 * fp8blk_kv_map -- block tables, slots and positions of one step, from the
 * requests' lengths.  For request s with ctx_lens[s] cached tokens and
 * new_lens[s] new ones (either may be 0):
 *   seq_lens[s] = ctx_lens[s] + new_lens[s];
 *   q_starts    = exclusive prefix sum of new_lens;
 *   table entries [ceil(ctx / B), ceil((ctx + new) / B)) are filled, requests in
 *   order, with the next ids of free_blocks from *free_head on; entries below
 *   are read and kept, entries above are left alone;
 *   positions[i] = the position of new token i in its request, and
 *   slots[i] = block_table[s][p / B] * B + p % B;
 *   *free_head_out = *free_head + the number of ids taken.
 * Entries i of slots and positions past the last new token are -1, so a step
 * captured once with max_tokens rows serves every batch that fits.
 * *free_head_out is the next call's *free_head (the two must not be the same
 * address).  Blocks are taken for all new tokens; where some of them may be
 * rejected afterwards (a verify step), the next call would take a rejected
 * token's block once more: such a loop calls fp8blk_kv_map_held.
 * When the free list runs out, the missing blocks' table entries and slots are
 * -1 and FP8BLK_STATUS_KV_EXHAUSTED is set.  Tokens beyond the table's width
 * get slot -1, starts beyond max_tokens stop there, negative lengths count as
 * 0; each sets FP8BLK_STATUS_BAD_KV.
 *   ctx_lens, new_lens   device, int32 [n_seqs]
 *   block_table          device, int32 [n_seqs, max_blocks], updated in place
 *   free_blocks          device, int32 [n_free]: ids in the order they are taken
 *                        (may be NULL if n_free is 0)
 *   free_head            device, int32 [1]: ids of free_blocks already taken
 *   seq_lens, q_starts   device, int32 [n_seqs], [n_seqs + 1]
 *   slots                device, int64 [max_tokens], 16-byte aligned
 *   positions            device, int32 [max_tokens], 16-byte aligned
 *   free_head_out        device, int32 [1]
 *   n_seqs 1 .. 65536; max_tokens 1 .. 2^31 - 1.
 * Outputs other than block_table must not overlap any input.
 * Errors: EINVAL, EALIGN, ERANGE, ECUDA.
 */
int fp8blk_kv_map(const int32_t *ctx_lens, const int32_t *new_lens, int32_t *block_table, const int32_t *free_blocks,
                  const int32_t *free_head, int32_t *seq_lens, int32_t *q_starts, int64_t *slots, int32_t *positions,
                  int32_t *free_head_out, int n_seqs, int max_blocks, int n_free, int block_tokens, int64_t max_tokens,
                  void *stream);

/*
 * fp8blk_kv_map_held -- the same for requests that may hold more blocks than
 * their context needs, because tokens of earlier steps were rejected.  Request
 * s holds the blocks of its table entries [0, h), h = max(held_blocks[s],
 * ceil(ctx / B)): these entries are read and kept, and [h, ceil((ctx + new) / B))
 * are filled.  held_out[s] is the number it holds afterwards, without those that
 * the free list could not give, and the next call's held_blocks[s]: every id of
 * the free list then lies in one table entry or in the rest of the list.
 * (A finished request's ids are its table's entries [0, held_out[s]).)
 *   held_blocks  device, int32 [n_seqs]; 0 for a new request.  A negative count
 *                is 0, one past max_blocks is max_blocks; both set
 *                FP8BLK_STATUS_BAD_KV
 *   held_out     device, int32 [n_seqs], not held_blocks itself
 * Both may be NULL: then this is fp8blk_kv_map.
 */
int fp8blk_kv_map_held(const int32_t *ctx_lens, const int32_t *new_lens, const int32_t *held_blocks, int32_t *block_table,
                       const int32_t *free_blocks, const int32_t *free_head, int32_t *seq_lens, int32_t *q_starts,
                       int64_t *slots, int32_t *positions, int32_t *free_head_out, int32_t *held_out, int n_seqs,
                       int max_blocks, int n_free, int block_tokens, int64_t max_tokens, void *stream);

/*
 * fp8blk_kv_append -- write new keys and values into the cache.  A run is a
 * maximal group of consecutive tokens whose slots are consecutive inside one
 * block; for each run and head
 *   s = the smallest power of two, at least 2^-126, with max|x| <= 448 s over
 *       the run (values that are not finite do not count); if the block holds
 *       earlier tokens (the run does not start at row 0), s = max(s, old scale);
 *   code = e4m3(x / s), nearest even; NaN and infinities become the NaN code;
 *   if s is larger than the old scale, the codes of the block's earlier rows
 *   become e4m3(e4m3(code) * old / s).  Each is rounded once, also where the
 *   old scale is no power of two.
 * So a block's scale never shrinks while it fills, and row 0 starts it afresh
 * (a block that is reused, or rolled back to empty, needs no clearing).
 *   k, v       device, f32 or bf16 [n_tokens, kv_heads, head_dim], tokens
 *              k_stride / v_stride elements apart (for instance slices of one
 *              fused projection), 16-byte aligned rows
 *   dtype      FP8BLK_F32 or FP8BLK_BF16, of k and v
 *   slots      device, int64 [n_tokens]; negative = skip the token
 * In one call, no two runs may lie in the same block (tokens of two requests
 * in turn, rows out of order, or a token skipped inside a block make two): what
 * such a block holds afterwards is undefined, and FP8BLK_STATUS_BAD_KV is set.
 * A slot at or past n_blocks * block_tokens is skipped and sets
 * FP8BLK_STATUS_BAD_KV.
 * Errors: EINVAL (also a stride that is no multiple of 16 bytes, or shorter
 * than a token), EALIGN, ERANGE, ECUDA.
 */
int fp8blk_kv_append(const void *k, const void *v, int dtype, const int64_t *slots, uint8_t *k_codes, float *k_scales,
                     uint8_t *v_codes, float *v_scales, int64_t n_tokens, int64_t k_stride, int64_t v_stride,
                     int64_t n_blocks, int kv_heads, int block_tokens, int head_dim, void *stream);

/* Workspace size (bytes) of fp8blk_kv_attn; 0 for invalid shapes. */
size_t fp8blk_kv_attn_ws_bytes(int n_seqs, int max_m, int q_heads, int kv_heads, int head_dim);

/*
 * fp8blk_kv_attn -- attention of each request's new rows over its cache.
 * Row i of the r = q_starts[s+1] - q_starts[s] rows of request s sits at
 * position p = seq_lens[s] - r + i and sees the positions 0 .. p; query head h
 * reads cache head h / (q_heads / kv_heads):
 *   a_t   = sm_scale * sum_d q[d] * k[t][d],       t = 0 .. p
 *   lse   = log sum_t exp(a_t),   out[d] = sum_t exp(a_t - lse) * v[t][d].
 * A row that sees nothing (p < 0) gives out = 0 and lse = -inf.  What a row
 * does not see has no part in it, whatever codes and scales are there.
 * Scores, softmax statistics and sums are f32; the codes go to the tensor
 * cores as stored, and q and the weights p s_v as sums of e4m3 values.  With
 * f32, each keeps 2^-16 of itself and 2^-24 of its row's largest (a weight's:
 * of the row's largest p |s_v| in the tile of 128 tokens).  With bf16, q loses
 * 2^-21 of its row's largest, and a weight 2^-8 of itself and 2^-20 of that
 * largest.  (Value scales more than 2^120 apart in one tile, or below 2^-119,
 * lose more.)
 *   q, out     device, f32 or bf16 (`dtype`) [total_rows, q_heads, head_dim],
 *              rows q_stride / out_stride elements apart, 16-byte aligned rows;
 *              rows outside q_starts are left alone
 *   lse        device, optional (NULL = not written): f32 [total_rows, q_heads]
 *   seq_lens   device, int32 [n_seqs]: tokens in the cache, this step's included
 *   max_m      most rows of one request, 1 .. FP8BLK_MAX_M
 *   q_heads    a multiple of kv_heads
 *   ws         device workspace of at least fp8blk_kv_attn_ws_bytes() bytes,
 *              16-byte aligned; zero-filled once before its first use, left
 *              ready by every call.  Calls that share it must be ordered.
 * A block id outside the pool (or a length past max_blocks) makes the rows
 * that see it NaN; a request with more than max_m rows, or rows outside
 * total_rows, is skipped; each sets FP8BLK_STATUS_BAD_KV.
 * Rows of a CTA that gave up on a wait are NaN in out and lse (see
 * fp8blk_set_wait_limit).
 * Errors: EINVAL, EALIGN, EWS, ERANGE (a size past the limits above, or more
 * than about 2^28 tiles of 128 tokens over all requests, heads and groups of 32
 * rows at max_blocks each), ECUDA.
 */
int fp8blk_kv_attn(const void *q, int dtype, const uint8_t *k_codes, const float *k_scales, const uint8_t *v_codes,
                   const float *v_scales, const int32_t *block_table, const int32_t *seq_lens, const int32_t *q_starts,
                   void *out, float *lse, void *ws, size_t ws_bytes, int n_seqs, int max_m, int64_t total_rows,
                   int q_heads, int kv_heads, int head_dim, int block_tokens, int64_t n_blocks, int max_blocks,
                   int64_t q_stride, int64_t out_stride, float sm_scale, void *stream);

/*
 * fp8blk_token_logprobs -- score given tokens under rows of logits: for row i
 * with x = logits[i], t = targets[i], lse = log sum_v exp(x_v)
 *   logprob[i] = x_t - lse
 *   rank[i]    = number of v that come before t in the order below
 *   entropy[i] = -sum_v p_v log p_v,  p = exp(x - lse)
 *   top_ids[i], top_logprobs[i] = the first `top` tokens of that order
 * Order: larger logits first, the lowest index first among equal ones (-0 and
 * +0 are equal), NaN last -- the order of fp8blk_gemv_argmax, so top_ids[i][0]
 * is its token.  Sums are f32.  The logits are read once, and the few words
 * that can hold top tokens twice; but a row (or an eighth of one, where rows are
 * few) in which fewer than about `top` tokens lie above a value that more than
 * 1024 share is read `top` times more: the top of masked rows with few tokens
 * allowed is slow (measured: 20 of 131072 with 5 or 100 allowed, 8 rows 71 us
 * instead of 7.7, 2048 rows 7.5 ms instead of 0.18; with 5000 allowed, or
 * without the top, no difference).
 * A row with a NaN or +inf, or with -inf alone, has NaN logprob, entropy and
 * top_logprobs; -inf among finite logits has probability 0.  Target -1 means
 * none: logprob NaN, rank -1; any other target outside [0, vocab) gives the
 * same and sets FP8BLK_STATUS_BAD_TARGET.
 *   logits   device, f32 or bf16 (`dtype`) [n_rows, vocab], rows `stride`
 *            elements apart (any stride >= vocab), aligned to one element
 *   targets  device, int32 [n_rows]
 *   logprob, entropy  device, f32 [n_rows];  rank  device, int32 [n_rows]
 *   top      0 .. FP8BLK_MAX_TOP, at most vocab; with 0, top_ids and
 *            top_logprobs may be NULL
 *   top_ids, top_logprobs  device, int32 / f32 [n_rows, top]
 *   vocab    1 .. FP8BLK_MAX_VOCAB
 * Errors: EINVAL, EALIGN, ERANGE, ECUDA.
 */
int fp8blk_token_logprobs(const void *logits, int dtype, const int32_t *targets, float *logprob, int32_t *rank,
                          float *entropy, int32_t *top_ids, float *top_logprobs, int64_t n_rows, int64_t vocab,
                          int64_t stride, int top, void *stream);

/*
 * fp8blk_set_launch_tuning -- process-wide launch-shape knobs for the
 * streaming GEMV kernels.  They change speed only: every output is reduced in
 * an order fixed by the column panel layout, so results are bit-identical
 * under any setting.  Pass 0 for a knob's default.
 *   target_stage_bytes  weight bytes per shared-memory pipeline stage (32 KiB)
 *   ctas_per_sm         resident CTAs per SM, 1..4 (2 for m <= 4, else 1)
 *   use_pdl             programmatic dependent launch on (nonzero) or off
 *   l2_prefetch         L2 prefetch, before the grid dependency wait, of the
 *                       stages after the first ring (e4m3) or of the first
 *                       stages (bf16), and of each CTA's first 192 KiB of
 *                       weight rows (tensor-core kernel), on (nonzero) or off
 *   max_stages          pipeline depth cap, 2..8 (8)
 * Not thread-safe against concurrent calls of the other entry points.
 * Errors: EINVAL.
 */
int fp8blk_set_launch_tuning(int target_stage_bytes, int ctas_per_sm, int use_pdl, int l2_prefetch,
                             int max_stages);

/*
 * fp8blk_set_wait_limit -- process-wide limit (nanoseconds, 0 ..
 * FP8BLK_WAIT_LIMIT_DEFAULT_NS) on how long a kernel thread of the CUDA-core
 * GEMVs (fp8blk_gemv / fp8blk_gemv_argmax below the tensor-core thresholds,
 * fp8blk_bf16_gemv, nvfp4_expert_gemv, mxfp4_expert_gemv) waits for a weight
 * tile, or a role of fp8blk_kv_attn for its operands, before it gives up,
 * sets FP8BLK_STATUS_WAIT_TIMEOUT and returns.  The
 * default is about one second; a healthy tile lands in microseconds, so any
 * shorter limit is for exercising the failure path (0 gives up on the first
 * tile that has not landed yet).  After a give-up the CTA still waits, with
 * the fixed one-second bound, for the copies it has in flight before it
 * exits, and still takes part in the argmax hand-off or the join of parts, so
 * the workspace stays consistent; the outputs of that call are invalid (those
 * of fp8blk_kv_attn NaN).  The tensor-core GEMV kernels and the dequant kernel
 * keep the fixed bound.  Not thread-safe against
 * concurrent calls of the other entry points.  Errors: EINVAL.
 */
#define FP8BLK_WAIT_LIMIT_DEFAULT_NS 1000000000ll
int fp8blk_set_wait_limit(int64_t limit_ns);

/*
 * fp8blk_set_m1_kernel -- which kernel serves m = 1 (speed only; results are
 * identical to within the stated error bound, and bit-identical run to run):
 *   choice 0 = by size (e4m3 from the tensor-core threshold of
 *   fp8blk_set_tensor_core_min_m, 48 MiB by default: the tensor-core kernel;
 *   otherwise -- below it, or a shape the tensor-core kernel does not take --
 *   row-per-warp when rows * cols * bytes_per_weight >= rowwarp_min_bytes,
 *   0 = default 96 MiB; the team kernel below that),
 *   1 = always row-per-warp, 2 = always the team kernel (both skip the tensor
 *   cores).  Errors: EINVAL.
 */
int fp8blk_set_m1_kernel(int choice, int64_t rowwarp_min_bytes);

/*
 * fp8blk_set_fp4_kernel -- which kernel serves nvfp4_expert_gemv and
 * mxfp4_expert_gemv (speed only;
 * both are within the stated error bound, each bit-identical run to run):
 *   0 = by shape: the tensor cores from 12288 active rows (n_active x rows)
 *   on, the CUDA cores below; 1 = CUDA cores (weights decoded to f32 in
 *   registers, one f32 FMA each); 2 = tensor cores (the e2m1 codes fed to
 *   tcgen05.mma kind::f8f6f4 as stored, x as five e4m3 planes per scale
 *   block -- 16 columns NVFP4, 32 MXFP4 -- the block scales applied to the
 *   f32 block sums).  The tensor cores also need 32-byte-aligned codes and
 *   room in shared memory for x's planes (16 bytes per column) beside four
 *   code stages (cols up to 4608 with 128-row slabs, more with shorter ones),
 *   else the CUDA cores serve the call; with an inf or NaN in x they return
 *   NaN in every output, the CUDA cores the IEEE result.
 *   Errors: EINVAL.
 */
int fp8blk_set_fp4_kernel(int choice);

/*
 * fp8blk_set_tensor_core_min_m -- route e4m3 GEMVs with m >= min_m activation
 * rows (1..8; 9 = never; 0 = the library default, 1) and at least min_bytes
 * of weights (rows * cols; 1 = any size; 0 = the library default, which
 * depends on m: 24 MiB for m >= 5, 32 MiB for m = 3..4, 48 MiB for m = 1..2) to
 * the tensor-core kernel ("Struct Dsv4Gpu" page, verify_batch_dev: the k+1
 * rows of a speculative verify; decode_step_greedy: the vocab head).  That
 * kernel feeds the stored e4m3 codes to the tensor cores unchanged, splits
 * x * S (S the 128-row tile's block scale) into five e4m3 planes with one
 * exponent per activation row and tile, and accumulates in f32 in tensor
 * memory.  The result stays within the e4m3 GEMV error bound but is not
 * bit-identical to the CUDA-core kernels.  Only for 128 <= cols <= 32768.
 * Speed only; process-wide; not thread-safe against concurrent calls of the
 * other entry points.  Errors: EINVAL.
 */
int fp8blk_set_tensor_core_min_m(int min_m, int64_t min_bytes);

/*
 * fp8blk_plan_query -- HOST, no CUDA calls: the launch geometry the streaming
 * GEMV would use for this shape on a device with the given SM count and
 * shared-memory limits (bytes), for inspection and bounds checks.
 *   bytes_per_weight  1 (e4m3) or 2 (bf16)
 *   out  host int64[13]: panels, panel_cols, team_warps, teams, row_batches,
 *        rows_per_batch, stage_rows, stage_bytes, stages, ctas_per_sm,
 *        n_groups, dynamic_smem_bytes, kernel (0 = team kernel, 1 = row-per-warp
 *        kernel (m = 1, large matrices); for kernel 1, stage_bytes and stages
 *        describe each warp's private ring and teams = warps per CTA)
 * Errors: EINVAL (bad shape or device facts).
 */
int fp8blk_plan_query(int m, int64_t rows, int64_t cols, int bytes_per_weight, int sms,
                      int smem_per_sm, int smem_per_block, int64_t *out);

/*
 * fp8blk_device_status -- read (and optionally clear) the library's device
 * status word on the current device (FP8BLK_STATUS_* bits; 0 = healthy).
 * SYNCHRONIZES the current device.  status_out is a host pointer.
 * Errors: EINVAL, ECUDA.
 */
int fp8blk_device_status(uint32_t *status_out, int clear);

#ifdef __cplusplus
}
#endif

#endif /* FP8BLK_H */
