/*
 * libfp8kv -- fp8 (E4M3) paged KV cache: quantise-on-append, single-query
 * (decode) grouped-query attention and chunked-prefill attention over the
 * cache, for NVIDIA GB300 (sm_103a).
 *
 * Sources the operations follow (the FP8 KV-cache web pages):
 *   [G] gpusmith.com, "FP8 KV Cache Quantization: Capacity Gains and Accuracy
 *       Risk": "What FP8 KV changes" (E4M3, 1 byte/element, max normal 448),
 *       "Scales and calibration" (divide by a per-tensor scale, then cast),
 *       "Attention backend interactions" (the kernel must read fp8 directly,
 *       dequantisation fused), "Why the KV cache sets long-context capacity"
 *       (paged, block-granular cache).
 *   [P] particula.tech, "KV Cache Quantization: What FP8 and q8_0 Cost in
 *       Accuracy", opening section (partial results accumulate in real FP32
 *       registers).
 *   [V] phantomic12 summary of the vLLM FP8 KV-cache blog: "ACCURACY AT LONG
 *       CONTEXT" (the P.V contraction runs over the context, >= 100K tokens),
 *       "DECODE COST" (sliding windows of 128 and 512).
 *   [A] phantomic12 record flops/ctx-fp8-kv-cache-long-context-accuracy:
 *       "Arithmetic intensity" (decode attention streams the cache at about
 *       2g flop per fp8 byte: memory-bound).
 *
 * Conventions for every entry point:
 *   - All pointers except `stream` are DEVICE pointers owned by the caller.
 *     The library allocates nothing and keeps no state between calls (the one
 *     exception is the fixed scratch array of fp8kv_paged_decode_noalloc).
 *     The entry points are safe to call from several host threads.
 *   - Work is enqueued asynchronously on `stream` (a cudaStream_t; NULL = the
 *     legacy default stream).  Nothing is synchronised.
 *   - Invalid arguments return an error status and launch nothing.  A failed
 *     launch returns FP8KV_ERR_CUDA.  Faults during execution surface at the
 *     caller's next synchronisation, as for any CUDA kernel.
 *   - bf16 means IEEE bfloat16 stored as 2-byte little-endian values.
 */
#ifndef FP8KV_H_
#define FP8KV_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FP8KV_OK = 0,
    FP8KV_ERR_INVALID_ARG = 1, /* null pointer, bad size, non-finite/<=0 scale, misalignment */
    FP8KV_ERR_UNSUPPORTED = 2, /* shape outside the supported set (see below)                */
    FP8KV_ERR_WORKSPACE = 3,   /* workspace missing or smaller than the required size         */
    FP8KV_ERR_CUDA = 4,        /* a CUDA runtime call or kernel launch failed                 */
    FP8KV_ERR_TIMEOUT = 5      /* a kernel gave up a bounded wait (read via fp8kv_read_error) */
} fp8kv_status;

/* Static, human-readable name of a status code. */
const char* fp8kv_status_string(fp8kv_status status);

/*
 * Quantise-on-append [G "Scales and calibration"; G "What FP8 KV changes"].
 *
 * For every token t < num_tokens, kv head h and dim i:
 *     code = E4M3( fp32(k_new[t][h][i]) / k_scale )     (same for V)
 * with one IEEE fp32 division followed by one round-to-nearest-even,
 * saturating-finite conversion (|x| >= 448 -> +-448, NaN -> NaN).  The code
 * is written at slot s = slot_mapping[t] = block * block_size + offset:
 *     k_cache[block][h][offset][i] = code.
 *
 *   k_new, v_new   bf16 [num_tokens][num_kv_heads][head_dim], contiguous,
 *                  16-byte aligned
 *   slot_mapping   int64 [num_tokens]; a negative slot skips the token (padding);
 *                  a slot >= num_blocks * block_size is out of range and is
 *                  skipped too (nothing is written for it)
 *   k_cache,       uint8 E4M3 [num_blocks][num_kv_heads][block_size][head_dim]
 *   v_cache        (one page = one (block, head) pair = block_size*head_dim
 *                  contiguous bytes), 16-byte aligned
 *   k_scale,       per-tensor scales, finite and > 0
 *   v_scale
 * Supported: head_dim % 16 == 0 and 16 <= head_dim <= 1024; block_size >= 1.
 * num_tokens == 0 is a no-op.
 */
fp8kv_status fp8kv_quant_append(const void* k_new, const void* v_new,
                                const int64_t* slot_mapping, int64_t num_tokens,
                                uint8_t* k_cache, uint8_t* v_cache, int64_t num_blocks,
                                int block_size, int num_kv_heads, int head_dim,
                                float k_scale, float v_scale, void* stream);

/*
 * Workspace bytes fp8kv_paged_decode needs for this problem on the CURRENT
 * device (the split-context plan depends on its SM count).  Returns 0 if the
 * arguments are invalid or no device is available.
 */
size_t fp8kv_paged_decode_workspace_size(int batch, int num_q_heads, int num_kv_heads,
                                         int head_dim, int max_seq_len, int block_size,
                                         int window);

/*
 * Zero-fills a workspace (asynchronously on `stream`).  A workspace must be
 * zero-filled once before its first fp8kv_paged_decode call; every call that
 * completes leaves it ready for the next one (its per-unit split counters
 * back at zero).  After a call that failed with
 * FP8KV_ERR_TIMEOUT the workspace must be zero-filled again.  Calls that share one workspace must be ordered (same
 * stream or explicit dependencies).
 */
fp8kv_status fp8kv_workspace_init(void* workspace, size_t workspace_bytes, void* stream);

/*
 * Reads (and clears) the workspace's error word: 0 = no error, otherwise an
 * fp8kv_status (FP8KV_ERR_TIMEOUT, or FP8KV_ERR_INVALID_ARG for an
 * out-of-range block id met on the device).  Synchronises `stream`.
 */
fp8kv_status fp8kv_read_error(void* workspace, uint32_t* code, void* stream);

/*
 * Paged fp8 decode attention [G "Attention backend interactions";
 * V "ACCURACY AT LONG CONTEXT"; P opening section].
 *
 * For batch b, query head h (kv head hk = h / g, g = num_q_heads/num_kv_heads),
 * with L = seq_lens[b] (the current token included) and the attended keys
 * t in [lo, L), lo = (window > 0 && L > window) ? L - window : 0:
 *     k^_t = decode(k_cache[page(t)][hk][t % bs][:]) * k_scale
 *     v^_t = decode(v_cache[page(t)][hk][t % bs][:]) * v_scale
 *     s_t  = sm_scale * sum_i q[b][h][i] * k^_t[i]
 *     out[b][h][:] = sum_t exp(s_t - max s) v^_t / sum_t exp(s_t - max s)
 * page(t) = block_tables[b][t / block_size].  Scores, the softmax and P.V are
 * accumulated in FP32; split-context partial results are merged in FP32; the
 * result is rounded to bf16 (RNE).  L == 0 writes zeros.
 *
 *   q              bf16 [batch][num_q_heads][head_dim], contiguous, 16-B aligned
 *   k_cache,       uint8 E4M3 [num_blocks][num_kv_heads][block_size][head_dim],
 *   v_cache        16-byte aligned (the layout fp8kv_quant_append writes)
 *   block_tables   int32 [batch][max_blocks_per_seq]; entries past a sequence's
 *                  last page are never read; an entry outside [0, num_blocks)
 *                  is replaced by block 0 and reported via fp8kv_read_error
 *   seq_lens       int32 [batch] on the device; each must satisfy
 *                  0 <= seq_lens[b] <= min(max_seq_len, max_blocks_per_seq*block_size)
 *   max_seq_len    host-side upper bound of seq_lens (sizes the split plan)
 *   sm_scale       softmax scale (usually 1/sqrt(head_dim)); finite
 *   window         <= 0: full attention; > 0: attend the last `window` keys
 *   out            bf16 [batch][num_q_heads][head_dim], 16-byte aligned
 *   workspace      >= fp8kv_paged_decode_workspace_size(...) bytes, 256-B
 *                  aligned, zero-filled before first use (fp8kv_workspace_init)
 * Supported: head_dim in {64, 128, 256}; block_size == 16;
 *            g in {1, 2, 4, 8, 16}; num_blocks * num_kv_heads < 2^31.  At g = 16
 *            each kv head runs as two units of 8 query heads, each reading the
 *            head's pages (the kernels put a unit's heads on the MMA's n side).
 */
fp8kv_status fp8kv_paged_decode(const void* q, const uint8_t* k_cache, const uint8_t* v_cache,
                                int64_t num_blocks, const int32_t* block_tables,
                                int max_blocks_per_seq, const int32_t* seq_lens,
                                int max_seq_len, int batch, int num_q_heads, int num_kv_heads,
                                int head_dim, int block_size, float k_scale, float v_scale,
                                float sm_scale, int window, void* out, void* workspace,
                                size_t workspace_bytes, void* stream);

/*
 * Per-attention-head scales [G "Scales and calibration": per-tensor or
 * per-attention-head k/v scales, [num_kv_heads] each].
 *
 * The same operations as fp8kv_quant_append, fp8kv_paged_decode and
 * fp8kv_decode_step, with one K scale and one V scale per kv head instead of
 * one per tensor: elements of kv head h are divided by k_scales[h]
 * (v_scales[h]) before the cast, and its codes stand for
 * decode(code) * scale[h] in the attention.
 *
 *   k_scales, v_scales  DEVICE fp32 [num_kv_heads], 4-byte aligned, finite and
 *                       > 0 (not checked on the device: other values give
 *                       unspecified codes and outputs); read by the kernels
 *                       after they wait for the previous work on the stream.
 *   all other arguments, the workspace and the errors as the per-tensor calls.
 * With every k_scales[h] == k_scale and v_scales[h] == v_scale the results
 * are bit-identical to the per-tensor calls.
 */
fp8kv_status fp8kv_quant_append_per_head(const void* k_new, const void* v_new, const int64_t* slot_mapping,
                                         int64_t num_tokens, uint8_t* k_cache, uint8_t* v_cache,
                                         int64_t num_blocks, int block_size, int num_kv_heads, int head_dim,
                                         const float* k_scales, const float* v_scales, void* stream);

fp8kv_status fp8kv_paged_decode_per_head(const void* q, const uint8_t* k_cache, const uint8_t* v_cache,
                                         int64_t num_blocks, const int32_t* block_tables,
                                         int max_blocks_per_seq, const int32_t* seq_lens, int max_seq_len,
                                         int batch, int num_q_heads, int num_kv_heads, int head_dim,
                                         int block_size, const float* k_scales, const float* v_scales,
                                         float sm_scale, int window, void* out, void* workspace,
                                         size_t workspace_bytes, void* stream);

fp8kv_status fp8kv_decode_step_per_head(const void* q, const void* k_new, const void* v_new,
                                        uint8_t* k_cache, uint8_t* v_cache, int64_t num_blocks,
                                        const int32_t* block_tables, int max_blocks_per_seq,
                                        const int32_t* seq_lens, int max_seq_len, int batch,
                                        int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                        const float* k_scales, const float* v_scales, float sm_scale,
                                        int window, void* out, void* workspace, size_t workspace_bytes,
                                        void* stream);

/*
 * The E5M2 cache [G "What FP8 KV changes": the other FP8 format, 2 mantissa
 * bits and a maximum of 57,344; E4M3 is the default].
 *
 * The same operations as fp8kv_quant_append, fp8kv_paged_decode and
 * fp8kv_decode_step with E5M2 codes (S.EEEEE.MM, exponent bias 15,
 * subnormals m * 2^-16): code = E5M2(fp32(x) / scale) with one IEEE fp32
 * division and one round-to-nearest-even, saturating-finite conversion
 * (|x| >= 57344 and infinities -> +-57344, NaN -> NaN).  A code stands for
 * its exact value times the scale; E5M2 values are exact in f16, so the
 * decode runs the same tensor-core path.  Arguments, layout, workspace and
 * errors as the E4M3 calls.
 */
fp8kv_status fp8kv_quant_append_e5m2(const void* k_new, const void* v_new, const int64_t* slot_mapping,
                                     int64_t num_tokens, uint8_t* k_cache, uint8_t* v_cache,
                                     int64_t num_blocks, int block_size, int num_kv_heads, int head_dim,
                                     float k_scale, float v_scale, void* stream);

fp8kv_status fp8kv_paged_decode_e5m2(const void* q, const uint8_t* k_cache, const uint8_t* v_cache,
                                     int64_t num_blocks, const int32_t* block_tables,
                                     int max_blocks_per_seq, const int32_t* seq_lens, int max_seq_len,
                                     int batch, int num_q_heads, int num_kv_heads, int head_dim,
                                     int block_size, float k_scale, float v_scale, float sm_scale,
                                     int window, void* out, void* workspace, size_t workspace_bytes,
                                     void* stream);

fp8kv_status fp8kv_decode_step_e5m2(const void* q, const void* k_new, const void* v_new,
                                    uint8_t* k_cache, uint8_t* v_cache, int64_t num_blocks,
                                    const int32_t* block_tables, int max_blocks_per_seq,
                                    const int32_t* seq_lens, int max_seq_len, int batch,
                                    int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                    float k_scale, float v_scale, float sm_scale, int window, void* out,
                                    void* workspace, size_t workspace_bytes, void* stream);

/* Which units perform the two contractions of the decode attention. */
typedef enum {
    FP8KV_ENGINE_DEFAULT = 0,      /* the library's choice for the shape (the faster one measured) */
    FP8KV_ENGINE_TENSOR_CORES = 1, /* m16n8k16 f16 MMA per stage tile, folded into FP32 registers */
    FP8KV_ENGINE_CUDA_CORES = 2    /* FP32 fma chains of exact f16 products on the CUDA cores     */
} fp8kv_engine;

/*
 * fp8kv_paged_decode with the contraction engine chosen by the caller
 * [P opening section (FP32 accumulation); A "Arithmetic intensity" (at M = g
 * the contractions are small next to the bytes streamed, so either unit may
 * keep up; the default is the one measured faster)].
 *
 * Same operation, arguments, workspace and errors as fp8kv_paged_decode; the
 * engines differ only in rounding order (both accumulate in FP32 and meet the
 * same tolerance).  An engine value outside fp8kv_engine is
 * FP8KV_ERR_INVALID_ARG.
 */
fp8kv_status fp8kv_paged_decode_engine(const void* q, const uint8_t* k_cache, const uint8_t* v_cache,
                                       int64_t num_blocks, const int32_t* block_tables,
                                       int max_blocks_per_seq, const int32_t* seq_lens,
                                       int max_seq_len, int batch, int num_q_heads, int num_kv_heads,
                                       int head_dim, int block_size, float k_scale, float v_scale,
                                       float sm_scale, int window, void* out, void* workspace,
                                       size_t workspace_bytes, void* stream, int engine);

/*
 * The bf16 twin of fp8kv_paged_decode: the same attention over a paged cache
 * that stores bf16 K and V instead of E4M3 codes -- the baseline the fp8 cache
 * is compared against [G "What FP8 KV changes" (1 byte per element against
 * bf16's 2); V "DECODE COST" (cost per cached token, fp8 against bf16)].
 *
 *   k_cache, v_cache  bf16 [num_blocks][num_kv_heads][block_size][head_dim],
 *                     16-byte aligned (no scales: the values are the cache)
 *   all other arguments, the workspace and the errors as fp8kv_paged_decode.
 *
 * Scores and P.V run on the tensor cores with bf16 operands (P rounded to
 * bf16) and FP32 accumulation, each stage's tile added into FP32 registers.
 * Supported: head_dim in {64, 128, 256}; block_size == 16; g in {1, 2, 4, 8, 16}.
 */
fp8kv_status fp8kv_paged_decode_bf16(const void* q, const void* k_cache, const void* v_cache,
                                     int64_t num_blocks, const int32_t* block_tables,
                                     int max_blocks_per_seq, const int32_t* seq_lens,
                                     int max_seq_len, int batch, int num_q_heads, int num_kv_heads,
                                     int head_dim, int block_size, float sm_scale, int window,
                                     void* out, void* workspace, size_t workspace_bytes, void* stream);

/*
 * One decode step: append, then attend [G "Scales and calibration";
 * G "Attention backend interactions"; V "ACCURACY AT LONG CONTEXT"].
 *
 * Equivalent to fp8kv_quant_append of each sequence's newest row followed by
 * fp8kv_paged_decode, in one launch: for every b with
 * L = seq_lens[b] > 0 the row k_new[b] (v_new[b]) is quantised exactly as
 * fp8kv_quant_append does and written at token L-1 of the sequence, i.e. at
 * page block_tables[b][(L-1)/block_size], offset (L-1) % block_size; then the
 * attention of fp8kv_paged_decode runs over the cache including that token.
 *
 *   k_new, v_new   bf16 [batch][num_kv_heads][head_dim], 16-byte aligned
 *   all other arguments as for fp8kv_paged_decode (k_cache / v_cache are
 *   written).  Sequences of length 0 append nothing; a page whose block id is
 *   out of range is not written (the error word reports it).
 */
fp8kv_status fp8kv_decode_step(const void* q, const void* k_new, const void* v_new, uint8_t* k_cache,
                               uint8_t* v_cache, int64_t num_blocks, const int32_t* block_tables,
                               int max_blocks_per_seq, const int32_t* seq_lens, int max_seq_len,
                               int batch, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                               float k_scale, float v_scale, float sm_scale, int window, void* out,
                               void* workspace, size_t workspace_bytes, void* stream);

/*
 * fp8kv_decode_step for a caller whose per-step inputs and result live in
 * host memory (an engine that computes q and the new K/V rows on the host, or
 * a test harness).  No counterpart on the pages: it only moves the step's
 * inputs and output across the host link around the step above.
 *
 * On `stream`, in order: one copy of in_bytes bytes from h_in to d_in, the
 * decode step, and the step's output (batch*num_q_heads*head_dim bf16) into
 * h_out.  When the device can address h_out (page-locked host memory under
 * unified addressing, e.g. cudaHostAlloc or a registered buffer) the step's
 * kernels store the output there directly, across the host link, and `out`
 * is not written; otherwise the output goes to `out` and one copy moves it
 * to h_out.  It returns once the work is enqueued; h_out is valid after the
 * caller synchronises the stream.
 *
 *   h_in    host buffer (page-locked for an asynchronous copy) holding the
 *           step's inputs exactly as they must appear at d_in
 *   d_in    device buffer of in_bytes bytes; q, k_new, v_new and seq_lens are
 *           device pointers, usually into d_in (the caller chooses the layout)
 *   h_out   host buffer for the output (page-locked for an asynchronous copy)
 *   all other arguments as for fp8kv_decode_step.
 * Errors: those of fp8kv_decode_step (checked before anything is enqueued);
 * null h_in, d_in or h_out with in_bytes > 0 is FP8KV_ERR_INVALID_ARG; a
 * failed copy is FP8KV_ERR_CUDA.
 */
fp8kv_status fp8kv_decode_step_host(const void* h_in, void* d_in, size_t in_bytes, void* h_out,
                                    const void* q, const void* k_new, const void* v_new, uint8_t* k_cache,
                                    uint8_t* v_cache, int64_t num_blocks, const int32_t* block_tables,
                                    int max_blocks_per_seq, const int32_t* seq_lens, int max_seq_len,
                                    int batch, int num_q_heads, int num_kv_heads, int head_dim,
                                    int block_size, float k_scale, float v_scale, float sm_scale, int window,
                                    void* out, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Allocation-free paged decode.  This entry point has no counterpart on the
 * pages: it exists for callers that cannot allocate device memory when they
 * decode -- e.g. a serving engine that reserved nearly all HBM for its own
 * paged KV pool, host code under a no-allocation rule, or a binding without a
 * CUDA allocator -- and so cannot provide the workspace fp8kv_paged_decode
 * takes.  It computes exactly what fp8kv_paged_decode computes, with the same
 * arguments minus the workspace.
 *
 * Scratch: a fixed 8 MiB array compiled into the library (every device that
 * loads the library keeps it until the process exits).  The call allocates
 * nothing and calls no allocating routine; it zeroes the array's header
 * (the error word) and its per-unit split counters (one cudaMemsetAsync on
 * `stream`), and then runs the decode.  The split partials need no clearing:
 * every call writes the ones it reads.
 *   - A problem whose split-merge scratch would exceed 8 MiB is rejected with
 *     FP8KV_ERR_WORKSPACE before anything is launched.
 *   - The first call on each device looks up the array's device address with
 *     that device current (cudaGetSymbolAddress); make that first call before
 *     any stream capture.  The address is kept for the life of the process:
 *     after a device reset (cudaDeviceReset) the array moves, so do not call
 *     this entry point on a device that was reset.
 *   - All calls share the one array: calls that overlap on the GPU (different
 *     streams without ordering, or different host threads) race and corrupt
 *     each other's results.  Order them.
 *   - Device-side errors (an out-of-range block id) are not reported by this
 *     variant; use fp8kv_paged_decode with a workspace to read them.
 */
fp8kv_status fp8kv_paged_decode_noalloc(const void* q, const uint8_t* k_cache, const uint8_t* v_cache,
                                        int64_t num_blocks, const int32_t* block_tables,
                                        int max_blocks_per_seq, const int32_t* seq_lens, int max_seq_len,
                                        int batch, int num_q_heads, int num_kv_heads, int head_dim,
                                        int block_size, float k_scale, float v_scale, float sm_scale,
                                        int window, void* out, void* stream);

/*
 * Chunked-prefill attention over the paged E4M3 cache [G "Attention backend
 * interactions" (the prefill pass reads the same fp8 cache as decode);
 * V "ACCURACY AT LONG CONTEXT" (P.V over the context in FP32)].
 *
 * Sequence b holds L = seq_lens[b] tokens in the cache, its n = q_len[b] =
 * q_starts[b+1] - q_starts[b] newest ones included (append them first with
 * fp8kv_quant_append).  Query row i < n of the sequence sits at position
 * p = L - n + i and attends the keys t in [lo(p), p], lo(p) = (window > 0 &&
 * p + 1 > window) ? p + 1 - window : 0 -- causal, optionally within a
 * sliding window; row by row this is fp8kv_paged_decode of a sequence of
 * length p + 1:
 *     s_t = sm_scale * sum_i q[r][h][i] * decode(k code of t)[i] * k_scale
 *     out[r][h][:] = sum_t exp(s_t - max s) decode(v code of t) * v_scale
 *                    / sum_t exp(s_t - max s)
 * with r = q_starts[b] + i.  Scores, the softmax and P.V accumulate in FP32
 * (key-range partials, when the call splits a long range over several CTAs,
 * are merged in FP32); the result is rounded to bf16 (RNE).
 *
 *   q              bf16 [num_q_tokens][num_q_heads][head_dim], the query rows of
 *                  all sequences packed in order, 16-byte aligned
 *   num_q_tokens   rows of q and out (q_starts[batch])
 *   k_cache,       uint8 E4M3 caches, layout as fp8kv_paged_decode
 *   v_cache
 *   block_tables   int32 [batch][max_blocks_per_seq]; only the pages a query
 *                  attends are read
 *   seq_lens       int32 [batch] on the device, 0 <= seq_lens[b] <= max_seq_len
 *   q_starts       int32 [batch + 1] on the device, non-decreasing, q_starts[0] = 0,
 *                  q_starts[b+1] - q_starts[b] <= min(seq_lens[b], max_q_len)
 *   max_q_len      host-side upper bound of the q_len (sizes the grid)
 *   window         <= 0: causal over the whole prefix; > 0: the last `window` keys
 *   out            bf16 [num_q_tokens][num_q_heads][head_dim], 16-byte aligned
 *   workspace      >= fp8kv_paged_prefill_workspace_size(...) bytes, 256-byte
 *                  aligned, zero-filled before first use (fp8kv_workspace_init);
 *                  its first word is the error word fp8kv_read_error reads: an
 *                  out-of-range block id (block 0 is read instead), or a
 *                  seq_lens / q_starts entry outside the bounds above (the
 *                  sequence is clamped, or skipped if its rows would fall
 *                  outside q / out).  Calls that share a workspace must be
 *                  ordered.  Missing or too small: FP8KV_ERR_WORKSPACE.
 * Supported: head_dim in {64, 128, 256}; block_size == 16; g in {1, 2, 4, 8, 16};
 *            num_blocks * num_kv_heads < 2^31.  batch == 0, max_q_len == 0 or
 *            num_q_tokens == 0 is a no-op.
 */
/*
 * Workspace bytes fp8kv_paged_prefill needs for this problem on the CURRENT
 * device: the key-range split plan depends on its SM count and on how many
 * prefill CTAs it holds at once.  At least 256 (the error word); larger
 * when the call splits key ranges.  Returns 0 if the arguments are invalid
 * or no device is available.  Enough for fp8kv_paged_prefill_block too.
 */
size_t fp8kv_paged_prefill_workspace_size(int batch, int max_q_len, int max_seq_len, int num_q_heads,
                                          int num_kv_heads, int head_dim, int block_size, int window);

fp8kv_status fp8kv_paged_prefill(const void* q, int64_t num_q_tokens, const uint8_t* k_cache,
                                 const uint8_t* v_cache, int64_t num_blocks, const int32_t* block_tables,
                                 int max_blocks_per_seq, const int32_t* seq_lens, const int32_t* q_starts,
                                 int max_q_len, int max_seq_len, int batch, int num_q_heads,
                                 int num_kv_heads, int head_dim, int block_size, float k_scale,
                                 float v_scale, float sm_scale, int window, void* out, void* workspace,
                                 size_t workspace_bytes, void* stream);

/* What a cache page holds (fp8kv_rope_append). */
typedef enum {
    FP8KV_CACHE_E4M3 = 0, /* the cache of fp8kv_quant_append, fp8kv_paged_decode, fp8kv_paged_prefill */
    FP8KV_CACHE_E5M2 = 1, /* the cache of fp8kv_quant_append_e5m2 and fp8kv_paged_decode_e5m2         */
    FP8KV_CACHE_BF16 = 2  /* the cache of fp8kv_paged_decode_bf16                                     */
} fp8kv_cache_format;

/* Which elements of a head a rotation pairs, R = rotary_dim. */
typedef enum {
    FP8KV_ROPE_HALVES = 0, /* frequency i turns elements i and i + R/2  */
    FP8KV_ROPE_PAIRS = 1   /* frequency i turns elements 2i and 2i + 1  */
} fp8kv_rope_style;

/*
 * Rotary positions on the way into the cache: q rotated into q_out, k rotated,
 * k and v quantised and written through a slot mapping.  No counterpart on the
 * pages, which start from rotated keys; it stands in front of every decode
 * and prefill call of this library.
 *
 * For token t and frequency i < rotary_dim / 2:
 *     angle = positions[axis(i)][t] * inv_freq[i]
 * as a real product (the kernels keep it to about 2^-48 of its size before
 * the fraction of a turn is taken, so positions of 2^20 lose nothing), and the pair (x, y) the
 * frequency owns (fp8kv_rope_style) becomes
 *     (x cos - y sin, y cos + x sin)
 * in fp32.  Elements from rotary_dim on pass unchanged.  q_out is rounded once
 * to bf16 (RNE).  k is not rounded before its conversion, which together with
 * v's is that of fp8kv_quant_append (E4M3: one fp32 division by the scale, one
 * RNE saturating conversion), fp8kv_quant_append_e5m2, or bf16 RNE.  With
 * rotary_dim 0 the cache bytes are exactly theirs.
 *
 *   q, q_out       bf16; token t's heads at q + t * q_stride elements, q_out
 *                  contiguous [num_tokens][num_q_heads][head_dim].  Both null:
 *                  no queries.  q_out may be q itself if q is contiguous; any
 *                  other overlap is undefined.
 *   k_new, v_new   bf16; token t's heads at k_new + t * k_stride elements.
 *                  Slices of one fused projection's output fit: the strides
 *                  are multiples of 8 and at least a row, the pointers
 *                  16-byte aligned.
 *   positions      int32 [num_axes][num_tokens]; num_axes 1..4.  One axis for
 *                  text; time, height and width for images and video.
 *   inv_freq       fp32 [rotary_dim / 2]
 *   freq_axis      uint8 [rotary_dim / 2], the axis of each frequency (in runs
 *                  or interleaved, as the model has them); null: axis 0.  A
 *                  value outside [0, num_axes) is read as axis 0.
 *   rotary_dim     0 (positions, inv_freq and freq_axis unused) or a multiple
 *                  of 16 up to head_dim
 *   slot_mapping   int64 [num_tokens], 8-byte aligned, as fp8kv_quant_append: a
 *                  negative or out-of-range slot skips the token's cache
 *                  write; its query is rotated all the same.  A slot given to
 *                  two tokens gets one of their rows, or a mix.
 *   k_cache,       [num_blocks][num_kv_heads][block_size][head_dim] of
 *   v_cache        cache_format, 16-byte aligned
 *   k_scale,       per-tensor scales, finite and > 0 (1 for a bf16 cache);
 *   v_scale        not used where k_scales, v_scales are given
 *   k_scales,      DEVICE fp32 [num_kv_heads] as fp8kv_quant_append_per_head,
 *   v_scales       or both null (null for a bf16 cache)
 * All of positions, inv_freq, freq_axis, slot_mapping, k_scales and v_scales
 * are device pointers.
 * Supported: head_dim in {64, 128, 256}; block_size >= 1; num_tokens < 2^31.
 * num_tokens == 0 is a no-op.
 */
fp8kv_status fp8kv_rope_append(const void* q, int64_t q_stride, void* q_out, const void* k_new, int64_t k_stride,
                               const void* v_new, int64_t v_stride, const int32_t* positions, int num_axes,
                               const float* inv_freq, const uint8_t* freq_axis, int rotary_dim, int rope_style,
                               const int64_t* slot_mapping, int64_t num_tokens, void* k_cache, void* v_cache,
                               int64_t num_blocks, int block_size, int num_q_heads, int num_kv_heads, int head_dim,
                               int cache_format, float k_scale, float v_scale, const float* k_scales,
                               const float* v_scales, void* stream);

/*
 * The block-scaled cache: E4M3 codes with one scale for each (page, kv head)
 * of K and one of V [below the granularities of G "Scales and calibration"].
 * No calibration: the append chooses the scales from the rows it writes.
 *
 *   k_scales, v_scales  DEVICE fp32 [num_blocks][num_kv_heads], 4-byte
 *                       aligned.  They may be the append's or the caller's
 *                       own (a page filled elsewhere).  Finite and within
 *                       [2^-40, 2^40] for every page that is attended or
 *                       appended to behind older rows; other values give
 *                       unspecified codes and outputs (not checked on the
 *                       device).  Need no initialisation: a page whose first
 *                       row is appended gets its scale then.
 *
 * fp8kv_rope_append_block rotates q and k as fp8kv_rope_append and appends
 * the newest n = q_starts[b+1] - q_starts[b] tokens of every sequence (of its
 * seq_lens[b], they included) to its pages.  For each page, kv head and each
 * of K (rotated) and V, with amax the largest finite magnitude of the new rows:
 *   - the page holds older rows of the sequence, and amax <= 448 * s for its
 *     scale s: the scale stays, the new rows are written under it;
 *   - otherwise the scale becomes 2^e (or stays, if larger), e the least whole
 *     number in [-40, 40] with amax <= 448 * 2^e, and the older rows' codes c
 *     become E4M3(decode(c) * (s_old / s_new)).
 * New codes are E4M3(x / s): one fp32 division, one RNE saturating conversion
 * (infinities saturate, NaN stays NaN; neither takes part in amax).
 *
 *   q .. rope_style     as fp8kv_rope_append; tokens packed by sequence
 *   num_tokens          rows of q, k_new, v_new and positions
 *   positions           null with num_axes 1: each token's place in its sequence
 *   block_tables        int32 [batch][max_blocks_per_seq], as fp8kv_paged_decode.
 *                       A page written must be in one place of one sequence's
 *                       row only: a page that one call appends to twice gets
 *                       unspecified codes and scales.
 *   seq_lens            int32 [batch] on the device
 *   q_starts            int32 [batch + 1] on the device, non-decreasing, or
 *                       null: a decode step, row b is sequence b's newest token
 *                       (num_tokens == batch; seq_lens[b] == 0 skips the row).
 *                       Rows of q_out outside [q_starts[0], q_starts[batch])
 *                       are left as they are.
 *   workspace           256-byte aligned, at least 256 bytes, zero-filled before
 *                       first use (fp8kv_workspace_init): the error word that
 *                       fp8kv_read_error reads.  Any workspace of this library
 *                       will do, in the order its calls share it.  Reported as
 *                       FP8KV_ERR_INVALID_ARG: a block id outside
 *                       [0, num_blocks) (the page is not written, its queries
 *                       are rotated), and a sequence whose seq_lens or q_starts
 *                       do not satisfy 0 <= n <= seq_lens[b] <= max_seq_len
 *                       and q_starts[b+1] <= num_tokens (it is skipped).
 * Supported: head_dim in {64, 128, 256}; block_size == 16; batch <= 65535;
 *            num_blocks * num_kv_heads < 2^31; num_tokens < 2^31.  batch == 0,
 *            num_tokens == 0 or max_seq_len == 0 is a no-op.
 */
fp8kv_status fp8kv_rope_append_block(const void* q, int64_t q_stride, void* q_out, const void* k_new,
                                     int64_t k_stride, const void* v_new, int64_t v_stride, int64_t num_tokens,
                                     const int32_t* positions, int num_axes, const float* inv_freq,
                                     const uint8_t* freq_axis, int rotary_dim, int rope_style, uint8_t* k_cache,
                                     uint8_t* v_cache, float* k_scales, float* v_scales, int64_t num_blocks,
                                     const int32_t* block_tables, int max_blocks_per_seq, const int32_t* seq_lens,
                                     const int32_t* q_starts, int max_seq_len, int batch, int num_q_heads,
                                     int num_kv_heads, int head_dim, int block_size, void* workspace,
                                     size_t workspace_bytes, void* stream);

/*
 * fp8kv_paged_decode over a block-scaled cache: key t's code stands for
 * decode(code) * k_scales[page(t)][hk], value t's for decode(code) *
 * v_scales[page(t)][hk].  Scores are scaled page by page in FP32; a key's weight
 * is its probability times its page's V scale, rounded to f16 (11 bits) for the
 * tensor cores: relative to itself where it is at least 2^-29 of the largest
 * such weight, in steps of 2^-39 of the largest below that.  So a page counts
 * by what it brings to the answer, whatever its scale and probability are for
 * themselves.  Sums are FP32.  All other arguments, the workspace
 * (fp8kv_paged_decode_workspace_size) and the errors as fp8kv_paged_decode.
 */
fp8kv_status fp8kv_paged_decode_block(const void* q, const uint8_t* k_cache, const uint8_t* v_cache,
                                      const float* k_scales, const float* v_scales, int64_t num_blocks,
                                      const int32_t* block_tables, int max_blocks_per_seq, const int32_t* seq_lens,
                                      int max_seq_len, int batch, int num_q_heads, int num_kv_heads, int head_dim,
                                      int block_size, float sm_scale, int window, void* out, void* workspace,
                                      size_t workspace_bytes, void* stream);

/*
 * fp8kv_paged_prefill over a block-scaled cache (append the chunk first, with
 * fp8kv_rope_append_block).  Weights are rounded as fp8kv_paged_decode_block's,
 * with less room: relative to themselves down to 2^-14 of a row's largest, in
 * steps of 2^-24 of it below.  Scores, in units of a factor of two, of up to
 * 2^26 in size; larger ones may give infinities.  All other arguments, the workspace
 * (fp8kv_paged_prefill_workspace_size) and the errors as fp8kv_paged_prefill.
 * What a row may not attend does not reach it, with one exception, as in
 * fp8kv_paged_prefill: a NaN code in V makes NaN of its dimension in every
 * row that shares a tile (up to 256 rows: token, query head) with one that
 * attends it, since a masked weight of zero still multiplies it.
 */
fp8kv_status fp8kv_paged_prefill_block(const void* q, int64_t num_q_tokens, const uint8_t* k_cache,
                                       const uint8_t* v_cache, const float* k_scales, const float* v_scales,
                                       int64_t num_blocks, const int32_t* block_tables, int max_blocks_per_seq,
                                       const int32_t* seq_lens, const int32_t* q_starts, int max_q_len,
                                       int max_seq_len, int batch, int num_q_heads, int num_kv_heads, int head_dim,
                                       int block_size, float sm_scale, int window, void* out, void* workspace,
                                       size_t workspace_bytes, void* stream);

/*
 * Attention of a tree of drafted tokens per sequence (speculative decoding:
 * a draft proposes several continuations at once, one call checks them all).
 * No counterpart on the pages; it stands beside fp8kv_paged_prefill, whose
 * chunk is the tree that is one chain.
 *
 * Sequence b holds L = seq_lens[b] tokens in the cache, the newest
 * n = q_starts[b+1] - q_starts[b] of them its drafted nodes, in any order that
 * has parents before children (append them first, at slots L - n + i, rotated
 * by the position c + depth(i) they stand for, c = L - n).  parents[q_starts[b]
 * + i] is the node's parent, a smaller number of the same tree, or -1: a root,
 * of depth 0; a child's depth is its parent's plus 1.  Node i attends
 *   - the context: token t < c with t > c + depth(i) - window;
 *   - itself and its ancestors j with depth(j) > depth(i) - window
 * (window <= 0: all of them), with the scores, softmax and rounding of
 * fp8kv_paged_prefill.  The newest keys before them in the cache are other
 * branches; they do not reach the row, but for a NaN or infinity in V, which
 * makes NaN of its dimension in every row that shares a tile (up to 256 rows:
 * node, query head), since a weight of zero still multiplies it.
 *
 *   q, out         bf16 [num_tokens][num_q_heads][head_dim], 16-byte aligned,
 *                  packed by sequence.  Rows that belong to no sequence are
 *                  left as they are.
 *   k_cache,       [num_blocks][num_kv_heads][block_size][head_dim] of
 *   v_cache        cache_format (fp8kv_cache_format), 16-byte aligned
 *   block_tables   as fp8kv_paged_decode
 *   seq_lens       int32 [batch] on the device
 *   q_starts       int32 [batch + 1] on the device, non-decreasing
 *   parents        int32 [num_tokens] on the device
 *   max_nodes      host-side bound of the trees' sizes, at most 256 and
 *                  max_seq_len
 *   k_scale ..     as fp8kv_rope_append: per-tensor scales (1 for a bf16 cache),
 *   v_scales       or DEVICE fp32 [num_kv_heads] arrays in their place (null
 *                  for a bf16 cache)
 *   window         as above
 *   workspace      >= fp8kv_paged_tree_workspace_size(...) bytes, 256-byte
 *                  aligned, zero-filled before first use (fp8kv_workspace_init).
 *                  Calls that share it must be ordered.  Its error word
 *                  (fp8kv_read_error) says FP8KV_ERR_INVALID_ARG for a block id
 *                  out of range (block 0 is read), for a parent that is neither
 *                  -1 nor a smaller node (it counts as -1), and for lengths or
 *                  starts out of bounds (0 <= n <= min(seq_lens[b], max_nodes),
 *                  seq_lens[b] <= max_seq_len, rows within num_tokens: the
 *                  sequence is clamped, or skipped if its rows do not exist).
 *                  FP8KV_ERR_TIMEOUT as for the other calls.
 * Queries enter an FP8 cache's score MMAs as two E4M3 numbers, which hold a
 * bf16 exactly down to 2^-15 of the row's largest element and to 2^-17 of that
 * below.  Weights are f16 (11 bits down to 2^-23 of the row's largest, steps of
 * 2^-33 of it below); over a bf16 cache two bf16 numbers.
 * Supported: head_dim in {64, 128, 256}; block_size == 16; g in {1, 2, 4, 8, 16};
 *            max_nodes <= 256; num_blocks * num_kv_heads < 2^31.  batch == 0,
 *            max_nodes == 0 or num_tokens == 0 is a no-op.
 */
fp8kv_status fp8kv_paged_tree_attention(const void* q, int64_t num_tokens, const void* k_cache, const void* v_cache,
                                        int64_t num_blocks, const int32_t* block_tables, int max_blocks_per_seq,
                                        const int32_t* seq_lens, const int32_t* q_starts, const int32_t* parents,
                                        int max_nodes, int max_seq_len, int batch, int num_q_heads, int num_kv_heads,
                                        int head_dim, int block_size, int cache_format, float k_scale, float v_scale,
                                        const float* k_scales, const float* v_scales, float sm_scale, int window,
                                        void* out, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes of fp8kv_paged_tree_attention on the CURRENT device; 0 if the
 * arguments are invalid or no device is available. */
size_t fp8kv_paged_tree_workspace_size(int batch, int max_nodes, int max_seq_len, int num_q_heads, int num_kv_heads,
                                       int head_dim, int block_size, int window);

/*
 * After a tree is checked: the accepted path's rows of K and V move behind the
 * context, in every kv head.  The path's i-th node lies at token c + accepted[i]
 * and moves to c + i (c = L - n as above); keys keep the rotation they were
 * stored with, which is that of their new place.  Rows from c + count on are
 * left as they are.
 *
 *   accepted       int32 [batch][max_accepted] on the device: node numbers in
 *                  strictly rising order, ended by the first negative entry
 *                  (or by max_accepted).  count is their number, 0 allowed.
 *   new_lens       int32 [batch] on the device, written: c + count.  Not
 *                  seq_lens itself, which the next layer's call still needs.
 *   k_cache ..     as fp8kv_paged_tree_attention (whose scales do not matter:
 *   max_seq_len    rows move as they are)
 *   workspace      256-byte aligned, at least 256 bytes, zero-filled before first
 *                  use: the error word.  FP8KV_ERR_INVALID_ARG: a block id out of
 *                  range (rows from it or to it are not moved), lengths or starts
 *                  out of bounds (clamped as above, n to at most 256), an entry
 *                  of accepted that does not rise or is not below n (it ends
 *                  the path).
 * Supported: head_dim in {64, 128, 256}; block_size == 16; batch <= 65535;
 *            num_kv_heads <= 65535; max_accepted <= 256; num_blocks * num_kv_heads
 *            < 2^31.  A page that two sequences share must hold no row that
 *            either moves.  batch == 0 or max_accepted == 0 is a no-op (new_lens is
 *            not written).
 */
fp8kv_status fp8kv_tree_commit(void* k_cache, void* v_cache, int64_t num_blocks, const int32_t* block_tables,
                               int max_blocks_per_seq, const int32_t* seq_lens, const int32_t* q_starts,
                               const int32_t* accepted, int max_accepted, int max_seq_len, int batch, int num_kv_heads,
                               int head_dim, int block_size, int cache_format, int32_t* new_lens, void* workspace,
                               size_t workspace_bytes, void* stream);

/*
 * A decode step that keeps account of attention, for caches that evict by it
 * (fp8kv_evict).  The output is that of the decode call of this cache format
 * (fp8kv_paged_decode, _per_head, _e5m2, _bf16), bit for bit.  Beside it, for every kv
 * head hk and attended token t of sequence b, with p_h(t) the probabilities that
 * sum to 1 over the attended tokens for each of the g query heads h of hk:
 *     weights[page(t)][hk][t % bs] = old(t) * decay + sum_h p_h(t)
 * in fp32; old is what was there, but 0 for the newest token, t = L - 1, whose
 * place may hold an earlier page's.  Tokens outside the window, and places past
 * the sequence, are left as they are.  Nothing depends on the order of atomics:
 * the same call gives the same bits.
 *
 *   weights        fp32 [num_blocks][num_kv_heads][block_size], 16-byte aligned.
 *                  Zero-fill what a prompt's tokens occupy before the first
 *                  call; a page in two sequences gets one of their sums.
 *   decay          finite, >= 0: 1 adds up, less forgets
 *   cache_format, k_scale, v_scale, k_scales, v_scales
 *                  as fp8kv_paged_tree_attention
 *   workspace      >= fp8kv_paged_decode_weights_workspace_size(...) bytes (the
 *                  scores of up to 64 MiB, or of one sequence), otherwise as
 *                  fp8kv_paged_decode.  The weights of a page whose block id is out
 *                  of range are not written, nor any after FP8KV_ERR_TIMEOUT.
 *   all other arguments, the shapes supported and the errors as fp8kv_paged_decode
 */
fp8kv_status fp8kv_paged_decode_weights(const void* q, const void* k_cache, const void* v_cache, int64_t num_blocks,
                                        const int32_t* block_tables, int max_blocks_per_seq, const int32_t* seq_lens,
                                        int max_seq_len, int batch, int num_q_heads, int num_kv_heads, int head_dim,
                                        int block_size, int cache_format, float k_scale, float v_scale,
                                        const float* k_scales, const float* v_scales, float sm_scale, int window,
                                        void* out, float* weights, float decay, void* workspace,
                                        size_t workspace_bytes, void* stream);

/* Workspace bytes of fp8kv_paged_decode_weights on the CURRENT device; 0 if the
 * arguments are invalid or no device is available. */
size_t fp8kv_paged_decode_weights_workspace_size(int batch, int num_q_heads, int num_kv_heads, int head_dim,
                                                 int max_seq_len, int block_size, int window);

/*
 * Cuts every sequence back to `budget` tokens by accumulated attention weight,
 * each kv head for itself (a page holds one head's rows, so heads may keep
 * different tokens).  Of sequence b's L = seq_lens[b] tokens, where L > budget, kv
 * head hk keeps the first `sinks`, the last `recent`, and of the others the
 * budget - sinks - recent of the largest weights[page(t)][hk][t % bs]; of equal
 * weights the earlier token (-0 equals 0, a NaN is below every number).  The kept
 * rows of K, V and weights move to places 0 .. budget - 1 of the sequence, in
 * their order; rows from there on are left as they are.  Where L <= budget
 * nothing moves.  Keys keep the rotation of their old position: later tokens are
 * rotated by their true positions, not by their place.
 *
 *   weights        fp32 [num_blocks][num_kv_heads][block_size], 16-byte aligned,
 *                  as fp8kv_paged_decode_weights keeps them
 *   budget         >= 1; sinks >= 0, recent >= 0, sinks + recent <= budget
 *   new_lens       int32 [batch] on the device, written: min(L, budget).  Not
 *                  seq_lens itself.
 *   kept           int32 [batch][num_kv_heads][budget] on the device, or null:
 *                  written with the places the kept tokens had, -1 past new_lens
 *   workspace      as fp8kv_tree_commit.  FP8KV_ERR_INVALID_ARG: a block id out of
 *                  range (its weights count as 0 and its rows are not moved,
 *                  nor any into its place), a length outside [0, max_seq_len]
 *                  (clamped).
 *   all other arguments as fp8kv_tree_commit
 * Supported: as fp8kv_tree_commit; max_seq_len <= 393,216.  A page must be in one
 * place of one sequence's row only.  batch == 0 is a no-op.
 */
fp8kv_status fp8kv_evict(void* k_cache, void* v_cache, float* weights, int64_t num_blocks, const int32_t* block_tables,
                         int max_blocks_per_seq, const int32_t* seq_lens, int max_seq_len, int budget, int sinks,
                         int recent, int batch, int num_kv_heads, int head_dim, int block_size, int cache_format,
                         int32_t* new_lens, int32_t* kept, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Failure-path test hooks.  No counterpart on the pages: the pages' failure
 * mode is silent (a wrong answer, no error), and these make the library's
 * answer to a stall observable.  A kernel wait that runs out writes
 * FP8KV_ERR_TIMEOUT into the workspace error word, waits (with the normal
 * limit) for the copies it has in flight, frees what it holds and returns.
 * Later calls on that workspace skip their work until it is zero-filled again
 * (fp8kv_workspace_init).  Nothing faults and nothing hangs: every wait is
 * bounded.
 *
 * fp8kv_debug_paged_decode_stall: fp8kv_paged_decode_engine with
 * FP8KV_ENGINE_CUDA_CORES (the engine whose copies run through barriers),
 * except that the K producer of CTA 0 never issues stage `stall_stage` and
 * every ring wait gives up after wait_limit_ns nanoseconds.
 *
 * fp8kv_debug_paged_prefill_stall: fp8kv_paged_prefill, except that CTA
 * (0, 0, 0) never issues the score MMAs of stage `stall_stage` and the MMA
 * waits give up after wait_limit_ns nanoseconds.
 *
 * Both: stall_stage >= 0 and 0 < wait_limit_ns <= 500,000,000, else
 * FP8KV_ERR_INVALID_ARG; all other arguments and errors as the wrapped call.
 */
fp8kv_status fp8kv_debug_paged_decode_stall(const void* q, const uint8_t* k_cache, const uint8_t* v_cache,
                                            int64_t num_blocks, const int32_t* block_tables,
                                            int max_blocks_per_seq, const int32_t* seq_lens, int max_seq_len,
                                            int batch, int num_q_heads, int num_kv_heads, int head_dim,
                                            int block_size, float k_scale, float v_scale, float sm_scale,
                                            int window, void* out, void* workspace, size_t workspace_bytes,
                                            void* stream, int stall_stage, uint64_t wait_limit_ns);

fp8kv_status fp8kv_debug_paged_prefill_stall(const void* q, int64_t num_q_tokens, const uint8_t* k_cache,
                                             const uint8_t* v_cache, int64_t num_blocks,
                                             const int32_t* block_tables, int max_blocks_per_seq,
                                             const int32_t* seq_lens, const int32_t* q_starts, int max_q_len,
                                             int max_seq_len, int batch, int num_q_heads, int num_kv_heads,
                                             int head_dim, int block_size, float k_scale, float v_scale,
                                             float sm_scale, int window, void* out, void* workspace,
                                             size_t workspace_bytes, void* stream, int stall_stage,
                                             uint64_t wait_limit_ns);

/* The same hook for fp8kv_paged_prefill_block. */
fp8kv_status fp8kv_debug_paged_prefill_block_stall(
    const void* q, int64_t num_q_tokens, const uint8_t* k_cache, const uint8_t* v_cache, const float* k_scales,
    const float* v_scales, int64_t num_blocks, const int32_t* block_tables, int max_blocks_per_seq,
    const int32_t* seq_lens, const int32_t* q_starts, int max_q_len, int max_seq_len, int batch, int num_q_heads,
    int num_kv_heads, int head_dim, int block_size, float sm_scale, int window, void* out, void* workspace,
    size_t workspace_bytes, void* stream, int stall_stage, uint64_t wait_limit_ns);

/* The same hook for fp8kv_paged_tree_attention: CTA 0 never issues the score
 * MMAs of its stage `stall_stage`. */
fp8kv_status fp8kv_debug_paged_tree_stall(const void* q, int64_t num_tokens, const void* k_cache, const void* v_cache,
                                          int64_t num_blocks, const int32_t* block_tables, int max_blocks_per_seq,
                                          const int32_t* seq_lens, const int32_t* q_starts, const int32_t* parents,
                                          int max_nodes, int max_seq_len, int batch, int num_q_heads,
                                          int num_kv_heads, int head_dim, int block_size, int cache_format,
                                          float k_scale, float v_scale, const float* k_scales, const float* v_scales,
                                          float sm_scale, int window, void* out, void* workspace,
                                          size_t workspace_bytes, void* stream, int stall_stage,
                                          uint64_t wait_limit_ns);

#ifdef __cplusplus
}
#endif

#endif /* FP8KV_H_ */
