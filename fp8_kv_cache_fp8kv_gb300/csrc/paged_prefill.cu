// Chunked-prefill attention over the paged fp8 (E4M3) KV cache, for sm_103a.
//
// What it computes: the new query tokens of each sequence (the last q_len of
// its seq_len tokens, already appended to the cache) attend causally over the
// sequence's cached keys, optionally within a sliding window: query position
// p reads keys [max(0, p + 1 - window), p].  This is the prefill pass that
// reads the same fp8 cache as decode (gpusmith.com, "FP8 KV Cache
// Quantization: Capacity Gains and Accuracy Risk", "Attention backend
// interactions"; phantomic12 vLLM-blog summary, "ACCURACY AT LONG CONTEXT":
// the P.V contraction runs over the context, so partial sums live in real
// FP32 registers).
//
// How: a unit is (tile of 128 query rows, kv head, sequence); a query row is
// a (token, query head) pair of the kv head's group.  Three kernels on the
// 5th-generation tensor cores (tcgen05.mma from swizzled f16 tiles in shared
// memory, S in tensor memory, one row per thread (TMEM lane) for the online
// softmax):
//  * paged_prefill_ws_kernel (d = 64 and 128, chunks of two or more tiles):
//    two tiles per CTA, 128-key stages, and warp roles -- converter warps,
//    one MMA-issuing thread, a softmax warpgroup per tile -- that overlap
//    through mbarriers.  P goes to tensor memory as the value MMA's A
//    operand, and the tensor cores carry O across stages in FP32;
//  * paged_prefill_ws1_kernel (d = 256): one tile per CTA with the same kind
//    of roles; each stage's P.V tile, computed in fresh FP32 accumulators, is
//    folded into an FP32 accumulator in tensor memory (O = O * alpha + tile,
//    IEEE FMA);
//  * paged_prefill_tc_kernel (single-tile chunks at d = 64 and 128): one
//    tile per CTA, its four warps taking each stage's steps in turn, the
//    fold into registers.
// See the comments above them.  When the units are too few to fill the GPU,
// each unit's key range is split over several CTAs whose FP32 partials (row
// maximum, row sum, unnormalised output) a second kernel merges (split plan:
// prefill_plan.h).
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "fp8kv.h"
#include "trace.cuh"
#include "prefill_kernels.cuh"

namespace fp8kv {
namespace prefill {

// Split plan: the tiles a sequence's chunk may need, how many CTAs share each
// unit's key range (choose_splits in prefill_plan.h) and the workspace layout.
struct Plan {
    int tiles = 0;
    int splits = 1;
    size_t ml = kHeader;   // offset of the (m, l) partials
    size_t o = kHeader;    // offset of the output partials
    size_t total = kHeader;
};

inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Query rows per tile (one TMEM lane each).
inline int rows_per_tile(int) { return kRowsTC; }

// Query tiles of 128 rows per (sequence, kv head) for a chunk of max_q_len.
inline int tiles_of(int max_q_len, int G) {
    return static_cast<int>((static_cast<int64_t>(max_q_len) * G + kRowsTC - 1) / kRowsTC);
}

// Which kernel runs: 2, the warp-specialised one-tile kernel, at d = 256;
// 1, the warp-specialised one with two tiles per CTA, at d = 64 and 128 when
// a sequence's chunk spans at least two tiles (at d = 64 it measured 617
// against 442 TFLOP/s for the one-tile kernel at 2048-token chunks); else 0,
// paged_prefill_tc_kernel, one tile per CTA.
inline int kernel_kind(int D, int tiles) {
    if (D == 256) return kKindWs1;
    return tiles >= 2 ? kKindWs : kKindTc;
}
// The same for a block-scaled cache: the two-tile kernel, or the one-tile
// kernel of paged_prefill_block.cu.
inline int block_kernel_kind(int D, int tiles) { return D == 256 || tiles == 1 ? kKindOne : kKindWs; }
inline int tiles_per_cta(int kind) { return kind == kKindWs ? ws::kTiles : 1; }

Plan make_plan(int batch, int max_q_len, int max_seq_len, int G, int Hkv, int D, int window, int sms, int per_sm,
               int kind) {
    Plan pl;
    const int rows = rows_per_tile(D);
    pl.tiles = tiles_of(max_q_len, G);
    const int tpc = tiles_per_cta(kind);
    const int64_t units = static_cast<int64_t>(pl.tiles) * Hkv * batch;
    const int64_t ctas = static_cast<int64_t>((pl.tiles + tpc - 1) / tpc) * Hkv * batch;
    int64_t pages = (static_cast<int64_t>(max_seq_len) + kBS - 1) / kBS;
    if (window > 0) pages = std::min<int64_t>(pages, (static_cast<int64_t>(window) + rows * tpc) / kBS + 2);
    pl.splits = choose_splits(ctas, pages, static_cast<int64_t>(sms) * per_sm);
    if (pl.splits > 1) {
        const size_t slots = static_cast<size_t>(units) * pl.splits * rows;
        pl.ml = kHeader;
        pl.o = pl.ml + align256(slots * sizeof(float2));
        pl.total = pl.o + align256(slots * D * sizeof(float));
    }
    return pl;
}

// The prefill kernel of a kind (kernel_kind) for (D, G), its dynamic shared
// memory and its threads.
template <int D, int G>
void kernel_of(int kind, void (**fn)(const Args), size_t* smem, int* threads) {
    if constexpr (D == 64 || D == 128) {
        if (kind == kKindWs) {
            *fn = paged_prefill_ws_kernel<D, G, false>;
            *smem = static_cast<size_t>(WsGeo<D>::SMEM) + 1024;
            *threads = ws::kThreads;
            return;
        }
    }
    if constexpr (D == 256) {   // kKindWs1 always
        *fn = paged_prefill_ws1_kernel<D, G>;
        *smem = static_cast<size_t>(Ws1Geo<D>::SMEM) + 1024;
        *threads = ws1::kThreads;
    } else {
        *fn = paged_prefill_tc_kernel<D, G>;
        *smem = static_cast<size_t>(TcGeo<D>::SMEM) + 1024;
        *threads = kThreads;
    }
}

template <int D>
bool kernel_of_g(int G, int kind, void (**fn)(const Args), size_t* smem, int* threads) {
    switch (G) {
        case 1: kernel_of<D, 1>(kind, fn, smem, threads); return true;
        case 2: kernel_of<D, 2>(kind, fn, smem, threads); return true;
        case 4: kernel_of<D, 4>(kind, fn, smem, threads); return true;
        case 8: kernel_of<D, 8>(kind, fn, smem, threads); return true;
        case 16: kernel_of<D, 16>(kind, fn, smem, threads); return true;
        default: return false;
    }
}

// Resident CTAs per SM of the prefill kernel for (D, G, kind) on the current
// device (the occupancy calculator, with the kernel's shared-memory opt-in
// applied); 0 on failure.  Cached per device.
int resident_per_sm(int D, int G, int kind) {
    static std::atomic<int> cache[3][3][5][64] = {};
    const int di = D == 64 ? 0 : (D == 128 ? 1 : 2);
    const int gi = G == 1 ? 0 : (G == 2 ? 1 : (G == 4 ? 2 : (G == 8 ? 3 : 4)));
    const int wi = kind;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (dev >= 0 && dev < 64) {
        const int c = cache[wi][di][gi][dev].load(std::memory_order_relaxed);
        if (c > 0) return c;
    }
    void (*fn)(const Args) = nullptr;
    size_t smem = 0;
    int threads = 0;
    const bool ok = D == 64 ? kernel_of_g<64>(G, kind, &fn, &smem, &threads)
                            : (D == 128 ? kernel_of_g<128>(G, kind, &fn, &smem, &threads)
                                        : kernel_of_g<256>(G, kind, &fn, &smem, &threads));
    if (!ok) return 0;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
        return 0;
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, fn, threads, smem) != cudaSuccess || n < 1) return 0;
    if (dev >= 0 && dev < 64) cache[wi][di][gi][dev].store(n, std::memory_order_relaxed);
    return n;
}

template <int D, int G>
cudaError_t launch(const Args& a, int batch, cudaStream_t s) {
    const int kind = kernel_kind(D, a.tiles);
    void (*kernel)(const Args) = nullptr;
    size_t smem = 0;
    int threads = 0;
    kernel_of<D, G>(kind, &kernel, &smem, &threads);
    static std::atomic<uint64_t> done_mask[3] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
    if (bit == 0 || !(done_mask[kind].load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
        done_mask[kind].fetch_or(bit, std::memory_order_release);
    }
    // Both grids may start before the previous work on the stream ends; each
    // waits (griddepcontrol.wait) before touching what that work wrote.
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    const int tpc = tiles_per_cta(kind);
    const int ctas_x = (a.tiles + tpc - 1) / tpc;
    cfg.gridDim = dim3(static_cast<unsigned>(ctas_x * a.splits), static_cast<unsigned>(a.num_kv_heads),
                       static_cast<unsigned>(batch));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kernel, a);
    if (e != cudaSuccess || a.splits == 1) return e;
    cfg.gridDim = dim3(static_cast<unsigned>(a.tiles * (a.rows / 8)), static_cast<unsigned>(a.num_kv_heads),
                       static_cast<unsigned>(batch));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, prefill_merge_kernel<D, G>, a);
}

template <int D>
cudaError_t launch_g(int G, const Args& a, int batch, cudaStream_t s) {
    switch (G) {
        case 1: return launch<D, 1>(a, batch, s);
        case 2: return launch<D, 2>(a, batch, s);
        case 4: return launch<D, 4>(a, batch, s);
        case 8: return launch<D, 8>(a, batch, s);
        case 16: return launch<D, 16>(a, batch, s);
        default: return cudaErrorInvalidValue;
    }
}

// Shape checks shared by the size query and the call.
fp8kv_status check_shape(int batch, int max_q_len, int max_seq_len, int num_q_heads, int num_kv_heads,
                         int head_dim, int block_size) {
    if (batch < 0 || batch > 65535 || num_kv_heads < 1 || num_kv_heads > 65535 || num_q_heads < 1 ||
        num_q_heads % num_kv_heads != 0 || max_seq_len < 0 || max_q_len < 0 || max_q_len > max_seq_len)
        return FP8KV_ERR_INVALID_ARG;
    const int G = num_q_heads / num_kv_heads;
    if (!(head_dim == 64 || head_dim == 128 || head_dim == 256) || block_size != kBS ||
        !(G == 1 || G == 2 || G == 4 || G == 8 || G == 16))
        return FP8KV_ERR_UNSUPPORTED;
    const int64_t tiles = (static_cast<int64_t>(max_q_len) * G + kRowsTC - 1) / kRowsTC;
    if (tiles * kMaxSplits > INT32_MAX) return FP8KV_ERR_UNSUPPORTED;
    return FP8KV_OK;
}

}  // namespace prefill
}  // namespace fp8kv

extern "C" size_t fp8kv_paged_prefill_workspace_size(int batch, int max_q_len, int max_seq_len, int num_q_heads,
                                                     int num_kv_heads, int head_dim, int block_size, int window) {
    using namespace fp8kv::prefill;
    if (check_shape(batch, max_q_len, max_seq_len, num_q_heads, num_kv_heads, head_dim, block_size) != FP8KV_OK)
        return 0;
    int sms = 0;
    if (fp8kv::device_sms(&sms) != 0) return 0;
    const int G = num_q_heads / num_kv_heads;
    const int per_sm = resident_per_sm(head_dim, G, kernel_kind(head_dim, tiles_of(max_q_len, G)));
    if (per_sm < 1) return 0;
    const int win = window > 0 ? window : 0, tiles = tiles_of(max_q_len, G);
    // enough for the block-scaled call too (its kernels and plan differ; one CTA per SM)
    return std::max(make_plan(batch, max_q_len, max_seq_len, G, num_kv_heads, head_dim, win, sms, per_sm,
                              kernel_kind(head_dim, tiles)).total,
                    make_plan(batch, max_q_len, max_seq_len, G, num_kv_heads, head_dim, win, sms, 1,
                              block_kernel_kind(head_dim, tiles)).total);
}

namespace {

fp8kv_status prefill_impl(const void* q, int64_t num_q_tokens, const uint8_t* k_cache, const uint8_t* v_cache,
                          int64_t num_blocks, const int32_t* block_tables, int max_blocks_per_seq,
                          const int32_t* seq_lens, const int32_t* q_starts, int max_q_len, int max_seq_len, int batch,
                          int num_q_heads, int num_kv_heads, int head_dim, int block_size, float k_scale,
                          float v_scale, float sm_scale, int window, void* out, void* workspace,
                          size_t workspace_bytes, void* stream, int stall_stage, uint64_t wait_ns,
                          const float* k_page_scales = nullptr, const float* v_page_scales = nullptr) {
    using namespace fp8kv::prefill;
    auto a16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
    const fp8kv_status sh = check_shape(batch, max_q_len, max_seq_len, num_q_heads, num_kv_heads, head_dim,
                                        block_size);
    if (sh != FP8KV_OK) return sh;
    if (num_blocks < 1 || max_blocks_per_seq < 0 || num_q_tokens < 0) return FP8KV_ERR_INVALID_ARG;
    if (!std::isfinite(k_scale) || !(k_scale > 0) || !std::isfinite(v_scale) || !(v_scale > 0) ||
        !std::isfinite(sm_scale))
        return FP8KV_ERR_INVALID_ARG;
    if (num_blocks >= (INT64_C(1) << 31) || num_blocks * num_kv_heads >= (INT64_C(1) << 31))
        return FP8KV_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(max_blocks_per_seq) * block_size < max_seq_len) return FP8KV_ERR_INVALID_ARG;
    if (batch == 0 || max_q_len == 0 || num_q_tokens == 0) return FP8KV_OK;
    if (!q || !k_cache || !v_cache || !block_tables || !seq_lens || !q_starts || !out) return FP8KV_ERR_INVALID_ARG;
    if (!a16(q) || !a16(k_cache) || !a16(v_cache) || !a16(out)) return FP8KV_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(block_tables) & 3u) || (reinterpret_cast<uintptr_t>(seq_lens) & 3u) ||
        (reinterpret_cast<uintptr_t>(q_starts) & 3u))
        return FP8KV_ERR_INVALID_ARG;
    int sms = 0;
    if (fp8kv::device_sms(&sms) != 0) return FP8KV_ERR_CUDA;
    const int G = num_q_heads / num_kv_heads;
    const bool block = k_page_scales != nullptr;
    const int tiles = tiles_of(max_q_len, G);
    const int kind = block ? block_kernel_kind(head_dim, tiles) : kernel_kind(head_dim, tiles);
    const int per_sm = block ? 1 : resident_per_sm(head_dim, G, kind);
    if (per_sm < 1) return FP8KV_ERR_CUDA;
    const Plan pl = make_plan(batch, max_q_len, max_seq_len, G, num_kv_heads, head_dim, window > 0 ? window : 0, sms,
                              per_sm, kind);
    if (!workspace || workspace_bytes < pl.total || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return FP8KV_ERR_WORKSPACE;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    Args a;
    a.q = static_cast<const uint16_t*>(q);
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.block_tables = block_tables;
    a.seq_lens = seq_lens;
    a.q_starts = q_starts;
    a.out = static_cast<uint16_t*>(out);
    a.err = reinterpret_cast<uint32_t*>(ws);
    a.part_ml = reinterpret_cast<float2*>(ws + pl.ml);
    a.part_o = reinterpret_cast<float*>(ws + pl.o);
    a.num_blocks = num_blocks;
    a.num_q_tokens = num_q_tokens;
    a.max_blocks_per_seq = max_blocks_per_seq;
    a.max_seq_len = max_seq_len;
    a.max_q_len = max_q_len;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = num_kv_heads;
    a.tiles = pl.tiles;
    a.rows = rows_per_tile(head_dim);
    a.splits = pl.splits;
    a.window = window > 0 ? window : 0;
    a.score_scale = sm_scale * k_scale * kLog2e;
    a.v_scale = v_scale;
    a.k_page_scales = k_page_scales;
    a.v_page_scales = v_page_scales;
    a.wait_ns = wait_ns;
    a.stall_stage = stall_stage;
    a.log2_group = 0;
    while ((1 << a.log2_group) < G) ++a.log2_group;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (block) e = launch_block(head_dim, G, kind, a, batch, s);
    else switch (head_dim) {
        case 64: e = launch_g<64>(G, a, batch, s); break;
        case 128: e = launch_g<128>(G, a, batch, s); break;
        default: e = launch_g<256>(G, a, batch, s); break;
    }
    return e == cudaSuccess ? FP8KV_OK : FP8KV_ERR_CUDA;
}

}  // namespace

extern "C" fp8kv_status fp8kv_paged_prefill(const void* q, int64_t num_q_tokens, const uint8_t* k_cache,
                                            const uint8_t* v_cache, int64_t num_blocks, const int32_t* block_tables,
                                            int max_blocks_per_seq, const int32_t* seq_lens, const int32_t* q_starts,
                                            int max_q_len, int max_seq_len, int batch, int num_q_heads,
                                            int num_kv_heads, int head_dim, int block_size, float k_scale,
                                            float v_scale, float sm_scale, int window, void* out, void* workspace,
                                            size_t workspace_bytes, void* stream) {
    FP8KV_TRACE("fp8kv_paged_prefill");
    return prefill_impl(q, num_q_tokens, k_cache, v_cache, num_blocks, block_tables, max_blocks_per_seq, seq_lens,
                        q_starts, max_q_len, max_seq_len, batch, num_q_heads, num_kv_heads, head_dim, block_size,
                        k_scale, v_scale, sm_scale, window, out, workspace, workspace_bytes, stream, -1,
                        fp8kv::prefill::tcg::kWaitNs);
}

namespace {

fp8kv_status prefill_block_impl(const void* q, int64_t num_q_tokens, const uint8_t* k_cache, const uint8_t* v_cache,
                                const float* k_scales, const float* v_scales, int64_t num_blocks,
                                const int32_t* block_tables, int max_blocks_per_seq, const int32_t* seq_lens,
                                const int32_t* q_starts, int max_q_len, int max_seq_len, int batch, int num_q_heads,
                                int num_kv_heads, int head_dim, int block_size, float sm_scale, int window, void* out,
                                void* workspace, size_t workspace_bytes, void* stream, int stall_stage,
                                uint64_t wait_ns) {
    if (batch > 0 && max_q_len > 0 && num_q_tokens > 0 &&
        (!k_scales || !v_scales || (reinterpret_cast<uintptr_t>(k_scales) & 3u) ||
         (reinterpret_cast<uintptr_t>(v_scales) & 3u)))
        return FP8KV_ERR_INVALID_ARG;
    return prefill_impl(q, num_q_tokens, k_cache, v_cache, num_blocks, block_tables, max_blocks_per_seq, seq_lens,
                        q_starts, max_q_len, max_seq_len, batch, num_q_heads, num_kv_heads, head_dim, block_size, 1.f,
                        1.f, sm_scale, window, out, workspace, workspace_bytes, stream, stall_stage, wait_ns, k_scales,
                        v_scales);
}

}  // namespace

extern "C" fp8kv_status fp8kv_paged_prefill_block(const void* q, int64_t num_q_tokens, const uint8_t* k_cache,
                                                  const uint8_t* v_cache, const float* k_scales,
                                                  const float* v_scales, int64_t num_blocks,
                                                  const int32_t* block_tables, int max_blocks_per_seq,
                                                  const int32_t* seq_lens, const int32_t* q_starts, int max_q_len,
                                                  int max_seq_len, int batch, int num_q_heads, int num_kv_heads,
                                                  int head_dim, int block_size, float sm_scale, int window, void* out,
                                                  void* workspace, size_t workspace_bytes, void* stream) {
    FP8KV_TRACE("fp8kv_paged_prefill_block");
    return prefill_block_impl(q, num_q_tokens, k_cache, v_cache, k_scales, v_scales, num_blocks, block_tables,
                              max_blocks_per_seq, seq_lens, q_starts, max_q_len, max_seq_len, batch, num_q_heads,
                              num_kv_heads, head_dim, block_size, sm_scale, window, out, workspace, workspace_bytes,
                              stream, -1, fp8kv::prefill::tcg::kWaitNs);
}

extern "C" fp8kv_status fp8kv_debug_paged_prefill_stall(
    const void* q, int64_t num_q_tokens, const uint8_t* k_cache, const uint8_t* v_cache, int64_t num_blocks,
    const int32_t* block_tables, int max_blocks_per_seq, const int32_t* seq_lens, const int32_t* q_starts,
    int max_q_len, int max_seq_len, int batch, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
    float k_scale, float v_scale, float sm_scale, int window, void* out, void* workspace, size_t workspace_bytes,
    void* stream, int stall_stage, uint64_t wait_limit_ns) {
    FP8KV_TRACE("fp8kv_debug_paged_prefill_stall");
    if (stall_stage < 0 || wait_limit_ns == 0 || wait_limit_ns > fp8kv::prefill::tcg::kWaitNs)
        return FP8KV_ERR_INVALID_ARG;
    return prefill_impl(q, num_q_tokens, k_cache, v_cache, num_blocks, block_tables, max_blocks_per_seq, seq_lens,
                        q_starts, max_q_len, max_seq_len, batch, num_q_heads, num_kv_heads, head_dim, block_size,
                        k_scale, v_scale, sm_scale, window, out, workspace, workspace_bytes, stream, stall_stage,
                        wait_limit_ns);
}

extern "C" fp8kv_status fp8kv_debug_paged_prefill_block_stall(
    const void* q, int64_t num_q_tokens, const uint8_t* k_cache, const uint8_t* v_cache, const float* k_scales,
    const float* v_scales, int64_t num_blocks, const int32_t* block_tables, int max_blocks_per_seq,
    const int32_t* seq_lens, const int32_t* q_starts, int max_q_len, int max_seq_len, int batch, int num_q_heads,
    int num_kv_heads, int head_dim, int block_size, float sm_scale, int window, void* out, void* workspace,
    size_t workspace_bytes, void* stream, int stall_stage, uint64_t wait_limit_ns) {
    FP8KV_TRACE("fp8kv_debug_paged_prefill_block_stall");
    if (stall_stage < 0 || wait_limit_ns == 0 || wait_limit_ns > fp8kv::prefill::tcg::kWaitNs)
        return FP8KV_ERR_INVALID_ARG;
    return prefill_block_impl(q, num_q_tokens, k_cache, v_cache, k_scales, v_scales, num_blocks, block_tables,
                              max_blocks_per_seq, seq_lens, q_starts, max_q_len, max_seq_len, batch, num_q_heads,
                              num_kv_heads, head_dim, block_size, sm_scale, window, out, workspace, workspace_bytes,
                              stream, stall_stage, wait_limit_ns);
}
