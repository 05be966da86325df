// Attention of a tree of drafted tokens per sequence over a paged cache: the calls
// and their plan (the kernels and the reasons for them: tree_kernel.cuh).
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "trace.cuh"
#include "tree_kernel.cuh"

namespace fp8kv {
namespace tree {

// Two tiles a CTA where a unit has more than 128 rows and their accumulators fit.
int tiles_of(int max_nodes, int G, int D) { return static_cast<int64_t>(max_nodes) * G > 128 && D <= 128 ? 2 : 1; }

// Copies of the rows in a tile where they leave room: the softmax of a stage is
// then shared by so many threads a row, 32 keys each at least.
int copies_of(int max_nodes, int G, int D, bool bf16) {
    const int64_t rows = static_cast<int64_t>(max_nodes) * G;
    return rows <= 32 && D <= 128 && !bf16 ? 4 : rows <= 64 ? 2 : 1;
}

Plan make_plan(int batch, int max_nodes, int max_seq_len, int G, int Hkv, int D, int window, int sms, bool bf16) {
    Plan p;
    p.tiles = tiles_of(max_nodes, G, D);
    p.copies = copies_of(max_nodes, G, D, bf16);
    p.rows = 128 / p.copies * p.tiles;
    p.blocks = static_cast<int>((static_cast<int64_t>(max_nodes) * G + p.rows - 1) / p.rows);
    // the most pages a unit may have: a window's keys, the tree's, and a page at either end
    int64_t pages = (static_cast<int64_t>(max_seq_len) + kBS - 1) / kBS;
    if (window > 0) pages = std::min<int64_t>(pages, (static_cast<int64_t>(window) + max_nodes) / kBS + 2);
    p.ctas = cta_count((pages + kLeadPages) * std::min(batch, kMaxBatch) * Hkv * p.blocks, sms, kMinPages);
    p.ml = 256;
    p.o = p.ml + static_cast<size_t>(2 * p.ctas) * p.rows * sizeof(float2);
    p.total = p.o + static_cast<size_t>(2 * p.ctas) * p.rows * D * sizeof(float);
    return p;
}

// Shape checks shared by the size query and the call.
static fp8kv_status check_shape(int batch, int max_nodes, int max_seq_len, int num_q_heads, int num_kv_heads,
                                int head_dim, int block_size) {
    if (batch < 0 || batch > 65535 || num_kv_heads < 1 || num_kv_heads > 65535 || num_q_heads < 1 ||
        num_q_heads % num_kv_heads != 0 || max_seq_len < 0 || max_nodes < 0 || max_nodes > max_seq_len)
        return FP8KV_ERR_INVALID_ARG;
    const int G = num_q_heads / num_kv_heads;
    if (!(head_dim == 64 || head_dim == 128 || head_dim == 256) || block_size != kBS ||
        !(G == 1 || G == 2 || G == 4 || G == 8 || G == 16) || max_nodes > kMaxNodes)
        return FP8KV_ERR_UNSUPPORTED;
    return FP8KV_OK;
}

static fp8kv_status tree_impl(const void* q, int64_t num_tokens, const void* k_cache, const void* v_cache,
                              int64_t num_blocks, const int32_t* block_tables, int max_blocks_per_seq,
                              const int32_t* seq_lens, const int32_t* q_starts, const int32_t* parents, int max_nodes,
                              int max_seq_len, int batch, int num_q_heads, int num_kv_heads, int head_dim,
                              int block_size, int cache_format, float k_scale, float v_scale, const float* k_scales,
                              const float* v_scales, float sm_scale, int window, void* out, void* workspace,
                              size_t workspace_bytes, void* stream, int stall_stage, uint64_t wait_ns) {
    auto a16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
    auto a4 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; };
    const fp8kv_status sh = check_shape(batch, max_nodes, max_seq_len, num_q_heads, num_kv_heads, head_dim, block_size);
    if (sh != FP8KV_OK) return sh;
    if (num_blocks < 1 || max_blocks_per_seq < 0 || num_tokens < 0 ||
        (cache_format != FP8KV_CACHE_E4M3 && cache_format != FP8KV_CACHE_E5M2 && cache_format != FP8KV_CACHE_BF16))
        return FP8KV_ERR_INVALID_ARG;
    if (!std::isfinite(k_scale) || !(k_scale > 0) || !std::isfinite(v_scale) || !(v_scale > 0) || !std::isfinite(sm_scale))
        return FP8KV_ERR_INVALID_ARG;
    if (cache_format == FP8KV_CACHE_BF16 && (k_scales || v_scales || k_scale != 1.f || v_scale != 1.f))
        return FP8KV_ERR_INVALID_ARG;
    if (num_blocks >= (INT64_C(1) << 31) || num_blocks * num_kv_heads >= (INT64_C(1) << 31)) return FP8KV_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(max_blocks_per_seq) * block_size < max_seq_len) return FP8KV_ERR_INVALID_ARG;
    if (batch == 0 || max_nodes == 0 || num_tokens == 0) return FP8KV_OK;
    if (!q || !k_cache || !v_cache || !block_tables || !seq_lens || !q_starts || !parents || !out)
        return FP8KV_ERR_INVALID_ARG;
    if (!a16(q) || !a16(k_cache) || !a16(v_cache) || !a16(out)) return FP8KV_ERR_INVALID_ARG;
    if (!a4(block_tables) || !a4(seq_lens) || !a4(q_starts) || !a4(parents) || !a4(k_scales) || !a4(v_scales))
        return FP8KV_ERR_INVALID_ARG;
    if ((k_scales == nullptr) != (v_scales == nullptr)) return FP8KV_ERR_INVALID_ARG;
    int sms = 0;
    if (device_sms(&sms) != 0) return FP8KV_ERR_CUDA;
    const int G = num_q_heads / num_kv_heads, win = window > 0 ? window : 0;
    const bool bf16 = cache_format == FP8KV_CACHE_BF16;
    const size_t need = make_plan(batch, max_nodes, max_seq_len, G, num_kv_heads, head_dim, win, sms, bf16).total;
    if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return FP8KV_ERR_WORKSPACE;
    // units of one launch, and the pages of one sequence's units, are counted in 31 bits
    if (((static_cast<int64_t>(max_seq_len) + kBS - 1) / kBS + kLeadPages) * num_kv_heads * (max_nodes * G / 32 + 1) >= (INT64_C(1) << 31))
        return FP8KV_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(std::min(batch, kMaxBatch)) * num_kv_heads * (max_nodes * G / 128 + 1) >= (INT64_C(1) << 31))
        return FP8KV_ERR_UNSUPPORTED;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    // Batches above kMaxBatch sequences run as consecutive launches, reusing the workspace.
    for (int b0 = 0; b0 < batch; b0 += kMaxBatch) {
        const int nb = std::min(kMaxBatch, batch - b0);
        const Plan p = make_plan(nb, max_nodes, max_seq_len, G, num_kv_heads, head_dim, win, sms, bf16);
        Args a;
        a.q = static_cast<const uint16_t*>(q);
        a.k_cache = static_cast<const uint8_t*>(k_cache);
        a.v_cache = static_cast<const uint8_t*>(v_cache);
        a.block_tables = block_tables + static_cast<int64_t>(b0) * max_blocks_per_seq;
        a.seq_lens = seq_lens + b0;
        a.q_starts = q_starts + b0;
        a.parents = parents;
        a.out = static_cast<uint16_t*>(out);
        a.err = reinterpret_cast<uint32_t*>(ws);
        a.part_ml = reinterpret_cast<float2*>(ws + p.ml);
        a.part_o = reinterpret_cast<float4*>(ws + p.o);
        a.k_scales = k_scales;
        a.v_scales = v_scales;
        a.num_blocks = num_blocks;
        a.num_tokens = num_tokens;
        a.k_scale = k_scale;
        a.v_scale = v_scale;
        a.sm_scale = sm_scale;
        a.max_blocks_per_seq = max_blocks_per_seq;
        a.max_seq_len = max_seq_len;
        a.max_nodes = max_nodes;
        a.batch = nb;
        a.num_q_heads = num_q_heads;
        a.num_kv_heads = num_kv_heads;
        a.log2_group = 0;
        while ((1 << a.log2_group) < G) ++a.log2_group;
        a.window = win;
        a.max_ctas = p.ctas;
        a.wait_ns = wait_ns;
        a.stall_stage = stall_stage;
        cudaStream_t s = static_cast<cudaStream_t>(stream);
        const cudaError_t e = cache_format == FP8KV_CACHE_BF16   ? launch_bf16(head_dim, a, p, s)
                              : cache_format == FP8KV_CACHE_E5M2 ? launch_e5m2(head_dim, a, p, s)
                                                                 : launch<1, false>(head_dim, a, p, s);
        if (e != cudaSuccess) return FP8KV_ERR_CUDA;
    }
    return FP8KV_OK;
}

}  // namespace tree
}  // namespace fp8kv

extern "C" size_t fp8kv_paged_tree_workspace_size(int batch, int max_nodes, int max_seq_len, int num_q_heads,
                                                  int num_kv_heads, int head_dim, int block_size, int window) {
    using namespace fp8kv::tree;
    if (check_shape(batch, max_nodes, max_seq_len, num_q_heads, num_kv_heads, head_dim, block_size) != FP8KV_OK) return 0;
    int sms = 0;
    if (fp8kv::device_sms(&sms) != 0) return 0;
    size_t most = 0;   // over the cache formats
    for (const bool bf16 : {false, true})
        most = std::max(most, make_plan(batch, max_nodes, max_seq_len, num_q_heads / num_kv_heads, num_kv_heads, head_dim,
                                        window > 0 ? window : 0, sms, bf16).total);
    return most;
}

extern "C" fp8kv_status fp8kv_paged_tree_attention(
    const void* q, int64_t num_tokens, const void* k_cache, const void* v_cache, int64_t num_blocks,
    const int32_t* block_tables, int max_blocks_per_seq, const int32_t* seq_lens, const int32_t* q_starts,
    const int32_t* parents, int max_nodes, int max_seq_len, int batch, int num_q_heads, int num_kv_heads, int head_dim,
    int block_size, int cache_format, float k_scale, float v_scale, const float* k_scales, const float* v_scales,
    float sm_scale, int window, void* out, void* workspace, size_t workspace_bytes, void* stream) {
    FP8KV_TRACE("fp8kv_paged_tree_attention");
    return fp8kv::tree::tree_impl(q, num_tokens, k_cache, v_cache, num_blocks, block_tables, max_blocks_per_seq, seq_lens,
                                  q_starts, parents, max_nodes, max_seq_len, batch, num_q_heads, num_kv_heads, head_dim,
                                  block_size, cache_format, k_scale, v_scale, k_scales, v_scales, sm_scale, window, out,
                                  workspace, workspace_bytes, stream, -1, fp8kv::tree::kWaitNs);
}

extern "C" fp8kv_status fp8kv_debug_paged_tree_stall(
    const void* q, int64_t num_tokens, const void* k_cache, const void* v_cache, int64_t num_blocks,
    const int32_t* block_tables, int max_blocks_per_seq, const int32_t* seq_lens, const int32_t* q_starts,
    const int32_t* parents, int max_nodes, int max_seq_len, int batch, int num_q_heads, int num_kv_heads, int head_dim,
    int block_size, int cache_format, float k_scale, float v_scale, const float* k_scales, const float* v_scales,
    float sm_scale, int window, void* out, void* workspace, size_t workspace_bytes, void* stream, int stall_stage,
    uint64_t wait_limit_ns) {
    FP8KV_TRACE("fp8kv_debug_paged_tree_stall");
    if (stall_stage < 0 || wait_limit_ns == 0 || wait_limit_ns > fp8kv::tree::kWaitNs) return FP8KV_ERR_INVALID_ARG;
    return fp8kv::tree::tree_impl(q, num_tokens, k_cache, v_cache, num_blocks, block_tables, max_blocks_per_seq, seq_lens,
                                  q_starts, parents, max_nodes, max_seq_len, batch, num_q_heads, num_kv_heads, head_dim,
                                  block_size, cache_format, k_scale, v_scale, k_scales, v_scales, sm_scale, window, out,
                                  workspace, workspace_bytes, stream, stall_stage, wait_limit_ns);
}
