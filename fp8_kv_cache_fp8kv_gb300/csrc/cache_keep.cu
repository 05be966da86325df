// Rows kept in a paged cache and moved to the front, in place and in their order:
// the accepted path of a checked tree of drafted tokens (fp8kv_tree_commit), and
// the tokens of the largest accumulated attention weight (fp8kv_evict).
//
// A unit is one (sequence, kv head): its rows lie in its own pages, so units never
// meet.  Kept row i comes from place s_i, s rising, and goes to place i <= s_i.  In
// place this is safe in rounds: a round reads a run of kept rows, waits until all
// of it is read, and writes them.  What a later round reads, s_j with j past the
// round, lies at or behind j, where no earlier round has written.
//
// Eviction chooses by a radix selection on the weights' bits (11, 11 and 10 of
// them): a pass counts the digits among the candidates and fixes one digit of the
// smallest kept weight.  A cluster of CTAs shares a unit: each holds its part of
// the weights in shared memory as sortable keys, read from HBM once, and the
// CTAs' counts and the kept tokens' places meet through distributed shared
// memory, so nothing goes back to global memory but what the call writes.
//
// Measured (GB300, graph of calls, 8 heads of 128, E4M3): 8 x 20K tokens to 4096
// 49.6 us, 15 of them the selection (4 CTAs a unit) and 30 the 134 MB of rows moved
// (4.5 TB/s); 1 x 128K to 8191 37 us (16 CTAs a unit, selection 17, rows 12); 16 x
// 1100 to 1024 24.1 us (2 CTAs a unit, selection 12, rows 9).  The selection is a
// chain of about ten meetings of a cluster, a microsecond each.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "fp8kv.h"
#include "ptx.cuh"
#include "trace.cuh"

namespace fp8kv {

int device_sms(int* sms);  // SM count of the current device (paged_decode.cu)

namespace keep {

namespace cg = cooperative_groups;

constexpr int kBS = 16;
constexpr int kMaxPath = 256;

struct Args {
    uint8_t* k_cache;
    uint8_t* v_cache;
    float* weights;               // evict
    const int32_t* block_tables;
    const int32_t* seq_lens;
    const int32_t* q_starts;      // commit
    const int32_t* accepted;
    int32_t* new_lens;
    int32_t* kept;
    uint32_t* err;
    int64_t num_blocks;
    int max_blocks_per_seq, max_seq_len, batch, num_kv_heads, max_accepted;
    int budget, sinks, recent;
    int per_cta;                  // evict: tokens a CTA of the cluster holds
};

__device__ __forceinline__ void report(uint32_t* err, uint32_t code) { atomicCAS(err, 0u, code); }

// Block of the page that holds token t, or -1 (reported).
__device__ __forceinline__ int block_of(const Args& a, const int32_t* row, int t) {
    const int id = ld_input(row + t / kBS);
    if (id < 0 || id >= a.num_blocks) {
        report(a.err, FP8KV_ERR_INVALID_ARG);
        return -1;
    }
    return id;
}

// Row t % 16 of kv head hk in a block, in rows.
__device__ __forceinline__ int64_t row_at(const Args& a, int block, int hk, int t) {
    return (static_cast<int64_t>(block) * a.num_kv_heads + hk) * kBS + t % kBS;
}

// ---------------------------------------------------------------- commit
//
// A CTA takes one (sequence, kv head).  A path is at most 256 rows, a few KB: one
// round of rows in registers, or a few.  What bounds it is a launch and a chain
// of three dependent reads (lengths and path, block ids, rows).
template <int RB>
__global__ void __launch_bounds__(256) commit_kernel(const Args a) {
    constexpr int CPR = RB / 16;             // 16-byte chunks per row
    constexpr int PER = 4;                   // chunks a thread holds in a round
    __shared__ int path[kMaxPath];
    __shared__ int count_sh;
    const int tid = threadIdx.x, hk = blockIdx.x, b = blockIdx.y;
    griddep_wait();
    griddep_launch_dependents();
    const int L_in = ld_input(a.seq_lens + b), n_in = ld_input(a.q_starts + b + 1) - ld_input(a.q_starts + b);
    const int L = L_in < 0 ? 0 : min(L_in, a.max_seq_len);
    const int n = n_in < 0 ? 0 : min(min(n_in, L), kMaxPath);
    const int ctx = L - n;
    const int mine = tid < a.max_accepted ? ld_input(a.accepted + static_cast<int64_t>(b) * a.max_accepted + tid) : -1;
    path[tid] = mine;
    if (tid == 0) count_sh = a.max_accepted;
    __syncthreads();
    // the path ends before its first entry that is negative, does not rise, or is past the tree
    if (mine < 0 || mine >= n || (tid > 0 && mine <= path[tid - 1])) atomicMin(&count_sh, tid);
    __syncthreads();
    const int count = count_sh;
    if (hk == 0 && tid == 0) {
        a.new_lens[b] = ctx + count;
        if (L != L_in || n != n_in) report(a.err, FP8KV_ERR_INVALID_ARG);
    }
    if (hk == 0 && tid == count && mine >= 0) report(a.err, FP8KV_ERR_INVALID_ARG);   // not ended by a negative entry
    const int32_t* row = a.block_tables + static_cast<int64_t>(b) * a.max_blocks_per_seq;
    const int chunks = count * CPR * 2;
    for (int c0 = 0; c0 < chunks; c0 += 256 * PER) {
        uint4 x[PER];
        uint8_t* to[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            // (K and V of a row beside each other, so that a round is a run of rows)
            const int c = c0 + j * 256 + tid, i = c / (2 * CPR), part = c % (2 * CPR);
            to[j] = nullptr;
            if (c < chunks && path[i] != i) {
                const int s = ctx + path[i], d = ctx + i;
                const int bs = block_of(a, row, s), bd = block_of(a, row, d);
                if (bs >= 0 && bd >= 0) {
                    uint8_t* cache = (part < CPR ? a.k_cache : a.v_cache) + (part % CPR) * 16;
                    x[j] = ld_input(reinterpret_cast<const uint4*>(cache + row_at(a, bs, hk, s) * RB));
                    to[j] = cache + row_at(a, bd, hk, d) * RB;
                }
            }
        }
        __syncthreads();                     // the round is read
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if (to[j]) *reinterpret_cast<uint4*>(to[j]) = x[j];
    }
}

// ---------------------------------------------------------------- evict

constexpr int kEvictThreads = 512;
constexpr int kBins = 2048;
constexpr int kChunks = 4;        // 16-byte chunks a thread moves in a round
constexpr int kStage = kEvictThreads * kChunks * 16;   // bytes of a CTA's round

// A weight as a key whose unsigned order is the weights': -0 is 0, a NaN is below all.
__device__ __forceinline__ uint32_t key_of(float w) {
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;   // (-inf is 0x007FFFFF)
}

// Exclusive prefix sum of one value per thread over the CTA; `total` of all.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    __syncthreads();              // (warp_sums of an earlier scan are read)
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kEvictThreads / 32; ++w) {
        const int y = warp_sums[w];
        before += w < warp ? y : 0;
        total += y;
    }
    return before + x - v;
}

// Words of the keys' place: they make way for two rounds of rows.
__host__ __device__ constexpr int keys_words(int per_cta) { return per_cta > kStage / 2 ? per_cta : kStage / 2; }

// One cluster per (kv head, sequence).  CTA r of it holds tokens
// [r * per_cta, (r + 1) * per_cta) of the sequence as keys, later their kept ones
// as a list of offsets.
template <int RB>
__global__ void __launch_bounds__(kEvictThreads) evict_kernel(const Args a) {
    cg::cluster_group cluster = cg::this_cluster();
    extern __shared__ __align__(16) uint32_t keys[];     // [per_cta], later two rounds' rows; then uint16 list[per_cta]
    __shared__ __align__(16) int hist[kBins], counted[kBins], sums[kBins];
    __shared__ int warp_sums[kEvictThreads / 32];
    __shared__ int found[2];                             // a pass's digit, and how many of its tokens stay
    __shared__ int counts[2];                            // this CTA's ties, and tokens that stay for sure
    __shared__ int place[17];                            // first kept place of each CTA's list; budget
    constexpr int CPR = RB / 16, ROW = 2 * CPR;          // chunks of a row: K's, with V's
    constexpr int RUN = kEvictThreads * kChunks / ROW;   // rows a CTA moves in a round
    static_assert(RUN <= kEvictThreads, "a thread looks up at most one row a round");
    static_assert(kBins == 4 * kEvictThreads, "a thread has four bins");
    __shared__ int64_t from[4][RUN], to[4][RUN];         // of round k in [k & 3]
    uint16_t* list = reinterpret_cast<uint16_t*>(keys + keys_words(a.per_cta));
    const int tid = threadIdx.x, rank = static_cast<int>(cluster.block_rank()), size = static_cast<int>(cluster.num_blocks());
    const int hk = blockIdx.x / size, b = blockIdx.y;
    griddep_wait();
    griddep_launch_dependents();
    const int L_in = ld_input(a.seq_lens + b), L = L_in < 0 ? 0 : min(L_in, a.max_seq_len);
    if (hk == 0 && rank == 0 && tid == 0) {
        if (L != L_in) report(a.err, FP8KV_ERR_INVALID_ARG);
        a.new_lens[b] = min(L, a.budget);
    }
    int32_t* kept = a.kept ? a.kept + (static_cast<int64_t>(b) * a.num_kv_heads + hk) * a.budget : nullptr;
    if (L <= a.budget) {                                 // (the whole cluster) nothing to choose
        if (kept)
            for (int64_t i = rank * kEvictThreads + tid; i < a.budget; i += size * kEvictThreads)
                kept[i] = i < L ? static_cast<int>(i) : -1;
        return;
    }
    const int32_t* table = a.block_tables + static_cast<int64_t>(b) * a.max_blocks_per_seq;
    const int t0 = rank * a.per_cta, n = max(0, min(a.per_cta, L - t0));
    auto is_fixed = [&](int i) { return t0 + i < a.sinks || t0 + i >= L - a.recent; };

    // ---- the keys (per_cta is a multiple of 16: four tokens lie in one page), and
    // the first pass's counts
    *reinterpret_cast<int4*>(hist + 4 * tid) = make_int4(0, 0, 0, 0);
    __syncthreads();
    constexpr int AT = 4;                                // reads of a thread at once
    for (int i0 = tid * 4; i0 < n; i0 += kEvictThreads * 4 * AT) {
        int id[AT];
        float4 w[AT];
#pragma unroll
        for (int j = 0; j < AT; ++j) {
            const int i = i0 + j * kEvictThreads * 4;
            id[j] = i < n ? block_of(a, table, t0 + i) : -1;
        }
#pragma unroll
        for (int j = 0; j < AT; ++j) {
            const int i = i0 + j * kEvictThreads * 4;
            w[j] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (id[j] >= 0) w[j] = ld_input(reinterpret_cast<const float4*>(a.weights + row_at(a, id[j], hk, t0 + i)));
        }
#pragma unroll
        for (int j = 0; j < AT; ++j) {
            const int i = i0 + j * kEvictThreads * 4;
            const uint32_t k[4] = {key_of(w[j].x), key_of(w[j].y), key_of(w[j].z), key_of(w[j].w)};
            if (i >= n) break;
            *reinterpret_cast<uint4*>(keys + i) = make_uint4(k[0], k[1], k[2], k[3]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (i + e < n && !is_fixed(i + e)) atomicAdd(&hist[k[e] >> 21], 1);
        }
    }
    // ---- the smallest kept key, digit by digit: `want` of the tokens that are not fixed stay
    int want = a.budget - a.sinks - a.recent;
    uint32_t least = want > 0 ? 0u : ~0u;                // (no weight has the key ~0)
    if (want > 0) {
        // Two CTAs read each other's counts.  More sum a share of the bins each, then
        // all read the sums: 16 KB a CTA, where every count is 8 KB a CTA of the
        // cluster (16 CTAs: a pass of 3 us, 8 us by reading every count; 2 CTAs: 2.4
        // and 2.0 us).
        const int nb = kBins / size;
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, mask = pass == 2 ? 1023 : 2047;
            if (pass > 0) {
                *reinterpret_cast<int4*>(hist + 4 * tid) = make_int4(0, 0, 0, 0);
                __syncthreads();
                for (int i = tid; i < n; i += kEvictThreads) {
                    const uint32_t k = keys[i];
                    if ((k >> (pass == 1 ? 21 : 10)) == least && !is_fixed(i)) atomicAdd(&hist[(k >> shift) & mask], 1);
                }
            }
            cluster.sync();                              // the counts are there
            // thread t has bins 2047 - 4 t and the three below
            int c[4] = {0, 0, 0, 0}, all;
            const int top = kBins - 1 - 4 * tid;
            auto add = [&](const int* from) {
                const int4 x = *reinterpret_cast<const int4*>(from);
                c[0] += x.w; c[1] += x.z; c[2] += x.y; c[3] += x.x;
            };
            if (size <= 2) {
                for (int r = 0; r < size; ++r) add(cluster.map_shared_rank(hist, r) + top - 3);
                cluster.sync();                          // every count is read
            } else {
                *reinterpret_cast<int4*>(counted + 4 * tid) =
                    *reinterpret_cast<const int4*>(cluster.map_shared_rank(hist, 4 * tid / nb) + rank * nb + 4 * tid % nb);
                __syncthreads();
                for (int i = tid; i < nb; i += kEvictThreads) {
                    int x = 0;
                    for (int r = 0; r < size; ++r) x += counted[r * nb + i];
                    sums[i] = x;
                }
                cluster.sync();                          // every count is read, and the sums are there
                add(cluster.map_shared_rank(sums, (top - 3) / nb) + (top - 3) % nb);
            }
            const int mine = (c[0] + c[1]) + (c[2] + c[3]);
            int above = block_scan(mine, warp_sums, all);
            if (above < want && want <= above + mine) {
                int j = 0;
#pragma unroll
                for (; j < 3; ++j) {
                    if (above + c[j] >= want) break;
                    above += c[j];
                }
                found[0] = top - j;
                found[1] = want - above;
            }
            __syncthreads();
            least = (least << (pass == 2 ? 10 : 11)) | static_cast<uint32_t>(found[0]);
            want = found[1];
        }
    } else {
        __syncthreads();
    }
    // Keys above `least` stay, and the first `want` of those equal to it.
    // ---- what of this CTA's tokens stays: each thread a run (of odd length: no bank conflicts)
    const int per = ((n + kEvictThreads - 1) / kEvictThreads) | 1, i0 = min(n, tid * per), i1 = min(n, i0 + per);
    uint64_t ties = 0, sure = 0;                         // bits of the run
    for (int i = i0; i < i1; ++i) {
        const uint64_t bit = 1ull << (i - i0);
        if (is_fixed(i) || keys[i] > least) sure |= bit;
        else if (keys[i] == least) ties |= bit;
    }
    int all;                                             // (two counts in one scan: each is below 2^16)
    const int before_me = block_scan(__popcll(ties) | __popcll(sure) << 16, warp_sums, all);
    const int ties_before = before_me & 0xFFFF, sure_before = before_me >> 16;
    if (tid == 0) {
        counts[0] = all & 0xFFFF;
        counts[1] = all >> 16;
    }
    cluster.sync();
    if (tid < 32) {
        // ties stay from the front: each CTA's share, and where its list begins
        int t = 0, k = 0;
        if (tid < size) {
            const int* c = cluster.map_shared_rank(counts, tid);
            t = c[0];
            k = c[1];
        }
        int x = t;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, off);
            if (tid >= off) x += y;
        }
        const int own = k + max(0, min(t, want - (x - t)));
        int y = own;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int z = __shfl_up_sync(0xffffffffu, y, off);
            if (tid >= off) y += z;
        }
        if (tid < size) place[tid] = y - own;
        if (tid == size - 1) place[size] = y;            // the budget
        const int before = __shfl_sync(0xffffffffu, x - t, rank);
        if (tid == 0) found[0] = max(0, want - before);  // ties that may stay from this CTA on
    }
    __syncthreads();
    const int ties_left = found[0];
    int at = sure_before + min(ties_left, ties_before), tie = ties_before;
    for (uint64_t left = sure | ties; left; left &= left - 1) {
        const uint64_t bit = left & (~left + 1);
        if ((sure & bit) || tie++ < ties_left) list[at++] = static_cast<uint16_t>(i0 + __ffsll(static_cast<long long>(bit)) - 1);
    }
    cluster.sync();                                      // the lists are there
    if (kept)
        for (int i = tid; i < place[rank + 1] - place[rank]; i += kEvictThreads) kept[place[rank] + i] = t0 + list[i];

    // ---- the rows, in rounds of the whole cluster: a round is read while the one
    // before it is written (see the top), and its rows' places are looked up a
    // round earlier still.
    // rows of this CTA's run of round k, a thread each: where they lie, where they go, their weight
    const int rounds = (a.budget + size * RUN - 1) / (size * RUN);
    auto look_up = [&](int k) {
        float w = 0.f;
        if (tid < RUN) {
            const int i = (k * size + rank) * RUN + tid;
            int64_t f = -1, t = 0;
            if (i < a.budget) {
                int r = 0;
                while (i >= place[r + 1]) ++r;
                const int src = r * a.per_cta + cluster.map_shared_rank(list, r)[i - place[r]];
                if (src != i) {
                    const int bs = block_of(a, table, src), bd = block_of(a, table, i);
                    if (bs >= 0 && bd >= 0) {
                        f = row_at(a, bs, hk, src);
                        t = row_at(a, bd, hk, i);
                        w = ld_input(a.weights + f);
                    }
                }
            }
            from[k & 3][tid] = f;
            to[k & 3][tid] = t;
        }
        return w;
    };
    // Chunk j of the thread is chunk (j * threads + tid) of the run, K's and V's of a
    // row beside each other; the thread that stages a chunk writes it.
    const uint32_t stage = smem_u32(keys);               // (the keys are done with)
    auto read = [&](int k) {
#pragma unroll
        for (int j = 0; j < kChunks; ++j) {
            const int c = j * kEvictThreads + tid, part = c % ROW;
            const int64_t f = from[k & 3][c / ROW];
            if (f >= 0)
                cp_async_16(stage + (k & 1) * kStage + c * 16,
                            (part < CPR ? a.k_cache : a.v_cache) + f * RB + (part % CPR) * 16);
        }
        cp_async_commit();
    };
    float w = look_up(0), w1 = look_up(1);
    __syncthreads();
    read(0);
    for (int k = 0; k < rounds; ++k) {
        if (k + 1 < rounds) read(k + 1); else cp_async_commit();
        const float w2 = k + 2 < rounds ? look_up(k + 2) : 0.f;
        cp_async_wait<1>();
        cluster.sync();                                  // round k is read
#pragma unroll
        for (int j = 0; j < kChunks; ++j) {
            const int c = j * kEvictThreads + tid, part = c % ROW, i = c / ROW;
            if (from[k & 3][i] >= 0)
                *reinterpret_cast<uint4*>((part < CPR ? a.k_cache : a.v_cache) + to[k & 3][i] * RB + (part % CPR) * 16) =
                    *reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(keys) + (k & 1) * kStage + c * 16);
        }
        if (tid < RUN && from[k & 3][tid] >= 0) a.weights[to[k & 3][tid]] = w;
        w = w1;
        w1 = w2;
    }
    cluster.sync();                                      // no CTA leaves while its list is read
}

// ---------------------------------------------------------------- host side

constexpr int kMaxCluster = 16;
constexpr int kMaxPerCta = 24576;   // tokens a CTA holds at most: 6 bytes each, 144 KB; 48 a thread

int evict_smem(int per_cta) { return keys_words(per_cta) * 4 + per_cta * 2; }

template <typename Kernel>
static cudaError_t launch(Kernel kernel, dim3 grid, int threads, int smem, int cluster, const Args& a, cudaStream_t s) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int RB>
static cudaError_t launch_evict(const Args& a, int cluster, int smem, cudaStream_t s) {
    static std::atomic<uint64_t> done_mask{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
    if (bit == 0 || !(done_mask.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(evict_kernel<RB>, cudaFuncAttributeMaxDynamicSharedMemorySize, evict_smem(kMaxPerCta));
        if (e == cudaSuccess) e = cudaFuncSetAttribute(evict_kernel<RB>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        done_mask.fetch_or(bit, std::memory_order_release);
    }
    return launch(evict_kernel<RB>, dim3(static_cast<unsigned>(a.num_kv_heads * cluster), static_cast<unsigned>(a.batch)),
                  kEvictThreads, smem, cluster, a, s);
}

// What both calls check.
static fp8kv_status check(const void* k_cache, const void* v_cache, int64_t num_blocks, const int32_t* block_tables,
                          int max_blocks_per_seq, const int32_t* seq_lens, int max_seq_len, int batch, int num_kv_heads,
                          int head_dim, int block_size, int cache_format, const int32_t* new_lens, const void* workspace,
                          size_t workspace_bytes) {
    auto off = [](const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; };
    if (batch < 0 || batch > 65535 || num_kv_heads < 1 || num_kv_heads > 65535 || max_seq_len < 0 || num_blocks < 1 ||
        max_blocks_per_seq < 0 ||
        (cache_format != FP8KV_CACHE_E4M3 && cache_format != FP8KV_CACHE_E5M2 && cache_format != FP8KV_CACHE_BF16))
        return FP8KV_ERR_INVALID_ARG;
    if (!(head_dim == 64 || head_dim == 128 || head_dim == 256) || block_size != kBS) return FP8KV_ERR_UNSUPPORTED;
    if (num_blocks >= (INT64_C(1) << 31) || num_blocks * num_kv_heads >= (INT64_C(1) << 31)) return FP8KV_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(max_blocks_per_seq) * block_size < max_seq_len) return FP8KV_ERR_INVALID_ARG;
    if (batch == 0) return FP8KV_OK;
    if (!k_cache || !v_cache || !block_tables || !seq_lens || !new_lens || off(k_cache, 16) || off(v_cache, 16) ||
        off(block_tables, 4) || off(seq_lens, 4) || off(new_lens, 4))
        return FP8KV_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < 256 || off(workspace, 256)) return FP8KV_ERR_WORKSPACE;
    return FP8KV_OK;
}

static Args args(void* k_cache, void* v_cache, int64_t num_blocks, const int32_t* block_tables, int max_blocks_per_seq,
                 const int32_t* seq_lens, int max_seq_len, int batch, int num_kv_heads, int32_t* new_lens, void* workspace) {
    Args a = {};
    a.k_cache = static_cast<uint8_t*>(k_cache);
    a.v_cache = static_cast<uint8_t*>(v_cache);
    a.num_blocks = num_blocks;
    a.block_tables = block_tables;
    a.max_blocks_per_seq = max_blocks_per_seq;
    a.seq_lens = seq_lens;
    a.max_seq_len = max_seq_len;
    a.batch = batch;
    a.num_kv_heads = num_kv_heads;
    a.new_lens = new_lens;
    a.err = static_cast<uint32_t*>(workspace);
    return a;
}

}  // namespace keep
}  // namespace fp8kv

extern "C" fp8kv_status fp8kv_tree_commit(void* k_cache, void* v_cache, int64_t num_blocks, const int32_t* block_tables,
                                          int max_blocks_per_seq, const int32_t* seq_lens, const int32_t* q_starts,
                                          const int32_t* accepted, int max_accepted, int max_seq_len, int batch,
                                          int num_kv_heads, int head_dim, int block_size, int cache_format,
                                          int32_t* new_lens, void* workspace, size_t workspace_bytes, void* stream) {
    using namespace fp8kv::keep;
    FP8KV_TRACE("fp8kv_tree_commit");
    if (max_accepted < 0) return FP8KV_ERR_INVALID_ARG;
    const fp8kv_status c = check(k_cache, v_cache, num_blocks, block_tables, max_blocks_per_seq, seq_lens, max_seq_len,
                                 max_accepted == 0 ? std::min(batch, 0) : batch, num_kv_heads, head_dim, block_size,
                                 cache_format, new_lens, workspace, workspace_bytes);
    if (c != FP8KV_OK) return c;
    if (max_accepted > kMaxPath) return FP8KV_ERR_UNSUPPORTED;
    if (batch == 0 || max_accepted == 0) return FP8KV_OK;
    if (!q_starts || !accepted || (reinterpret_cast<uintptr_t>(q_starts) & 3u) || (reinterpret_cast<uintptr_t>(accepted) & 3u))
        return FP8KV_ERR_INVALID_ARG;
    Args a = args(k_cache, v_cache, num_blocks, block_tables, max_blocks_per_seq, seq_lens, max_seq_len, batch, num_kv_heads,
                  new_lens, workspace);
    a.q_starts = q_starts;
    a.accepted = accepted;
    a.max_accepted = max_accepted;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const dim3 grid(static_cast<unsigned>(num_kv_heads), static_cast<unsigned>(batch));
    const int rb = head_dim * (cache_format == FP8KV_CACHE_BF16 ? 2 : 1);
    const cudaError_t e = rb == 64    ? launch(commit_kernel<64>, grid, 256, 0, 1, a, s)
                          : rb == 128 ? launch(commit_kernel<128>, grid, 256, 0, 1, a, s)
                          : rb == 256 ? launch(commit_kernel<256>, grid, 256, 0, 1, a, s)
                                      : launch(commit_kernel<512>, grid, 256, 0, 1, a, s);
    return e == cudaSuccess ? FP8KV_OK : FP8KV_ERR_CUDA;
}

extern "C" fp8kv_status fp8kv_evict(void* k_cache, void* v_cache, float* weights, int64_t num_blocks,
                                    const int32_t* block_tables, int max_blocks_per_seq, const int32_t* seq_lens,
                                    int max_seq_len, int budget, int sinks, int recent, int batch, int num_kv_heads,
                                    int head_dim, int block_size, int cache_format, int32_t* new_lens, int32_t* kept,
                                    void* workspace, size_t workspace_bytes, void* stream) {
    using namespace fp8kv::keep;
    FP8KV_TRACE("fp8kv_evict");
    if (budget < 1 || sinks < 0 || recent < 0 || static_cast<int64_t>(sinks) + recent > budget) return FP8KV_ERR_INVALID_ARG;
    const fp8kv_status c = check(k_cache, v_cache, num_blocks, block_tables, max_blocks_per_seq, seq_lens, max_seq_len, batch,
                                 num_kv_heads, head_dim, block_size, cache_format, new_lens, workspace, workspace_bytes);
    if (c != FP8KV_OK) return c;
    if (max_seq_len > kMaxCluster * kMaxPerCta) return FP8KV_ERR_UNSUPPORTED;
    if (batch == 0) return FP8KV_OK;
    if (!weights || (reinterpret_cast<uintptr_t>(weights) & 15u) || (reinterpret_cast<uintptr_t>(kept) & 3u))
        return FP8KV_ERR_INVALID_ARG;
    int sms = 0;
    if (fp8kv::device_sms(&sms) != 0) return FP8KV_ERR_CUDA;
    // CTAs of a cluster: as many as hold the longest sequence, and while there is
    // room for more on the SMs, two on each, twice as many each time
    int cluster = 1;
    const int64_t units = static_cast<int64_t>(batch) * num_kv_heads;
    auto per_cta = [&](int n) { return ((max_seq_len + n - 1) / n + 15) & ~15; };
    while (cluster < kMaxCluster && (per_cta(cluster) > kMaxPerCta || (units * cluster <= sms && per_cta(cluster) > 256)))
        cluster *= 2;
    Args a = args(k_cache, v_cache, num_blocks, block_tables, max_blocks_per_seq, seq_lens, max_seq_len, batch, num_kv_heads,
                  new_lens, workspace);
    a.weights = weights;
    a.kept = kept;
    a.budget = budget;
    a.sinks = sinks;
    a.recent = recent;
    a.per_cta = per_cta(cluster);
    const int smem = evict_smem(a.per_cta);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int rb = head_dim * (cache_format == FP8KV_CACHE_BF16 ? 2 : 1);
    const cudaError_t e = rb == 64    ? launch_evict<64>(a, cluster, smem, s)
                          : rb == 128 ? launch_evict<128>(a, cluster, smem, s)
                          : rb == 256 ? launch_evict<256>(a, cluster, smem, s)
                                      : launch_evict<512>(a, cluster, smem, s);
    return e == cudaSuccess ? FP8KV_OK : FP8KV_ERR_CUDA;
}
