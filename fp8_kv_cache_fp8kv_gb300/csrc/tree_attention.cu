// Attention of a tree of drafted tokens per sequence over a paged cache
// (speculative decoding: a draft model proposes a tree, this checks all of it at
// once).  The drafted tokens are the sequence's newest; node i attends the
// context before them, its ancestors and itself.
//
// With row r = (node, query head of the group), 128 rows to a tile, and per key t
// the codes ck_t, cv_t:
//     s_rt = sm ks (q_r . ck_t),   out_r = vs sum_t w_rt cv_t / sum_t w_rt,
//     w_rt = 2^(s_rt log2 e - m_r) for the keys that r attends.
//
// The work is between decode and prefill: g rows of a node times 1 to 256 nodes
// share every key, so the tensor cores have to run a 128-row tile at the rate
// HBM delivers keys.  Two things keep them fed:
//   * FP8 keys are MMA operands as they lie in the cache.  kind::f8f6f4 takes them
//     beside a Q of two E4M3 numbers, q = hi + lo: E4M3 has 4 significant bits,
//     bf16 has 8, so the split is exact but for elements below 2^-15 of the row's
//     largest, which are rounded to 2^-17 of it.  Keys need no conversion and half
//     the shared memory; the two MMAs of hi and lo take the time of one in f16.
//   * V goes to f16 (exact) row by row, without a transpose: the value MMA reads
//     it MN-major.  P is f16 in tensor memory, as the prefill kernels have it: 11
//     bits down to 2^-23 of a row's largest weight, steps of 2^-33 of it below, where two E4M3 numbers
//     would lose everything below 2^-18 of it (2^17 such keys are half the answer).
// A bf16 cache is used as it lies on both sides; its P is two bf16 numbers (16
// bits), since one alone would round as coarsely as the output is rounded.
//
// Scores, the softmax and P.V accumulate in FP32.  The reference m_r of a row is a
// whole number, moved only where 64 keys' weights grow too large for f16 (or at
// masked keys), so scaling what was summed under another is exact.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "fp8kv.h"
#include "partition.cuh"
#include "ptx.cuh"
#include "tcgen05.cuh"
#include "trace.cuh"
#include "tree_walk.h"

namespace fp8kv {

int device_sms(int* sms);  // SM count of the current device (paged_decode.cu)

namespace tree {

constexpr int kBS = 16;
constexpr int kMaxNodes = 256;
constexpr int kMaxBatch = 256;                   // sequences per launch; larger batches run in chunks
constexpr int kMinPages = 16;                    // pages a CTA takes at least
constexpr uint64_t kWaitNs = 500000000ull;       // bounded waits
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRoom = 9.f;                     // a new reference lies this far below the largest score (log2),
constexpr float kMaxSum = 60000.f;               // and moves when 64 keys' weights sum to more (f16 ends at 65504):
                                                 // 64 equal scores sum to 2^15

struct Args {
    const uint16_t* q;           // bf16 [num_tokens, Hq, D]
    const uint8_t* k_cache;
    const uint8_t* v_cache;
    const int32_t* block_tables;
    const int32_t* seq_lens;
    const int32_t* q_starts;     // [B + 1]
    const int32_t* parents;      // [num_tokens]
    uint16_t* out;
    uint32_t* err;
    float2* part_ml;             // [2 * ctas][rows]         (reference, sum)
    float4* part_o;              // [2 * ctas][D / 4][rows]  unnormalised outputs
    const float* k_scales;       // [Hkv] or null
    const float* v_scales;
    int64_t num_blocks;
    int64_t num_tokens;
    float k_scale, v_scale, sm_scale;
    int max_blocks_per_seq, max_seq_len, max_nodes, batch, num_q_heads, num_kv_heads, log2_group, window;
    int max_ctas;
    uint64_t wait_ns;            // failure-path hook: see fp8kv_debug_paged_tree_stall
    int stall_stage;
};

// D elements a head, ES bytes an element, T tiles of 128 rows a CTA.
template <int D, int ES, int T>
struct Geo {
    static constexpr int KEYS = ES == 1 && D < 256 ? 128 : 64;   // keys per stage
    static constexpr int PAGES = KEYS / kBS;
    static constexpr int RB = D * ES;                            // bytes of a row
    static constexpr int PAGE = kBS * RB;
    static constexpr int TILE = KEYS * RB;                       // K bytes (and V bytes) of a stage
    static constexpr int COL = KEYS * 128;                       // one 128-byte atom column of a tile
    static constexpr int QB = 128 * 2 * D;                     // Q tile: hi and lo E4M3, or bf16
    static constexpr int VB = ES == 1 ? KEYS * 2 * D : 0;        // f16 V tile
    static constexpr int R = ES == 1 ? (D == 64 ? 4 : D == 128 ? (T == 1 ? 3 : 2) : 2) : D == 64 ? 6 : D == 128 ? (T == 1 ? 5 : 4) : 2;
    static constexpr int LAG = R - 2 > 2 ? 2 : R - 2;            // copies of this many younger stages are in flight
    static constexpr int HALVES = KEYS / 64;
    // shared memory: Q tiles, the ring, V tiles, tables
    static constexpr int RING = T * QB, V16 = RING + R * 2 * TILE, MASKS = V16 + 2 * VB;
    static constexpr int PRE = MASKS + 8 * T * 128 * 4;          // int64 [kMaxBatch + 1]
    static constexpr int LENS = PRE + (kMaxBatch + 1) * 8;       // int32 [3][kMaxBatch]: L, n, q0
    static constexpr int SMEM = LENS + 3 * kMaxBatch * 4 + 1024;
    // TMEM columns: T = 1: two S buffers and O; T = 2: each tile S and O.  P lies over S.
    static constexpr int OC = T == 1 ? 256 : 128;
    static_assert(T == 1 ? 2 * KEYS <= OC && OC + D <= 512 : KEYS <= OC && OC + D <= 256, "TMEM columns");
    static_assert(SMEM <= 227 * 1024 - 512, "shared memory");
    static constexpr int SW = 4 * T;                             // softmax warps
    static constexpr int CW0 = SW, CW = ES == 1 ? 4 : 0;         // converter warps
    static constexpr int PW0 = CW0 + CW, PW = 3;                 // copy warps
    static constexpr int MW = PW0 + PW;                          // the MMA warp
    static constexpr int THREADS = (MW + 1) * 32;
};

__device__ __forceinline__ void report(uint32_t* err, uint32_t code) { atomicCAS(err, 0u, code); }

__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, uint64_t limit_ns, volatile int* abort_flag) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (true) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (global_timer_ns() - t0 > limit_ns) {
            *abort_flag = 1;
            return false;
        }
    }
}

// 16-byte cp.async of `bytes` (16 or 0) bytes, the rest zeros.
__device__ __forceinline__ void cp_async_16z(uint32_t dst, const void* src, int bytes, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(bytes),
                 "l"(policy)
                 : "memory");
}
__device__ __forceinline__ uint64_t l2_policy_normal() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}

// Place of chunk c (16 bytes) of row k in an operand tile of KEYS rows.
template <int RB, int COL>
__device__ __forceinline__ uint32_t tile_at(int k, int c) {
    if constexpr (RB == 64) return k * 64 + ((c ^ ((k >> 1) & 3)) << 4);
    else return (c >> 3) * COL + k * 128 + (((c & 7) ^ (k & 7)) << 4);
}

// d = a * b + c of two values in one instruction, and d += a.
__device__ __forceinline__ void fma2(float& d0, float& d1, float b, float c) {
    asm("{\n\t.reg .b64 ra, rb, rc;\n\t"
        "mov.b64 ra, {%0, %1};\n\tmov.b64 rb, {%2, %2};\n\tmov.b64 rc, {%3, %3};\n\t"
        "fma.rn.f32x2 ra, ra, rb, rc;\n\tmov.b64 {%0, %1}, ra;\n\t}"
        : "+f"(d0), "+f"(d1)
        : "f"(b), "f"(c));
}
__device__ __forceinline__ void add2(float& d0, float& d1, float a0, float a1) {
    asm("{\n\t.reg .b64 ra, rb;\n\t"
        "mov.b64 ra, {%0, %1};\n\tmov.b64 rb, {%2, %3};\n\t"
        "add.rn.f32x2 ra, ra, rb;\n\tmov.b64 {%0, %1}, ra;\n\t}"
        : "+f"(d0), "+f"(d1)
        : "f"(a0), "f"(a1));
}

__device__ __forceinline__ uint64_t ones(int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1; }

// What a sequence's entries say, clamped to their bounds.
struct Seq {
    int L, n, q0;
    bool bad;
};
__device__ __forceinline__ Seq read_seq(const Args& a, int b) {
    Seq s;
    s.q0 = ld_input(a.q_starts + b);
    const int n_in = ld_input(a.q_starts + b + 1) - s.q0, L_in = ld_input(a.seq_lens + b);
    s.L = L_in < 0 ? 0 : min(L_in, a.max_seq_len);
    s.n = n_in < 0 ? 0 : min(n_in, min(s.L, a.max_nodes));
    if (s.q0 < 0 || s.q0 + static_cast<int64_t>(s.n) > a.num_tokens) s.n = 0;   // never rows outside q / out
    s.bad = s.L != L_in || s.n != n_in;
    return s;
}
__device__ __forceinline__ int row_blocks(int n, int lg, int rows) { return ((n << lg) + rows - 1) / rows; }

// ---------------------------------------------------------------- the kernel
//
// One CTA per SM, persistent over its range of pages (tree_walk.h).  Roles hand
// over through mbarriers, stage by stage (g counts stages over all segments):
//   * copy warps: 16-byte cp.async copies of a stage's pages, K swizzled as the
//     MMA reads it, zeros past the sequence's end; block ids a stage ahead;
//   * converter warps (FP8): V rows to the f16 tile g & 1;
//   * the MMA thread: S = Q K^T a stage ahead, then O += P V;
//   * softmax warps, thread = row = TMEM lane: S to P over itself, O rescaled
//     where a reference moves; they also build the Q tiles, between segments,
//     and write out what a segment ends with.
// With T = 1 the S of two stages alternate in two buffers; with T = 2 the two
// tiles share the stage's keys and alternate on the tensor cores.
template <int D, int ES, bool E5M2, int T>
__global__ void __launch_bounds__(Geo<D, ES, T>::THREADS, 1) tree_kernel(const Args a) {
    using G = Geo<D, ES, T>;
    constexpr int KEYS = G::KEYS, PAGES = G::PAGES, R = G::R, ROWS = 128 * T;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[R], empty[R], v_full[2], o_done[2], s_full[2], p_full[2], q_full, end_bar;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_sh, timed_out;
    volatile int* abort_flag = &abort_sh;
    uint8_t* sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const uint32_t sb = smem_u32(sm);
    uint32_t* masks = reinterpret_cast<uint32_t*>(sm + G::MASKS);      // [8][ROWS], a column per row thread
    int64_t* pre = reinterpret_cast<int64_t*>(sm + G::PRE);
    int32_t* lens = reinterpret_cast<int32_t*>(sm + G::LENS);
    int32_t *nodes = lens + kMaxBatch, *firsts = nodes + kMaxBatch;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int lg = a.log2_group, B = a.batch, H = a.num_kv_heads;

    if (tid == 0) {
        for (int j = 0; j < R; ++j) {
            mbar_init(&full[j], G::PW);
            mbar_init(&empty[j], ES == 1 ? 1 + G::CW : 1);   // the score MMAs and the converters; or the value MMAs
        }
        for (int j = 0; j < 2; ++j) {
            mbar_init(&v_full[j], 128);
            mbar_init(&o_done[j], 1);
            mbar_init(&s_full[j], 1);
            mbar_init(&p_full[j], 128);
        }
        mbar_init(&q_full, ROWS);
        mbar_init(&end_bar, 1);
        abort_sh = 0;
        fence_barrier_init();
    }
    if (warp == G::MW) tc::alloc(&tmem_base, 512);
    griddep_wait();
    griddep_launch_dependents();
    if (warp == 0) {
        int64_t run = 0;
        for (int b0 = 0; b0 < B; b0 += 32) {
            const int b = b0 + lane;
            int64_t pages = 0;
            if (b < B) {
                const Seq s = read_seq(a, b);
                if (s.bad && blockIdx.x == 0) report(a.err, FP8KV_ERR_INVALID_ARG);
                lens[b] = s.L;
                nodes[b] = s.n;
                firsts[b] = s.q0;
                pages = static_cast<int64_t>(unit_pages(s.L, s.n, a.window)) * H * row_blocks(s.n, lg, ROWS);
            }
            int64_t x = pages;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, x, off);
                if (lane >= off) x += y;
            }
            if (b < B) pre[b] = run + x - pages;
            run += __shfl_sync(0xffffffffu, x, 31);
        }
        if (lane == 0) {
            pre[B] = run;
            timed_out = *reinterpret_cast<volatile uint32_t*>(a.err) == FP8KV_ERR_TIMEOUT;
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = tmem_base;
    const int64_t P = pre[B];
    const int C = cta_count(P, a.max_ctas, kMinPages);
    const Partition part = make_partition(P, C);
    const bool work = P > 0 && static_cast<int>(blockIdx.x) < C && !timed_out;
    const int64_t range0 = work ? range_start(part, blockIdx.x) : 0, range1 = work ? range_start(part, blockIdx.x + 1) : 0;
    auto blocks_of = [&](int b) { return row_blocks(nodes[b], lg, ROWS); };

    if (warp < G::SW) {
        // ------------------------------------------------------------ softmax
        const int tile = T == 1 ? 0 : warp >> 2;
        const uint32_t trow = tm + (static_cast<uint32_t>((warp & 3) * 32) << 16) + tile * 256;
        uint8_t* qt = sm + tile * G::QB;
        const int myrow = tid & 127;
        // The Q tile's row of this thread for a segment; returns the multiplier of
        // its raw scores (>= 0: the sign of the score scale goes into Q).
        auto build_q = [&](const Segment& s) {
            const int r = s.rb * ROWS + tid;
            const bool rv = r < (nodes[s.b] << lg);
            const uint16_t* src = a.q + (static_cast<int64_t>(firsts[s.b] + (rv ? r >> lg : 0)) * a.num_q_heads +
                                         (s.hk << lg) + (rv ? r & ((1 << lg) - 1) : 0)) * D;
            const float ks = a.k_scales ? ld_input(a.k_scales + s.hk) : a.k_scale;
            float cs = fabsf(a.sm_scale) * ks * kLog2e;
            const uint32_t flip = a.sm_scale < 0.f ? 0x80008000u : 0u;
            uint8_t* row = qt + myrow * 128;
            if constexpr (ES == 2) {
#pragma unroll 4
                for (int c = 0; c < D / 8; ++c) {
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (rv) x = ld_input(reinterpret_cast<const uint4*>(src) + c);
                    x.x ^= flip; x.y ^= flip; x.z ^= flip; x.w ^= flip;
                    *reinterpret_cast<uint4*>(row + (c >> 3) * 16384 + (((c & 7) ^ (myrow & 7)) << 4)) = x;
                }
            } else {
                float top = 0.f;
#pragma unroll 8
                for (int c = 0; c < D / 8; ++c) {
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (rv) x = ld_input(reinterpret_cast<const uint4*>(src) + c);
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xFFFF0000u))));
                }
                int shift = 0;   // the largest element to [2^7, 2^8)
                if (top > 0.f) shift = max(-126, min(126, 7 - (static_cast<int>((__float_as_uint(top) >> 23) & 0xFF) - 127)));
                const float up = __uint_as_float(static_cast<uint32_t>(127 + shift) << 23);
                cs *= __uint_as_float(static_cast<uint32_t>(127 - shift) << 23);
                const float none = __uint_as_float(0x7FC00000u);
#pragma unroll 2
                for (int c = 0; c < D / 16; ++c) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        uint4 x = make_uint4(0, 0, 0, 0);
                        if (rv) x = ld_input(reinterpret_cast<const uint4*>(src) + 2 * c + hf);
                        const uint32_t w[4] = {x.x ^ flip, x.y ^ flip, x.z ^ flip, x.w ^ flip};
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t h = 0, l = 0;
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const uint32_t u = w[2 * i + e];
                                float x0 = __uint_as_float(u << 16) * up, x1 = __uint_as_float(u & 0xFFFF0000u) * up;
                                if (!(fabsf(x0) < 512.f)) x0 = none;   // an infinity must not saturate
                                if (!(fabsf(x1) < 512.f)) x1 = none;
                                const uint32_t hh = f32x2_to_e4m3x2_satfinite(x0, x1);
                                const uint32_t back = e4m3x2_to_f16x2(static_cast<uint16_t>(hh));
                                const __half2 b2 = *reinterpret_cast<const __half2*>(&back);
                                const uint32_t ll = f32x2_to_e4m3x2_satfinite(x0 - __low2float(b2), x1 - __high2float(b2));
                                h |= hh << (16 * e);
                                l |= ll << (16 * e);
                            }
                            hi[2 * hf + i] = h;
                            lo[2 * hf + i] = l;
                        }
                    }
                    const int ch = c, cl = c + D / 16;   // chunks of the row's hi and lo halves
                    *reinterpret_cast<uint4*>(row + (ch >> 3) * 16384 + (((ch & 7) ^ (myrow & 7)) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4*>(row + (cl >> 3) * 16384 + (((cl & 7) ^ (myrow & 7)) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            }
            tc::fence_proxy_async_smem();   // the tile is read by the tensor cores
            mbar_arrive(&q_full);
            return cs;
        };

        int g = 0;
        bool ok = true;
        float cs = 0.f;
        if (work) cs = build_q(segment_at(range0, range1, pre, B, H, blocks_of));
        for (int64_t pos = range0; pos < range1 && ok;) {
            const Segment s = segment_at(pos, range1, pre, B, H, blocks_of);
            pos = s.base + s.lp1;
            const int L = lens[s.b], n = nodes[s.b], ctx = L - n;
            const int page0 = first_key(L, n, a.window) / kBS;
            const int t_first = (page0 + s.lp0) * kBS, t_end = min((page0 + s.lp1) * kBS, L);
            const int nst = (s.lp1 - s.lp0 + PAGES - 1) / PAGES;
            const int rows = n << lg, r = s.rb * ROWS + tid;
            const bool rv = r < rows;
            const bool warp_rows = s.rb * ROWS + warp * 32 < rows;   // a warp of no rows only keeps the handshake
            // ---- which drafted tokens the row's node attends, and its depth
            int lo = 0;
            if (warp_rows && (t_end > ctx || a.window > 0)) {
                uint32_t* mine = masks + tid;
#pragma unroll
                for (int w = 0; w < 8; ++w) mine[w * ROWS] = 0;
                int depth = -1;
                for (int i = rv ? r >> lg : -1; i >= 0;) {
                    ++depth;
                    if (a.window <= 0 || depth < a.window) mine[(i >> 5) * ROWS] |= 1u << (i & 31);
                    const int p = ld_input(a.parents + firsts[s.b] + i);
                    if (p >= i || p < -1) {
                        report(a.err, FP8KV_ERR_INVALID_ARG);
                        break;
                    }
                    i = p;
                }
                if (a.window > 0) lo = max(0, ctx + depth + 1 - a.window);
            }
            const int wlo = __reduce_max_sync(0xffffffffu, rv ? lo : 0);

            float m = rv ? -INFINITY : 0.f, l = 0.f;   // (the tile's rows past the last: zero scores)
            for (int st = 0; st < nst && ok; ++st, ++g) {
                const int buf = T == 1 ? g & 1 : tile, ph = T == 1 ? (g >> 1) & 1 : g & 1;
                const uint32_t scol = trow + (T == 1 ? buf * KEYS : 0);
                ok = __all_sync(0xffffffffu, wait_or_abort(&s_full[buf], ph, a.wait_ns, abort_flag));
                if (!ok) break;
                if (warp_rows) {
                    tc::fence_after_sync();
                    const int t0 = t_first + st * KEYS;
                    const bool masked = t0 + KEYS > min(ctx, t_end) || t0 < wlo;
#pragma unroll 1
                    for (int h = 0; h < G::HALVES; ++h) {
                        float x[64];
                        float sum[4];
                        auto load = [&]() {
                            tc::ld32(scol + 64 * h, *reinterpret_cast<float(*)[32]>(x));
                            tc::ld32(scol + 64 * h + 32, *reinterpret_cast<float(*)[32]>(x + 32));
                            tc::wait_ld(*reinterpret_cast<float(*)[32]>(x));
                            tc::wait_ld(*reinterpret_cast<float(*)[32]>(x + 32));
                        };
                        load();
                        bool slow = masked || __any_sync(0xffffffffu, m == -INFINITY && rv);
                        if (!slow) {
                            sum[0] = sum[1] = sum[2] = sum[3] = 0.f;
#pragma unroll
                            for (int i = 0; i < 64; i += 2) {
                                fma2(x[i], x[i + 1], cs, -m);
                                x[i] = fast_exp2(x[i]);
                                x[i + 1] = fast_exp2(x[i + 1]);
                                add2(sum[i & 2], sum[(i & 2) + 1], x[i], x[i + 1]);
                            }
                            slow = __any_sync(0xffffffffu, (sum[0] + sum[1]) + (sum[2] + sum[3]) > kMaxSum);
                            if (slow) load();
                        }
                        if (slow) {
                            // the row's keys of this half, and where its reference belongs
                            const int th = t0 + 64 * h;
                            uint64_t keep = ~0ull;
                            if (masked) {
                                keep = ones(min(ctx, t_end) - th) & ~ones(lo - th);
                                if (t_end > ctx && th + 64 > ctx) {
                                    const uint32_t* mine = masks + tid;
                                    const int off = max(0, th - ctx), w = off >> 5, sh = off & 31;
                                    const uint32_t w0 = w < 8 ? mine[w * ROWS] : 0, w1 = w < 7 ? mine[(w + 1) * ROWS] : 0,
                                                   w2 = w < 6 ? mine[(w + 2) * ROWS] : 0;
                                    const uint64_t bits = static_cast<uint64_t>(__funnelshift_r(w0, w1, sh)) |
                                                          (static_cast<uint64_t>(__funnelshift_r(w1, w2, sh)) << 32);
                                    keep |= (th < ctx ? bits << (ctx - th) : bits) & ones(t_end - th);
                                }
                            }
                            float top = -INFINITY;
#pragma unroll
                            for (int i = 0; i < 64; ++i)
                                if ((i < 32 ? static_cast<uint32_t>(keep) >> i : static_cast<uint32_t>(keep >> 32) >> (i - 32)) & 1)
                                    top = fmaxf(top, x[i]);
                            if (top > -INFINITY) top = ceilf(top * cs - kRoom);
                            const float mn = fmaxf(m, top);
                            const float alpha = m > -INFINITY ? fast_exp2(m - mn) : 1.f;   // a power of two
                            l *= alpha;
                            m = mn;
                            if (__any_sync(0xffffffffu, alpha < 1.f)) {
                                if (h > 0) {   // the stage's first half is already weighed: 64 keys, in 32 or 64 columns
#pragma unroll 1
                                    for (int c = 0; c < (ES == 1 ? 2 : 4); ++c) {
                                        float y[16];
                                        tc::ld16(scol + 16 * c, y);
                                        tc::wait_ld(y);
                                        const __half2 a2 = __float2half2_rn(alpha);
#pragma unroll
                                        for (int j = 0; j < 16; ++j) {
                                            __half2 v = *reinterpret_cast<__half2*>(&y[j]);
                                            v = __hmul2(v, a2);
                                            y[j] = *reinterpret_cast<float*>(&v);
                                        }
                                        tc::st16(scol + 16 * c, y);
                                    }
                                }
                                if (st > 0) {  // O of the stages before, once their value MMAs are in
                                    ok = __all_sync(0xffffffffu, wait_or_abort(&o_done[(g - 1) & 1], ((g - 1) >> 1) & 1, a.wait_ns, abort_flag));
                                    if (!ok) break;
                                    tc::fence_after_sync();
#pragma unroll 1
                                    for (int c = 0; c < D / 16; ++c) {
                                        float y[16];
                                        tc::ld16(trow + G::OC + 16 * c, y);
                                        tc::wait_ld(y);
#pragma unroll
                                        for (int j = 0; j < 16; ++j) y[j] *= alpha;
                                        tc::st16(trow + G::OC + 16 * c, y);
                                    }
                                }
                            }
                            const float mu = m == -INFINITY ? 0.f : m;
                            sum[0] = sum[1] = sum[2] = sum[3] = 0.f;
#pragma unroll
                            for (int i = 0; i < 64; ++i) {
                                const bool in = (i < 32 ? static_cast<uint32_t>(keep) >> i : static_cast<uint32_t>(keep >> 32) >> (i - 32)) & 1;
                                x[i] = in ? fast_exp2(fmaf(x[i], cs, -mu)) : 0.f;
                                sum[i & 3] += x[i];
                            }
                        }
                        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                        float y[32];
                        if constexpr (ES == 1) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) y[i] = __uint_as_float(pack_f16x2(x[2 * i], x[2 * i + 1]));
                            tc::st32(scol + 64 * h, y);
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                const uint32_t u = pack_bf16x2(x[2 * i], x[2 * i + 1]);
                                y[i] = __uint_as_float(u);
                                x[i] = __uint_as_float(pack_bf16x2(x[2 * i] - __uint_as_float(u << 16),
                                                                   x[2 * i + 1] - __uint_as_float(u & 0xFFFF0000u)));
                            }
                            tc::st32(scol + 64 * h, y);
                            tc::st32(scol + 64 * h + 32, *reinterpret_cast<float(*)[32]>(x));
                        }
                    }
                    if (!ok) break;
                    tc::wait_st();
                    tc::fence_before_sync();
                }
                mbar_arrive(&p_full[buf]);
            }
            if (!ok) break;
            // ---- the next segment's Q (every score MMA of this tile has completed), then what this one gave
            const float vs = a.v_scales ? ld_input(a.v_scales + s.hk) : a.v_scale;
            if (pos < range1) cs = build_q(segment_at(pos, range1, pre, B, H, blocks_of));
            ok = __all_sync(0xffffffffu, wait_or_abort(&o_done[(g - 1) & 1], ((g - 1) >> 1) & 1, a.wait_ns, abort_flag));
            if (!ok) break;
            if (!warp_rows) continue;
            tc::fence_after_sync();
            const bool whole = s.lp0 == 0 && s.lp1 == s.np;
            const int64_t slot = partial_slot(part, blockIdx.x, s.base);
            const float so = l > 0.f ? vs / l : l;   // NaN stays NaN
            uint4* orow = reinterpret_cast<uint4*>(a.out + (static_cast<int64_t>(firsts[s.b] + (rv ? r >> lg : 0)) * a.num_q_heads +
                                                            (s.hk << lg) + (rv ? r & ((1 << lg) - 1) : 0)) * D);
            float4* po = a.part_o + slot * (D / 4) * ROWS + tid;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                float x[32];
                tc::ld32(trow + G::OC + 32 * c, x);
                tc::wait_ld(x);
                if (!rv) continue;
                if (whole) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        orow[4 * c + i] = make_uint4(pack_bf16x2(x[8 * i] * so, x[8 * i + 1] * so),
                                                     pack_bf16x2(x[8 * i + 2] * so, x[8 * i + 3] * so),
                                                     pack_bf16x2(x[8 * i + 4] * so, x[8 * i + 5] * so),
                                                     pack_bf16x2(x[8 * i + 6] * so, x[8 * i + 7] * so));
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        po[(8 * c + i) * ROWS] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                }
            }
            if (rv && !whole) a.part_ml[slot * ROWS + tid] = make_float2(m, l);
            tc::fence_before_sync();   // (O is read before the next segment's first P is handed over)
        }
    } else if (ES == 1 && warp < G::PW0) {
        // ------------------------------------------------------------ converters: V rows to f16
        if constexpr (ES == 1) {
            constexpr int CPR = D / 16;          // chunks per row
            constexpr int STEP = 128 / CPR;      // rows at a time
            const int ct = tid - G::CW0 * 32, c = ct % CPR, k0 = ct / CPR;
            int g = 0;
            bool ok = true;
            for (int64_t pos = range0; pos < range1 && ok;) {
                const Segment s = segment_at(pos, range1, pre, B, H, blocks_of);
                pos = s.base + s.lp1;
                const int nst = (s.lp1 - s.lp0 + PAGES - 1) / PAGES;
                for (int st = 0; st < nst; ++st, ++g) {
                    const int slot = g % R;
                    ok = wait_or_abort(&full[slot], (g / R) & 1, a.wait_ns, abort_flag) &&
                         (g < 2 || wait_or_abort(&o_done[g & 1], ((g >> 1) + 1) & 1, a.wait_ns, abort_flag));
                    if (!ok) break;
                    const uint8_t* src = sm + G::RING + slot * 2 * G::TILE + G::TILE + c * 16;
                    uint8_t* dst = sm + G::V16 + (g & 1) * G::VB + (c >> 2) * G::COL;
                    const int odd = (c >> 2) & 1;   // which of its two chunks a lane writes first: no bank conflicts
#pragma unroll 4
                    for (int i = 0; i < KEYS / STEP; ++i) {
                        const int k = k0 + i * STEP;
                        const uint4 x = *reinterpret_cast<const uint4*>(src + k * D);
                        uint32_t f[8];
                        if constexpr (E5M2) {
                            e5m2x4_to_f16x2x2(x.x, f[0], f[1]);
                            e5m2x4_to_f16x2x2(x.y, f[2], f[3]);
                            e5m2x4_to_f16x2x2(x.z, f[4], f[5]);
                            e5m2x4_to_f16x2x2(x.w, f[6], f[7]);
                        } else {
                            e4m3x4_to_f16x2x2(x.x, f[0], f[1]);
                            e4m3x4_to_f16x2x2(x.y, f[2], f[3]);
                            e4m3x4_to_f16x2x2(x.z, f[4], f[5]);
                            e4m3x4_to_f16x2x2(x.w, f[6], f[7]);
                        }
                        const uint4 first = make_uint4(f[0], f[1], f[2], f[3]), second = make_uint4(f[4], f[5], f[6], f[7]);
                        uint8_t* row = dst + k * 128;
                        const int j = 2 * (c & 3);
                        *reinterpret_cast<uint4*>(row + (((j + odd) ^ (k & 7)) << 4)) = odd ? second : first;
                        *reinterpret_cast<uint4*>(row + (((j + 1 - odd) ^ (k & 7)) << 4)) = odd ? first : second;
                    }
                    tc::fence_proxy_async_smem();
                    mbar_arrive(&v_full[g & 1]);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&empty[slot]);
                }
            }
        }
    } else if (warp < G::MW) {
        // ------------------------------------------------------------ copies
        const int pw = warp - G::PW0;
        const uint64_t pol = (static_cast<int64_t>(a.max_nodes) << lg) <= ROWS ? l2_policy_evict_first() : l2_policy_normal();
        int g = 0;
        bool ok = true;
        // Signals stage x, whose copies are in but for the LAG younger stages'.
        auto signal = [&](int x) {
            tc::fence_proxy_async_smem();   // the tensor cores read what was copied
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[x % R]);
        };
        for (int64_t pos = range0; pos < range1 && ok;) {
            const Segment s = segment_at(pos, range1, pre, B, H, blocks_of);
            pos = s.base + s.lp1;
            const int L = lens[s.b];
            const int page0 = first_key(L, nodes[s.b], a.window) / kBS + s.lp0, np_all = s.lp1 - s.lp0;
            const int nst = (np_all + PAGES - 1) / PAGES;
            const int32_t* bt = a.block_tables + static_cast<int64_t>(s.b) * a.max_blocks_per_seq + page0;
            auto ids_of = [&](int st) { return lane < PAGES && st * PAGES + lane < np_all ? ld_input(bt + st * PAGES + lane) : 0; };
            int ids = ids_of(0), next = ids_of(1);
            for (int st = 0; st < nst; ++st, ++g) {
                const int slot = g % R;
                if (g >= R) {
                    ok = __all_sync(0xffffffffu, wait_or_abort(&empty[slot], (g / R + 1) & 1, a.wait_ns, abort_flag));
                    if (!ok) break;
                }
                if (ids < 0 || ids >= a.num_blocks) {   // block 0 is read instead
                    report(a.err, FP8KV_ERR_INVALID_ARG);
                    ids = 0;
                }
                const int after = ids_of(st + 2);
                const uint32_t dst = sb + G::RING + slot * 2 * G::TILE;
                const int np = np_all - st * PAGES;     // pages left, this stage's included
#pragma unroll
                for (int j0 = 0; j0 < 2 * PAGES; j0 += G::PW) {
                    const int j = j0 + pw, p = j >> 1, is_v = j & 1;
                    const int id = __shfl_sync(0xffffffffu, ids, p & 31);
                    if (j < 2 * PAGES) {
                        const uint8_t* src = (is_v ? a.v_cache : a.k_cache) + (static_cast<int64_t>(id) * H + s.hk) * G::PAGE + lane * 16;
                        const int valid = p < np ? min(kBS, L - (page0 + st * PAGES + p) * kBS) : 0;   // rows of the page
                        constexpr int CPR = G::RB / 16;
#pragma unroll
                        for (int i = 0; i < kBS * CPR / 32; ++i) {
                            const int ci = lane + 32 * i, k = ci / CPR, c = ci % CPR, row = p * kBS + k;
                            uint32_t at;
                            if (ES == 1 && is_v) at = G::TILE + row * G::RB + c * 16;
                            else at = (is_v ? G::TILE : 0) + tile_at<G::RB, G::COL>(row, c);
                            cp_async_16z(dst + at, src + 512 * i, k < valid ? 16 : 0, pol);
                        }
                    }
                }
                cp_async_commit();
                ids = next;
                next = after;
                cp_async_wait<G::LAG>();
                if (g >= G::LAG) signal(g - G::LAG);
            }
        }
        cp_async_wait<0>();                // no copy lands after the CTA is gone
        if (ok)
            for (int x = max(0, g - G::LAG); x < g; ++x) signal(x);
    } else if (lane == 0 && work) {
        // ------------------------------------------------------------ MMA issuer
        constexpr uint32_t id_s = ES == 1 ? tc::idesc_fp8(128, KEYS, E5M2) : tc::idesc_16bit(128, KEYS, true, false);
        constexpr uint32_t id_o = tc::idesc_16bit(128, D, ES == 2, true);
        bool ok = true;
        int g = 0, nseg = 0;
        auto issue_s = [&](int x, int t) {   // S of stage x, tile t
            const uint32_t kt = sb + G::RING + (x % R) * 2 * G::TILE;
            const uint32_t dcol = tm + (T == 1 ? (x & 1) * KEYS : t * 256);
            const uint64_t qd = tc::desc_k_sw128(sb + t * G::QB);
            if constexpr (ES == 1) {
                const uint64_t kd = D == 64 ? tc::desc_k_sw64(kt) : tc::desc_k_sw128(kt);
#pragma unroll
                for (int j = 0; j < 2 * D / 32; ++j) {       // hi, then lo
                    const int jk = j % (D / 32);
                    tc::mma_fp8(dcol, tc::desc_at(qd, (j >> 2) * 16384 + (j & 3) * 32),
                                tc::desc_at(kd, D == 64 ? jk * 32 : (jk >> 2) * G::COL + (jk & 3) * 32), id_s, j > 0);
                }
            } else {
                const uint64_t kd = tc::desc_k_sw128(kt);
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
                    tc::mma_f16(dcol, tc::desc_at(qd, (j >> 2) * 16384 + (j & 3) * 32),
                                tc::desc_at(kd, (j >> 2) * G::COL + (j & 3) * 32), id_s, j > 0);
            }
            tc::commit(&s_full[T == 1 ? x & 1 : t]);
        };
        auto issue_o = [&](int x, int t, bool first) {
            const uint32_t pcol = tm + (T == 1 ? (x & 1) * KEYS : t * 256), ocol = tm + t * 256 + G::OC;
            const uint32_t vt = ES == 1 ? sb + G::V16 + (x & 1) * G::VB : sb + G::RING + (x % R) * 2 * G::TILE + G::TILE;
            const uint64_t vd = tc::desc_mn_sw128(vt, G::COL);
#pragma unroll
            for (int j = 0; j < KEYS / 16; ++j) {
                const uint32_t pc = pcol + (j >> 2) * 64 + (j & 3) * 8;
                tc::mma_f16_ts(ocol, pc, tc::desc_at(vd, j * 2048), id_o, !(first && j == 0));
                if constexpr (ES == 2) tc::mma_f16_ts(ocol, pc + 32, tc::desc_at(vd, j * 2048), id_o, 1);
            }
        };
        auto wait_k = [&](int x) {
            ok = wait_or_abort(&full[x % R], (x / R) & 1, a.wait_ns, abort_flag);
            if (!ok) return false;
            if (x == a.stall_stage && blockIdx.x == 0) {   // test hook: this stage's S never arrives
                mbar_wait_bounded(&end_bar, 0, a.wait_ns);
                ok = false;
                *abort_flag = 1;
                return false;
            }
            tc::fence_after_sync();
            return true;
        };
        for (int64_t pos = range0; pos < range1 && ok; ++nseg) {
            const Segment s = segment_at(pos, range1, pre, B, H, blocks_of);
            pos = s.base + s.lp1;
            const int nst = (s.lp1 - s.lp0 + PAGES - 1) / PAGES;
            ok = wait_or_abort(&q_full, nseg & 1, a.wait_ns, abort_flag);
            if (!ok || !wait_k(g)) break;
            for (int t = 0; t < T; ++t) issue_s(g, t);
            if (ES == 1) tc::commit(&empty[g % R]);
            for (int st = 0; st < nst; ++st, ++g) {
                const bool more = st + 1 < nst;
                if (T == 1 && more) {
                    if (!wait_k(g + 1)) break;
                    issue_s(g + 1, 0);
                    if (ES == 1) tc::commit(&empty[(g + 1) % R]);
                }
                if (ES == 1 && !(ok = wait_or_abort(&v_full[g & 1], (g >> 1) & 1, a.wait_ns, abort_flag))) break;
                for (int t = 0; t < T; ++t) {
                    const int buf = T == 1 ? g & 1 : t, ph = T == 1 ? (g >> 1) & 1 : g & 1;
                    if (!(ok = wait_or_abort(&p_full[buf], ph, a.wait_ns, abort_flag))) break;
                    tc::fence_after_sync();
                    issue_o(g, t, st == 0);
                    if (t == T - 1) {
                        tc::commit(&o_done[g & 1]);
                        if (ES == 2) tc::commit(&empty[g % R]);
                    }
                    if (T == 2 && more) {
                        if (t == 0 && !wait_k(g + 1)) break;
                        issue_s(g + 1, t);
                        if (ES == 1 && t == T - 1) tc::commit(&empty[(g + 1) % R]);
                    }
                }
                if (!ok) break;
            }
        }
        // every MMA this thread issued completes before TMEM is released
        tc::commit(&end_bar);
        mbar_wait_bounded(&end_bar, 0, kWaitNs);
    }
    tc::fence_before_sync();
    __syncthreads();
    if (tid == 0 && *abort_flag) report(a.err, FP8KV_ERR_TIMEOUT);
    if (warp == G::MW) {
        __syncwarp();
        tc::fence_after_sync();
        tc::dealloc(tm, 512);
    }
}

// Joins the partials of the units that several CTAs shared: a block takes 32
// rows of one unit, a lane a row and a warp D / 8 dimensions.
template <int D, int T>
__global__ void __launch_bounds__(256) tree_merge_kernel(const Args a, int blocks) {
    constexpr int ROWS = 128 * T, F4 = D / 32;   // float4 groups per warp
    __shared__ int64_t red[2][8];
    griddep_launch_dependents();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, lg = a.log2_group;
    const int u = blockIdx.x, rb = u % blocks, hk = u / blocks % a.num_kv_heads, b = u / blocks / a.num_kv_heads;
    int64_t before = 0, total = 0;
    for (int i = tid; i < a.batch; i += 256) {
        const Seq s = read_seq(a, i);
        const int64_t pages = static_cast<int64_t>(unit_pages(s.L, s.n, a.window)) * a.num_kv_heads * row_blocks(s.n, lg, ROWS);
        total += pages;
        before += i < b ? pages : 0;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        before += __shfl_xor_sync(0xffffffffu, before, off);
        total += __shfl_xor_sync(0xffffffffu, total, off);
    }
    if (lane == 0) {
        red[0][warp] = before;
        red[1][warp] = total;
    }
    __syncthreads();
    before = total = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        before += red[0][w];
        total += red[1][w];
    }
    const Seq s = read_seq(a, b);
    griddep_wait();   // every block waits: this grid must not complete before the attention has
    if (*reinterpret_cast<volatile uint32_t*>(a.err) == FP8KV_ERR_TIMEOUT) return;
    const int rbs = row_blocks(s.n, lg, ROWS), np = unit_pages(s.L, s.n, a.window);
    const int lrow = blockIdx.y * 32 + lane, r = rb * ROWS + lrow;
    if (rb >= rbs || rb * ROWS + static_cast<int>(blockIdx.y) * 32 >= (s.n << lg)) return;
    const Partition part = make_partition(total, cta_count(total, a.max_ctas, kMinPages));
    const int64_t base = before + (static_cast<int64_t>(hk) * rbs + rb) * np;
    const int c0 = cta_of(part, base), c1 = cta_of(part, base + np - 1);
    if (c0 == c1 || r >= (s.n << lg)) return;    // written by its only CTA
    float M = -INFINITY;
    for (int c = c0; c <= c1; ++c) M = fmaxf(M, a.part_ml[partial_slot(part, c, base) * ROWS + lrow].x);
    const float mu = M == -INFINITY ? 0.f : M;
    float l = 0.f;
    float4 acc[F4];
#pragma unroll
    for (int i = 0; i < F4; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int c = c0; c <= c1; ++c) {
        const int64_t slot = partial_slot(part, c, base);
        const float2 ml = a.part_ml[slot * ROWS + lrow];
        const float f = fast_exp2(ml.x - mu);
        l = fmaf(f, ml.y, l);
        if (f == 0.f && ml.y == 0.f) continue;   // no keys of this row there: its O was never written
#pragma unroll
        for (int i = 0; i < F4; ++i) {
            const float4 x = a.part_o[(slot * (D / 4) + warp * F4 + i) * ROWS + lrow];
            acc[i].x = fmaf(f, x.x, acc[i].x);
            acc[i].y = fmaf(f, x.y, acc[i].y);
            acc[i].z = fmaf(f, x.z, acc[i].z);
            acc[i].w = fmaf(f, x.w, acc[i].w);
        }
    }
    const float vs = a.v_scales ? ld_input(a.v_scales + hk) : a.v_scale;
    const float so = l > 0.f ? vs / l : l;
    uint2* orow = reinterpret_cast<uint2*>(a.out + (static_cast<int64_t>(s.q0 + (r >> lg)) * a.num_q_heads + (hk << lg) +
                                                    (r & ((1 << lg) - 1))) * D) + warp * F4;
#pragma unroll
    for (int i = 0; i < F4; ++i)
        orow[i] = make_uint2(pack_bf16x2(acc[i].x * so, acc[i].y * so), pack_bf16x2(acc[i].z * so, acc[i].w * so));
}

// ---------------------------------------------------------------- host side

// Two tiles a CTA where a unit has more than 128 rows and their accumulators fit.
int tiles_of(int max_nodes, int G, int D) { return static_cast<int64_t>(max_nodes) * G > 128 && D <= 128 ? 2 : 1; }

struct Plan {
    int tiles, blocks, ctas;   // tiles per CTA, row blocks per (sequence, kv head), CTAs
    size_t ml, o, total;       // workspace offsets
};

Plan make_plan(int batch, int max_nodes, int max_seq_len, int G, int Hkv, int D, int window, int sms) {
    Plan p;
    p.tiles = tiles_of(max_nodes, G, D);
    const int rows = 128 * p.tiles;
    p.blocks = static_cast<int>((static_cast<int64_t>(max_nodes) * G + rows - 1) / rows);
    // the most pages a unit may have: a window's keys, the tree's, and a page at either end
    int64_t pages = (static_cast<int64_t>(max_seq_len) + kBS - 1) / kBS;
    if (window > 0) pages = std::min<int64_t>(pages, (static_cast<int64_t>(window) + max_nodes) / kBS + 2);
    p.ctas = cta_count(pages * std::min(batch, kMaxBatch) * Hkv * p.blocks, sms, kMinPages);
    p.ml = 256;
    p.o = p.ml + static_cast<size_t>(2 * p.ctas) * rows * sizeof(float2);
    p.total = p.o + static_cast<size_t>(2 * p.ctas) * rows * D * sizeof(float);
    return p;
}

template <int D, int ES, bool E5M2, int T>
static cudaError_t launch_t(const Args& a, const Plan& p, cudaStream_t s) {
    using G = Geo<D, ES, T>;
    static std::atomic<uint64_t> done_mask{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
    if (bit == 0 || !(done_mask.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(tree_kernel<D, ES, E5M2, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM);
        if (e != cudaSuccess) return e;
        done_mask.fetch_or(bit, std::memory_order_release);
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.ctas);
    cfg.blockDim = dim3(G::THREADS);
    cfg.dynamicSmemBytes = G::SMEM;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, tree_kernel<D, ES, E5M2, T>, a);
    if (e != cudaSuccess || p.ctas == 1) return e;
    cudaLaunchConfig_t mcfg = {};
    mcfg.gridDim = dim3(static_cast<unsigned>(a.batch * a.num_kv_heads * p.blocks), 4 * T);
    mcfg.blockDim = dim3(256);
    mcfg.stream = s;
    mcfg.attrs = attr;
    mcfg.numAttrs = 1;
    return cudaLaunchKernelEx(&mcfg, tree_merge_kernel<D, T>, a, p.blocks);
}

template <int ES, bool E5M2>
static cudaError_t launch(int D, const Args& a, const Plan& p, cudaStream_t s) {
    if (D == 64) return p.tiles == 1 ? launch_t<64, ES, E5M2, 1>(a, p, s) : launch_t<64, ES, E5M2, 2>(a, p, s);
    if (D == 128) return p.tiles == 1 ? launch_t<128, ES, E5M2, 1>(a, p, s) : launch_t<128, ES, E5M2, 2>(a, p, s);
    return launch_t<256, ES, E5M2, 1>(a, p, s);
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
    const size_t need = make_plan(batch, max_nodes, max_seq_len, G, num_kv_heads, head_dim, win, sms).total;
    if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return FP8KV_ERR_WORKSPACE;
    // units of one launch are counted in 31 bits
    if (static_cast<int64_t>(std::min(batch, kMaxBatch)) * num_kv_heads * (max_nodes * G / 128 + 1) >= (INT64_C(1) << 31))
        return FP8KV_ERR_UNSUPPORTED;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    // Batches above kMaxBatch sequences run as consecutive launches, reusing the workspace.
    for (int b0 = 0; b0 < batch; b0 += kMaxBatch) {
        const int nb = std::min(kMaxBatch, batch - b0);
        const Plan p = make_plan(nb, max_nodes, max_seq_len, G, num_kv_heads, head_dim, win, sms);
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
        const cudaError_t e = cache_format == FP8KV_CACHE_BF16   ? launch<2, false>(head_dim, a, p, s)
                              : cache_format == FP8KV_CACHE_E5M2 ? launch<1, true>(head_dim, a, p, s)
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
    return make_plan(batch, max_nodes, max_seq_len, num_q_heads / num_kv_heads, num_kv_heads, head_dim,
                     window > 0 ? window : 0, sms).total;
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
