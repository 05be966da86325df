// The kernels of the tree attention, as templates.  tree_attention.cu has the calls
// and the E4M3 cache's instances, tree_attention_e5m2.cu and _bf16.cu the others'.
//
// Speculative decoding: a draft model proposes a tree, this checks all of it at
// once.  The drafted tokens are the sequence's newest; node i attends the
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
//
// Measured (GB300, graph of calls, 32 over 8 heads of 128, E4M3): 8 x 20K tokens,
// 12 to 20 nodes 84.3 us (3.9 TB/s, 503 TFLOP/s; tensor pipe 47% active), 48 to 80
// nodes 223 us (760 TFLOP/s, tensor pipe 56%), 128 nodes 356 us (953 TFLOP/s); 1 x
// 4096, 8 nodes 18.7 us.  What bounds it is the round of a stage,
// S -> weights -> P V -> the next S of the same tile: of 3480 cycles (two tiles,
// 128 keys) 2048 are MMAs.  Alone, no part of it sets the pace: without copies 214
// us instead of 223, without the exponentials 219, without the conversion of V 216,
// with one MMA of each product 190.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "fp8kv.h"
#include "partition.cuh"
#include "ptx.cuh"
#include "tcgen05.cuh"
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

// D elements a head, ES bytes an element, T tiles of 128 rows a CTA, REP copies of
// the rows in a tile.
template <int D, int ES, int T, int REP>
struct Geo {
    static constexpr bool F8 = ES == 1;
    static constexpr int NG = D < 256 ? 2 : 1;                   // softmax groups (warpgroups)
    static constexpr bool ALT = T == 1 && NG == 2;               // the groups take the stages in turn
    static constexpr int KEYS = F8 && D < 256 ? 128 : 64;        // keys per stage
    static constexpr int PAGES = KEYS / kBS;
    static constexpr int RT = 128 / REP;                         // rows in a tile
    static constexpr int ROWS = RT * T;                          // rows of a block (CTA)
    static constexpr int KP = KEYS / REP;                        // keys of a stage that one thread weighs
    static constexpr int HK = KP > 64 ? 64 : KP;                 // ... of which at once
    static constexpr int PIECES = KP / HK;                       // (P is handed over piece by piece)
    static constexpr int RB = D * ES;                            // bytes of a row
    static constexpr int PAGE = kBS * RB;
    static constexpr int TILE = KEYS * RB;                       // K bytes (and V bytes) of a stage
    static constexpr int COL = KEYS * 128;                       // one 128-byte atom column of a tile
    static constexpr int QB = 128 * 2 * D;                       // Q tile: hi and lo E4M3, or bf16
    static constexpr int VB = F8 ? KEYS * 2 * D : 0;             // f16 V tile
    // The ring of staged (K, V): slots.
    static constexpr int R = F8 ? (D == 64 ? 4 : D == 128 && T == 1 ? 3 : 2) : D == 64 ? 6 : D == 128 ? 6 - T : 2;
    // shared memory: Q tiles, the ring, V tiles, tables
    static constexpr int RING = T * QB, V16 = RING + R * 2 * TILE, MASKS = V16 + 2 * VB;
    static constexpr int PRE = MASKS + 8 * NG * 128 * 4;         // int64 [kMaxBatch + 1]
    static constexpr int LENS = PRE + (kMaxBatch + 1) * 8;       // int32 [3][kMaxBatch]: L, n, q0
    static constexpr int PARENTS = LENS + 3 * kMaxBatch * 4;     // uint8 [warps][kMaxNodes]
    static constexpr int SMEM = PARENTS + 4 * NG * kMaxNodes + 1024;
    static_assert(SMEM <= 227 * 1024 - 512, "shared memory");
    // TMEM columns.  Two groups: group i has S at 256 i and O behind it; one: S of
    // two stages, then O.  P lies over S.
    static constexpr int OC = NG == 2 ? 128 : 256;
    static_assert(NG == 2 ? KEYS <= OC && OC + D <= 256 : 2 * KEYS <= OC && OC + D <= 512, "TMEM columns");
    static constexpr int SW = 4 * NG;                            // softmax warps
    static constexpr int CW0 = SW, CW = F8 ? 4 : 0;              // converter warps
    static constexpr int PW0 = CW0 + CW, PW = 3;                 // copy warps
    static constexpr int MW = PW0 + PW;                          // the MMA warp
    static constexpr int THREADS = (MW + 1) * 32;
    // 16 warps are launched with 128 registers a thread, which the softmax, 64 scores
    // in hand, would spill; the warpgroups share them out.
    static constexpr bool SPLIT = THREADS == 512;
    static constexpr int REGS = 128, SOFT_REGS = 160, AUX_REGS = 96;
    static_assert(!SPLIT || 2 * SOFT_REGS + 2 * AUX_REGS == 4 * REGS, "register shares");
};

__device__ __forceinline__ void report(uint32_t* err, uint32_t code) { atomicCAS(err, 0u, code); }

// Barriers by their shared address, which the kernel holds in one register.
__device__ __forceinline__ void arrive_at(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void copies_arrive_at(uint32_t bar) {   // when this thread's copies have landed
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// One look, which may sleep for up to 2 us in the barrier.
__device__ __forceinline__ bool try_wait_at(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 2000;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ uint32_t flag_at(uint32_t at) {
    uint32_t v;
    asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void set_flag_at(uint32_t at) { asm volatile("st.volatile.shared.u32 [%0], 1;" ::"r"(at) : "memory"); }

// A bounded wait that also gives up as soon as another thread of the CTA has (the
// shared abort flag); the first to run out sets it.  It counts the SM's own
// cycles, two to a nanosecond (the clock ends at 2.07 GHz).
__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, uint64_t limit_ns, uint32_t abort_flag) {
    if (try_wait_at(bar, parity)) return true;
    const int64_t t0 = clock64();
    while (true) {
        if (try_wait_at(bar, parity)) return true;
        if (flag_at(abort_flag)) return false;
        if (clock64() - t0 > static_cast<int64_t>(2 * limit_ns)) {
            set_flag_at(abort_flag);
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

// Raises or lowers the calling warpgroup's registers a thread.
template <int N>
__device__ __forceinline__ void more_regs() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void fewer_regs() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// Named barrier over n threads that also ORs a predicate across them.
__device__ __forceinline__ bool bar_or(int id, int n, bool pred) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.red.or.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(pred)), "r"(id), "r"(n)
        : "memory");
    return r != 0;
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

// Row r of a block's Q (zeros from `rows` on) into its row of the Q tile, 16-byte
// chunks swizzled by sw; where PARTS threads share a row, one writes its part.
// Returns the multiplier of the row's raw scores, > 0: the sign of the score scale
// goes into Q, and a scale of zero makes Q zero.
template <int D, int ES, int PARTS>
__device__ __forceinline__ float build_q(const Args& a, int hk, int r, int rows, int q0, int part, uint8_t* to, int sw) {
    const int lg = a.log2_group;
    const bool rv = r < rows;
    const uint4* src = reinterpret_cast<const uint4*>(
        a.q + (static_cast<int64_t>(q0 + (rv ? r >> lg : 0)) * a.num_q_heads + (hk << lg) + (rv ? r & ((1 << lg) - 1) : 0)) * D);
    const float ks = a.k_scales ? ld_input(a.k_scales + hk) : a.k_scale;
    float cs = fabsf(a.sm_scale) * ks * kLog2e;
    const uint32_t flip = a.sm_scale < 0.f ? 0x80008000u : 0u;
    auto put = [&](int c, uint4 x) { *reinterpret_cast<uint4*>(to + (c >> 3) * 16384 + (((c & 7) ^ sw) << 4)) = x; };
    constexpr int CH = D / 8, MINE = CH / PARTS;   // 16-byte chunks of a row, of this thread
    const uint4 zero = make_uint4(0, 0, 0, 0);
    if constexpr (ES == 2) {
        const bool none = !(cs > 0.f);
        if (none) cs = 1.f;
#pragma unroll 8
        for (int i = 0; i < MINE; ++i) {
            const int c = i + part * MINE;
            uint4 x = rv && !none ? ld_input(src + c) : zero;
            x.x ^= flip; x.y ^= flip; x.z ^= flip; x.w ^= flip;
            put(c, x);
        }
    } else {
        // the largest element's exponent (as bits: magnitudes of bf16 order as
        // integers).  All of the row is read at once; d <= 128: what this thread
        // converts stays in registers.
        constexpr bool kHeld = D <= 128;
        uint4 held[kHeld ? MINE : 1];
        uint32_t top = 0;
        auto look = [&](const uint4& x) {
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) top = __vmaxu2(top, w[j] & 0x7FFF7FFFu);
        };
        if constexpr (kHeld) {
            uint4 other[PARTS > 1 ? MINE : 1];
#pragma unroll
            for (int i = 0; i < MINE; ++i) held[i] = rv ? ld_input(src + i + part * MINE) : zero;
            if constexpr (PARTS > 1) {
#pragma unroll
                for (int i = 0; i < MINE; ++i) other[i] = rv ? ld_input(src + i + (part ^ 1) * MINE) : zero;
#pragma unroll
                for (int i = 0; i < MINE; ++i) look(other[i]);
            }
#pragma unroll
            for (int i = 0; i < MINE; ++i) look(held[i]);
        } else {
#pragma unroll 16
            for (int i = 0; i < CH; ++i) look(rv ? ld_input(src + i) : zero);
        }
        top = max(top & 0xFFFFu, top >> 16);
        int shift = 0;   // the largest element to [2^7, 2^8)
        if (top > 0) shift = max(-126, min(126, 7 - (static_cast<int>(top >> 7) - 127)));
        const float up = __uint_as_float(static_cast<uint32_t>(127 + shift) << 23);
        cs *= __uint_as_float(static_cast<uint32_t>(127 - shift) << 23);
        const bool none = !(cs > 0.f);
        if (none) cs = 1.f;
        const float nan = __uint_as_float(0x7FC00000u);
#pragma unroll kHeld ? MINE / 2 : 1
        for (int i = 0; i < MINE / 2; ++i) {       // 16 elements
            const int c = i + part * (MINE / 2);
            uint4 x0 = zero, x1 = zero;
            if constexpr (kHeld) {
                x0 = none ? zero : held[2 * i];
                x1 = none ? zero : held[2 * i + 1];
            } else if (rv && !none) {
                x0 = ld_input(src + 2 * c);
                x1 = ld_input(src + 2 * c + 1);
            }
            const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                hi[j] = lo[j] = 0;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t u = w[2 * j + e] ^ flip;
                    float y0 = __uint_as_float(u << 16) * up, y1 = __uint_as_float(u & 0xFFFF0000u) * up;
                    if (!(fabsf(y0) < 512.f)) y0 = nan;   // an infinity must not saturate
                    if (!(fabsf(y1) < 512.f)) y1 = nan;
                    const uint32_t h = f32x2_to_e4m3x2_satfinite(y0, y1);
                    const uint32_t back = e4m3x2_to_f16x2(static_cast<uint16_t>(h));
                    const __half2 b2 = *reinterpret_cast<const __half2*>(&back);
                    const uint32_t l = f32x2_to_e4m3x2_satfinite(y0 - __low2float(b2), y1 - __high2float(b2));
                    hi[j] |= h << (16 * e);
                    lo[j] |= l << (16 * e);
                }
            }
            put(c, make_uint4(hi[0], hi[1], hi[2], hi[3]));
            put(c + D / 16, make_uint4(lo[0], lo[1], lo[2], lo[3]));
        }
    }
    return cs;
}

// ---------------------------------------------------------------- the kernel
//
// One CTA per SM, persistent over its range of pages (tree_walk.h).  Roles hand
// over through mbarriers, stage by stage (g counts stages over all segments):
//   * copy warps: 16-byte cp.async copies of a stage's pages, K swizzled as the
//     MMA reads it, zeros past the sequence's end; block ids two stages ahead;
//   * converter warps (FP8): V rows to the f16 tile g & 1;
//   * the MMA thread: O += P V of a stage, then S = Q K^T of a later one over the
//     columns that P leaves;
//   * softmax warps, thread = row = TMEM lane: S to P over itself, O rescaled
//     where a reference moves; they also build the Q tiles, between segments,
//     and write out what a segment ends with.
// A row's way through a stage (S, weights, P V) is longer than any one unit's work
// in it, so two groups of softmax warps are under way at once: with T = 2 each has
// a tile of its own and both share the stage's keys; with T = 1 (at most 128 rows)
// they take the stages in turn, each with an O and a reference of its own for the
// same rows, joined where the segment ends.  (d = 256: TMEM holds one O; one group,
// S a stage ahead.)
template <int D, int ES, bool E5M2, int T, int REP>
__global__ void __launch_bounds__(Geo<D, ES, T, REP>::THREADS, 1) tree_kernel(const Args a) {
    using G = Geo<D, ES, T, REP>;
    constexpr int KEYS = G::KEYS, PAGES = G::PAGES, ROWS = G::ROWS, ST = G::NG * 128;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bars[2 * G::R + 14];
    __shared__ int64_t range_sh[2];
    __shared__ uint32_t tmem_base;
    __shared__ int abort_sh;
    uint8_t* sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const uint32_t sb = smem_u32(sm);
    uint32_t* masks = reinterpret_cast<uint32_t*>(sm + G::MASKS);      // [8][ST], a column per softmax thread
    int64_t* pre = reinterpret_cast<int64_t*>(sm + G::PRE);
    int32_t* lens = reinterpret_cast<int32_t*>(sm + G::LENS);
    int32_t *nodes = lens + kMaxBatch, *firsts = nodes + kMaxBatch;
    // between segments, over the masks: (reference, sum) of every softmax thread,
    // then what the copies of a row hand over
    float2* joined = reinterpret_cast<float2*>(sm + G::MASKS);         // [ST]
    float* handed = reinterpret_cast<float*>(sm + G::MASKS) + 2 * ST;  // [NG][REP - 1][RT][.]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int lg = a.log2_group, B = a.batch, H = a.num_kv_heads;

    // the barriers, by address (8 bytes each)
    uint32_t bar0 = smem_u32(bars), abort_flag = smem_u32(&abort_sh);
    asm volatile("" : "+r"(bar0), "+r"(abort_flag));   // (taken once)
    auto full = [&](int j) { return bar0 + 8 * j; };
    auto empty = [&](int j) { return bar0 + 8 * (G::R + j); };
    const uint32_t pairs = bar0 + 16 * G::R;
    auto v_full = [&](int j) { return pairs + 8 * j; };
    auto o_done = [&](int j) { return pairs + 16 + 8 * j; };
    auto s_full = [&](int j) { return pairs + 32 + 8 * j; };
    auto p_full = [&](int j, int piece) { return pairs + 48 + 8 * j + 16 * piece; };
    auto piece_done = [&](int j) { return pairs + 80 + 8 * j; };
    const uint32_t q_full = pairs + 96, end_bar = pairs + 104;
    if (tid == 0) {
        uint64_t* b = bars;
        for (int j = 0; j < G::R; ++j) mbar_init(b + j, G::PW * 32);                        // full: the copying threads, as their copies land
        for (int j = 0; j < G::R; ++j) mbar_init(b + G::R + j, ES == 1 ? 1 + G::CW : 1);    // empty: the score MMAs and the converters; or the value MMAs
        b += 2 * G::R;
        for (int j = 0; j < 2; ++j) {
            mbar_init(b + j, 128);       // v_full: the converters
            mbar_init(b + 2 + j, 1);     // o_done: the value MMAs
            mbar_init(b + 4 + j, 1);     // s_full: the score MMAs
            mbar_init(b + 6 + j, 128);   // p_full: the softmax threads, a stage's first piece,
            mbar_init(b + 8 + j, 128);   // and its second
            mbar_init(b + 10 + j, 1);    // piece_done: the value MMAs of a first piece
        }
        mbar_init(b + 12, ST);           // q_full
        mbar_init(b + 13, 1);            // end
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
                if (s.n > 0) pages = static_cast<int64_t>(unit_pages(s.L, s.n, a.window) + kLeadPages) * H * row_blocks(s.n, lg, ROWS);
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
            const bool timed_out = *reinterpret_cast<volatile uint32_t*>(a.err) == FP8KV_ERR_TIMEOUT;
            const int C = cta_count(run, a.max_ctas, kMinPages);
            const bool work = run > 0 && static_cast<int>(blockIdx.x) < C && !timed_out;
            const Partition part = make_partition(run, C);
            range_sh[0] = work ? range_start(part, blockIdx.x) : 0;
            range_sh[1] = work ? range_start(part, blockIdx.x + 1) : 0;
        }
        __syncwarp();
        if (lane == 0 && range_sh[1] > range_sh[0]) {   // a range that ends in a unit's lead ends before that unit
            const Segment s = segment_at(range_sh[1] - 1, range_sh[1], pre, B, [&](int b) { return row_blocks(nodes[b], lg, ROWS); },
                                         [&](int b) { return unit_pages(lens[b], nodes[b], a.window); });
            if (s.lp1 == 0) range_sh[1] = s.base;
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = tmem_base;
    const int64_t range0 = range_sh[0], range1 = range_sh[1];
    const bool work = range0 < range1;
    auto segment_of = [&](int64_t pos) {
        return segment_at(pos, range1, pre, B, [&](int b) { return row_blocks(nodes[b], lg, ROWS); },
                          [&](int b) { return unit_pages(lens[b], nodes[b], a.window); });
    };

    if (warp < G::SW) {
        // ------------------------------------------------------------ softmax
        if constexpr (G::SPLIT) more_regs<G::SOFT_REGS>();
        constexpr int RT = G::RT, KP = G::KP, HK = G::HK;
        const int grp = warp >> 2, tile = T == 1 ? 0 : grp;
        const uint32_t trow = tm + (static_cast<uint32_t>((warp & 3) * 32) << 16) + grp * 256;
        uint8_t* qt = sm + tile * G::QB;
        const int myrow = tid & 127;                                   // row of the tile
        const int lrow = tile * RT + myrow % RT, copy = myrow / RT;    // row of the block; which copy of it (the same for a warp)
        // (the threads of a row in two groups share its Q and its output, a half each)
        const int half = G::ALT ? grp : 0;
        constexpr int PARTS = G::ALT ? 2 : 1;
        constexpr bool kShared = G::ALT || REP > 1;
        uint8_t* my_parents = sm + G::PARENTS + warp * kMaxNodes;
        // One turn a segment: its stages; the next one's Q; what it gave.  (The
        // first turn has a Q to build only.)
        int g = 0;
        bool ok = true;
        float cs = 0.f;
        int64_t pos = range0;
        Segment s = {};
#pragma unroll 1
        for (bool first = true; work; first = false) {
            float m = 0.f, l = 0.f, f0 = 1.f, f1 = 0.f;
            int nst = 0, g0 = 0;
            if (!first) {
            const int L = lens[s.b], n = nodes[s.b], ctx = L - n;
            const int page0 = first_key(L, n, a.window) / kBS;
            const int t_first = (page0 + s.lp0) * kBS, t_end = min((page0 + s.lp1) * kBS, L);
            nst = (s.lp1 - s.lp0 + PAGES - 1) / PAGES;
            const int rows = n << lg, r = s.rb * ROWS + lrow;
            const bool rv = r < rows;
            const bool warp_rows = s.rb * ROWS + tile * RT + (warp & 3) * 32 % RT < rows;   // a warp of no rows only keeps the handshake
            // ---- which drafted tokens the row's node attends, and its depth
            int lo = 0;
            if (warp_rows && (t_end > ctx || a.window > 0)) {
                // the tree's parents, a byte each (a parent is below 255; 255: a root)
                for (int i = lane; i < n; i += 32) {
                    const int p = ld_input(a.parents + firsts[s.b] + i);
                    if (p >= i || p < -1) report(a.err, FP8KV_ERR_INVALID_ARG);
                    my_parents[i] = static_cast<uint8_t>(p >= i || p < 0 ? 255 : p);
                }
                __syncwarp();
                uint32_t* mine = masks + tid;
#pragma unroll
                for (int w = 0; w < 8; ++w) mine[w * ST] = 0;
                int depth = -1;
                for (int i = rv ? r >> lg : -1; i >= 0;) {
                    ++depth;
                    if (a.window <= 0 || depth < a.window) mine[(i >> 5) * ST] |= 1u << (i & 31);
                    const int p = my_parents[i];
                    i = p == 255 ? -1 : p;
                }
                if (a.window > 0) lo = max(0, ctx + depth + 1 - a.window);
            }
            const int wlo = __reduce_max_sync(0xffffffffu, rv ? lo : 0);

            m = rv ? -INFINITY : 0.f;   // (the tile's rows past the last: zero scores)
            g0 = g;
            bool fresh = true;          // a row of the warp has met no key yet
            for (int st = 0; st < nst && ok; ++st, ++g) {
                if (G::ALT && (g & 1) != grp) continue;
                const int buf = T == 1 ? g & 1 : tile, ph = T == 1 ? (g >> 1) & 1 : g & 1;
                const uint32_t scol = trow + (G::NG == 1 ? buf * KEYS : 0);
                ok = __all_sync(0xffffffffu, wait_or_abort(s_full(buf), ph, a.wait_ns, abort_flag));
                if (!ok) break;
                if (warp_rows) {
                    tc::fence_after_sync();
                    const int t0 = t_first + st * KEYS;
                    const bool masked = t0 + KEYS > min(ctx, t_end) || t0 < wlo;
#pragma unroll 1
                    for (int h = 0; h < G::PIECES; ++h) {
                        const int k0 = copy * KP + HK * h;     // first key of the stage that is weighed here
                        float x[HK];
                        float sum[4];
                        auto load = [&]() {
#pragma unroll
                            for (int c = 0; c < HK / 32; ++c) tc::ld32(scol + k0 + 32 * c, *reinterpret_cast<float(*)[32]>(x + 32 * c));
#pragma unroll
                            for (int c = 0; c < HK / 32; ++c) tc::wait_ld(*reinterpret_cast<float(*)[32]>(x + 32 * c));
                        };
                        auto weigh = [&](float ref) {
                            sum[0] = sum[1] = sum[2] = sum[3] = 0.f;
#pragma unroll
                            for (int i = 0; i < HK; i += 2) {
                                fma2(x[i], x[i + 1], cs, -ref);
                                x[i] = fast_exp2(x[i]);
                                x[i + 1] = fast_exp2(x[i + 1]);
                                add2(sum[i & 2], sum[(i & 2) + 1], x[i], x[i + 1]);
                            }
                        };
                        // A row's first keys, masked keys, and weights that grew too large are
                        // looked at first, for where the reference belongs; then the scores
                        // are read again (they are not in registers while O is rescaled).
                        bool look = masked || fresh, settled = false;
#pragma unroll 1
                        while (true) {
                            load();
                            if (masked) {   // the keys that the row attends
                                int th = t0 + k0;
                                asm volatile("" : "+r"(th));   // (not worked out ahead: 5 x 9K tokens in bf16, d 64, 90.3 us, 95.7 without)
                                uint64_t keep = ones(min(ctx, t_end) - th) & ~ones(lo - th);
                                if (t_end > ctx && th + HK > ctx) {
                                    const uint32_t* mine = masks + tid;
                                    const int off = max(0, th - ctx), w = off >> 5, sh = off & 31;
                                    const uint32_t w0 = w < 8 ? mine[w * ST] : 0, w1 = w < 7 ? mine[(w + 1) * ST] : 0,
                                                   w2 = w < 6 ? mine[(w + 2) * ST] : 0;
                                    const uint64_t bits = static_cast<uint64_t>(__funnelshift_r(w0, w1, sh)) |
                                                          (static_cast<uint64_t>(__funnelshift_r(w1, w2, sh)) << 32);
                                    keep |= (th < ctx ? bits << (ctx - th) : bits) & ones(t_end - th);
                                }
                                const uint32_t k_lo = static_cast<uint32_t>(keep), k_hi = static_cast<uint32_t>(keep >> 32);
#pragma unroll
                                for (int i = 0; i < HK; ++i)
                                    if (!(((i < 32 ? k_lo : k_hi) >> (i & 31)) & 1)) x[i] = -INFINITY;
                            }
                            if (!look) {
                                weigh(m == -INFINITY ? 0.f : m);
                                if (settled) break;
                                look = __any_sync(0xffffffffu, (sum[0] + sum[1]) + (sum[2] + sum[3]) > kMaxSum);
                                if (!look) break;
                                continue;
                            }
                            float big[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                            for (int i = 4; i < HK; ++i) big[i & 3] = fmaxf(big[i & 3], x[i]);
                            float top = fmaxf(fmaxf(big[0], big[1]), fmaxf(big[2], big[3]));
                            if (top > -INFINITY) top = ceilf(top * cs - kRoom);
                            const float mn = fmaxf(m, top);
                            const float alpha = m > -INFINITY ? fast_exp2(m - mn) : 1.f;   // a power of two
                            l *= alpha;
                            m = mn;
                            look = false;
                            settled = true;
                            fresh = __any_sync(0xffffffffu, m == -INFINITY);
                            if (!__any_sync(0xffffffffu, alpha < 1.f)) continue;
                            // O of what was summed before, once its value MMAs are in: up to the
                            // stage before (of this group), or this stage's first piece
                            const int gp = G::ALT ? g - 2 : g - 1;
                            if (h > 0 || gp >= g0) {
                                ok = __all_sync(0xffffffffu, h > 0 ? wait_or_abort(piece_done(buf), ph, a.wait_ns, abort_flag)
                                                                   : wait_or_abort(o_done(gp & 1), (gp >> 1) & 1, a.wait_ns, abort_flag));
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
                        if (!ok) break;
                        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                        // P: 64 keys in 64 columns of theirs, f16 in the first 32, or bf16
                        // and what it rounds off; 32 keys at a time (a store takes
                        // consecutive registers).  A copy's other keys weigh nothing.
                        auto put_p = [&](int key, int off, const float (&y)[16]) {
                            tc::st16(scol + key / 64 * 64 + key % 64 / 2 + off, y);
                        };
#pragma unroll
                        for (int c = 0; c < HK; c += 32) {
                            float y[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                y[i] = __uint_as_float(ES == 1 ? pack_f16x2(x[c + 2 * i], x[c + 2 * i + 1]) : pack_bf16x2(x[c + 2 * i], x[c + 2 * i + 1]));
                            put_p(k0 + c, 0, y);
                            if constexpr (ES == 2) {
#pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    const uint32_t u = __float_as_uint(y[i]);
                                    y[i] = __uint_as_float(pack_bf16x2(x[c + 2 * i] - __uint_as_float(u << 16),
                                                                       x[c + 2 * i + 1] - __uint_as_float(u & 0xFFFF0000u)));
                                }
                                put_p(k0 + c, 32, y);
                            }
                        }
                        if constexpr (REP > 1) {
                            float y[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) y[i] = 0.f;
#pragma unroll
                            for (int c = KP; c < KEYS; c += 32) {
                                const int key = (copy * KP + c) % KEYS;
                                put_p(key, 0, y);
                                if constexpr (ES == 2) put_p(key, 32, y);
                            }
                        }
                        tc::wait_st();
                        tc::fence_before_sync();
                        arrive_at(p_full(buf, h));
                    }
                    if (!ok) break;
                } else {
                    for (int h = 0; h < G::PIECES; ++h) arrive_at(p_full(buf, h));
                }
            }
            // ---- what the segment gave, once its value MMAs are in.  Threads that share
            // a row (two groups, copies) meet here, and every softmax thread comes here
            // once a segment, whatever became of its waits.
            if (ok) ok = __all_sync(0xffffffffu, wait_or_abort(o_done((g - 1) & 1), ((g - 1) >> 1) & 1, a.wait_ns, abort_flag));
            if constexpr (kShared) {
                if (G::ALT && ok && nst > 1)
                    ok = __all_sync(0xffffffffu, wait_or_abort(o_done(g & 1), ((g - 2) >> 1) & 1, a.wait_ns, abort_flag));
                ok = !bar_or(1, ST, !ok);            // (the masks are done with)
                if (!ok) break;
                joined[tid] = make_float2(m, l);
                bar_or(1, ST, false);
                m = -INFINITY;
                l = 0.f;
#pragma unroll
                for (int i = 0; i < REP; ++i)
#pragma unroll
                    for (int j = 0; j < PARTS; ++j) m = fmaxf(m, joined[j * 128 + i * RT + myrow % RT].x);
                const float mu = m == -INFINITY ? 0.f : m;
#pragma unroll
                for (int i = 0; i < REP; ++i)
#pragma unroll
                    for (int j = 0; j < PARTS; ++j) {
                        const float2 x = joined[j * 128 + i * RT + myrow % RT];
                        const float f = fast_exp2(x.x - mu);     // a power of two
                        l = fmaf(f, x.y, l);
                        if (i == copy && j == 0) f0 = f;
                        if (i == copy && j == 1) f1 = f;
                    }
            } else if (!ok) {
                break;
            }
            }
            // the next segment's Q (every score MMA of this one has completed)
            const bool more = pos < range1;
            Segment after = {};
            if (more) {
                after = segment_of(pos);
                cs = build_q<D, ES, PARTS>(a, after.hk, after.rb * ROWS + lrow, nodes[after.b] << lg, firsts[after.b], half,
                                           qt + myrow * 128, myrow & 7);
                tc::fence_proxy_async_smem();   // the tile is read by the tensor cores
                arrive_at(q_full);
                pos = unit_end(after);
            }
            if (!first) {
            tc::fence_after_sync();
            const int r = s.rb * ROWS + lrow, rows = nodes[s.b] << lg;
            const bool rv = r < rows, warp_rows = s.rb * ROWS + tile * RT + (warp & 3) * 32 % RT < rows;
            const float vs = a.v_scales ? ld_input(a.v_scales + s.hk) : a.v_scale;
            const bool whole = s.lp0 == 0 && s.lp1 == s.np;
            const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (s.base + kLeadPages >= range0);   // (partial_slot)
            const float so = whole ? (l > 0.f ? vs / l : l) : 1.f;   // NaN stays NaN
            uint4* orow = reinterpret_cast<uint4*>(a.out + (static_cast<int64_t>(firsts[s.b] + (rv ? r >> lg : 0)) * a.num_q_heads +
                                                            (s.hk << lg) + (rv ? r & ((1 << lg) - 1) : 0)) * D);
            float4* po = a.part_o + slot * (D / 4) * ROWS + lrow;
            const bool has0 = !G::ALT || nst > 1 || (g0 & 1) == 0, has1 = G::ALT && (nst > 1 || (g0 & 1) == 1);
            const uint32_t ocol = (G::ALT ? trow - grp * 256 : trow) + G::OC;
            f0 *= so;
            f1 *= so;
            constexpr int EC = 16;                                   // columns at a time
#pragma unroll 1
            for (int c = half * (D / EC / PARTS); c < (half + 1) * (D / EC / PARTS); ++c) {
                float x[EC];
                if (warp_rows) {
                    if (has0) {
                        tc::ld16(ocol + EC * c, x);
                        tc::wait_ld(x);
#pragma unroll
                        for (int i = 0; i < EC; ++i) x[i] *= f0;
                    }
                    if constexpr (G::ALT) {
                        if (has1) {
                            float y[EC];
                            tc::ld16(ocol + 256 + EC * c, y);
                            tc::wait_ld(y);
#pragma unroll
                            for (int i = 0; i < EC; ++i) x[i] = has0 ? fmaf(y[i], f1, x[i]) : y[i] * f1;
                        }
                    }
                }
                if constexpr (REP > 1) {
                    // copies 1 .. hand over, copy 0 adds: in two steps of EC / 2 columns
                    constexpr int HC = EC / 2;
                    float4* mine = reinterpret_cast<float4*>(handed) + ((half * (REP - 1) + copy - 1) * RT + myrow % RT) * (HC / 4);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if (copy > 0)
#pragma unroll
                            for (int i = 0; i < HC / 4; ++i)
                                mine[i] = make_float4(x[HC * e + 4 * i], x[HC * e + 4 * i + 1], x[HC * e + 4 * i + 2], x[HC * e + 4 * i + 3]);
                        bar_or(2 + half, 128, false);
                        if (copy == 0)
#pragma unroll
                            for (int o = 1; o < REP; ++o) {
                                const float4* from = reinterpret_cast<const float4*>(handed) + ((half * (REP - 1) + o - 1) * RT + myrow % RT) * (HC / 4);
#pragma unroll
                                for (int i = 0; i < HC / 4; ++i) {
                                    const float4 y = from[i];
                                    x[HC * e + 4 * i] += y.x;
                                    x[HC * e + 4 * i + 1] += y.y;
                                    x[HC * e + 4 * i + 2] += y.z;
                                    x[HC * e + 4 * i + 3] += y.w;
                                }
                            }
                        bar_or(2 + half, 128, false);
                    }
                }
                if (!rv || copy > 0) continue;
                if (whole) {
#pragma unroll
                    for (int i = 0; i < EC / 8; ++i)
                        orow[EC / 8 * c + i] = make_uint4(pack_bf16x2(x[8 * i], x[8 * i + 1]), pack_bf16x2(x[8 * i + 2], x[8 * i + 3]),
                                                          pack_bf16x2(x[8 * i + 4], x[8 * i + 5]), pack_bf16x2(x[8 * i + 6], x[8 * i + 7]));
                } else {
#pragma unroll
                    for (int i = 0; i < EC / 4; ++i)
                        po[(EC / 4 * c + i) * ROWS] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                }
            }
            if (rv && !whole && half == 0 && copy == 0) a.part_ml[slot * ROWS + lrow] = make_float2(m, l);
            tc::fence_before_sync();   // (O is read before the next segment's first P is handed over ...
            if constexpr (kShared) bar_or(1, ST, false);   // ... by every thread of the row, and the masks may be written)
            }
            if (!more) break;
            s = after;
        }
    } else {
    if constexpr (G::SPLIT) fewer_regs<G::AUX_REGS>();
    if (ES == 1 && warp < G::PW0) {
        // ------------------------------------------------------------ converters: V rows to f16
        if constexpr (ES == 1) {
            constexpr int CPR = D / 16;          // chunks per row (staged swizzled, as K)
            constexpr int STEP = 128 / CPR;      // rows at a time
            const int ct = tid - G::CW0 * 32, c = ct % CPR, k0 = ct / CPR;
            int g = 0;
            bool ok = true;
            for (int64_t pos = range0; pos < range1 && ok;) {
                const Segment s = segment_of(pos);
                pos = unit_end(s);
                const int nst = (s.lp1 - s.lp0 + PAGES - 1) / PAGES;
                for (int st = 0; st < nst; ++st, ++g) {
                    const int slot = g % G::R;
                    ok = wait_or_abort(full(slot), (g / G::R) & 1, a.wait_ns, abort_flag) &&
                         (g < 2 || wait_or_abort(o_done(g & 1), ((g >> 1) + 1) & 1, a.wait_ns, abort_flag));
                    if (!ok) break;
                    const uint8_t* src = sm + G::RING + slot * 2 * G::TILE + G::TILE;
                    uint8_t* dst = sm + G::V16 + (g & 1) * G::VB + (c >> 2) * G::COL;
                    const int odd = (c >> 2) & 1;   // which of its two chunks a lane writes first: no bank conflicts
#pragma unroll 4
                    for (int i = 0; i < KEYS / STEP; ++i) {
                        const int k = k0 + i * STEP;
                        const uint4 x = *reinterpret_cast<const uint4*>(src + tile_at<D, G::COL>(k, c));
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
                    arrive_at(v_full(g & 1));
                    __syncwarp();
                    if (lane == 0) arrive_at(empty(slot));
                }
            }
        }
    } else if (warp < G::MW) {
        // ------------------------------------------------------------ copies
        const int pw = warp - G::PW0;
        const uint64_t pol = (static_cast<int64_t>(a.max_nodes) << lg) <= ROWS ? l2_policy_evict_first() : l2_policy_normal();
        int g = 0;
        bool ok = true;
        for (int64_t pos = range0; pos < range1 && ok;) {
            const Segment s = segment_of(pos);
            pos = unit_end(s);
            const int L = lens[s.b], page0 = first_key(L, nodes[s.b], a.window) / kBS + s.lp0, np = s.lp1 - s.lp0;
            const int32_t* table = a.block_tables + static_cast<int64_t>(s.b) * a.max_blocks_per_seq + page0;
            // block ids, a lane a page, two stages ahead
            auto ids_at = [&](int p) { return lane < PAGES && p + lane < np ? ld_input(table + p + lane) : 0; };
            int ids = ids_at(0), next = ids_at(PAGES);
            for (int p0 = 0; p0 < np; p0 += PAGES, ++g) {
                const int slot = g % G::R;
                if (g >= G::R) {
                    ok = __all_sync(0xffffffffu, wait_or_abort(empty(slot), (g / G::R + 1) & 1, a.wait_ns, abort_flag));
                    if (!ok) break;
                }
                if (ids < 0 || ids >= a.num_blocks) {   // block 0 is read instead
                    report(a.err, FP8KV_ERR_INVALID_ARG);
                    ids = 0;
                }
                const int after = ids_at(p0 + 2 * PAGES);
                const uint32_t dst = sb + G::RING + slot * 2 * G::TILE;
#pragma unroll 1
                for (int p = pw; p < PAGES; p += G::PW) {
                    const int64_t at = (static_cast<int64_t>(__shfl_sync(0xffffffffu, ids, p)) * H + s.hk) * G::PAGE + lane * 16;
                    const int valid = p0 + p < np ? min(kBS, L - (page0 + p0 + p) * kBS) : 0;   // rows of the page
                    constexpr int CPR = G::RB / 16, STEPS = kBS * CPR / 32;
                    const uint8_t* ks = a.k_cache + at;
                    const uint8_t* vs = a.v_cache + at;
#pragma unroll
                    for (int i = 0; i < STEPS; ++i) {
                        const int ci = lane + 32 * i, k = ci / CPR, c = ci % CPR;
                        const uint32_t to = dst + tile_at<G::RB, G::COL>(p * kBS + k, c);
                        const int bytes = k < valid ? 16 : 0;
                        cp_async_16z(to, ks + 512 * i, bytes, pol);
                        cp_async_16z(to + G::TILE, vs + 512 * i, bytes, pol);
                    }
                }
                copies_arrive_at(full(slot));
                ids = next;
                next = after;
            }
        }
        cp_async_wait_all();               // no copy lands after the CTA is gone
    } else if (work) {
        // ------------------------------------------------------------ MMA issuer
        // (the whole warp: what it branches on is the same in every lane)
        constexpr uint32_t id_s = ES == 1 ? tc::idesc_fp8(128, KEYS, E5M2) : tc::idesc_16bit(128, KEYS, true, false);
        constexpr uint32_t id_o = tc::idesc_16bit(128, D, ES == 2, true);
        const uint32_t tmu = __shfl_sync(0xffffffffu, tm, 0), sbu = __shfl_sync(0xffffffffu, sb, 0);
        const uint64_t q_desc = tc::desc_k_sw128(sbu);
        const uint64_t k_desc = ES == 1 && D == 64 ? tc::desc_k_sw64(sbu + G::RING) : tc::desc_k_sw128(sbu + G::RING);
        const uint64_t v_desc = tc::desc_mn_sw128(sbu + (ES == 1 ? G::V16 : G::RING + G::TILE), G::COL);
        bool ok = true;
        int g = 0, nseg = 0;
        auto wait = [&](uint32_t bar, uint32_t parity) {
            ok = __all_sync(0xffffffffu, wait_or_abort(bar, parity, a.wait_ns, abort_flag));
            return ok;
        };
        // Where stage x of tile t has its S and P, and its O.
        auto s_col = [&](int x, int t) { return tmu + (G::NG == 1 ? (x & 1) * KEYS : (T == 1 ? x & 1 : t) * 256); };
        auto o_col = [&](int x, int t) { return tmu + (G::NG == 1 ? 0 : (T == 1 ? x & 1 : t) * 256) + G::OC; };
        auto issue_s = [&](int x, int t) {   // S of stage x, tile t
            const uint32_t dcol = s_col(x, t);
            const uint64_t qd = tc::desc_at(q_desc, t * G::QB), kd = tc::desc_at(k_desc, x % G::R * 2 * G::TILE);
            if constexpr (ES == 1) {
#pragma unroll
                for (int j = 0; j < 2 * D / 32; ++j) {       // hi, then lo
                    const int jk = j % (D / 32);
                    tc::warp_mma_fp8(dcol, tc::desc_at(qd, (j >> 2) * 16384 + (j & 3) * 32),
                                     tc::desc_at(kd, D == 64 ? jk * 32 : (jk >> 2) * G::COL + (jk & 3) * 32), id_s, j > 0);
                }
            } else {
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
                    tc::warp_mma_f16(dcol, tc::desc_at(qd, (j >> 2) * 16384 + (j & 3) * 32),
                                     tc::desc_at(kd, (j >> 2) * G::COL + (j & 3) * 32), id_s, j > 0);
            }
            tc::warp_commit_at(s_full(T == 1 ? x & 1 : t));
            if (ES == 1 && t == T - 1) tc::warp_commit_at(empty(x % G::R));
        };
        auto issue_o = [&](int x, int t, int piece, bool first) {   // a piece of P V
            constexpr int N = KEYS / 16 / G::PIECES;               // MMAs of a piece (16 keys each)
            const int key = piece * (KEYS / G::PIECES);
            const uint32_t pcol = s_col(x, t) + key, ocol = o_col(x, t);   // (64 keys in 64 columns)
            const uint64_t vd = tc::desc_at(v_desc, (ES == 1 ? (x & 1) * G::VB : x % G::R * 2 * G::TILE) + key * 128);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const uint32_t pc = pcol + (j >> 2) * 64 + (j & 3) * 8;
                tc::warp_mma_f16_ts(ocol, pc, tc::desc_at(vd, j * 2048), id_o, !(first && piece == 0 && j == 0));
                if constexpr (ES == 2) tc::warp_mma_f16_ts(ocol, pc + 32, tc::desc_at(vd, j * 2048), id_o, 1);
            }
        };
        auto wait_k = [&](int x) {
            if (!wait(full(x % G::R), (x / G::R) & 1)) return false;
            if (x == a.stall_stage && blockIdx.x == 0) {   // test hook: this stage's S never arrives
                wait_or_abort(end_bar, 0, a.wait_ns, abort_flag);
                set_flag_at(abort_flag);
                __syncwarp();
                ok = false;
            }
            return ok;
        };
        // S runs ahead of P V by two stages, over the columns that the P V before it
        // has read (by one with two tiles, which alternate).
        constexpr int AHEAD = T == 1 ? 2 : 1;
        for (int64_t pos = range0; pos < range1 && ok; ++nseg) {
            const Segment s = segment_of(pos);
            pos = unit_end(s);
            const int nst = __shfl_sync(0xffffffffu, (s.lp1 - s.lp0 + PAGES - 1) / PAGES, 0);
            if (!wait(q_full, nseg & 1)) break;
#pragma unroll 1
            for (int i = 0; i < nst + AHEAD && ok; ++i) {
                const int xs = g + i, xo = xs - AHEAD;      // the stage of S, of P V
                const bool has_o = i >= AHEAD, has_s = i < nst;
                if (has_o && !(ES == 1 ? wait(v_full(xo & 1), (xo >> 1) & 1) : wait(full(xo % G::R), (xo / G::R) & 1))) break;
                if (ES == 2 && has_o) tc::fence_proxy_async_smem();   // the copies are generic writes, the tensor cores read them
#pragma unroll 1
                for (int t = 0; t < T; ++t) {
                    if (has_o) {
                        const int buf = T == 1 ? xo & 1 : t, ph = T == 1 ? (xo >> 1) & 1 : xo & 1;
#pragma unroll 1
                        for (int piece = 0; piece < G::PIECES; ++piece) {
                            if (!wait(p_full(buf, piece), ph)) break;
                            tc::fence_after_sync();
                            issue_o(xo, t, piece, G::ALT ? i < 4 : i == AHEAD);
                            if (piece + 1 < G::PIECES) tc::warp_commit_at(piece_done(buf));
                        }
                        if (!ok) break;
                        if (t == T - 1) {
                            tc::warp_commit_at(o_done(xo & 1));
                            if (ES == 2) tc::warp_commit_at(empty(xo % G::R));
                        }
                    }
                    if (has_s) {
                        if (t == 0) {
                            if (!wait_k(xs)) break;
                            tc::fence_proxy_async_smem();
                        }
                        issue_s(xs, t);
                    }
                }
            }
            g += nst;
        }
        // every MMA this warp issued completes before TMEM is released
        tc::warp_commit_at(end_bar);
        for (const int64_t t0 = clock64(); !try_wait_at(end_bar, 0) && clock64() - t0 < static_cast<int64_t>(2 * kWaitNs);) {}
        __syncwarp();
    }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (tid == 0 && flag_at(abort_flag)) report(a.err, FP8KV_ERR_TIMEOUT);
    if (warp == G::MW) {
        __syncwarp();
        tc::fence_after_sync();
        tc::dealloc(tm, 512);
    }
}

// Joins the partials of the units that several CTAs shared: a block takes 32
// rows of one unit, a lane a row and a warp D / 8 dimensions.
template <int D>
__global__ void __launch_bounds__(256) tree_merge_kernel(const Args a, int blocks, int block_rows) {
    constexpr int F4 = D / 32;           // float4 groups per warp
    constexpr int AT = D == 256 ? 4 : 8; // partials read at once
    __shared__ int64_t red[2][8];
    __shared__ float2 ml[AT][32];
    __shared__ bool timed_out;
    griddep_launch_dependents();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, lg = a.log2_group;
    const int u = blockIdx.x, rb = u % blocks, hk = u / blocks % a.num_kv_heads, b = u / blocks / a.num_kv_heads;
    int64_t before = 0, total = 0;
    for (int i = tid; i < a.batch; i += 256) {
        const Seq s = read_seq(a, i);
        const int64_t pages = s.n > 0 ? static_cast<int64_t>(unit_pages(s.L, s.n, a.window) + kLeadPages) * a.num_kv_heads * row_blocks(s.n, lg, block_rows) : 0;
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
    const int rbs = row_blocks(s.n, lg, block_rows), np = unit_pages(s.L, s.n, a.window);
    const int lrow = blockIdx.y * 32 + lane, r = rb * block_rows + lrow;
    const bool some = rb < rbs && rb * block_rows + static_cast<int>(blockIdx.y) * 32 < (s.n << lg);
    int c0 = 0, c1 = 0;
    if (some) {
        const Partition part = make_partition(total, cta_count(total, a.max_ctas, kMinPages));
        const int64_t base = before + (static_cast<int64_t>(hk) * rbs + rb) * (np + kLeadPages) + kLeadPages;   // its first page
        c0 = cta_of(part, base);
        c1 = cta_of(part, base + np - 1);
    }
    griddep_wait();   // every block waits: this grid must not complete before the attention has
    if (c0 == c1) return;   // no rows, or written by its only CTA
    if (tid == 0) timed_out = *reinterpret_cast<volatile uint32_t*>(a.err) == FP8KV_ERR_TIMEOUT;
    // c0 began the unit in its range's last segment, the others have it in their first (partial_slot)
    auto slot_of = [&](int c) { return 2 * static_cast<int64_t>(c) + (c == c0); };
    float M = -INFINITY, l = 0.f;
    float4 acc[F4];
#pragma unroll
    for (int i = 0; i < F4; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = c0; c <= c1; c += AT) {
        const int k = min(AT, c1 - c + 1);
        if (warp < k) ml[warp][lane] = a.part_ml[slot_of(c + warp) * block_rows + lrow];
        float4 x[AT][F4];
#pragma unroll
        for (int j = 0; j < AT; ++j)
            if (j < k)
#pragma unroll
                for (int i = 0; i < F4; ++i) x[j][i] = a.part_o[(slot_of(c + j) * (D / 4) + warp * F4 + i) * block_rows + lrow];
        __syncthreads();
        float top = M;
        for (int j = 0; j < k; ++j) top = fmaxf(top, ml[j][lane].x);
        const float mu = top == -INFINITY ? 0.f : top;
        const float f = fast_exp2(M - mu);
        M = top;
        l *= f;
#pragma unroll
        for (int i = 0; i < F4; ++i) {
            acc[i].x *= f; acc[i].y *= f; acc[i].z *= f; acc[i].w *= f;
        }
#pragma unroll
        for (int j = 0; j < AT; ++j)
            if (j < k) {
                const float2 y = ml[j][lane];
                const float w = fast_exp2(y.x - mu);
                l = fmaf(w, y.y, l);
#pragma unroll
                for (int i = 0; i < F4; ++i) {
                    acc[i].x = fmaf(w, x[j][i].x, acc[i].x);
                    acc[i].y = fmaf(w, x[j][i].y, acc[i].y);
                    acc[i].z = fmaf(w, x[j][i].z, acc[i].z);
                    acc[i].w = fmaf(w, x[j][i].w, acc[i].w);
                }
            }
        __syncthreads();
    }
    if (timed_out || r >= (s.n << lg)) return;   // (the loop has met once at least)
    const float vs = a.v_scales ? ld_input(a.v_scales + hk) : a.v_scale;
    const float so = l > 0.f ? vs / l : l;
    uint2* orow = reinterpret_cast<uint2*>(a.out + (static_cast<int64_t>(s.q0 + (r >> lg)) * a.num_q_heads + (hk << lg) +
                                                    (r & ((1 << lg) - 1))) * D) + warp * F4;
#pragma unroll
    for (int i = 0; i < F4; ++i)
        orow[i] = make_uint2(pack_bf16x2(acc[i].x * so, acc[i].y * so), pack_bf16x2(acc[i].z * so, acc[i].w * so));
}

// ---------------------------------------------------------------- launch

// How a call is cut (make_plan, tree_attention.cu): tiles a CTA, copies of the rows
// in a tile, rows of a block, blocks per (sequence, kv head), CTAs; workspace offsets.
struct Plan {
    int tiles, copies, rows, blocks, ctas;
    size_t ml, o, total;
};

template <int D, int ES, bool E5M2, int T, int REP>
static cudaError_t launch_t(const Args& a, const Plan& p, cudaStream_t s) {
    using G = Geo<D, ES, T, REP>;
    static std::atomic<uint64_t> done_mask{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
    if (bit == 0 || !(done_mask.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(tree_kernel<D, ES, E5M2, T, REP>, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM);
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
    e = cudaLaunchKernelEx(&cfg, tree_kernel<D, ES, E5M2, T, REP>, a);
    if (e != cudaSuccess || p.ctas == 1) return e;
    cudaLaunchConfig_t mcfg = {};
    mcfg.gridDim = dim3(static_cast<unsigned>(a.batch * a.num_kv_heads * p.blocks), static_cast<unsigned>(p.rows / 32));
    mcfg.blockDim = dim3(256);
    mcfg.stream = s;
    mcfg.attrs = attr;
    mcfg.numAttrs = 1;
    return cudaLaunchKernelEx(&mcfg, tree_merge_kernel<D>, a, p.blocks, p.rows);
}

template <int D, int ES, bool E5M2>
static cudaError_t launch_d(const Args& a, const Plan& p, cudaStream_t s) {
    if constexpr (D <= 128) {
        if (p.tiles == 2) return launch_t<D, ES, E5M2, 2, 1>(a, p, s);
        if constexpr (ES == 1)
            if (p.copies == 4) return launch_t<D, ES, E5M2, 1, 4>(a, p, s);
    }
    return p.copies == 2 ? launch_t<D, ES, E5M2, 1, 2>(a, p, s) : launch_t<D, ES, E5M2, 1, 1>(a, p, s);
}

template <int ES, bool E5M2>
static cudaError_t launch(int D, const Args& a, const Plan& p, cudaStream_t s) {
    return D == 64 ? launch_d<64, ES, E5M2>(a, p, s) : D == 128 ? launch_d<128, ES, E5M2>(a, p, s) : launch_d<256, ES, E5M2>(a, p, s);
}

cudaError_t launch_e5m2(int head_dim, const Args& a, const Plan& p, cudaStream_t s);
cudaError_t launch_bf16(int head_dim, const Args& a, const Plan& p, cudaStream_t s);

}  // namespace tree
}  // namespace fp8kv
