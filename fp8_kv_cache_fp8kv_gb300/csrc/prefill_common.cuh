// What the chunked-prefill kernels share: their arguments, what a CTA covers,
// the conversion of staged fp8 pages into f16 operand tiles, bounded waits, and
// the merge of split partials.  paged_prefill.cu holds the kernels of the
// per-tensor scales, paged_prefill_block.cu those of block scales.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "fp8kv.h"
#include "ptx.cuh"
#include "tcgen05.cuh"
#include "prefill_plan.h"

namespace fp8kv {

int device_sms(int* sms);  // SM count of the current device (paged_decode.cu)

namespace prefill {

constexpr int kBS = 16;
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kRowsTC = 128;            // query rows per unit of the tcgen05 kernel (one per TMEM lane)
constexpr size_t kHeader = 256;         // error word, then the partials
constexpr float kLog2e = 1.4426950408889634f;

struct Args {
    const uint16_t* q;           // bf16 [num_q_tokens, Hq, D], packed by sequence
    const uint8_t* k_cache;      // E4M3 [num_blocks, Hkv, 16, D]
    const uint8_t* v_cache;
    const int32_t* block_tables; // [B, max_blocks_per_seq]
    const int32_t* seq_lens;     // [B]
    const int32_t* q_starts;     // [B + 1] cumulative query-row offsets
    uint16_t* out;               // bf16 [num_q_tokens, Hq, D]
    uint32_t* err;               // error word
    float* part_o;               // [units][splits][rows][D] unnormalised FP32 outputs
    float2* part_ml;             // [units][splits][rows] (row maximum in log2 units, row sum)
    int64_t num_blocks;
    int64_t num_q_tokens;
    int max_blocks_per_seq;
    int max_seq_len;
    int max_q_len;
    int num_q_heads;
    int num_kv_heads;
    int tiles;                   // query tiles per (sequence, kv head)
    int rows;                    // query rows per tile (kRowsTC)
    int splits;                  // CTAs per unit
    int window;
    float score_scale;           // sm_scale * k_scale * log2(e)
    float v_scale;
    const float* k_page_scales;  // [num_blocks, Hkv] of a block-scaled cache (null otherwise)
    const float* v_page_scales;
    // Failure-path test hook of the tcgen05 kernel (fp8kv_debug_paged_prefill_stall):
    // CTA (0, 0, 0) never issues the score MMAs of stage stall_stage (-1: none),
    // and the MMA waits give up after wait_ns (normally 0.5 s).
    uint64_t wait_ns;
    int stall_stage;
    int log2_group;              // log2 of the query heads per kv head (the block-scaled kernels)
};

__device__ __forceinline__ float bf16_to_f32(uint32_t h) { return __uint_as_float(h << 16); }

__device__ __forceinline__ void cp_async16(uint32_t smem, const void* gmem) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(gmem) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void report(uint32_t* err, uint32_t code) { atomicCAS(err, 0u, code); }

// What one (tile, kv head, sequence) covers: its query rows and the key
// range the rows attend, from the device-side lengths (clamped; an entry
// outside the documented bounds is reported when `report_errors`).
struct Unit {
    int q0;          // first packed query row of the sequence
    int L;           // keys in the cache
    int n;           // query tokens of the sequence
    int rows;        // n * G
    int R0;          // first row of the tile
    int kmin, kmax;  // keys the tile attends (inclusive)
};

// G: the query heads per kv head, or 0: 2^a.log2_group of them.
template <int G>
__device__ __forceinline__ bool make_unit(const Args& a, int b, int tile, bool report_errors, Unit& u) {
    auto times_g = [&](int n) {
        if constexpr (G > 0) return n * G;
        else return n << a.log2_group;
    };
    auto over_g = [&](int r) {
        if constexpr (G > 0) return r / G;
        else return r >> a.log2_group;
    };
    u.q0 = ld_input(a.q_starts + b);
    const int L_in = ld_input(a.seq_lens + b);
    u.L = L_in < 0 ? 0 : min(L_in, a.max_seq_len);
    const int n_in = ld_input(a.q_starts + b + 1) - u.q0;
    int n = n_in < 0 ? 0 : min(n_in, min(u.L, a.max_q_len));
    if (u.q0 < 0 || u.q0 + static_cast<int64_t>(n) > a.num_q_tokens) n = 0;  // never touch rows outside q / out
    if (report_errors && (u.L != L_in || n != n_in)) report(a.err, FP8KV_ERR_INVALID_ARG);
    u.n = n;
    u.rows = times_g(n);
    u.R0 = tile * a.rows;
    if (u.R0 >= u.rows) return false;
    const int p_first = u.L - n + over_g(u.R0);
    u.kmax = u.L - n + over_g(min(u.R0 + a.rows, u.rows) - 1);
    u.kmin = (a.window > 0 && p_first + 1 > a.window) ? p_first + 1 - a.window : 0;
    return true;
}

namespace tcg {
constexpr int kKeys = 64;                       // keys per stage
constexpr int kPages = kKeys / kBS;             // 4 pages per stage
constexpr uint64_t kWaitNs = 500000000ull;      // bounded waits on the MMA barriers
}  // namespace tcg

// Staged key row k, 16-byte chunk c: the XOR keeps the conversions' reads free
// of bank conflicts (8 consecutive keys per K read; 8 keys 8 apart per V read).
// (At d = 256 a key row is 256 bytes: the XOR of the low 3 chunk bits keeps
// each 128-byte half's chunks apart in the same way.)
template <int D>
__device__ __forceinline__ uint32_t stg_k(int k, int c) {
    if constexpr (D >= 128) return k * D + ((c ^ (k & 7)) << 4);
    else return k * 64 + ((c ^ ((k >> 1) & 3)) << 4);
}
template <int D>
__device__ __forceinline__ uint32_t stg_v(int k, int c) {
    if constexpr (D >= 128) return k * D + ((c ^ ((k >> 3) & 7)) << 4);
    else return k * 64 + ((c ^ ((k >> 3) & 3)) << 4);
}
// The same address for a key k = 8 kb + i of key block kb.
template <int D>
__device__ __forceinline__ uint32_t stg_v_kb(int k, int kb, int c) {
    if constexpr (D >= 128) return k * D + ((c ^ kb) << 4);
    else return k * 64 + ((c ^ (kb & 3)) << 4);
}

// One stage's operand tiles, by 128 threads (thread index ct): the staged
// fp8 K rows of the stage's 64 keys into the f16 K tile at kt (64 keys x d,
// K-major, 128-byte swizzle) and the staged V rows, transposed, into the f16
// V^T tile at vt (d rows x 64 keys).  Keys outside [kmin, kmax] or past the
// stage's np pages become zeros in V^T (their scores are masked).
// NT: threads that share the work (128 or 256).
template <int D, int KS = tcg::kKeys * 128, int NT = 128>   // KS: bytes between the K tile's 128-byte atom columns
__device__ __forceinline__ void convert_stage_k(const uint8_t* stg, uint8_t* kt, int ct) {
    // K: thread ct converts CH staged chunks (16 dims each) of key ct & 63
    {
        constexpr int CH = D / 16 * 64 / NT;              // of 128 threads: 8 at d = 256, 4 at 128, 2 at 64
        const int k = ct & 63, part = ct >> 6;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = part * CH + i;                   // staged chunk: dims 16c .. 16c + 15
            const uint4 x = *reinterpret_cast<const uint4*>(stg + stg_k<D>(k, c));
            uint32_t f[8];
            e4m3x4_to_f16x2x2(x.x, f[0], f[1]);
            e4m3x4_to_f16x2x2(x.y, f[2], f[3]);
            e4m3x4_to_f16x2x2(x.z, f[4], f[5]);
            e4m3x4_to_f16x2x2(x.w, f[6], f[7]);
            const int j = 2 * (c & 3);                     // f16 chunk within the 64-dim block c / 4
            uint8_t* dst = kt + (c >> 2) * KS + k * 128;
            *reinterpret_cast<uint4*>(dst + ((j ^ (k & 7)) << 4)) = make_uint4(f[0], f[1], f[2], f[3]);
            *reinterpret_cast<uint4*>(dst + (((j + 1) ^ (k & 7)) << 4)) = make_uint4(f[4], f[5], f[6], f[7]);
        }
    }
}

template <int D, int NT = 128>
__device__ __forceinline__ void convert_stage_v(const uint8_t* stg, uint8_t* vt, int ct, int t0, int np, int kmin,
                                                int kmax) {
    constexpr int VPASS = D > NT ? D / NT : 1;
    // V^T: thread ct (ct < d) converts keys [8kb, 8kb + 8) x dims [8db, 8db + 8)
#pragma unroll
    for (int vp = 0; vp < VPASS; ++vp)
        if (D >= NT || ct < D) {
            const int kb = ct & 7, db = (ct >> 3) + NT / 8 * vp;
            uint32_t w[8][2];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int k = 8 * kb + i, key = t0 + k;
                uint2 x = make_uint2(0, 0);
                if (k < np * kBS && key >= kmin && key <= kmax)
                    x = *reinterpret_cast<const uint2*>(stg + tcg::kKeys * D + stg_v_kb<D>(k, kb, db >> 1) +
                                                        8 * (db & 1));
                w[i][0] = x.x;
                w[i][1] = x.y;
            }
            uint32_t vt4[8][4];   // [dim][key pair]
#pragma unroll
            for (int i2 = 0; i2 < 4; ++i2)
#pragma unroll
                for (int hw = 0; hw < 2; ++hw) {
                    e4m3x4_to_f16x2x2(byte_perm(w[2 * i2][hw], w[2 * i2 + 1][hw], 0x5140u), vt4[4 * hw + 0][i2],
                                      vt4[4 * hw + 1][i2]);
                    e4m3x4_to_f16x2x2(byte_perm(w[2 * i2][hw], w[2 * i2 + 1][hw], 0x7362u), vt4[4 * hw + 2][i2],
                                      vt4[4 * hw + 3][i2]);
                }
#pragma unroll
            for (int dd = 0; dd < 8; ++dd)
                *reinterpret_cast<uint4*>(vt + (8 * db + dd) * 128 + ((kb ^ dd) << 4)) =
                    make_uint4(vt4[dd][0], vt4[dd][1], vt4[dd][2], vt4[dd][3]);
        }
}

__device__ __forceinline__ void named_bar_sync(int id, int n) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}

// Named barrier over n threads that also ORs a predicate across them.
__device__ __forceinline__ bool named_bar_or(int id, int n, bool pred) {
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

// Packed FP32 pairs (sm_100 family): d = a * b + c and d += a, lane by lane,
// one instruction for two values.
__device__ __forceinline__ void fma_f32x2(float& d0, float& d1, float a0, float a1, float b0, float b1, float c0,
                                          float c1) {
    asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
        "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void add_f32x2(float& d0, float& d1, float a0, float a1) {
    asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
        "mov.b64 ra, {%0, %1};\n\tmov.b64 rb, {%2, %3};\n\t"
        "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "+f"(d0), "+f"(d1)
        : "f"(a0), "f"(a1));
}

// A bounded mbarrier wait that also gives up as soon as another thread of the
// CTA has given up (the shared abort flag); the first to run out sets it.
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, uint64_t limit_ns,
                                              volatile int* abort_flag) {
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

// Combines a unit's split partials row by row in FP32: with M the largest
// row maximum, weight_s = 2^(m_s - M), out = v_scale * sum_s weight_s o_s /
// sum_s weight_s l_s, rounded to bf16.  A CTA covers 8 rows of a unit, a
// warp one row; each lane owns D/32 dimensions and keeps 8 splits' loads in
// flight.  Every split writes its partial (zeros and m = -inf when it has no
// keys for the row), so all loads are of written values.
template <int D, int G>
__global__ void __launch_bounds__(256) prefill_merge_kernel(const Args a) {
    constexpr int PER = D / 32;   // dimensions per lane: 2, 4 or 8
    __shared__ float wsm[8][kMaxSplits];
    const int b = blockIdx.z, hk = blockIdx.y;
    const int groups = a.rows / 8;
    const int tile = blockIdx.x / groups, grp = blockIdx.x % groups;
    Unit u;
    const bool ok = make_unit<G>(a, b, tile, false, u);  // only the lengths: read before the wait
    griddep_wait();                                      // the partials are complete and visible
    if (!ok) return;
    // a CTA of this call gave up a wait: its partials are missing, and the
    // error word says so
    if (*reinterpret_cast<volatile uint32_t*>(a.err) == FP8KV_ERR_TIMEOUT) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rr = grp * 8 + warp;                       // row within the tile
    const int r = u.R0 + rr;
    if (r >= u.rows) return;                             // whole warp; no CTA-wide sync follows
    const int64_t unit = (static_cast<int64_t>(b) * a.num_kv_heads + hk) * a.tiles + tile;
    const int64_t slot0 = unit * a.splits * a.rows + rr;  // split s at slot0 + s * rows
    float mmax = -INFINITY;
    for (int sp = lane; sp < a.splits; sp += 32) mmax = fmaxf(mmax, a.part_ml[slot0 + sp * a.rows].x);
#pragma unroll
    for (int off = 16; off; off >>= 1) mmax = fmaxf(mmax, __shfl_xor_sync(0xffffffffu, mmax, off));
    float lsum = 0.f;
    for (int sp = lane; sp < a.splits; sp += 32) {
        const float2 ml = a.part_ml[slot0 + sp * a.rows];
        const float wgt = ml.x == -INFINITY ? 0.f : fast_exp2(ml.x - mmax);
        wsm[warp][sp] = wgt;
        lsum += wgt * ml.y;
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) lsum += __shfl_xor_sync(0xffffffffu, lsum, off);
    __syncwarp();
    const float so = lsum > 0.f ? a.v_scale / lsum : 0.f;
    const float* po = a.part_o + slot0 * D + lane * PER;
    const int64_t stride = static_cast<int64_t>(a.rows) * D;
    float acc[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] = 0.f;
    int sp = 0;
    for (; sp + 8 <= a.splits; sp += 8) {
        float v[8][PER];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int e = 0; e < PER; e += 2) {
                const float2 x = *reinterpret_cast<const float2*>(po + (sp + i) * stride + e);
                v[i][e] = x.x;
                v[i][e + 1] = x.y;
            }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float wgt = wsm[warp][sp + i];
#pragma unroll
            for (int e = 0; e < PER; ++e) acc[e] = fmaf(wgt, v[i][e], acc[e]);
        }
    }
    for (; sp < a.splits; ++sp) {
        const float wgt = wsm[warp][sp];
#pragma unroll
        for (int e = 0; e < PER; e += 2) {
            const float2 x = *reinterpret_cast<const float2*>(po + sp * stride + e);
            acc[e] = fmaf(wgt, x.x, acc[e]);
            acc[e + 1] = fmaf(wgt, x.y, acc[e + 1]);
        }
    }
    uint16_t* orow = a.out + (static_cast<int64_t>(u.q0 + r / G) * a.num_q_heads + hk * G + r % G) * D + lane * PER;
#pragma unroll
    for (int e = 0; e < PER; e += 2)
        *reinterpret_cast<uint32_t*>(orow + e) = pack_bf16x2(acc[e] * so, acc[e + 1] * so);
}

// Kernel kinds (kernel_kind in paged_prefill.cu).
constexpr int kKindTc = 0, kKindWs = 1, kKindWs1 = 2, kKindOne = 3;

// Launches a block-scaled prefill of kind kKindWs or kKindOne and, when its
// key ranges are split, the merge (paged_prefill_block.cu).
cudaError_t launch_block(int head_dim, int G, int kind, const Args& a, int batch, cudaStream_t s);

}  // namespace prefill
}  // namespace fp8kv
