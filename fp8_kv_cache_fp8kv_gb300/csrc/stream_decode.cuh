// The streaming decode kernel (per-warp cp.async rings, tensor-core engine),
// the merge of its split partials and their launch, as templates: the
// translation units that instantiate them are paged_decode.cu (per-tensor and
// per-head scales, E5M2, bf16) and paged_decode_block.cu (block scales).
// paged_decode.cu's opening comment describes the whole.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "fp8kv.h"
#include "partition.cuh"
#include "ptx.cuh"
#include "walk.cuh"

namespace fp8kv {

constexpr int kBS = 16;                    // tokens per page (block_size)
constexpr int kNCW = 4;                    // consumer warps per CTA
constexpr int kNPW = 2;                    // producer warps: one issues K copies, one V copies
constexpr int kThreads = (kNCW + kNPW) * 32;
constexpr int kStageHalf = 4096;           // K bytes (and V bytes) per stage
constexpr int kStageBytes = 2 * kStageHalf;
constexpr int kCtasPerSm = 2;
constexpr int kMaxBatch = 512;             // sequences per launch; larger batches run in chunks
constexpr int kMaxMergeSplits = 1024;      // CTAs per launch are capped at this (the merge keeps one weight each)
constexpr int kMinPagesPerCta = 16;
constexpr int kMaxG = 16;                  // query heads per kv head at most (partial (max, sum) entries per slot)
constexpr uint64_t kWaitLimitNs = 500000000ull;  // 0.5 s: far beyond any legitimate wait
constexpr float kLog2e = 1.4426950408889634f;

struct DecodeArgs {
    const uint16_t* q;          // bf16 [B, Hq, D]
    const uint16_t* k_new;      // bf16 [B, Hkv, D] newest rows to append first, or null
    const uint16_t* v_new;
    uint8_t* k_cache;           // the caches (written only when appending)
    uint8_t* v_cache;
    float k_scale_raw;          // per-tensor scales (the append divides by them)
    float v_scale_raw;
    const float* k_scales;      // [Hkv] per-kv-head scales, or null for the per-tensor ones
    const float* v_scales;
    const float* k_page_scales; // [num_blocks][cache kv heads] scales of a block-scaled cache
    const float* v_page_scales; // (read by the BS kernels only)
    float sm_scale;
    const int32_t* block_tables;
    const int32_t* seq_lens;
    uint16_t* out;              // bf16 [B, Hq, D]
    uint32_t* err;              // workspace error word
    int decode_ctas;            // grid size of the decode kernel (the merge recomputes its split)
    float2* part_ml;            // [B*Hkv + ctas][kMaxG] (max, sum) in log2 units
    float* part_o;              // [B*Hkv + ctas][G][D]  unnormalised partial outputs
    int32_t* split_cnt;         // [B*Hkv] partials written so far per split unit (tensor-core engine);
                                // zero between calls: the CTA that completes a unit resets it
    int inline_merge;           // 1: the CTA that completes a split unit merges it; 0: the merge kernel does
    int64_t num_blocks;
    int max_blocks_per_seq;
    int max_seq_len;
    int batch;
    int num_q_heads;
    int num_kv_heads;           // units per sequence: the cache's kv heads << kv_shift
    int kv_shift;               // 1 when g = 16 runs as two units of 8 query heads per cache head
    int window;
    float score_scale;          // sm_scale * k_scale * log2(e)
    float v_scale;
    // Failure-path test hook of the CUDA-core engine (fp8kv_debug_paged_decode_stall):
    // the K producer of CTA 0 never issues stage stall_stage (-1: none), and
    // the ring waits give up after wait_ns (normally kWaitLimitNs).
    uint64_t wait_ns;
    int stall_stage;
};

// Geometry of one head dimension D with ES-byte elements (1: E4M3 codes,
// 2: bf16 for the bf16 twin).  Pages, boxes, stages and per-thread loads are
// in bytes; k-steps and m-tiles in elements.
template <int D, int ES = 1>
struct Geo {
    static constexpr int RB = D * ES;                   // bytes of one token row of one head
    static constexpr int PAGE = kBS * RB;               // bytes of one K (or V) page
    static constexpr int SH = PAGE > kStageHalf ? PAGE : kStageHalf;  // K bytes (and V bytes) per stage
    static constexpr int SB = 2 * SH;                   // bytes per stage
    static constexpr int PPS = SH / PAGE;               // pages per stage: 4, 2, 1
    static constexpr int HALVES = RB >= 128 ? RB / 128 : 1;
    static constexpr int ROWB = RB >= 128 ? 128 : RB;   // bytes per smem row of one TMA box
    static constexpr int BOX = kBS * ROWB;              // bytes of one TMA box
    static constexpr int DBOX = ROWB / ES;              // elements per box row
    static constexpr int KS = D / 16;                   // k-steps of the score MMA
    static constexpr int MT = D / 16;                   // m-tiles of the value MMA
    static constexpr int KW = ROWB / 4;                 // K bytes a thread reads per row per box
    static constexpr int KSH = KW / (4 * ES);           // k-steps per box
    static constexpr int VW = ROWB / 8;                 // V bytes a thread reads per token per box
    static constexpr int VWD = VW / ES;                 // ... in elements
    static constexpr int MTH = VWD / 2;                 // m-tiles per box
    static constexpr int XW = MT * 4 + 4;               // per-lane words exchanged in the warp merge
    static constexpr int STAGES = XW > 40 ? 8 : 12;     // ring slots (a multiple of kNCW)
    static_assert(PPS >= 1 && PPS * PAGE == SH, "stage must hold whole pages");
    static_assert(STAGES % kNCW == 0, "every consumer warp owns whole ring slots");
    static_assert(32 % PPS == 0, "a 32-page block-id batch holds whole stages");
    static_assert(KSH * HALVES == KS && MTH * HALVES == MT, "boxes cover the head dimension");
};

// Byte offset of (row r, byte o) inside one TMA box written with the 128-byte
// (rows of 128 B) or 64-byte (rows of 64 B) swizzle: the 16-byte chunk index
// is XORed with address bits 7.. of the row start.
template <int ROWB>
__device__ __forceinline__ uint32_t swz(int r, int o) {
    if constexpr (ROWB == 128)
        return r * 128 + ((((o >> 4) ^ (r & 7)) << 4) | (o & 15));
    else
        return r * 64 + ((((o >> 4) ^ ((r >> 1) & 3)) << 4) | (o & 15));
}

// The streaming kernel's own layout of a staged page (its cp.async copies and
// its fragment loads are the only users, so it need not match TMA's): rows of
// 128 bytes as swz<128>; rows of 64 bytes (d = 64) go in pairs into 128-byte
// lines whose eight 16-byte chunks are XOR-permuted per line, the halves
// swapped on every other line.  Measured on the gpt-oss-like step: 0.2 us
// faster than swz<64>.  Its 8-byte value loads still take 4 wavefronts instead
// of 2 (a half-warp reads pieces of four rows, two of them in the same half
// of their lines); a permutation that makes them conflict-free (chunk bits
// 2, 1, 0 flipped by line bits 0, 1, 2) measured 0.14 us slower, so the
// shared-memory wavefronts are not what bounds this kernel.
template <int ROWB>
__device__ __forceinline__ uint32_t sswz(int r, int o) {
    if constexpr (ROWB == 128) {
        return swz<128>(r, o);
    } else {
        const int line = r >> 1;
        const int c = ((r & 1) << 2) | (o >> 4);
        const int g = ((line & 1) << 2) | ((line >> 1) & 3);
        return static_cast<uint32_t>(line * 128 + ((c ^ g) << 4) + (o & 15));
    }
}

__device__ __forceinline__ void report(uint32_t* err, uint32_t code) { atomicCAS(err, 0u, code); }

__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kNCW * 32) : "memory"); }

// Named barrier 1 over the first NW warps of the CTA.
template <int NW>
__device__ __forceinline__ void consumer_sync_n() { asm volatile("bar.sync 1, %0;" ::"n"(NW * 32) : "memory"); }

__device__ __forceinline__ float bf16_to_f32(uint16_t h) { return __uint_as_float(static_cast<uint32_t>(h) << 16); }

__device__ __forceinline__ uint16_t f32_to_bf16(float x) {
    __nv_bfloat16 h = __float2bfloat16_rn(x);
    return *reinterpret_cast<uint16_t*>(&h);
}

// Per-sequence geometry: the attended keys of a length-L sequence are
// [first_token, L); they occupy pages first_token/16 .. (L-1)/16.
__device__ __forceinline__ int clamp_len(int L, int max_len) { return L < 0 ? 0 : (L > max_len ? max_len : L); }
__device__ __forceinline__ int first_token(int L, int window) { return (window > 0 && L > window) ? L - window : 0; }
__device__ __forceinline__ int attended_pages(int L, int window) {
    return L > 0 ? (L - 1) / kBS - first_token(L, window) / kBS + 1 : 0;
}

// Block id of page `lane` of a batch; an id outside [0, num_blocks) is
// reported and returned as -1 (its page is then read from block 0 and never
// written).
__device__ __forceinline__ int load_block_id(const int32_t* row, int lane, int count, int64_t num_blocks,
                                             uint32_t* err) {
    int id = 0;
    if (lane < count) {
        id = ld_input(row + lane);
        if (id < 0 || id >= num_blocks) {
            report(err, FP8KV_ERR_INVALID_ARG);
            id = -1;
        }
    }
    return id;
}

// One new K or V row (D bf16 values) held by a warp: lane l owns elements
// [l*D/32, (l+1)*D/32).
template <int D>
struct NewRow {
    uint32_t w[D / 64];
};

template <int D>
__device__ __forceinline__ void load_new_row(NewRow<D>& r, const uint16_t* src_row, int lane) {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(src_row + lane * (D / 32));
#pragma unroll
    for (int i = 0; i < D / 64; ++i) r.w[i] = ld_input(p + i);
}

// Quantise-on-append of the warp's row: code = E4M3_satfinite(fp32(x) / scale)
// with one IEEE divide and one RNE conversion (the same arithmetic as the
// quant_append kernel), stored at dst_row.
template <int D, bool E5M2 = false>
__device__ __forceinline__ void store_new_row(const NewRow<D>& r, uint8_t* dst_row, int lane, float scale) {
    uint16_t c[D / 64];
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
        const float e0 = __uint_as_float(r.w[i] << 16), e1 = __uint_as_float(r.w[i] & 0xFFFF0000u);
        c[i] = E5M2 ? f32x2_to_e5m2x2_satfinite(__fdiv_rn(e0, scale), __fdiv_rn(e1, scale))
                    : f32x2_to_e4m3x2_satfinite(__fdiv_rn(e0, scale), __fdiv_rn(e1, scale));
    }
    uint8_t* dst = dst_row + lane * (D / 32);
    if constexpr (D == 64) {
        *reinterpret_cast<uint16_t*>(dst) = c[0];
    } else if constexpr (D == 128) {
        *reinterpret_cast<uint32_t*>(dst) = static_cast<uint32_t>(c[0]) | (static_cast<uint32_t>(c[1]) << 16);
    } else {
        *reinterpret_cast<uint2*>(dst) =
            make_uint2(static_cast<uint32_t>(c[0]) | (static_cast<uint32_t>(c[1]) << 16),
                       static_cast<uint32_t>(c[2]) | (static_cast<uint32_t>(c[3]) << 16));
    }
}

// Query fragments of one (sequence, kv head): the B operand of the score MMA,
// pre-scaled per head by a power of two so the f16 copy is exact (largest |q|
// in [2^14, 2^15)); cs[j] scales the raw score of head 2*tig+j back and into
// log2 units.
// Four FP8 codes (one 32-bit word, code 0 in the low byte) -> two f16x2:
// codes 0,1 in lo and 2,3 in hi; exact for both formats.
template <bool E5M2>
__device__ __forceinline__ void codes4_to_f16x2x2(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if constexpr (E5M2)
        e5m2x4_to_f16x2x2(w, lo, hi);
    else
        e4m3x4_to_f16x2x2(w, lo, hi);
}

// Score multiplier (sm_scale * k_scale * log2 e, multiplied in that order as
// the host does for the per-tensor scale) and V scale of kv head hk.
__device__ __forceinline__ float unit_score_scale(const DecodeArgs& a, int hk) {
    return a.k_scales ? (a.sm_scale * ld_input(a.k_scales + (hk >> a.kv_shift))) * kLog2e : a.score_scale;
}

__device__ __forceinline__ float unit_v_scale(const DecodeArgs& a, int hk) {
    return a.v_scales ? ld_input(a.v_scales + (hk >> a.kv_shift)) : a.v_scale;
}

template <int D, int G>
__device__ __forceinline__ void load_query(const DecodeArgs& a, int b, int hk, int gid, int tig,
                                           uint32_t (&qf)[Geo<D>::KS][2], float (&cs)[2], int h0 = 0) {
    using Gm = Geo<D>;
    uint32_t qw[Gm::HALVES][Gm::KSH][2];
    float qmax = 0.f;
#pragma unroll
    for (int hh = 0; hh < Gm::HALVES; ++hh) {
#pragma unroll
        for (int c = 0; c < Gm::KW / 8; ++c) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (h0 + gid < G)
                v = ld_input(reinterpret_cast<const uint4*>(a.q + (static_cast<int64_t>(b) * a.num_q_heads + hk * G + h0 + gid) * D +
                                                         hh * 128 + tig * Gm::KW) + c);
            const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                qw[hh][c * 2 + e / 2][e % 2] = w4[e];
                qmax = fmaxf(qmax, fmaxf(fabsf(bf16_to_f32(w4[e] & 0xFFFF)), fabsf(bf16_to_f32(w4[e] >> 16))));
            }
        }
    }
    qmax = fmaxf(qmax, __shfl_xor_sync(0xffffffffu, qmax, 1));
    qmax = fmaxf(qmax, __shfl_xor_sync(0xffffffffu, qmax, 2));
    int shift = 0;
    if (qmax > 0.f) {
        const int e = static_cast<int>((__float_as_uint(qmax) >> 23) & 0xFF) - 127;
        shift = max(-100, min(100, 14 - e));
    }
    const float up = __uint_as_float(static_cast<uint32_t>(127 + shift) << 23);
#pragma unroll
    for (int hh = 0; hh < Gm::HALVES; ++hh)
#pragma unroll
        for (int kk = 0; kk < Gm::KSH; ++kk)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t w = qw[hh][kk][e];
                qf[hh * Gm::KSH + kk][e] = pack_f16x2(bf16_to_f32(w & 0xFFFF) * up, bf16_to_f32(w >> 16) * up);
            }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int sh = __shfl_sync(0xffffffffu, shift, (2 * tig + j) * 4);
        cs[j] = unit_score_scale(a, hk) * __uint_as_float(static_cast<uint32_t>(127 - sh) << 23);
    }
}

// bf16 twin: the g query rows of kv head hk as bf16 B fragments of the score
// MMA (no scaling: the cache is bf16 too), in the k order that matches how a
// thread reads its K bytes: MMA k = 2*tig + e and 2*tig + 8 + e of k-step kk
// of box hh are elements hh*64 + tig*16 + 4*kk + e and ... + 2 + e.
template <int D, int G>
__device__ __forceinline__ void load_query_bf16(const DecodeArgs& a, int b, int hk, int gid, int tig,
                                                uint32_t (&qf)[Geo<D, 2>::KS][2], float (&cs)[2], int h0 = 0) {
    using Gm = Geo<D, 2>;
#pragma unroll
    for (int hh = 0; hh < Gm::HALVES; ++hh) {
        uint4 v0 = make_uint4(0, 0, 0, 0), v1 = make_uint4(0, 0, 0, 0);
        if (h0 + gid < G) {
            const uint4* src = reinterpret_cast<const uint4*>(
                a.q + (static_cast<int64_t>(b) * a.num_q_heads + hk * G + h0 + gid) * D + hh * Gm::DBOX + tig * 16);
            v0 = ld_input(src);
            v1 = ld_input(src + 1);
        }
        const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
        for (int kk = 0; kk < Gm::KSH; ++kk) {
            qf[hh * Gm::KSH + kk][0] = w[2 * kk];
            qf[hh * Gm::KSH + kk][1] = w[2 * kk + 1];
        }
    }
    cs[0] = cs[1] = a.score_scale;
}

// The V bytes one thread feeds to the value MMA from one box of a page:
// token rows 2*tig, 2*tig+1, 2*tig+8, 2*tig+9, VW bytes each at column
// gid*VW.  Rows outside [lo, L) (or a page past the stage's last) read as
// zero codes, so stale NaN codes never meet a zero probability.
template <int D, int ES>
__device__ __forceinline__ void load_v_box(const uint8_t* box, int gid, int tig, int t0, int lo, int L, bool page_ok,
                                           uint32_t (&v)[4][Geo<D, ES>::VW / 4]) {
    using Gm = Geo<D, ES>;
    const bool edge = t0 < lo || t0 + kBS > L;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int row = 2 * tig + (r & 1) + 8 * (r >> 1);
        if (page_ok) {
            if constexpr (Gm::VW == 16) {
                const uint4 x = *reinterpret_cast<const uint4*>(box + sswz<Gm::ROWB>(row, gid * 16));
                v[r][0] = x.x; v[r][1] = x.y; v[r][2] = x.z; v[r][3] = x.w;
            } else {
                const uint2 x = *reinterpret_cast<const uint2*>(box + sswz<Gm::ROWB>(row, gid * 8));
                v[r][0] = x.x; v[r][1] = x.y;
            }
        }
        if (!page_ok || (edge && (t0 + row < lo || t0 + row >= L))) {
#pragma unroll
            for (int ww = 0; ww < Gm::VW / 4; ++ww) v[r][ww] = 0u;
        }
    }
}

// Folds state (m2, l2, o2) into (m, l, o): the FP32 softmax-merge identity.
template <int MT>
__device__ __forceinline__ void combine(float (&m)[2], float (&l)[2], float (&o)[MT][4], const float (&m2)[2],
                                        const float (&l2)[2], const float (&o2)[MT][4]) {
    float f1[2], f2[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const float M = fmaxf(m[j], m2[j]);
        const float Mu = M == -INFINITY ? 0.f : M;
        f1[j] = fast_exp2(m[j] - Mu);
        f2[j] = fast_exp2(m2[j] - Mu);
        l[j] = l[j] * f1[j] + l2[j] * f2[j];
        m[j] = M;
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        o[mt][0] = o[mt][0] * f1[0] + o2[mt][0] * f2[0];
        o[mt][1] = o[mt][1] * f1[1] + o2[mt][1] * f2[1];
        o[mt][2] = o[mt][2] * f1[0] + o2[mt][2] * f2[0];
        o[mt][3] = o[mt][3] * f1[1] + o2[mt][3] * f2[1];
    }
}

template <int MT>
__device__ __forceinline__ void publish(float* x, int lane, const float (&m)[2], const float (&l)[2],
                                        const float (&o)[MT][4]) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int r = 0; r < 4; ++r) x[(mt * 4 + r) * 32 + lane] = o[mt][r];
    x[(MT * 4 + 0) * 32 + lane] = m[0];
    x[(MT * 4 + 1) * 32 + lane] = m[1];
    x[(MT * 4 + 2) * 32 + lane] = l[0];
    x[(MT * 4 + 3) * 32 + lane] = l[1];
}

template <int MT>
__device__ __forceinline__ void absorb(const float* x, int lane, float (&m)[2], float (&l)[2], float (&o)[MT][4]) {
    float m2[2], l2[2], o2[MT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int r = 0; r < 4; ++r) o2[mt][r] = x[(mt * 4 + r) * 32 + lane];
    m2[0] = x[(MT * 4 + 0) * 32 + lane];
    m2[1] = x[(MT * 4 + 1) * 32 + lane];
    l2[0] = x[(MT * 4 + 2) * 32 + lane];
    l2[1] = x[(MT * 4 + 3) * 32 + lane];
    combine<MT>(m, l, o, m2, l2, o2);
}

// ---------------------------------------------------------------- streaming decode (per-warp rings)
//
// The same split-context flash-decoding step with a different copy pipeline:
// there are no producer warps.  Every consumer warp streams its own pages
// with 16-byte cp.async copies into a private ring of R stages in shared
// memory, R-1 stages ahead of the stage it computes.  Each warp takes one
// contiguous share of every segment of its CTA (the segment's pages cut into
// NW equal runs), so its block ids are consecutive entries of one block-table
// row; they are read 32 at a time, one window ahead.  Copies complete by
// themselves (no barrier handshake, no bounded waits); the warps of a CTA
// meet only at segment ends, to merge their partial softmax states.

// One stage: the np (<= PPS) pages of K at kst and V at vst, holding tokens
// [tok_base, tok_base + 16*np) of a sequence attended on [lo, L), folded into
// the running state (m, l, o) of the warp.  The query heads sit on the MMA's
// n side, 8 per n-tile: NT = 2 n-tiles carry g = 16 heads, and the converted
// K and V fragments feed both tiles' MMAs, so each page is read once.
// BS: with ks, vs = psc[p] the scales of page p, a key's weight is
// w = 2^(s ks + log2 vs - m), so the V scale costs an addend of the score's FMA;
// the row sum takes w / vs, and out = o / l.  m is the largest s ks + log2 vs
// less kRoom, rounded up so that no weight passes 2^15 (f16 ends at 65504) at
// any size of the scores.  P is the f16 of w: what it rounds is relative to the
// largest p vs, as the answer is; 2^-29 of that still has 11 bits, and below
// 2^-40 of it nothing is left.  (Relative to the largest p, with the page's P.V
// tile multiplied by vs, a page of 2^26 times the others' V scale and 2^-26 of
// their probability, half the answer, was lost.)
// Measured against a factor per page in FP32 (the page's V scale times
// 2^(page maximum - m), P relative to the page): 8 x 20K, d = 128, g = 4: 62.2 us
// both; 8 x 16K, d = 64, g = 8: 32.4 and 34.8; 4 x 32K, d = 128, g = 16: 69.1 and
// 70.3; 8 x 8K, d = 256: 20.7 and 20.2.  The kernel that lost such pages took 61.7,
// 32.4, 65.7 and 19.9 (g = 16 at d = 128 now has 255 registers and spills 16 bytes).
constexpr float kRoom = 15.f;

template <int D, int ES, bool E5M2, int NT, bool BS>
__device__ __forceinline__ void tc_stage(const uint8_t* kst, const uint8_t* vst, const float2* psc, int np,
                                         int tok_base, int lo, int L,
                                         int gid, int tig, const uint32_t (&qf)[NT][Geo<D, ES>::KS][2],
                                         const float (&cs)[NT][2], float (&m)[NT][2], float (&l)[NT][2],
                                         float (&o)[NT][Geo<D, ES>::MT][4]) {
    using Gm = Geo<D, ES>;
    constexpr bool kEarlyV = Gm::MT == 8 && NT == 1;
    // ---- (d = 128) the stage's V fragments into registers first, so their
    // shared-memory latency overlaps the score math
    uint32_t vr[kEarlyV ? Gm::PPS : 1][kEarlyV ? Gm::HALVES : 1][4][Gm::VW / 4];
    if constexpr (kEarlyV) {
#pragma unroll
        for (int p = 0; p < Gm::PPS; ++p)
#pragma unroll
            for (int hh = 0; hh < Gm::HALVES; ++hh)
                load_v_box<D, ES>(vst + p * Gm::PAGE + hh * Gm::BOX, gid, tig, tok_base + p * kBS, lo, L, p < np,
                                  vr[p][hh]);
    }

    // ---- scores S^T[token][head] = K Q^T, two accumulator chains per page
    // and n-tile (even and odd k-steps) to halve the dependent MMA latency
    float sc[Gm::PPS][NT][4];
#pragma unroll
    for (int p = 0; p < Gm::PPS; ++p) {
        float s1[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) sc[p][t][r] = s1[t][r] = 0.f;
        if (p < np) {
#pragma unroll
            for (int hh = 0; hh < Gm::HALVES; ++hh) {
                const uint8_t* box = kst + p * Gm::PAGE + hh * Gm::BOX;
                uint32_t w0[Gm::KW / 4], w1[Gm::KW / 4];
#pragma unroll
                for (int cc = 0; cc < Gm::KW / 16; ++cc) {
                    const uint4 x = *reinterpret_cast<const uint4*>(box + sswz<Gm::ROWB>(gid, tig * Gm::KW + 16 * cc));
                    const uint4 y = *reinterpret_cast<const uint4*>(box + sswz<Gm::ROWB>(gid + 8, tig * Gm::KW + 16 * cc));
                    w0[4 * cc + 0] = x.x; w0[4 * cc + 1] = x.y; w0[4 * cc + 2] = x.z; w0[4 * cc + 3] = x.w;
                    w1[4 * cc + 0] = y.x; w1[4 * cc + 1] = y.y; w1[4 * cc + 2] = y.z; w1[4 * cc + 3] = y.w;
                }
#pragma unroll
                for (int kk = 0; kk < Gm::KSH; ++kk) {
                    const int ks = hh * Gm::KSH + kk;
                    uint32_t af[4];
                    if constexpr (ES == 1) {
                        codes4_to_f16x2x2<E5M2>(w0[kk], af[0], af[2]);
                        codes4_to_f16x2x2<E5M2>(w1[kk], af[1], af[3]);
                    } else {
                        af[0] = w0[2 * kk];
                        af[2] = w0[2 * kk + 1];
                        af[1] = w1[2 * kk];
                        af[3] = w1[2 * kk + 1];
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        float(&acc)[4] = (ks & 1) ? s1[t] : sc[p][t];
                        if constexpr (ES == 1)
                            mma_16816(acc, af, qf[t][ks][0], qf[t][ks][1], acc);
                        else
                            mma_16816_bf16(acc, af, qf[t][ks][0], qf[t][ks][1], acc);
                    }
                }
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) sc[p][t][r] += s1[t][r];
    }

    float kscale[BS ? Gm::PPS : 1], vlog[BS ? Gm::PPS : 1], vinv[BS ? Gm::PPS : 1];
    if constexpr (BS) {
#pragma unroll
        for (int p = 0; p < Gm::PPS; ++p) {
            const float2 ps = p < np ? psc[p] : make_float2(1.f, 1.f);
            kscale[p] = ps.x;
            vlog[p] = fast_log2(ps.y);
            vinv[p] = fast_rcp(ps.y);
        }
    }

    // ---- mask, scale to log2 units, stage maximum
    float mx[NT][2];
    const bool interior = tok_base >= lo && tok_base + np * kBS <= L && np == Gm::PPS;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        mx[t][0] = mx[t][1] = -INFINITY;
#pragma unroll
        for (int p = 0; p < Gm::PPS; ++p)
#pragma unroll
            for (int e2 = 0; e2 < 2; ++e2) {
                const int tok = tok_base + p * kBS + gid + 8 * e2;
                const bool valid = interior || ((p < np) && tok >= lo && tok < L);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float raw = sc[p][t][2 * e2 + j];
                    const float x = !valid ? -INFINITY : BS ? fmaf(raw, cs[t][j] * kscale[p], vlog[p]) : raw * cs[t][j];
                    sc[p][t][2 * e2 + j] = x;
                    mx[t][j] = fmaxf(mx[t][j], x);
                }
            }
    }
    float alpha[NT][2], muse[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            mx[t][j] = fmaxf(mx[t][j], __shfl_xor_sync(0xffffffffu, mx[t][j], 4));
            mx[t][j] = fmaxf(mx[t][j], __shfl_xor_sync(0xffffffffu, mx[t][j], 8));
            mx[t][j] = fmaxf(mx[t][j], __shfl_xor_sync(0xffffffffu, mx[t][j], 16));
            const float mn = fmaxf(m[t][j], BS ? __fadd_ru(mx[t][j], -kRoom) : mx[t][j]);
            muse[t][j] = mn == -INFINITY ? 0.f : mn;
            alpha[t][j] = fast_exp2(m[t][j] - muse[t][j]);
            m[t][j] = mn;
        }

    // ---- probabilities -> f16 (bf16 for the bf16 twin) B fragments of the value MMA
    uint32_t pb[Gm::PPS][NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        float lsum[2] = {0.f, 0.f};
#pragma unroll
        for (int p = 0; p < Gm::PPS; ++p) {
            const float p00 = fast_exp2(sc[p][t][0] - muse[t][0]);
            const float p01 = fast_exp2(sc[p][t][1] - muse[t][1]);
            const float p10 = fast_exp2(sc[p][t][2] - muse[t][0]);
            const float p11 = fast_exp2(sc[p][t][3] - muse[t][1]);
            if constexpr (BS) {
                lsum[0] = fmaf(p00 + p10, vinv[p], lsum[0]);
                lsum[1] = fmaf(p01 + p11, vinv[p], lsum[1]);
            } else {
                lsum[0] += p00 + p10;
                lsum[1] += p01 + p11;
            }
            if constexpr (ES == 1) {
                pb[p][t][0] = movmatrix_trans(pack_f16x2(p00, p01));
                pb[p][t][1] = movmatrix_trans(pack_f16x2(p10, p11));
            } else {
                pb[p][t][0] = movmatrix_trans(pack_bf16x2(p00, p01));
                pb[p][t][1] = movmatrix_trans(pack_bf16x2(p10, p11));
            }
        }
        l[t][0] = l[t][0] * alpha[t][0] + lsum[0];
        l[t][1] = l[t][1] * alpha[t][1] + lsum[1];
    }

    // ---- P.V tile of this stage: O^T[dim][head] = V^T P^T
    float ot[NT][Gm::MT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int mt = 0; mt < Gm::MT; ++mt) ot[t][mt][0] = ot[t][mt][1] = ot[t][mt][2] = ot[t][mt][3] = 0.f;
#pragma unroll
    for (int p = 0; p < Gm::PPS; ++p) {
        if (p < np) {
#pragma unroll
            for (int hh = 0; hh < Gm::HALVES; ++hh) {
                uint32_t v[4][Gm::VW / 4];
                if constexpr (kEarlyV) {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
#pragma unroll
                        for (int ww = 0; ww < Gm::VW / 4; ++ww) v[r][ww] = vr[p][hh][r][ww];
                } else {
                    load_v_box<D, ES>(vst + p * Gm::PAGE + hh * Gm::BOX, gid, tig, tok_base + p * kBS, lo, L, true, v);
                }
#pragma unroll
                for (int mtl = 0; mtl < Gm::MTH; ++mtl) {
                    uint32_t af[4];
                    if constexpr (ES == 1) {
                        const uint32_t sel = (mtl & 1) ? 0x7362u : 0x5140u;
                        const uint32_t x01 = byte_perm(v[0][mtl >> 1], v[1][mtl >> 1], sel);
                        const uint32_t x23 = byte_perm(v[2][mtl >> 1], v[3][mtl >> 1], sel);
                        codes4_to_f16x2x2<E5M2>(x01, af[0], af[1]);
                        codes4_to_f16x2x2<E5M2>(x23, af[2], af[3]);
                    } else {
                        af[0] = byte_perm(v[0][mtl], v[1][mtl], 0x5410u);
                        af[1] = byte_perm(v[0][mtl], v[1][mtl], 0x7632u);
                        af[2] = byte_perm(v[2][mtl], v[3][mtl], 0x5410u);
                        af[3] = byte_perm(v[2][mtl], v[3][mtl], 0x7632u);
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        float(&acc)[4] = ot[t][hh * Gm::MTH + mtl];
                        if constexpr (ES == 1)
                            mma_16816(acc, af, pb[p][t][0], pb[p][t][1], acc);
                        else
                            mma_16816_bf16(acc, af, pb[p][t][0], pb[p][t][1], acc);
                    }
                }
            }
        }
    }

    // ---- fold the tile into the FP32 accumulators
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int mt = 0; mt < Gm::MT; ++mt) {
            o[t][mt][0] = fmaf(o[t][mt][0], alpha[t][0], ot[t][mt][0]);
            o[t][mt][1] = fmaf(o[t][mt][1], alpha[t][1], ot[t][mt][1]);
            o[t][mt][2] = fmaf(o[t][mt][2], alpha[t][0], ot[t][mt][2]);
            o[t][mt][3] = fmaf(o[t][mt][3], alpha[t][1], ot[t][mt][3]);
        }
}

// Combines the k_u partials of unit u (slots u + c_first ...) into its output
// rows, with all NTHR threads of the CTA.  The partials come from other CTAs
// of the grid, so they are read through L2: the unit's slots are contiguous,
// and chunks of them are copied into `stage` (shared memory the streaming no
// longer needs) by 16-byte cp.async copies issued all at once; thread i then
// folds (query head, 4 dims) items i, i + NTHR, ... over the chunk (max, then
// rescale and accumulate).
template <int D, int G, int NTHR, int STAGE_BYTES>
__device__ __forceinline__ void merge_unit(const DecodeArgs& a, int u, int c_first, int k_u, int tid,
                                           uint8_t* stage) {
    constexpr int NG = D / 4;                      // float4 groups per head
    constexpr int ITEMS = G * NG;
    constexpr int IT = (ITEMS + NTHR - 1) / NTHR;  // items per thread
    constexpr int OB = G * D * 4;                  // bytes of one partial's outputs
    constexpr int MB = kMaxG * 8;                  // bytes of one partial's (max, sum) entries
    constexpr int cap = STAGE_BYTES / (OB + MB);   // partials per chunk
    static_assert(cap >= 1, "the staging area holds at least one partial");
    const int Hkv = a.num_kv_heads, b = u / Hkv, hk = u - b * Hkv;
    const int64_t s0 = static_cast<int64_t>(u) + c_first;
    const float4* so = reinterpret_cast<const float4*>(stage);             // [cap][G][NG]
    const float2* sml = reinterpret_cast<const float2*>(stage + cap * OB);  // [cap][kMaxG]
    const uint32_t so_s = smem_u32(stage), sml_s = smem_u32(stage + cap * OB);
    float M[IT], Lh[IT];
    float4 acc[IT];
#pragma unroll
    for (int j = 0; j < IT; ++j) {
        M[j] = -INFINITY;
        Lh[j] = 0.f;
        acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int k0 = 0; k0 < k_u; k0 += cap) {
        const int kc = min(cap, k_u - k0);
        const uint8_t* go = reinterpret_cast<const uint8_t*>(a.part_o + (s0 + k0) * G * D);
        const uint8_t* gml = reinterpret_cast<const uint8_t*>(a.part_ml + (s0 + k0) * kMaxG);
        for (int i = tid; i < kc * (OB / 16); i += NTHR) cp_async_16(so_s + i * 16, go + i * 16);
        for (int i = tid; i < kc * (MB / 16); i += NTHR) cp_async_16(sml_s + i * 16, gml + i * 16);
        cp_async_commit();
        cp_async_wait<0>();
        __syncthreads();
#pragma unroll
        for (int j = 0; j < IT; ++j) {
            const int it = tid + j * NTHR;
            if (it < ITEMS) {
                const int h = it / NG, g4 = it - (it / NG) * NG;
                float Mb = M[j];
                for (int k = 0; k < kc; ++k) Mb = fmaxf(Mb, sml[k * kMaxG + h].x);
                const float Mbu = Mb == -INFINITY ? 0.f : Mb;
                const float r = fast_exp2(M[j] - Mbu);
                float4 x = acc[j];
                float lx = Lh[j] * r;
                x.x *= r; x.y *= r; x.z *= r; x.w *= r;
                for (int k = 0; k < kc; ++k) {
                    const float2 ml = sml[k * kMaxG + h];
                    const float f = fast_exp2(ml.x - Mbu);
                    const float4 v = so[(k * G + h) * NG + g4];
                    x.x += f * v.x; x.y += f * v.y; x.z += f * v.z; x.w += f * v.w;
                    lx += f * ml.y;
                }
                acc[j] = x;
                Lh[j] = lx;
                M[j] = Mb;
            }
        }
        __syncthreads();  // the chunk is consumed before the next one lands
    }
    const float vsc = unit_v_scale(a, hk);
#pragma unroll
    for (int j = 0; j < IT; ++j) {
        const int it = tid + j * NTHR;
        if (it < ITEMS) {
            const int h = it / NG, g4 = it - (it / NG) * NG;
            const float sc_out = Lh[j] > 0.f ? vsc / Lh[j] : 0.f;
            uint16_t* out = a.out + (static_cast<int64_t>(b) * a.num_q_heads + hk * G + h) * D;
            const uint32_t lo2 =
                f32_to_bf16(acc[j].x * sc_out) | (static_cast<uint32_t>(f32_to_bf16(acc[j].y * sc_out)) << 16);
            const uint32_t hi2 =
                f32_to_bf16(acc[j].z * sc_out) | (static_cast<uint32_t>(f32_to_bf16(acc[j].w * sc_out)) << 16);
            *reinterpret_cast<uint2*>(out + g4 * 4) = make_uint2(lo2, hi2);
        }
    }
}

// Warps and ring depth of the streaming kernel.  Two CTAs share an SM
// (228 KB of shared memory, 64K registers).  At d = 256 the larger merge
// buffers leave room for two ring stages per warp, elsewhere three.  At
// d = 64 (g <= 8, whose registers allow it) 6 warps with two stages each
// measured 7% faster than 4 warps with three: more warps issuing copies.
// The bf16 cache at d = 256 has 8 KB pages: a stage is one page of K and one
// of V (16 KB), and three warps with two stages each fit.
template <int D, int ES, int G>
struct StreamCfg {
    static constexpr bool kWide = D == 64 && ES == 1 && G <= 8;
    static constexpr bool kBigPage = Geo<D, ES>::SH > kStageHalf;            // bf16 at d = 256: 8 KB pages
    static constexpr int NW = kWide ? 6 : kBigPage ? 3 : 4;                  // warps per CTA
    static constexpr int R = (Geo<D, ES>::XW > 40 || kWide) ? 2 : 3;         // ring stages per warp
    static constexpr int NBUF = NW / 2;                                      // merge exchange buffers
    static constexpr int CPP = Geo<D, ES>::PAGE / 512;                       // 16-byte copies per lane per page
};

// int32 words of the per-sequence tables behind the rings (an even count, so
// that the float2 page scales behind them are aligned).
constexpr int kTableWords = 2 * kMaxBatch + 1 + 8 + 1;

// BS: each ring stage also holds the (K, V) scales of its pages.
template <int D, int ES, int G, bool BS>
constexpr size_t stream_smem_bytes() {
    using Sc = StreamCfg<D, ES, G>;
    return 128 + static_cast<size_t>(Sc::NW) * Sc::R * Geo<D, ES>::SB + Sc::NBUF * Geo<D, ES>::XW * 32 * sizeof(float) +
           kTableWords * sizeof(int32_t) + (BS ? Sc::NW * Sc::R * Geo<D, ES>::PPS * sizeof(float2) : 0);
}

// Dynamic shared memory one of kCtasPerSm resident CTAs may take (228 KB per
// SM, 1 KB of it reserved per CTA).
constexpr size_t kSmemPerCta = (228u * 1024u) / kCtasPerSm - 1024u;

template <int D, int G, int ES, bool E5M2, bool BS = false>
__global__ void __launch_bounds__(StreamCfg<D, ES, G>::NW * 32, kCtasPerSm)
    stream_decode_kernel(const DecodeArgs a) {
    using Gm = Geo<D, ES>;
    using Sc = StreamCfg<D, ES, G>;
    constexpr int NW = Sc::NW, R = Sc::R, CPP = Sc::CPP;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* rings = smem_raw + ((128u - (smem_u32(smem_raw) & 127u)) & 127u);
    float* xbuf = reinterpret_cast<float*>(rings + NW * R * Gm::SB);                 // [NBUF][XW][32]
    int32_t* pre = reinterpret_cast<int32_t*>(xbuf + Sc::NBUF * Gm::XW * 32);         // [kMaxBatch + 1]
    int32_t* lens = pre + kMaxBatch + 1;                                              // [kMaxBatch]
    volatile int* flag = reinterpret_cast<volatile int*>(lens + kMaxBatch);            // [1] earlier timeout
    int32_t* mlist = lens + kMaxBatch + 1;  // [0]: units this CTA completes; then (u, c_first, k_u) each
    float2* scale_ring = reinterpret_cast<float2*>(pre + kTableWords);                // BS: [NW][R][PPS]

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // This grid may have started before the previous one on the stream
    // finished (programmatic launch): wait for it before reading any input.
    griddep_wait();
    // The next grid on the stream may start its set-up now; it waits for
    // this grid's completion before it reads anything this grid writes.
    griddep_launch_dependents();
    const int B = a.batch, Hkv = a.num_kv_heads, C = gridDim.x, c = blockIdx.x;

    // ---- attended pages per sequence and their exclusive prefix; the error
    // word is read alongside (a call that gave up a wait fails every later
    // call on the workspace until it is re-initialised)
    if (warp == 0) {
        uint32_t prev_err = 0;
        if (lane == 0) prev_err = *reinterpret_cast<volatile uint32_t*>(a.err);
        int run = 0;
        for (int b0 = 0; b0 < B; b0 += 32) {
            const int b = b0 + lane;
            int n = 0;
            if (b < B) {
                const int Lraw = ld_input(a.seq_lens + b);
                if (Lraw < 0 || Lraw > a.max_seq_len) report(a.err, FP8KV_ERR_INVALID_ARG);
                lens[b] = clamp_len(Lraw, a.max_seq_len);
                n = attended_pages(lens[b], a.window);
            }
            int x = n;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, off);
                if (lane >= off) x += y;
            }
            if (b < B) pre[b] = run + x - n;
            run += __shfl_sync(0xffffffffu, x, 31);
        }
        if (lane == 0) {
            pre[B] = run;
            flag[0] = prev_err == FP8KV_ERR_TIMEOUT;
            mlist[0] = 0;
        }
    }
    __syncthreads();
    if (flag[0]) return;

    const int64_t P = static_cast<int64_t>(Hkv) * pre[B];
    for (int b = c; b < B; b += C) {  // sequences with nothing to attend produce zeros
        if (pre[b + 1] == pre[b]) {
            uint16_t* ob = a.out + static_cast<int64_t>(b) * a.num_q_heads * D;
            for (int i = tid; i < a.num_q_heads * D; i += NW * 32) ob[i] = 0;
        }
    }
    const int Ce = static_cast<int>(P < C ? P : C);
    if (c >= Ce) return;
    const Partition part = make_partition(P, Ce);
    const int64_t s = range_start(part, c);
    const int64_t e = range_start(part, c + 1);

    // ---- this warp's ring and its per-lane copy offsets: lane l copies the
    // 16-byte chunks l, l+32, ... of a page, stored at their swizzled place
    uint8_t* ring = rings + warp * R * Gm::SB;
    const uint32_t ring_s = smem_u32(ring);
    float2* scales = scale_ring + warp * R * Gm::PPS;
    const uint32_t scales_s = smem_u32(scales);
    uint32_t soff[CPP];
#pragma unroll
    for (int i = 0; i < CPP; ++i) {
        const int byte = (lane + 32 * i) * 16;
        const int r = byte / Gm::RB, b = byte % Gm::RB;
        soff[i] = (b / Gm::ROWB) * Gm::BOX + sswz<Gm::ROWB>(r, b % Gm::ROWB);
    }
    const uint64_t pol = l2_policy_evict_first();
    const bool appending = ES == 1 && a.k_new != nullptr;
    const int kvs = a.kv_shift, Hc = Hkv >> kvs;

    // ---- issue side: a cursor over this warp's pages in windows of up to 32
    // pages that never straddle a segment (walk.cuh).  Lane l holds the block
    // id of page start + l of the window; the window after the current one is
    // read one window ahead, with the newest K/V rows when it holds a unit's
    // last page and this is a decode step.
    struct Win {
        WinPos pos;
        int id;     // lane-held block id
        bool last;  // the window holds its unit's last page, which gets the new rows first
        NewRow<D> krow, vrow;
    };
    auto load_win = [&](Win& x) {
        x.id = 0;
        x.last = false;
        if (!x.pos.valid) return;
        const int32_t* row = a.block_tables + static_cast<int64_t>(x.pos.w.b) * a.max_blocks_per_seq +
                             first_token(lens[x.pos.w.b], a.window) / kBS + (x.pos.w.g - x.pos.w.base);
        x.id = load_block_id(row + x.pos.start, lane, x.pos.n, a.num_blocks, a.err);
        x.last = appending && window_holds_unit_end(x.pos, e);
        if (x.last) {
            const int64_t nr = static_cast<int64_t>(x.pos.w.b) * Hc + (x.pos.w.hk >> kvs);
            load_new_row<D>(x.krow, a.k_new + nr * D, lane);
            load_new_row<D>(x.vrow, a.v_new + nr * D, lane);
        }
    };
    Win cur, nxt;
    {
        Walker w0;
        walk_start(w0, pre, B, Hkv, s);
        cur.pos = first_window_from(w0, true, pre, Hkv, e, warp, NW);
        load_win(cur);
        nxt.pos = next_window(cur.pos, pre, Hkv, e, warp, NW);
        load_win(nxt);
    }
    int cpos = 0;   // pages of the current window already issued
    int ist = 0;    // stages issued
    // Issues this warp's next stage (up to PPS pages of K and V) into ring
    // slot ist % R, or an empty copy group once its pages are exhausted.
    auto issue_stage = [&]() {
        if (cur.pos.valid) {
            const int n = min(Gm::PPS, cur.pos.n - cpos);
            const uint32_t slot = ring_s + (ist % R) * Gm::SB;
            if constexpr (BS) {
                // the stage's page scales travel with its pages, in the same
                // copy group: lane 2p copies page p's K scale, lane 2p + 1 its V scale
                const int id = __shfl_sync(0xffffffffu, cur.id, (cpos + (lane >> 1)) & 31);
                if (lane < 2 * n) {
                    const int64_t page = static_cast<int64_t>(max(id, 0)) * Hc + (cur.pos.w.hk >> kvs);
                    cp_async_4(scales_s + ((ist % R) * Gm::PPS * 2 + lane) * 4,
                               ((lane & 1) ? a.v_page_scales : a.k_page_scales) + page);
                }
            }
            for (int p = 0; p < n; ++p) {
                const int id = __shfl_sync(0xffffffffu, cur.id, cpos + p);
                const int64_t page = static_cast<int64_t>(max(id, 0)) * Hc + (cur.pos.w.hk >> kvs);
                const uint8_t* ksrc = a.k_cache + page * Gm::PAGE;
                const uint8_t* vsrc = a.v_cache + page * Gm::PAGE;
                if (cur.last && cur.pos.start + cpos + p == cur.pos.hi - 1 && id >= 0) {
                    // the unit's last page: write the sequence's newest K and
                    // V rows into it first (the same quantisation as the
                    // append kernel), then copy it
                    const int L = lens[cur.pos.w.b];
                    const int64_t roff = static_cast<int64_t>((L - 1) % kBS) * D;
                    const float ksc = a.k_scales ? ld_input(a.k_scales + (cur.pos.w.hk >> kvs)) : a.k_scale_raw;
                    const float vsc = a.v_scales ? ld_input(a.v_scales + (cur.pos.w.hk >> kvs)) : a.v_scale_raw;
                    store_new_row<D, E5M2>(cur.krow, a.k_cache + page * Gm::PAGE + roff, lane, ksc);
                    store_new_row<D, E5M2>(cur.vrow, a.v_cache + page * Gm::PAGE + roff, lane, vsc);
                    __threadfence();
                    __syncwarp();
                }
#pragma unroll
                for (int i = 0; i < CPP; ++i) {
                    cp_async_16(slot + p * Gm::PAGE + soff[i], ksrc + (lane + 32 * i) * 16, pol);
                    cp_async_16(slot + Gm::SH + p * Gm::PAGE + soff[i], vsrc + (lane + 32 * i) * 16, pol);
                }
            }
            cpos += n;
            if (cpos == cur.pos.n) {
                cur = nxt;
                cpos = 0;
                nxt.pos = next_window(cur.pos, pre, Hkv, e, warp, NW);
                load_win(nxt);
            }
        }
        cp_async_commit();
        ++ist;
    };
#pragma unroll
    for (int i = 0; i < R - 1; ++i) issue_stage();

    // ---- compute side: the segments of the CTA's range in order; in each,
    // this warp's share stage by stage, then the CTA's warps merge
    const int gid = lane >> 2, tig = lane & 3;
    constexpr int NT = G > 8 ? 2 : 1;  // n-tiles of 8 query heads
    uint32_t qf[NT][Gm::KS][2];
    float cs[NT][2];
    float m[NT][2], l[NT][2];
    float o[NT][Gm::MT][4];
    int kst = 0;  // stages computed
    Walker w;
    walk_start(w, pre, B, Hkv, s);
    while (true) {
        const int64_t seg_end = min(e, w.base + w.n);
        const int lp0 = static_cast<int>(w.g - w.base);
        int q0, q1;
        warp_share(w, e, warp, NW, q0, q1);
        const int L = lens[w.b];
        const int lo = first_token(L, a.window);
        const int pg_first = lo / kBS + lp0;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if constexpr (ES == 1)
                load_query<D, G>(a, w.b, w.hk, gid, tig, qf[t], cs[t], 8 * t);
            else
                load_query_bf16<D, G>(a, w.b, w.hk, gid, tig, qf[t], cs[t], 8 * t);
            m[t][0] = m[t][1] = -INFINITY;
            l[t][0] = l[t][1] = 0.f;
#pragma unroll
            for (int mt = 0; mt < Gm::MT; ++mt) o[t][mt][0] = o[t][mt][1] = o[t][mt][2] = o[t][mt][3] = 0.f;
        }

        for (int p0 = q0; p0 < q1; p0 += Gm::PPS) {
            issue_stage();
            cp_async_wait<R - 1>();
            __syncwarp();
            const uint8_t* kst_p = ring + (kst % R) * Gm::SB;
            tc_stage<D, ES, E5M2, NT, BS>(kst_p, kst_p + Gm::SH, scales + (kst % R) * Gm::PPS, min(Gm::PPS, q1 - p0),
                                          (pg_first + p0) * kBS, lo, L, gid, tig, qf, cs, m, l, o);
            __syncwarp();  // every lane is done with the slot before it is refilled
            ++kst;
        }

#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                l[t][j] += __shfl_xor_sync(0xffffffffu, l[t][j], 4);
                l[t][j] += __shfl_xor_sync(0xffffffffu, l[t][j], 8);
                l[t][j] += __shfl_xor_sync(0xffffffffu, l[t][j], 16);
            }

        // ---- merge the warps' states into warp 0 (tree through smem), one
        // n-tile after the other through the same buffers
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int n = NW; n > 1; n -= n / 2) {
                const int h = n / 2;
                if (warp >= n - h && warp < n)
                    publish<Gm::MT>(xbuf + (warp - (n - h)) * Gm::XW * 32, lane, m[t], l[t], o[t]);
                consumer_sync_n<NW>();
                if (warp < h) absorb<Gm::MT>(xbuf + warp * Gm::XW * 32, lane, m[t], l[t], o[t]);
                consumer_sync_n<NW>();
            }

        // ---- emit: the whole unit in this CTA -> output; else a partial
        const int u = w.b * Hkv + w.hk;
        const int c_first = cta_of(part, w.base);
        const int c_last = cta_of(part, w.base + w.n - 1);
        if (warp == 0) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (c_first == c_last) {
                    uint16_t* out_u = a.out + (static_cast<int64_t>(w.b) * a.num_q_heads + w.hk * G) * D;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int h = 8 * t + 2 * tig + j;
                        const float sc_out = l[t][j] > 0.f ? unit_v_scale(a, w.hk) / l[t][j] : 0.f;
                        if (h < G) {
#pragma unroll
                            for (int mt = 0; mt < Gm::MT; ++mt) {
                                // dimensions dim and dim + 1 together (one 4-byte store)
                                const int dim = (mt / Gm::MTH) * Gm::DBOX + Gm::VWD * gid + 2 * (mt % Gm::MTH);
                                *reinterpret_cast<uint32_t*>(out_u + h * D + dim) =
                                    static_cast<uint32_t>(f32_to_bf16(o[t][mt][j] * sc_out)) |
                                    (static_cast<uint32_t>(f32_to_bf16(o[t][mt][2 + j] * sc_out)) << 16);
                            }
                        }
                    }
                } else {
                    const int64_t slot_idx = static_cast<int64_t>(u) + c;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int h = 8 * t + 2 * tig + j;
                        if (h < G) {
                            float* po = a.part_o + (slot_idx * G + h) * D;
#pragma unroll
                            for (int mt = 0; mt < Gm::MT; ++mt)
#pragma unroll
                                for (int e2 = 0; e2 < 2; ++e2)
                                    po[(mt / Gm::MTH) * Gm::DBOX + Gm::VWD * gid + 2 * (mt % Gm::MTH) + e2] = o[t][mt][2 * e2 + j];
                            if (gid == 0) a.part_ml[slot_idx * kMaxG + h] = make_float2(m[t][j], l[t][j]);
                        }
                    }
                }
            }
            if (c_first != c_last && a.inline_merge) {
                // Publish the partial, then count it.  The CTA that brings the
                // count to k_u merges the unit once its own range is done (a
                // range holds at most two split units: its first and its last
                // segment).
                __threadfence();
                __syncwarp();
                if (lane == 0) {
                    const int k_u = c_last - c_first + 1;
                    if (atomicAdd(a.split_cnt + u, 1) == k_u - 1) {
                        a.split_cnt[u] = 0;  // every partial is in: ready for the next call
                        __threadfence();
                        const int i = mlist[0];
                        mlist[1 + 3 * i] = u;
                        mlist[2 + 3 * i] = c_first;
                        mlist[3 + 3 * i] = k_u;
                        mlist[0] = i + 1;
                    }
                }
            }
        }
        if (seg_end >= e) break;
        walk_next(w, pre, Hkv);
    }
    cp_async_wait<0>();

    // ---- the units this CTA completed: combine their partials into the output
    // (the rings and the exchange buffers, contiguous, stage the partials)
    __syncthreads();
    const int nm = mlist[0];
    for (int i = 0; i < nm; ++i)
        merge_unit<D, G, NW * 32, NW * R * Gm::SB + Sc::NBUF * Gm::XW * 32 * static_cast<int>(sizeof(float))>(
            a, mlist[1 + 3 * i], mlist[2 + 3 * i], mlist[3 + 3 * i], tid, rings);
}

// Combines the partials of every (sequence, kv head) unit that was split over
// several CTAs, when the decode grid does not (see merge_inline): one CTA per
// (unit, query head of the group).  Its 4 * D threads split the unit's
// partials into 16 slices (8 loads in flight per thread, one online
// softmax-merge pass), then combine the slices in shared memory.  It starts as
// a programmatic dependent of the decode grid and waits for that grid's
// completion before reading.
template <int D>
__host__ __device__ constexpr int merge_threads() { return 4 * D; }

template <int D, int G>
__global__ void __launch_bounds__(merge_threads<D>()) merge_kernel(const DecodeArgs a) {
    constexpr int kMergeThreads = merge_threads<D>();
    constexpr int NG = D / 4;                // float4 groups per head: 16, 32, 64
    constexpr int KS = kMergeThreads / NG;   // slices of the partial list: 16
    __shared__ float sm_m[KS][NG], sm_l[KS][NG];
    __shared__ float4 sm_o[KS][NG];
    griddep_launch_dependents();  // the next call's set-up may overlap this merge
    const int u = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
    const int g4 = tid % NG, ks = tid / NG;
    // Where this unit's partials are: the decode grid's page split, recomputed
    // from the lengths while that grid finishes (they are final: the decode
    // CTAs trigger this grid only after their own wait).
    __shared__ long long red[2][kMergeThreads / 32];
    const int Hkv = a.num_kv_heads, b = u / Hkv, hk = u - b * Hkv;
    long long before = 0, total = 0;
    for (int i = tid; i < a.batch; i += kMergeThreads) {
        const int n = attended_pages(clamp_len(ld_input(a.seq_lens + i), a.max_seq_len), a.window);
        total += n;
        before += i < b ? n : 0;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        before += __shfl_xor_sync(0xffffffffu, before, off);
        total += __shfl_xor_sync(0xffffffffu, total, off);
    }
    if ((tid & 31) == 0) {
        red[0][tid >> 5] = before;
        red[1][tid >> 5] = total;
    }
    __syncthreads();
    before = total = 0;
#pragma unroll
    for (int w = 0; w < kMergeThreads / 32; ++w) {
        before += red[0][w];
        total += red[1][w];
    }
    const int nb = attended_pages(clamp_len(ld_input(a.seq_lens + b), a.max_seq_len), a.window);
    int k_u = 0, c_first = 0;
    if (nb > 0) {
        const int64_t P = static_cast<int64_t>(Hkv) * total;
        const Partition part = make_partition(P, static_cast<int>(P < a.decode_ctas ? P : a.decode_ctas));
        const int64_t base = static_cast<int64_t>(Hkv) * before + static_cast<int64_t>(hk) * nb;
        c_first = cta_of(part, base);
        k_u = cta_of(part, base + nb - 1) - c_first + 1;
    }
    // Every CTA waits, even one with nothing to merge: this grid must not
    // complete (and release the next grid on the stream) before the decode
    // grid has.
    griddep_wait();
    if (k_u <= 1) return;  // empty (zeros), or written directly by its only CTA
    // a decode CTA gave up a wait (in this call or an earlier one on this
    // workspace): the partials are incomplete, and the error word says so
    if (*reinterpret_cast<volatile uint32_t*>(a.err) == FP8KV_ERR_TIMEOUT) return;
    const int64_t s0 = static_cast<int64_t>(u) + c_first;
    float M = -INFINITY, Lh = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = ks; k0 < k_u; k0 += 8 * KS) {
        float2 ml[8];
        float4 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int k = k0 + j * KS;
            if (k < k_u) {
                ml[j] = a.part_ml[(s0 + k) * kMaxG + h];
                v[j] = *(reinterpret_cast<const float4*>(a.part_o + ((s0 + k) * G + h) * D) + g4);
            } else {
                ml[j] = make_float2(-INFINITY, 0.f);
                v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
        float Mb = M;
#pragma unroll
        for (int j = 0; j < 8; ++j) Mb = fmaxf(Mb, ml[j].x);
        const float Mbu = Mb == -INFINITY ? 0.f : Mb;
        const float r = fast_exp2(M - Mbu);
        acc.x *= r; acc.y *= r; acc.z *= r; acc.w *= r;
        Lh *= r;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float f = fast_exp2(ml[j].x - Mbu);
            acc.x += f * v[j].x; acc.y += f * v[j].y; acc.z += f * v[j].z; acc.w += f * v[j].w;
            Lh += f * ml[j].y;
        }
        M = Mb;
    }
    sm_m[ks][g4] = M;
    sm_l[ks][g4] = Lh;
    sm_o[ks][g4] = acc;
    __syncthreads();
    if (ks != 0) return;
    float Mt = -INFINITY;
#pragma unroll
    for (int j = 0; j < KS; ++j) Mt = fmaxf(Mt, sm_m[j][g4]);
    const float Mtu = Mt == -INFINITY ? 0.f : Mt;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float Lt = 0.f;
#pragma unroll
    for (int j = 0; j < KS; ++j) {
        const float f = fast_exp2(sm_m[j][g4] - Mtu);
        o.x += f * sm_o[j][g4].x; o.y += f * sm_o[j][g4].y; o.z += f * sm_o[j][g4].z; o.w += f * sm_o[j][g4].w;
        Lt += f * sm_l[j][g4];
    }
    const float sc_out = Lt > 0.f ? unit_v_scale(a, hk) / Lt : 0.f;
    uint16_t* out = a.out + (static_cast<int64_t>(b) * a.num_q_heads + hk * G + h) * D;
    const uint32_t lo2 = f32_to_bf16(o.x * sc_out) | (static_cast<uint32_t>(f32_to_bf16(o.y * sc_out)) << 16);
    const uint32_t hi2 = f32_to_bf16(o.z * sc_out) | (static_cast<uint32_t>(f32_to_bf16(o.w * sc_out)) << 16);
    *reinterpret_cast<uint2*>(out + g4 * 4) = make_uint2(lo2, hi2);
}

// ---------------------------------------------------------------- launch

template <int D, int G, int ES = 1, bool E5M2 = false, bool BS = false>
cudaError_t launch_stream(const DecodeArgs& a, int ctas, cudaStream_t stream) {
    static_assert(stream_smem_bytes<D, ES, G, BS>() <= kSmemPerCta, "two CTAs must fit on one SM");
    static std::atomic<uint64_t> done_mask{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
    if (bit == 0 || !(done_mask.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(stream_decode_kernel<D, G, ES, E5M2, BS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(stream_smem_bytes<D, ES, G, BS>()));
        if (e != cudaSuccess) return e;
        done_mask.fetch_or(bit, std::memory_order_release);
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(StreamCfg<D, ES, G>::NW * 32);
    cfg.dynamicSmemBytes = stream_smem_bytes<D, ES, G, BS>();
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, stream_decode_kernel<D, G, ES, E5M2, BS>, a);
    if (e != cudaSuccess || ctas == 1 || a.inline_merge) return e;  // merged inside the decode grid
    cudaLaunchConfig_t mcfg = {};
    mcfg.gridDim = dim3(a.batch * a.num_kv_heads, G);
    mcfg.blockDim = dim3(merge_threads<D>());
    mcfg.dynamicSmemBytes = 0;
    mcfg.stream = stream;
    mcfg.attrs = attr;
    mcfg.numAttrs = 1;
    return cudaLaunchKernelEx(&mcfg, merge_kernel<D, G>, a);
}

template <int D, int ES = 1, bool E5M2 = false, bool BS = false>
cudaError_t launch_stream_g(int G, const DecodeArgs& a, int ctas, cudaStream_t s) {
    switch (G) {
        case 1: return launch_stream<D, 1, ES, E5M2, BS>(a, ctas, s);
        case 2: return launch_stream<D, 2, ES, E5M2, BS>(a, ctas, s);
        case 4: return launch_stream<D, 4, ES, E5M2, BS>(a, ctas, s);
        case 8: return launch_stream<D, 8, ES, E5M2, BS>(a, ctas, s);
        case 16:
            if constexpr (D <= 128) return launch_stream<D, 16, ES, E5M2, BS>(a, ctas, s);
            else return cudaErrorInvalidValue;  // g = 16 at d = 256 runs as two units of 8 (head_map)
        default: return cudaErrorInvalidValue;
    }
}

// The decode over a block-scaled cache (paged_decode_block.cu).
cudaError_t launch_stream_block(int head_dim, int G, const DecodeArgs& a, int ctas, cudaStream_t s);

}  // namespace fp8kv
