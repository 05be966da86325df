// Paged fp8 (E4M3) decode attention for sm_103a.
//
// What it computes: single-query grouped-query softmax attention over a paged
// KV cache stored as E4M3 codes with per-tensor K and V scales, the fp8 cache
// read directly with dequantisation fused into the attention (gpusmith.com,
// "FP8 KV Cache Quantization: Capacity Gains and Accuracy Risk", sections
// "What FP8 KV changes" and "Attention backend interactions"), with scores,
// softmax and P.V accumulated in real FP32 registers however long the context
// (particula.tech, "KV Cache Quantization: What FP8 and q8_0 Cost in
// Accuracy", opening section; phantomic12 vLLM-blog summary, "ACCURACY AT
// LONG CONTEXT": the P.V contraction runs over the context length), and an
// optional sliding window (same summary, "DECODE COST": windows 128, 512).
//
// How (persistent CTAs over a flattened, evenly split page list):
//  * All g query heads of a kv head are handled together, so every cache byte
//    is read from HBM once.  Decode attention is bandwidth-bound (2g flop per
//    fp8 byte), so the kernel is built around streaming pages at HBM speed.
//  * The attended pages of every (sequence, kv head) unit are laid end to end
//    and cut into one equal contiguous range per CTA (2 CTAs per SM), so all
//    CTAs finish together whatever the mix of sequence lengths.  A CTA walks
//    the units its range overlaps ("segments").
//  * Tensor-core engine (the default; stream_decode.cuh): no producer
//    warps.  Each of the 4 warps of a CTA (6 at d = 64) takes one contiguous
//    share of every segment and streams it with 16-byte cp.async copies
//    (evict-first L2 policy) into a private ring of 3 stages (2 at d = 64
//    and d = 256), up to two stages ahead of the one it computes (one with
//    a two-stage ring); its block ids are consecutive entries of
//    one block-table row, read 32 at a time one window ahead.  Copies end by
//    themselves, so there is no barrier handshake and no wait to bound.  In a
//    decode step (fp8kv_decode_step) the warp whose share holds a unit's last
//    page first quantises the sequence's newest K and V rows into it, fences,
//    and only then copies it.  Many warps issuing small copies streamed the
//    random 2 KB pages faster than two TMA-issuing producer warps per CTA.
//  * CUDA-core engine (comparison only, paged_decode_kernel): two producer
//    warps stream the pages with TMA tensor copies into a ring guarded by
//    mbarriers (every wait bounded), four consumer warps own every fourth
//    stage.
//  * Per stage a consumer warp converts codes to f16 (exact) and runs the
//    score contraction S^T = K Q^T and the value contraction O^T += V^T P^T on
//    the tensor cores (mma m16n8k16, fp32 accumulators): the g <= 8 query
//    heads form the n=8 side.  The stage's P.V tile is then added into
//    separate FP32 registers (O = O*alpha + tile), so the long contraction is
//    summed in IEEE FP32, not inside the MMA.  The CUDA-core engine instead
//    sums FP32 fma chains of exact f16 products; it is slower at every
//    supported g and is used only when asked for.
//  * The softmax max/sum use warp shuffles; P is rounded to f16 for the MMA.
//  * At the end of a segment the CTA's warps merge through shared memory; a
//    unit split over several CTAs leaves FP32 partials.  When the plan gives
//    units few partials, each such CTA of the tensor-core engine counts its
//    partial on a per-unit counter in the workspace, and the CTA whose partial
//    completes the count combines the unit's partials at the end of its range
//    (one launch per call).  Otherwise, and always in the CUDA-core engine, a
//    small merge kernel combines them, launched as a programmatic dependent:
//    it derives the split from the lengths while the decode grid finishes,
//    then waits for that grid and reads the partials.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "fp8kv.h"
#include "trace.cuh"
#include "partition.cuh"
#include "ptx.cuh"
#include "stream_decode.cuh"
#include "walk.cuh"

namespace fp8kv {

// The CUDA-core consumers also keep the segment's f16 queries ([G][D]) and
// their shifts ([8]) in shared memory.
template <int D, int G>
constexpr size_t smem_bytes() {
    return 1024 + Geo<D>::STAGES * kStageBytes + 2 * Geo<D>::XW * 32 * sizeof(float) +
           4 * Geo<D>::STAGES * sizeof(uint64_t) + (2 * kMaxBatch + 1 + 4 + 32 * kNPW) * sizeof(int32_t) + 16 +
           G * D * sizeof(uint16_t) + 8 * sizeof(int);
}

// ---------------------------------------------------------------- CUDA-core consumers
//
// The same split-context flash-decoding step with both contractions on the
// CUDA cores: every score and every P.V sum is an FP32 fma chain of exact f16
// products (K, V and P are f16-exact: E4M3 codes, the f16-rounded
// probabilities; q is the same power-of-two-scaled f16 copy the tensor-core
// consumers use).  Scores: lane = token (D = 256: two lanes per token, one per
// 128-dim half), q broadcast from shared memory.  P.V: lane = D/32 output
// dims, the stage's probabilities broadcast from shared memory.
template <int D, int G>
struct SimtGeo {
    using Gm = Geo<D>;
    static constexpr int TS = Gm::PPS * kBS;              // tokens per stage: 64, 32, 16
    static constexpr int TPL = TS >= 32 ? TS / 32 : 1;     // tokens per lane in the score pass
    static constexpr int DSPLIT = TS >= 32 ? 1 : 32 / TS;  // lanes sharing one token (D = 256: 2)
    static constexpr int DPL = D / 32;                     // output dims per lane in the value pass
    static constexpr int CH = Gm::ROWB / 16;               // 16-byte chunks per box row
    static constexpr int XW = G * DPL + 2;                 // words per lane in the warp merge
    static constexpr int PSM = TS * G * 2;                 // bytes of one warp's f16 probabilities
    static_assert(XW <= Gm::XW, "merge state fits the exchange buffer");
    static_assert(kNCW * PSM <= 2 * Gm::XW * 32 * 4, "probabilities fit the exchange buffer");
    static_assert(DSPLIT == 1 || DSPLIT == Gm::HALVES, "split lanes cover one 128-dim box each");
};

template <int N>
__device__ __forceinline__ void load_f16s(const uint8_t* p, uint16_t (&h)[N]) {
    if constexpr (N == 1) {
        h[0] = *reinterpret_cast<const uint16_t*>(p);
    } else if constexpr (N == 2) {
        const uint32_t x = *reinterpret_cast<const uint32_t*>(p);
        h[0] = x & 0xFFFF; h[1] = x >> 16;
    } else if constexpr (N == 4) {
        const uint2 x = *reinterpret_cast<const uint2*>(p);
        h[0] = x.x & 0xFFFF; h[1] = x.x >> 16; h[2] = x.y & 0xFFFF; h[3] = x.y >> 16;
    } else {
        const uint4 x = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) { h[2 * i] = w[i] & 0xFFFF; h[2 * i + 1] = w[i] >> 16; }
    }
}

template <int N>
__device__ __forceinline__ void store_f16s(uint8_t* p, const float (&v)[N]) {
    if constexpr (N == 1) {
        const __half h = __float2half_rn(v[0]);
        *reinterpret_cast<uint16_t*>(p) = *reinterpret_cast<const uint16_t*>(&h);
    } else if constexpr (N == 2) {
        *reinterpret_cast<uint32_t*>(p) = pack_f16x2(v[0], v[1]);
    } else if constexpr (N == 4) {
        *reinterpret_cast<uint2*>(p) = make_uint2(pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]));
    } else {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]),
                                                  pack_f16x2(v[4], v[5]), pack_f16x2(v[6], v[7]));
    }
}

template <int G, int DPL>
__device__ __forceinline__ void simt_combine(float (&m)[G], float (&l)[G], float (&o)[G][DPL], const float (&m2)[G],
                                             const float (&l2)[G], const float (&o2)[G][DPL]) {
#pragma unroll
    for (int j = 0; j < G; ++j) {
        const float M = fmaxf(m[j], m2[j]);
        const float Mu = M == -INFINITY ? 0.f : M;
        const float f1 = fast_exp2(m[j] - Mu), f2 = fast_exp2(m2[j] - Mu);
        l[j] = l[j] * f1 + l2[j] * f2;
        m[j] = M;
#pragma unroll
        for (int d = 0; d < DPL; ++d) o[j][d] = o[j][d] * f1 + o2[j][d] * f2;
    }
}

// Lane-major exchange of a warp's (m, l, o); m and l are warp-uniform and go
// one head per lane.
template <int G, int DPL>
__device__ __forceinline__ void simt_publish(float* x, int lane, const float (&m)[G], const float (&l)[G],
                                             const float (&o)[G][DPL]) {
#pragma unroll
    for (int j = 0; j < G; ++j)
#pragma unroll
        for (int d = 0; d < DPL; ++d) x[(j * DPL + d) * 32 + lane] = o[j][d];
#pragma unroll
    for (int j = 0; j < G; ++j)
        if (lane == j) {
            x[(G * DPL) * 32 + j] = m[j];
            x[(G * DPL + 1) * 32 + j] = l[j];
        }
}

template <int G, int DPL>
__device__ __forceinline__ void simt_absorb(const float* x, int lane, float (&m)[G], float (&l)[G],
                                            float (&o)[G][DPL]) {
    float m2[G], l2[G], o2[G][DPL];
#pragma unroll
    for (int j = 0; j < G; ++j) {
#pragma unroll
        for (int d = 0; d < DPL; ++d) o2[j][d] = x[(j * DPL + d) * 32 + lane];
        m2[j] = x[(G * DPL) * 32 + j];
        l2[j] = x[(G * DPL + 1) * 32 + j];
    }
    simt_combine<G, DPL>(m, l, o, m2, l2, o2);
}

// Byte offset, inside one V page, of the D/32 codes lane `lane` reads from a
// row whose swizzle phase is k (the row's address bits 7-9 for 128-byte rows,
// 7-8 for 64-byte rows), minus the row start.
template <int D>
__device__ __forceinline__ int simt_v_offset(int lane, int k) {
    using Gm = Geo<D>;
    const int o = D == 256 ? (lane % 16) * 8 : lane * (D / 32);   // offset inside the box row
    const int box = D == 256 ? (lane / 16) * Gm::BOX : 0;
    return box + ((((o >> 4) ^ k) << 4) | (o & 15));
}

// One token of the P.V pass: o[j][d] += P[j] * V[d] for the lane's D/32 dims.
template <int D, int G>
__device__ __forceinline__ void simt_pv_row(const uint8_t* vrow, const uint8_t* prow, float (&o)[G][D / 32]) {
    constexpr int DPL = D / 32;
    uint32_t vh[DPL / 2];
    if constexpr (DPL == 2) {
        vh[0] = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(vrow));
    } else if constexpr (DPL == 4) {
        e4m3x4_to_f16x2x2(*reinterpret_cast<const uint32_t*>(vrow), vh[0], vh[1]);
    } else {
        const uint2 c8 = *reinterpret_cast<const uint2*>(vrow);
        e4m3x4_to_f16x2x2(c8.x, vh[0], vh[1]);
        e4m3x4_to_f16x2x2(c8.y, vh[2], vh[3]);
    }
    uint16_t ph[G];
    load_f16s<G>(prow, ph);
#pragma unroll
    for (int j = 0; j < G; ++j)
#pragma unroll
        for (int k = 0; k < DPL / 2; ++k) fma_f16x2_f16_f32(o[j][2 * k], o[j][2 * k + 1], vh[k], ph[j]);
}

// Shared state of one CTA that the consumer warps read.
struct CtaView {
    uint8_t* ring;
    float* xbuf;
    uint64_t* full_bar;   // [S] K half of a slot landed; V: full_bar + S
    uint64_t* empty_bar;  // [S] K half of a slot consumed; V: empty_bar + S
    const int32_t* pre;
    const int32_t* lens;
    volatile int* flag;
    uint16_t* qsm;   // [G][D] f16 scaled queries of the current segment
    int* qsh;        // [G] their power-of-two shifts
    int64_t s, e;
    Partition part;
    int c;
};

template <int D, int G>
__device__ __forceinline__ void simt_consumers(const DecodeArgs& a, const CtaView& v, int warp, int lane) {
    using Gm = Geo<D>;
    using Sg = SimtGeo<D, G>;
    constexpr int S = Gm::STAGES;
    constexpr int DPL = Sg::DPL;
    const int B = a.batch, Hkv = a.num_kv_heads;
    uint8_t* psm = reinterpret_cast<uint8_t*>(v.xbuf) + warp * Sg::PSM;  // this warp's probabilities
    float m[G], l[G], o[G][DPL], cs[G];
    constexpr int NK = Gm::ROWB == 128 ? 8 : 4;  // swizzle phases of a box row
    int vo[NK];
#pragma unroll
    for (int k = 0; k < NK; ++k) vo[k] = simt_v_offset<D>(lane, k);
    int st_base = 0;
    Walker w;
    walk_start(w, v.pre, B, Hkv, v.s);
    while (true) {
        const int64_t seg_end = min(v.e, w.base + w.n);
        const int lp0 = static_cast<int>(w.g - w.base);
        const int np_seg = static_cast<int>(seg_end - w.g);
        const int nst = (np_seg + Gm::PPS - 1) / Gm::PPS;
        const int L = v.lens[w.b];
        const int lo = first_token(L, a.window);
        const int pg_first = lo / kBS + lp0;

        // ---- the segment's queries -> scaled f16 in shared memory (one warp per head)
        for (int j = warp; j < G; j += kNCW) {
            const uint16_t* src = a.q + (static_cast<int64_t>(w.b) * a.num_q_heads + w.hk * G + j) * D + lane * DPL;
            float x[DPL];
            if constexpr (DPL == 2) {
                const uint32_t u = ld_input(reinterpret_cast<const uint32_t*>(src));
                x[0] = bf16_to_f32(u & 0xFFFF); x[1] = bf16_to_f32(u >> 16);
            } else if constexpr (DPL == 4) {
                const uint2 u = ld_input(reinterpret_cast<const uint2*>(src));
                x[0] = bf16_to_f32(u.x & 0xFFFF); x[1] = bf16_to_f32(u.x >> 16);
                x[2] = bf16_to_f32(u.y & 0xFFFF); x[3] = bf16_to_f32(u.y >> 16);
            } else {
                const uint4 u = ld_input(reinterpret_cast<const uint4*>(src));
                const uint32_t ww[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) { x[2 * i] = bf16_to_f32(ww[i] & 0xFFFF); x[2 * i + 1] = bf16_to_f32(ww[i] >> 16); }
            }
            float qmax = 0.f;
#pragma unroll
            for (int d = 0; d < DPL; ++d) qmax = fmaxf(qmax, fabsf(x[d]));
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) qmax = fmaxf(qmax, __shfl_xor_sync(0xffffffffu, qmax, off));
            int shift = 0;
            if (qmax > 0.f) {
                const int ex = static_cast<int>((__float_as_uint(qmax) >> 23) & 0xFF) - 127;
                shift = max(-100, min(100, 14 - ex));
            }
            const float up = __uint_as_float(static_cast<uint32_t>(127 + shift) << 23);
#pragma unroll
            for (int d = 0; d < DPL; ++d) x[d] *= up;
            store_f16s<DPL>(reinterpret_cast<uint8_t*>(v.qsm + j * D + lane * DPL), x);
            if (lane == 0) v.qsh[j] = shift;
        }
        if (seg_end < v.e) {  // warm L2 with the next segment's queries
            Walker nw = w;
            walk_next(nw, v.pre, Hkv);
            if (lane < G * D * 2 / 128)
                prefetch_l2(reinterpret_cast<const uint8_t*>(a.q + (static_cast<int64_t>(nw.b) * a.num_q_heads + nw.hk * G) * D) +
                            lane * 128);
        }
        consumer_sync();
#pragma unroll
        for (int j = 0; j < G; ++j) {
            cs[j] = unit_score_scale(a, w.hk) * __uint_as_float(static_cast<uint32_t>(127 - v.qsh[j]) << 23);
            m[j] = -INFINITY;
            l[j] = 0.f;
#pragma unroll
            for (int d = 0; d < DPL; ++d) o[j][d] = 0.f;
        }

        for (int i = (warp - st_base % kNCW + kNCW) % kNCW; i < nst; i += kNCW) {
            const int st = st_base + i;
            const int slot = st % S;
            if (v.flag[1]) break;
            if (!mbar_wait_bounded(&v.full_bar[slot], (st / S) & 1, a.wait_ns)) {
                report(a.err, FP8KV_ERR_TIMEOUT);
                v.flag[1] = 1;
                break;
            }
            const int p0 = i * Gm::PPS;
            const int np = min(Gm::PPS, np_seg - p0);
            const uint8_t* kst = v.ring + slot * kStageBytes;
            const uint8_t* vst = kst + kStageHalf;
            const int tok_base = (pg_first + p0) * kBS;

            // ---- scores: s[t][j] = sum_d K[t][d] q_j[d]
            float sc[Sg::TPL][G];
            {
                const int hb = Sg::DSPLIT == 1 ? 0 : lane / Sg::TS;
                float acc[Sg::TPL][G][2];
#pragma unroll
                for (int t = 0; t < Sg::TPL; ++t)
#pragma unroll
                    for (int j = 0; j < G; ++j) acc[t][j][0] = acc[t][j][1] = 0.f;
#pragma unroll
                for (int cc = 0; cc < Sg::CH; ++cc) {
                    uint4 x[Sg::TPL];
#pragma unroll
                    for (int t = 0; t < Sg::TPL; ++t) {
                        const int tl = Sg::DSPLIT == 1 ? t * 32 + lane : lane % Sg::TS;
                        const uint8_t* box = kst + (tl / kBS) * Gm::PAGE + hb * Gm::BOX;
                        x[t] = *reinterpret_cast<const uint4*>(box + swz<Gm::ROWB>(tl % kBS, 16 * cc));
                    }
#pragma unroll
                    for (int j = 0; j < G; ++j) {
                        const uint16_t* qj = v.qsm + j * D + hb * 128 + 16 * cc;
                        const uint4 qa = *reinterpret_cast<const uint4*>(qj);
                        const uint4 qb = *reinterpret_cast<const uint4*>(qj + 8);
#pragma unroll
                        for (int t = 0; t < Sg::TPL; ++t) {
                            uint32_t k0, k1, k2, k3, k4, k5, k6, k7;
                            e4m3x4_to_f16x2x2(x[t].x, k0, k1);
                            e4m3x4_to_f16x2x2(x[t].y, k2, k3);
                            e4m3x4_to_f16x2x2(x[t].z, k4, k5);
                            e4m3x4_to_f16x2x2(x[t].w, k6, k7);
                            fma_f16x2_f32(acc[t][j][0], acc[t][j][1], k0, qa.x);
                            fma_f16x2_f32(acc[t][j][0], acc[t][j][1], k1, qa.y);
                            fma_f16x2_f32(acc[t][j][0], acc[t][j][1], k2, qa.z);
                            fma_f16x2_f32(acc[t][j][0], acc[t][j][1], k3, qa.w);
                            fma_f16x2_f32(acc[t][j][0], acc[t][j][1], k4, qb.x);
                            fma_f16x2_f32(acc[t][j][0], acc[t][j][1], k5, qb.y);
                            fma_f16x2_f32(acc[t][j][0], acc[t][j][1], k6, qb.z);
                            fma_f16x2_f32(acc[t][j][0], acc[t][j][1], k7, qb.w);
                        }
                    }
                }
#pragma unroll
                for (int t = 0; t < Sg::TPL; ++t)
#pragma unroll
                    for (int j = 0; j < G; ++j) {
                        float sv = acc[t][j][0] + acc[t][j][1];
                        if constexpr (Sg::DSPLIT == 2) sv += __shfl_xor_sync(0xffffffffu, sv, 16);
                        sc[t][j] = sv;
                    }
            }

            __syncwarp();
            if (lane == 0) mbar_arrive(&v.empty_bar[slot]);  // the K half is free again

            // ---- mask, scale to log2 units, stage maximum
            float mx[G];
#pragma unroll
            for (int j = 0; j < G; ++j) mx[j] = -INFINITY;
#pragma unroll
            for (int t = 0; t < Sg::TPL; ++t) {
                const int tl = Sg::DSPLIT == 1 ? t * 32 + lane : lane % Sg::TS;
                const int tok = tok_base + tl;
                const bool valid = tl < np * kBS && tok >= lo && tok < L;
#pragma unroll
                for (int j = 0; j < G; ++j) {
                    sc[t][j] = valid ? sc[t][j] * cs[j] : -INFINITY;
                    mx[j] = fmaxf(mx[j], sc[t][j]);
                }
            }
            float alpha[G], muse[G];
#pragma unroll
            for (int j = 0; j < G; ++j) {
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], off));
                const float mn = fmaxf(m[j], mx[j]);
                muse[j] = mn == -INFINITY ? 0.f : mn;
                alpha[j] = fast_exp2(m[j] - muse[j]);
                m[j] = mn;
            }

            // ---- probabilities -> f16 in this warp's shared slice; each lane's
            // share of l moves to the new maximum first
#pragma unroll
            for (int j = 0; j < G; ++j) l[j] *= alpha[j];
            __syncwarp();  // the previous stage's readers are done with the slice
#pragma unroll
            for (int t = 0; t < Sg::TPL; ++t) {
                const int tl = Sg::DSPLIT == 1 ? t * 32 + lane : lane % Sg::TS;
                float pr[G];
#pragma unroll
                for (int j = 0; j < G; ++j) pr[j] = fast_exp2(sc[t][j] - muse[j]);
                if (Sg::DSPLIT == 1 || lane < Sg::TS) {
#pragma unroll
                    for (int j = 0; j < G; ++j) l[j] += pr[j];
                    store_f16s<G>(psm + tl * G * 2, pr);
                }
            }
            __syncwarp();

            // ---- P.V: o[j][d] += sum_t P[t][j] V[t][d] over the stage's valid tokens
            if (!mbar_wait_bounded(&v.full_bar[S + slot], (st / S) & 1, a.wait_ns)) {
                report(a.err, FP8KV_ERR_TIMEOUT);
                v.flag[1] = 1;
                break;
            }
#pragma unroll
            for (int j = 0; j < G; ++j)
#pragma unroll
                for (int d = 0; d < DPL; ++d) o[j][d] *= alpha[j];
            const int t_lo = max(lo - tok_base, 0);
            const int t_hi = min(L - tok_base, np * kBS);
            if (t_lo == 0 && t_hi == np * kBS) {
                // every token of the stage attended: fully unrolled rows with
                // the swizzled lane offsets taken from vo[]
#pragma unroll
                for (int p = 0; p < Gm::PPS; ++p) {
                    if (p < np) {
#pragma unroll
                        for (int r = 0; r < kBS; ++r)
                            simt_pv_row<D, G>(vst + p * Gm::PAGE + r * Gm::ROWB + vo[Gm::ROWB == 128 ? (r & 7) : ((r >> 1) & 3)],
                                              psm + (p * kBS + r) * G * 2, o);
                    }
                }
            } else {
#pragma unroll 2
                for (int t = t_lo; t < t_hi; ++t) {
                    const int r = t % kBS;
                    simt_pv_row<D, G>(vst + (t / kBS) * Gm::PAGE + r * Gm::ROWB +
                                          simt_v_offset<D>(lane, Gm::ROWB == 128 ? (r & 7) : ((r >> 1) & 3)),
                                      psm + t * G * 2, o);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&v.empty_bar[S + slot]);
        }
        st_base += nst;

#pragma unroll
        for (int j = 0; j < G; ++j)
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) l[j] += __shfl_xor_sync(0xffffffffu, l[j], off);

        // ---- merge the four warps' states into warp 0 (the exchange buffer
        // also holds the probability slices: every warp leaves its stages first)
        consumer_sync();
        if (warp >= 2) simt_publish<G, DPL>(v.xbuf + (warp - 2) * Sg::XW * 32, lane, m, l, o);
        consumer_sync();
        if (warp < 2) simt_absorb<G, DPL>(v.xbuf + warp * Sg::XW * 32, lane, m, l, o);
        consumer_sync();
        if (warp == 1) simt_publish<G, DPL>(v.xbuf, lane, m, l, o);
        consumer_sync();
        if (warp == 0) simt_absorb<G, DPL>(v.xbuf, lane, m, l, o);

        // ---- emit (as the tensor-core consumers do)
        const int u = w.b * Hkv + w.hk;
        const int c_first = cta_of(v.part, w.base);
        const int c_last = cta_of(v.part, w.base + w.n - 1);
        const int k_u = c_last - c_first + 1;
        if (warp == 0) {
            if (k_u == 1) {
                uint16_t* out_u = a.out + (static_cast<int64_t>(w.b) * a.num_q_heads + w.hk * G) * D + lane * DPL;
#pragma unroll
                for (int j = 0; j < G; ++j) {
                    const float sc_out = l[j] > 0.f ? unit_v_scale(a, w.hk) / l[j] : 0.f;
                    uint32_t pk[DPL / 2];
#pragma unroll
                    for (int k = 0; k < DPL / 2; ++k)
                        pk[k] = static_cast<uint32_t>(f32_to_bf16(o[j][2 * k] * sc_out)) |
                                (static_cast<uint32_t>(f32_to_bf16(o[j][2 * k + 1] * sc_out)) << 16);
                    if constexpr (DPL == 2) *reinterpret_cast<uint32_t*>(out_u + j * D) = pk[0];
                    else if constexpr (DPL == 4) *reinterpret_cast<uint2*>(out_u + j * D) = make_uint2(pk[0], pk[1]);
                    else *reinterpret_cast<uint4*>(out_u + j * D) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                }
            } else {
                const int64_t slot_idx = static_cast<int64_t>(u) + v.c;
#pragma unroll
                for (int j = 0; j < G; ++j) {
                    float* po = a.part_o + (slot_idx * G + j) * D + lane * DPL;
#pragma unroll
                    for (int d = 0; d < DPL; d += 2) *reinterpret_cast<float2*>(po + d) = make_float2(o[j][d], o[j][d + 1]);
                    if (lane == 0) a.part_ml[slot_idx * kMaxG + j] = make_float2(m[j], l[j]);
                }
            }
        }
        consumer_sync();  // warp 0 is done with the exchange buffer
        if (seg_end >= v.e) break;
        walk_next(w, v.pre, Hkv);
    }
}

// The CUDA-core engine: TMA producers, an mbarrier-guarded ring, CUDA-core
// consumers (simt_consumers).  E4M3 cache, per-tensor or per-head scales.
template <int D, int G>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                        const DecodeArgs a) {
    using Gm = Geo<D>;
    constexpr int S = Gm::STAGES;
    extern __shared__ uint8_t smem_raw[];
    // 1024-byte aligned ring (the swizzle pattern is a function of address
    // bits 4..9); offsetting the shared array keeps the address space known.
    uint8_t* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    float* xbuf = reinterpret_cast<float*>(ring + S * kStageBytes);  // [2][XW][32]
    // Each ring slot holds a K half and a V half with a barrier pair each:
    // full_bar[s] / full_bar[S + s] complete when the K / V copies land,
    // empty_bar[s] / empty_bar[S + s] when the consumer is done with them, so
    // the K half returns to its producer as soon as the scores are computed.
    uint64_t* full_bar = reinterpret_cast<uint64_t*>(xbuf + 2 * Gm::XW * 32);  // [2][S]
    uint64_t* empty_bar = full_bar + 2 * S;                                     // [2][S]
    int32_t* pre = reinterpret_cast<int32_t*>(empty_bar + 2 * S);    // [kMaxBatch + 1] page prefix
    int32_t* lens = pre + kMaxBatch + 1;                             // [kMaxBatch] clamped lengths
    volatile int* flag = reinterpret_cast<volatile int*>(lens + kMaxBatch);  // [1] abort
    int32_t* ids = lens + kMaxBatch + 4;                             // [kNPW][32] block ids per producer
    uint16_t* qsm = reinterpret_cast<uint16_t*>(                     // CUDA-core consumers: [G][D] f16 q
        ring + ((reinterpret_cast<uint8_t*>(ids + 32 * kNPW) - ring + 15) & ~static_cast<intptr_t>(15)));
    int* qsh = reinterpret_cast<int*>(qsm + G * D);                  // [8] q shifts

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // Set-up that reads no input: the ring barriers (shared memory) and the
    // tensor-map descriptors (kernel parameters).
    if (tid == 0) {
        for (int st0 = 0; st0 < 2 * S; ++st0) {
            mbar_init(&full_bar[st0], 1);
            mbar_init(&empty_bar[st0], 1);
        }
        flag[1] = 0;
        fence_barrier_init();
    }
    if (warp == kNCW && lane == 0) prefetch_tmap(&tmK);
    if (warp == kNCW + 1 && lane == 0) prefetch_tmap(&tmV);
    // This grid may have started before the previous one on the stream
    // finished (programmatic launch): wait for it before reading any input,
    // since that grid may have produced them (q, lengths, tables, the cache).
    griddep_wait();
    // The merge kernel that follows may start now: it reads the lengths (final,
    // since every CTA of this grid is past its wait) and waits for this grid's
    // completion before reading anything this grid writes.
    griddep_launch_dependents();
    const int B = a.batch, Hkv = a.num_kv_heads, C = gridDim.x, c = blockIdx.x;

    // ---- attended pages per sequence and their exclusive prefix; the error
    // word is read alongside (a CTA of an earlier call that gave up a wait
    // fails every later call until the workspace is re-initialised)
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
            flag[2] = prev_err == FP8KV_ERR_TIMEOUT;
        }
    }
    __syncthreads();
    if (flag[2]) return;

    const int64_t P = static_cast<int64_t>(Hkv) * pre[B];
    // sequences with nothing to attend (length 0) produce zeros
    for (int b = c; b < B; b += C) {
        if (pre[b + 1] == pre[b]) {
            uint16_t* ob = a.out + static_cast<int64_t>(b) * a.num_q_heads * D;
            for (int i = tid; i < a.num_q_heads * D; i += kThreads) ob[i] = 0;
        }
    }
    const int Ce = static_cast<int>(P < C ? P : C);  // CTAs with work: every one gets >= 1 page
    if (c >= Ce) return;
    const Partition part = make_partition(P, Ce);
    const int64_t s = range_start(part, c);
    const int64_t e = range_start(part, c + 1);

    if (warp >= kNCW) {
        // ------------------------------------------------------------ producers
        // Two producer warps walk the same pages: the first issues the K
        // copies (and posts each stage's byte count), the second the V copies,
        // so their issue latencies overlap.  In each, lane 0 alone issues;
        // once per 32 pages the warp hands it the next 32 block ids through
        // shared memory and loads the 32 after those while lane 0 works.
        const int pw = warp - kNCW;
        const CUtensorMap* tm = pw == 0 ? &tmK : &tmV;
        int32_t* my_ids = ids + pw * 32;
        const uint64_t pol = l2_policy_evict_first();
        int st = 0;
        bool ok = true;
        // Batches of up to 32 pages never straddle a segment; the ids of the
        // batch after the current one (in the same or the next segment) are
        // loaded while lane 0 issues the current one.
        //
        // With a row to append (a decode step), the producer that owns a
        // unit's last page first writes that sequence's newest K (or V) row
        // into the page, orders the write before its own copies
        // (fence.proxy.async), and only then issues the page.
        const bool appending = a.k_new != nullptr;
        const uint16_t* new_rows = pw == 0 ? a.k_new : a.v_new;
        uint8_t* cache = pw == 0 ? a.k_cache : a.v_cache;
        const float scale_raw = pw == 0 ? a.k_scale_raw : a.v_scale_raw;  // per-tensor; per head below
        const float* head_scales = pw == 0 ? a.k_scales : a.v_scales;
        Walker w;
        walk_start(w, pre, B, Hkv, s);
        auto seg_pages = [&](const Walker& x) { return static_cast<int>(min(e, x.base + x.n) - x.g); };
        auto seg_row = [&](const Walker& x) {
            return a.block_tables + static_cast<int64_t>(x.b) * a.max_blocks_per_seq +
                   first_token(lens[x.b], a.window) / kBS + (x.g - x.base);
        };
        auto seg_reaches_end = [&](const Walker& x) { return min(e, x.base + x.n) == x.base + x.n; };
        int np_seg = seg_pages(w);
        const int32_t* row = seg_row(w);
        int p0 = 0;
        int nxt = load_block_id(row, lane, np_seg, a.num_blocks, a.err);
        int seg_b = w.b, seg_hk = w.hk;
        bool seg_last = appending && seg_reaches_end(w);
        NewRow<D> nrow;
        // the cache (and the new rows) have Hkv >> kv_shift heads; unit hk reads head hk >> kv_shift
        const int kvs = a.kv_shift, Hc = Hkv >> kvs;
        if (seg_last) load_new_row<D>(nrow, new_rows + (static_cast<int64_t>(w.b) * Hc + (w.hk >> kvs)) * D, lane);
        bool more = true;
        while (ok && more) {
            const int cur = nxt;
            const int hk = seg_hk;
            const int nb = min(32, np_seg - p0);
            const bool batch_has_last = seg_last && p0 + nb == np_seg;
            const int batch_b = seg_b;
            const NewRow<D> batch_row = nrow;
            __syncwarp();  // lane 0 is done with the previous batch
            my_ids[lane] = cur;
            p0 += 32;
            if (p0 >= np_seg) {
                if (min(e, w.base + w.n) >= e) {
                    more = false;
                } else {
                    walk_next(w, pre, Hkv);
                    np_seg = seg_pages(w);
                    row = seg_row(w);
                    p0 = 0;
                    seg_b = w.b;
                    seg_hk = w.hk;
                    seg_last = appending && seg_reaches_end(w);
                    if (seg_last)
                        load_new_row<D>(nrow, new_rows + (static_cast<int64_t>(w.b) * Hc + (w.hk >> kvs)) * D, lane);
                }
            }
            nxt = more ? load_block_id(row + p0, lane, np_seg - p0, a.num_blocks, a.err) : 0;
            __syncwarp();
            if (batch_has_last) {
                const int id = my_ids[nb - 1];
                if (id >= 0) {
                    const int L = lens[batch_b];
                    // with two units per cache head both write the same bytes: identical values
                    uint8_t* dst_row = cache + ((static_cast<int64_t>(id) * Hc + (hk >> kvs)) * kBS + (L - 1) % kBS) * D;
                    store_new_row<D>(batch_row, dst_row, lane,
                                           head_scales ? ld_input(head_scales + (hk >> kvs)) : scale_raw);
                    fence_proxy_async_global();
                }
                __syncwarp();
            }
            if (lane == 0) {
                for (int q = 0; q < nb && ok; q += Gm::PPS) {
                    const int np = min(Gm::PPS, nb - q);
                    const int slot = st % S;
                    if (flag[1] || (st >= S && !mbar_wait_bounded(&empty_bar[pw * S + slot], ((st / S) & 1) ^ 1,
                                                                   a.wait_ns))) {
                        report(a.err, FP8KV_ERR_TIMEOUT);
                        flag[1] = 1;
                        ok = false;
                        break;
                    }
                    if (c == 0 && pw == 0 && st == a.stall_stage) {  // test hook: this stage never arrives
                        ++st;
                        continue;
                    }
                    // this producer's half of the stage (K or V)
                    mbar_arrive_expect_tx(&full_bar[pw * S + slot], static_cast<uint32_t>(np * Gm::PAGE));
                    uint8_t* dst = ring + slot * kStageBytes + pw * kStageHalf;
                    for (int p = 0; p < np; ++p) {
                        const int id = max(my_ids[q + p], 0);
#pragma unroll
                        for (int h = 0; h < Gm::HALVES; ++h)
                            tma_load_4d(dst + p * Gm::PAGE + h * Gm::BOX, tm, &full_bar[pw * S + slot], h * 128, 0,
                                        hk >> kvs, id, pol);
                    }
                    ++st;
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
        }
        // The CTA must not exit with copies in flight, and consumers that gave
        // up a wait no longer wait for them: before leaving, the producer waits
        // (with the normal limit) for the last ring's worth of stages it
        // issued.  Normally those have landed or are about to.
        if (lane == 0) {
            for (int t = st > S ? st - S : 0; t < st; ++t)
                if (!(c == 0 && pw == 0 && t == a.stall_stage))  // a stage the test hook skipped has no copies
                    mbar_wait_bounded(&full_bar[pw * S + t % S], (t / S) & 1, kWaitLimitNs);
        }
        return;
    }

    // ---------------------------------------------------------------- consumers
    const CtaView v{ring, xbuf, full_bar, empty_bar, pre, lens, flag, qsm, qsh, s, e, part, c};
    simt_consumers<D, G>(a, v, warp, lane);
}

// ---------------------------------------------------------------- host side

struct Plan {
    int batch;  // sequences per launch (batches above kMaxBatch run in chunks)
    int ctas;   // CTAs per launch
};

Plan make_plan(int batch, int num_kv_heads, int D, int max_seq_len, int window, int sms) {
    (void)D;
    Plan p{std::max(1, std::min(batch, kMaxBatch)), 1};
    if (max_seq_len <= 0) return p;
    const int64_t all_pages = (max_seq_len + kBS - 1) / kBS;
    int64_t max_pages = all_pages;
    if (window > 0 && window < max_seq_len) max_pages = std::min<int64_t>(all_pages, (window + kBS - 1) / kBS + 1);
    const int64_t pmax = static_cast<int64_t>(p.batch) * num_kv_heads * max_pages;
    const int64_t want = (pmax + kMinPagesPerCta - 1) / kMinPagesPerCta;
    p.ctas = static_cast<int>(std::max<int64_t>(
        1, std::min<int64_t>(std::min<int64_t>(want, static_cast<int64_t>(sms) * kCtasPerSm), kMaxMergeSplits)));
    return p;
}

// Who merges the split units of a tensor-core launch.  The CTA that completes
// a unit merges it when the unit's partials are few (one SM reads them all
// through L2: about 25 GB/s measured); otherwise the merge kernel, whose CTAs
// (one per unit and query head) spread the reading over many SMs.  The
// partials per unit are estimated from the plan with every sequence at
// max_seq_len: a unit of n pages meets at most ceil(n / pages per CTA) + 1
// CTAs.  Shorter sequences only change the speed of the chosen merge.
constexpr int64_t kInlineMergeBytes = 16 << 10;

bool merge_inline(const Plan& p, int batch, int units_per_seq, int G, int D, int max_seq_len, int window) {
    if (p.ctas <= 1 || max_seq_len <= 0) return true;
    const int64_t all_pages = (max_seq_len + kBS - 1) / kBS;
    int64_t n = all_pages;
    if (window > 0 && window < max_seq_len) n = std::min<int64_t>(all_pages, (window + kBS - 1) / kBS + 1);
    const int64_t total = static_cast<int64_t>(batch) * units_per_seq * n;
    const int64_t per_cta = std::max<int64_t>(1, total / p.ctas);
    const int64_t k_est = std::min<int64_t>(p.ctas, (n + per_cta - 1) / per_cta + 1);
    return k_est * G * D * static_cast<int64_t>(sizeof(float)) <= kInlineMergeBytes;
}

struct WsLayout {
    size_t cnt, ml, o, total;  // byte offsets of the split counters, the partial (max, sum), the partial outputs
};

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

WsLayout ws_layout(int batch, int num_q_heads, int num_kv_heads, int D, const Plan& p) {
    (void)batch;
    const size_t units = static_cast<size_t>(p.batch) * num_kv_heads;
    const size_t slots = units + p.ctas;
    const int G = num_q_heads / num_kv_heads;
    WsLayout w;
    w.cnt = 256;  // after the header (the error word)
    w.ml = w.cnt + align256(units * sizeof(int32_t));
    w.o = w.ml + align256(slots * kMaxG * sizeof(float2));
    w.total = w.o + align256(slots * G * D * sizeof(float));
    return w;
}

// SM count of the current device (queried once per device).
int device_sms(int* sms) {
    static std::atomic<int> cache[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return -1;
    if (dev >= 0 && dev < 64) {
        const int c = cache[dev].load(std::memory_order_relaxed);
        if (c > 0) {
            *sms = c;
            return 0;
        }
    }
    if (cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return -1;
    if (dev >= 0 && dev < 64) cache[dev].store(*sms, std::memory_order_relaxed);
    return 0;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// The cache as a 4-D tensor {D, 16 tokens, kv heads, blocks} of bytes; one box
// is one page (or one 128-byte-wide half of a D=256 page).
bool encode_cache_map(CUtensorMap* m, const void* base, int64_t num_blocks, int Hkv, int D) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(kBS),
                                static_cast<cuuint64_t>(Hkv), static_cast<cuuint64_t>(num_blocks)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(kBS) * D,
                                   static_cast<cuuint64_t>(kBS) * D * Hkv};
    const cuuint32_t box[4] = {static_cast<cuuint32_t>(D >= 128 ? 128 : D), static_cast<cuuint32_t>(kBS), 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    const CUtensorMapSwizzle sw = D >= 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Encoding a tensor map is pure host work on its arguments; the last few
// (pointer, shape) -> map results are kept so repeated decode calls over the
// same cache skip it.
bool make_cache_map(CUtensorMap* m, const void* base, int64_t num_blocks, int Hkv, int D) {
    struct Entry {
        const void* base;
        int64_t num_blocks;
        int Hkv, D;
        CUtensorMap map;
    };
    constexpr int kEntries = 8;
    static std::mutex mu;
    static Entry entries[kEntries];
    static int used = 0, next = 0;
    {
        std::lock_guard<std::mutex> lock(mu);
        for (int i = 0; i < used; ++i) {
            const Entry& e = entries[i];
            if (e.base == base && e.num_blocks == num_blocks && e.Hkv == Hkv && e.D == D) {
                *m = e.map;
                return true;
            }
        }
    }
    if (!encode_cache_map(m, base, num_blocks, Hkv, D)) return false;
    std::lock_guard<std::mutex> lock(mu);
    Entry& e = entries[next];
    e.base = base;
    e.num_blocks = num_blocks;
    e.Hkv = Hkv;
    e.D = D;
    e.map = *m;
    next = (next + 1) % kEntries;
    if (used < kEntries) ++used;
    return true;
}

template <int D, int G>
cudaError_t launch(const CUtensorMap& mk, const CUtensorMap& mv, const DecodeArgs& a, int ctas,
                   cudaStream_t stream) {
    // The shared-memory opt-in is per device; remember which devices have it.
    static std::atomic<uint64_t> done_mask{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
    if (bit == 0 || !(done_mask.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(paged_decode_kernel<D, G>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(smem_bytes<D, G>()));
        if (e != cudaSuccess) return e;
        done_mask.fetch_or(bit, std::memory_order_release);
    }
    // Both grids may start before the previous work on the stream ends; each
    // waits (griddepcontrol.wait) before touching what that work wrote.
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_bytes<D, G>();
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, paged_decode_kernel<D, G>, mk, mv, a);
    if (e != cudaSuccess || ctas == 1) return e;  // one CTA: every unit is written directly
    cudaLaunchConfig_t mcfg = {};
    mcfg.gridDim = dim3(a.batch * a.num_kv_heads, G);
    mcfg.blockDim = dim3(merge_threads<D>());
    mcfg.dynamicSmemBytes = 0;
    mcfg.stream = stream;
    mcfg.attrs = attr;
    mcfg.numAttrs = 1;
    return cudaLaunchKernelEx(&mcfg, merge_kernel<D, G>, a);
}

template <int D>
cudaError_t launch_g(int G, const CUtensorMap& mk, const CUtensorMap& mv, const DecodeArgs& a, int ctas,
                     cudaStream_t s) {
    switch (G) {
        case 1: return launch<D, 1>(mk, mv, a, ctas, s);
        case 2: return launch<D, 2>(mk, mv, a, ctas, s);
        case 4: return launch<D, 4>(mk, mv, a, ctas, s);
        case 8: return launch<D, 8>(mk, mv, a, ctas, s);
        default: return cudaErrorInvalidValue;
    }
}

// The contraction engine a call uses when the caller leaves it open.
bool default_is_cuda_cores(int /*head_dim*/, int /*G*/) { return false; }

bool supported(int head_dim, int block_size, int G) {
    return (head_dim == 64 || head_dim == 128 || head_dim == 256) && block_size == kBS &&
           (G == 1 || G == 2 || G == 4 || G == 8 || G == 16);
}

// How the kernels see the heads.  The streaming kernel at d <= 128 carries
// g = 16 natively (two MMA n-tiles of 8 heads on the same K and V fragments:
// each page is read once).  At d = 256, and on the CUDA-core engine, g = 16
// runs as two units of 8 query heads per cache head (each reads the head's
// pages): two n-tiles' accumulators do not fit beside the rest there.
struct HeadMap {
    int units_per_seq;  // kv-head units per sequence
    int g;              // query heads per unit
    int shift;          // unit -> cache head: hk >> shift
};

HeadMap head_map(int num_q_heads, int num_kv_heads, int head_dim, bool simt) {
    const int G = num_q_heads / num_kv_heads;
    if (G == 16 && (simt || head_dim > 128)) return {2 * num_kv_heads, 8, 1};
    return {num_kv_heads, G, 0};
}

}  // namespace fp8kv

using namespace fp8kv;

extern "C" size_t fp8kv_paged_decode_workspace_size(int batch, int num_q_heads, int num_kv_heads, int head_dim,
                                                    int max_seq_len, int block_size, int window) {
    if (batch < 0 || num_kv_heads < 1 || num_q_heads < 1 || num_q_heads % num_kv_heads != 0 || max_seq_len < 0)
        return 0;
    if (!supported(head_dim, block_size, num_q_heads / num_kv_heads)) return 0;
    int sms = 0;
    if (device_sms(&sms) != 0) return 0;
    // enough for either engine (their head mappings differ at g = 16)
    size_t total = 0;
    for (const bool simt : {false, true}) {
        const HeadMap hm = head_map(num_q_heads, num_kv_heads, head_dim, simt);
        const Plan p = make_plan(batch, hm.units_per_seq, head_dim, max_seq_len, window, sms);
        total = std::max(total, ws_layout(batch, hm.units_per_seq * hm.g, hm.units_per_seq, head_dim, p).total);
    }
    return total;
}

namespace {

// Host-side staging around a decode call: the inputs copied in before it, the
// output copied out after it (fp8kv_decode_step_host).
struct HostStage {
    const void* h_in;
    void* d_in;
    size_t in_bytes;
    void* h_out;
};

// The failure-path test hook's settings (fp8kv_debug_paged_decode_stall).
struct StallHook {
    int stall_stage;
    uint64_t wait_ns;
};

// What fp8kv_paged_decode_weights adds to a decode.
struct WeightsOut {
    float* weights;
    float decay;
};

// Sequences per launch of such a decode, and what it needs behind the decode's
// workspace.  A launch's scores stay within kScoreBytes (they are read back once,
// so they should not leave the L2), or are one sequence's.
constexpr int64_t kScoreBytes = INT64_C(64) << 20;

struct ScorePlan {
    int batch;        // sequences per launch
    int tokens;       // places a unit's scores take
    size_t softmax, scores, total;   // bytes from the end of the decode's workspace
};

ScorePlan score_plan(int batch, int num_q_heads, int max_seq_len, int window) {
    ScorePlan p;
    int64_t pages = (static_cast<int64_t>(max_seq_len) + kBS - 1) / kBS;
    if (window > 0) pages = std::min<int64_t>(pages, (static_cast<int64_t>(window) + kBS - 1) / kBS + 1);
    p.tokens = static_cast<int>(pages * kBS);
    const int64_t each = std::max<int64_t>(1, pages * kBS * num_q_heads * static_cast<int64_t>(sizeof(float)));
    p.batch = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(std::min(batch, kMaxBatch), kScoreBytes / each)));
    p.softmax = 0;
    p.scores = align256(static_cast<size_t>(p.batch) * num_q_heads * sizeof(float2));
    p.total = p.scores + align256(static_cast<size_t>(p.batch) * static_cast<size_t>(each));
    return p;
}

fp8kv_status decode_impl(const void* q, const void* k_new, const void* v_new, const uint8_t* k_cache,
                         const uint8_t* v_cache, int64_t num_blocks, const int32_t* block_tables,
                         int max_blocks_per_seq, const int32_t* seq_lens, int max_seq_len, int batch,
                         int num_q_heads, int num_kv_heads, int head_dim, int block_size, float k_scale,
                         float v_scale, float sm_scale, int window, void* out, void* workspace,
                         size_t workspace_bytes, void* stream, int engine, int es = 1,
                         const float* k_scales = nullptr, const float* v_scales = nullptr, bool e5m2 = false,
                         const HostStage* hs = nullptr, const StallHook* dbg = nullptr,
                         const float* k_page_scales = nullptr, const float* v_page_scales = nullptr,
                         const WeightsOut* wout = nullptr) {
    auto a16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
    if (batch < 0 || batch > 65535 || num_kv_heads < 1 || num_kv_heads > 65535 || num_q_heads < 1 ||
        num_q_heads % num_kv_heads != 0 || max_seq_len < 0 || num_blocks < 1 || max_blocks_per_seq < 0)
        return FP8KV_ERR_INVALID_ARG;
    if (!std::isfinite(k_scale) || !(k_scale > 0) || !std::isfinite(v_scale) || !(v_scale > 0) ||
        !std::isfinite(sm_scale))
        return FP8KV_ERR_INVALID_ARG;
    if (!supported(head_dim, block_size, num_q_heads / num_kv_heads)) return FP8KV_ERR_UNSUPPORTED;
    if (engine != FP8KV_ENGINE_DEFAULT && engine != FP8KV_ENGINE_TENSOR_CORES && engine != FP8KV_ENGINE_CUDA_CORES)
        return FP8KV_ERR_INVALID_ARG;
    const bool simt = engine == FP8KV_ENGINE_CUDA_CORES ||
                      (engine == FP8KV_ENGINE_DEFAULT && default_is_cuda_cores(head_dim, num_q_heads / num_kv_heads));
    const HeadMap hm = head_map(num_q_heads, num_kv_heads, head_dim, simt);
    const int G = hm.g;
    if (num_blocks >= (INT64_C(1) << 31) || num_blocks * num_kv_heads >= (INT64_C(1) << 31))
        return FP8KV_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(max_blocks_per_seq) * block_size < max_seq_len) return FP8KV_ERR_INVALID_ARG;
    // total (sequence, kv head, page) triples of one launch must stay far inside int64 index math
    if (static_cast<int64_t>(std::min(batch, kMaxBatch)) * num_kv_heads * ((max_seq_len + kBS - 1) / kBS + 1) >=
        (INT64_C(1) << 40))
        return FP8KV_ERR_UNSUPPORTED;
    if (batch == 0) return FP8KV_OK;
    if (!q || !k_cache || !v_cache || !block_tables || !seq_lens || !out) return FP8KV_ERR_INVALID_ARG;
    if (!a16(q) || !a16(k_cache) || !a16(v_cache) || !a16(out)) return FP8KV_ERR_INVALID_ARG;
    if ((k_new == nullptr) != (v_new == nullptr)) return FP8KV_ERR_INVALID_ARG;
    if (k_new && (!a16(k_new) || !a16(v_new))) return FP8KV_ERR_INVALID_ARG;
    if ((k_scales == nullptr) != (v_scales == nullptr)) return FP8KV_ERR_INVALID_ARG;
    if (k_scales && ((reinterpret_cast<uintptr_t>(k_scales) & 3u) || (reinterpret_cast<uintptr_t>(v_scales) & 3u)))
        return FP8KV_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(block_tables) & 3u) || (reinterpret_cast<uintptr_t>(seq_lens) & 3u))
        return FP8KV_ERR_INVALID_ARG;
    int sms = 0;
    if (device_sms(&sms) != 0) return FP8KV_ERR_CUDA;
    const ScorePlan sp = wout ? score_plan(batch, num_q_heads, max_seq_len, window) : ScorePlan{kMaxBatch, 0, 0, 0, 0};
    const WsLayout w = ws_layout(batch, num_q_heads, hm.units_per_seq, head_dim,
                                 make_plan(std::min(batch, sp.batch), hm.units_per_seq, head_dim, max_seq_len, window, sms));
    if (!workspace || workspace_bytes < w.total + sp.total || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return FP8KV_ERR_WORKSPACE;

    CUtensorMap mk, mv;  // the CUDA-core engine's TMA view of the caches (rows of head_dim bytes)
    if (simt && (!make_cache_map(&mk, k_cache, num_blocks, num_kv_heads, head_dim) ||
                 !make_cache_map(&mv, v_cache, num_blocks, num_kv_heads, head_dim)))
        return FP8KV_ERR_CUDA;

    uint8_t* ws = static_cast<uint8_t*>(workspace);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (hs && hs->in_bytes > 0 &&
        cudaMemcpyAsync(hs->d_in, hs->h_in, hs->in_bytes, cudaMemcpyHostToDevice, s) != cudaSuccess)
        return FP8KV_ERR_CUDA;
    // A host output buffer that the device can address (page-locked memory,
    // mapped under unified addressing) receives the result directly from the
    // kernels' stores, across the host link; otherwise the result goes to
    // `out` and is copied to h_out after the step.
    bool direct_out = false;
    if (hs && hs->h_out) {
        cudaPointerAttributes pa;
        if (cudaPointerGetAttributes(&pa, hs->h_out) == cudaSuccess && pa.type == cudaMemoryTypeHost &&
            pa.devicePointer != nullptr && a16(pa.devicePointer)) {
            out = pa.devicePointer;
            direct_out = true;
        } else {
            (void)cudaGetLastError();  // not a registered host buffer: copy instead
        }
    }
    // Batches above kMaxBatch sequences (or whose scores take more room) run as
    // consecutive launches on the stream, reusing the workspace.
    for (int b0 = 0; b0 < batch; b0 += sp.batch) {
        const int nb = std::min(sp.batch, batch - b0);
        const Plan p = make_plan(nb, hm.units_per_seq, head_dim, max_seq_len, window, sms);
        DecodeArgs a;
        a.q = static_cast<const uint16_t*>(q) + static_cast<int64_t>(b0) * num_q_heads * head_dim;
        a.k_new = k_new ? static_cast<const uint16_t*>(k_new) + static_cast<int64_t>(b0) * num_kv_heads * head_dim
                        : nullptr;
        a.v_new = v_new ? static_cast<const uint16_t*>(v_new) + static_cast<int64_t>(b0) * num_kv_heads * head_dim
                        : nullptr;
        a.k_cache = const_cast<uint8_t*>(k_cache);
        a.v_cache = const_cast<uint8_t*>(v_cache);
        a.k_scale_raw = k_scale;
        a.v_scale_raw = v_scale;
        a.k_scales = k_scales;
        a.v_scales = v_scales;
        a.k_page_scales = k_page_scales;
        a.v_page_scales = v_page_scales;
        a.sm_scale = sm_scale;
        a.block_tables = block_tables + static_cast<int64_t>(b0) * max_blocks_per_seq;
        a.seq_lens = seq_lens + b0;
        a.out = static_cast<uint16_t*>(out) + static_cast<int64_t>(b0) * num_q_heads * head_dim;
        a.err = reinterpret_cast<uint32_t*>(ws);
        a.decode_ctas = p.ctas;
        a.part_ml = reinterpret_cast<float2*>(ws + w.ml);
        a.part_o = reinterpret_cast<float*>(ws + w.o);
        a.split_cnt = reinterpret_cast<int32_t*>(ws + w.cnt);
        a.inline_merge = !simt && merge_inline(p, nb, hm.units_per_seq, G, head_dim, max_seq_len, window);
        a.num_blocks = num_blocks;
        a.max_blocks_per_seq = max_blocks_per_seq;
        a.max_seq_len = max_seq_len;
        a.batch = nb;
        a.num_q_heads = num_q_heads;
        a.num_kv_heads = hm.units_per_seq;
        a.kv_shift = hm.shift;
        a.window = window > 0 ? window : 0;
        a.score_scale = sm_scale * k_scale * kLog2e;
        a.v_scale = v_scale;
        a.wait_ns = dbg ? dbg->wait_ns : kWaitLimitNs;
        a.stall_stage = dbg ? dbg->stall_stage : -1;
        a.scores = wout ? reinterpret_cast<float*>(ws + w.total + sp.scores) : nullptr;
        a.softmax = wout ? reinterpret_cast<float2*>(ws + w.total + sp.softmax) : nullptr;
        a.score_tokens = sp.tokens;
        a.weights = wout ? wout->weights : nullptr;
        a.decay = wout ? wout->decay : 0.f;
        cudaError_t e;
        if (wout) {
            e = launch_stream_weights(head_dim, G, es, e5m2, a, p.ctas, s);
        } else if (!simt) {
            if (k_page_scales)
                e = launch_stream_block(head_dim, G, a, p.ctas, s);
            else if (es == 2)
                e = head_dim == 64 ? launch_stream_g<64, 2>(G, a, p.ctas, s)
                    : head_dim == 128 ? launch_stream_g<128, 2>(G, a, p.ctas, s)
                                      : launch_stream_g<256, 2>(G, a, p.ctas, s);
            else if (e5m2)
                e = head_dim == 64 ? launch_stream_g<64, 1, true>(G, a, p.ctas, s)
                    : head_dim == 128 ? launch_stream_g<128, 1, true>(G, a, p.ctas, s)
                                      : launch_stream_g<256, 1, true>(G, a, p.ctas, s);
            else
                e = head_dim == 64 ? launch_stream_g<64>(G, a, p.ctas, s)
                    : head_dim == 128 ? launch_stream_g<128>(G, a, p.ctas, s)
                                      : launch_stream_g<256>(G, a, p.ctas, s);
        } else {
            e = head_dim == 64 ? launch_g<64>(G, mk, mv, a, p.ctas, s)
                : head_dim == 128 ? launch_g<128>(G, mk, mv, a, p.ctas, s)
                                  : launch_g<256>(G, mk, mv, a, p.ctas, s);
        }
        if (e != cudaSuccess) return FP8KV_ERR_CUDA;
    }
    if (hs && !direct_out &&
        cudaMemcpyAsync(hs->h_out, out, static_cast<size_t>(batch) * num_q_heads * head_dim * 2,
                        cudaMemcpyDeviceToHost, s) != cudaSuccess)
        return FP8KV_ERR_CUDA;
    return FP8KV_OK;
}

}  // namespace

extern "C" fp8kv_status fp8kv_paged_decode(const void* q, const uint8_t* k_cache, const uint8_t* v_cache,
                                           int64_t num_blocks, const int32_t* block_tables, int max_blocks_per_seq,
                                           const int32_t* seq_lens, int max_seq_len, int batch, int num_q_heads,
                                           int num_kv_heads, int head_dim, int block_size, float k_scale,
                                           float v_scale, float sm_scale, int window, void* out, void* workspace,
                                           size_t workspace_bytes, void* stream) {
    FP8KV_TRACE("fp8kv_paged_decode");
    return decode_impl(q, nullptr, nullptr, k_cache, v_cache, num_blocks, block_tables, max_blocks_per_seq,
                       seq_lens, max_seq_len, batch, num_q_heads, num_kv_heads, head_dim, block_size, k_scale,
                       v_scale, sm_scale, window, out, workspace, workspace_bytes, stream, FP8KV_ENGINE_DEFAULT);
}

extern "C" fp8kv_status fp8kv_paged_decode_engine(const void* q, const uint8_t* k_cache, const uint8_t* v_cache,
                                                  int64_t num_blocks, const int32_t* block_tables,
                                                  int max_blocks_per_seq, const int32_t* seq_lens, int max_seq_len,
                                                  int batch, int num_q_heads, int num_kv_heads, int head_dim,
                                                  int block_size, float k_scale, float v_scale, float sm_scale,
                                                  int window, void* out, void* workspace, size_t workspace_bytes,
                                                  void* stream, int engine) {
    FP8KV_TRACE("fp8kv_paged_decode_engine");
    return decode_impl(q, nullptr, nullptr, k_cache, v_cache, num_blocks, block_tables, max_blocks_per_seq,
                       seq_lens, max_seq_len, batch, num_q_heads, num_kv_heads, head_dim, block_size, k_scale,
                       v_scale, sm_scale, window, out, workspace, workspace_bytes, stream, engine);
}

extern "C" fp8kv_status fp8kv_paged_decode_bf16(const void* q, const void* k_cache, const void* v_cache,
                                                int64_t num_blocks, const int32_t* block_tables,
                                                int max_blocks_per_seq, const int32_t* seq_lens, int max_seq_len,
                                                int batch, int num_q_heads, int num_kv_heads, int head_dim,
                                                int block_size, float sm_scale, int window, void* out,
                                                void* workspace, size_t workspace_bytes, void* stream) {
    FP8KV_TRACE("fp8kv_paged_decode_bf16");
    return decode_impl(q, nullptr, nullptr, static_cast<const uint8_t*>(k_cache), static_cast<const uint8_t*>(v_cache),
                       num_blocks, block_tables, max_blocks_per_seq, seq_lens, max_seq_len, batch, num_q_heads,
                       num_kv_heads, head_dim, block_size, 1.0f, 1.0f, sm_scale, window, out, workspace,
                       workspace_bytes, stream, FP8KV_ENGINE_TENSOR_CORES, 2);
}

extern "C" fp8kv_status fp8kv_paged_decode_per_head(const void* q, const uint8_t* k_cache, const uint8_t* v_cache,
                                                    int64_t num_blocks, const int32_t* block_tables,
                                                    int max_blocks_per_seq, const int32_t* seq_lens,
                                                    int max_seq_len, int batch, int num_q_heads, int num_kv_heads,
                                                    int head_dim, int block_size, const float* k_scales,
                                                    const float* v_scales, float sm_scale, int window, void* out,
                                                    void* workspace, size_t workspace_bytes, void* stream) {
    FP8KV_TRACE("fp8kv_paged_decode_per_head");
    if (batch > 0 && (!k_scales || !v_scales)) return FP8KV_ERR_INVALID_ARG;
    return decode_impl(q, nullptr, nullptr, k_cache, v_cache, num_blocks, block_tables, max_blocks_per_seq,
                       seq_lens, max_seq_len, batch, num_q_heads, num_kv_heads, head_dim, block_size, 1.0f, 1.0f,
                       sm_scale, window, out, workspace, workspace_bytes, stream, FP8KV_ENGINE_DEFAULT, 1, k_scales,
                       v_scales);
}

extern "C" fp8kv_status fp8kv_paged_decode_block(const void* q, const uint8_t* k_cache, const uint8_t* v_cache,
                                                 const float* k_scales, const float* v_scales, int64_t num_blocks,
                                                 const int32_t* block_tables, int max_blocks_per_seq,
                                                 const int32_t* seq_lens, int max_seq_len, int batch, int num_q_heads,
                                                 int num_kv_heads, int head_dim, int block_size, float sm_scale,
                                                 int window, void* out, void* workspace, size_t workspace_bytes,
                                                 void* stream) {
    FP8KV_TRACE("fp8kv_paged_decode_block");
    if (batch > 0 && (!k_scales || !v_scales || (reinterpret_cast<uintptr_t>(k_scales) & 3u) ||
                      (reinterpret_cast<uintptr_t>(v_scales) & 3u)))
        return FP8KV_ERR_INVALID_ARG;
    return decode_impl(q, nullptr, nullptr, k_cache, v_cache, num_blocks, block_tables, max_blocks_per_seq, seq_lens,
                       max_seq_len, batch, num_q_heads, num_kv_heads, head_dim, block_size, 1.0f, 1.0f, sm_scale,
                       window, out, workspace, workspace_bytes, stream, FP8KV_ENGINE_TENSOR_CORES, 1, nullptr, nullptr,
                       false, nullptr, nullptr, k_scales, v_scales);
}

extern "C" size_t fp8kv_paged_decode_weights_workspace_size(int batch, int num_q_heads, int num_kv_heads, int head_dim,
                                                            int max_seq_len, int block_size, int window) {
    if (batch < 0 || num_kv_heads < 1 || num_q_heads < 1 || num_q_heads % num_kv_heads != 0 || max_seq_len < 0)
        return 0;
    if (!supported(head_dim, block_size, num_q_heads / num_kv_heads)) return 0;
    int sms = 0;
    if (device_sms(&sms) != 0) return 0;
    const HeadMap hm = head_map(num_q_heads, num_kv_heads, head_dim, false);
    const ScorePlan sp = score_plan(batch, num_q_heads, max_seq_len, window > 0 ? window : 0);
    const Plan p = make_plan(std::min(batch, sp.batch), hm.units_per_seq, head_dim, max_seq_len, window, sms);
    return ws_layout(batch, num_q_heads, hm.units_per_seq, head_dim, p).total + sp.total;
}

extern "C" fp8kv_status fp8kv_paged_decode_weights(
    const void* q, const void* k_cache, const void* v_cache, int64_t num_blocks, const int32_t* block_tables,
    int max_blocks_per_seq, const int32_t* seq_lens, int max_seq_len, int batch, int num_q_heads, int num_kv_heads,
    int head_dim, int block_size, int cache_format, float k_scale, float v_scale, const float* k_scales,
    const float* v_scales, float sm_scale, int window, void* out, float* weights, float decay, void* workspace,
    size_t workspace_bytes, void* stream) {
    FP8KV_TRACE("fp8kv_paged_decode_weights");
    const bool bf16 = cache_format == FP8KV_CACHE_BF16;
    if (cache_format != FP8KV_CACHE_E4M3 && cache_format != FP8KV_CACHE_E5M2 && !bf16) return FP8KV_ERR_INVALID_ARG;
    if (!std::isfinite(decay) || decay < 0.f) return FP8KV_ERR_INVALID_ARG;
    if (bf16 && (k_scales || v_scales || k_scale != 1.f || v_scale != 1.f)) return FP8KV_ERR_INVALID_ARG;
    if (batch > 0 && (!weights || (reinterpret_cast<uintptr_t>(weights) & 15u))) return FP8KV_ERR_INVALID_ARG;
    const WeightsOut wo{weights, decay};
    return decode_impl(q, nullptr, nullptr, static_cast<const uint8_t*>(k_cache), static_cast<const uint8_t*>(v_cache),
                       num_blocks, block_tables, max_blocks_per_seq, seq_lens, max_seq_len, batch, num_q_heads,
                       num_kv_heads, head_dim, block_size, k_scale, v_scale, sm_scale, window > 0 ? window : 0, out,
                       workspace, workspace_bytes, stream, FP8KV_ENGINE_TENSOR_CORES, bf16 ? 2 : 1, k_scales, v_scales,
                       cache_format == FP8KV_CACHE_E5M2, nullptr, nullptr, nullptr, nullptr, &wo);
}

extern "C" fp8kv_status fp8kv_decode_step_per_head(const void* q, const void* k_new, const void* v_new,
                                                   uint8_t* k_cache, uint8_t* v_cache, int64_t num_blocks,
                                                   const int32_t* block_tables, int max_blocks_per_seq,
                                                   const int32_t* seq_lens, int max_seq_len, int batch,
                                                   int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                                   const float* k_scales, const float* v_scales, float sm_scale,
                                                   int window, void* out, void* workspace, size_t workspace_bytes,
                                                   void* stream) {
    FP8KV_TRACE("fp8kv_decode_step_per_head");
    if (batch > 0 && (!k_new || !v_new || !k_scales || !v_scales)) return FP8KV_ERR_INVALID_ARG;
    return decode_impl(q, k_new, v_new, k_cache, v_cache, num_blocks, block_tables, max_blocks_per_seq, seq_lens,
                       max_seq_len, batch, num_q_heads, num_kv_heads, head_dim, block_size, 1.0f, 1.0f, sm_scale,
                       window, out, workspace, workspace_bytes, stream, FP8KV_ENGINE_DEFAULT, 1, k_scales, v_scales);
}

extern "C" fp8kv_status fp8kv_paged_decode_e5m2(const void* q, const uint8_t* k_cache, const uint8_t* v_cache,
                                                int64_t num_blocks, const int32_t* block_tables,
                                                int max_blocks_per_seq, const int32_t* seq_lens, int max_seq_len,
                                                int batch, int num_q_heads, int num_kv_heads, int head_dim,
                                                int block_size, float k_scale, float v_scale, float sm_scale,
                                                int window, void* out, void* workspace, size_t workspace_bytes,
                                                void* stream) {
    FP8KV_TRACE("fp8kv_paged_decode_e5m2");
    return decode_impl(q, nullptr, nullptr, k_cache, v_cache, num_blocks, block_tables, max_blocks_per_seq,
                       seq_lens, max_seq_len, batch, num_q_heads, num_kv_heads, head_dim, block_size, k_scale,
                       v_scale, sm_scale, window, out, workspace, workspace_bytes, stream, FP8KV_ENGINE_TENSOR_CORES,
                       1, nullptr, nullptr, true);
}

extern "C" fp8kv_status fp8kv_decode_step_e5m2(const void* q, const void* k_new, const void* v_new,
                                               uint8_t* k_cache, uint8_t* v_cache, int64_t num_blocks,
                                               const int32_t* block_tables, int max_blocks_per_seq,
                                               const int32_t* seq_lens, int max_seq_len, int batch,
                                               int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                               float k_scale, float v_scale, float sm_scale, int window, void* out,
                                               void* workspace, size_t workspace_bytes, void* stream) {
    FP8KV_TRACE("fp8kv_decode_step_e5m2");
    if (batch > 0 && (!k_new || !v_new)) return FP8KV_ERR_INVALID_ARG;
    return decode_impl(q, k_new, v_new, k_cache, v_cache, num_blocks, block_tables, max_blocks_per_seq, seq_lens,
                       max_seq_len, batch, num_q_heads, num_kv_heads, head_dim, block_size, k_scale, v_scale,
                       sm_scale, window, out, workspace, workspace_bytes, stream, FP8KV_ENGINE_TENSOR_CORES, 1,
                       nullptr, nullptr, true);
}

extern "C" fp8kv_status fp8kv_decode_step(const void* q, const void* k_new, const void* v_new, uint8_t* k_cache,
                                          uint8_t* v_cache, int64_t num_blocks, const int32_t* block_tables,
                                          int max_blocks_per_seq, const int32_t* seq_lens, int max_seq_len,
                                          int batch, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                          float k_scale, float v_scale, float sm_scale, int window, void* out,
                                          void* workspace, size_t workspace_bytes, void* stream) {
    FP8KV_TRACE("fp8kv_decode_step");
    if (batch > 0 && (!k_new || !v_new)) return FP8KV_ERR_INVALID_ARG;
    return decode_impl(q, k_new, v_new, k_cache, v_cache, num_blocks, block_tables, max_blocks_per_seq, seq_lens,
                       max_seq_len, batch, num_q_heads, num_kv_heads, head_dim, block_size, k_scale, v_scale,
                       sm_scale, window, out, workspace, workspace_bytes, stream, FP8KV_ENGINE_DEFAULT);
}

extern "C" fp8kv_status fp8kv_decode_step_host(const void* h_in, void* d_in, size_t in_bytes, void* h_out,
                                               const void* q, const void* k_new, const void* v_new,
                                               uint8_t* k_cache, uint8_t* v_cache, int64_t num_blocks,
                                               const int32_t* block_tables, int max_blocks_per_seq,
                                               const int32_t* seq_lens, int max_seq_len, int batch,
                                               int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                               float k_scale, float v_scale, float sm_scale, int window, void* out,
                                               void* workspace, size_t workspace_bytes, void* stream) {
    FP8KV_TRACE("fp8kv_decode_step_host");
    if (batch > 0 && (!k_new || !v_new)) return FP8KV_ERR_INVALID_ARG;
    if ((in_bytes > 0 && (!h_in || !d_in)) || (batch > 0 && !h_out)) return FP8KV_ERR_INVALID_ARG;
    if (batch == 0) {  // nothing to attend: only the inputs move
        if (in_bytes > 0 && cudaMemcpyAsync(d_in, h_in, in_bytes, cudaMemcpyHostToDevice,
                                            static_cast<cudaStream_t>(stream)) != cudaSuccess)
            return FP8KV_ERR_CUDA;
        return FP8KV_OK;
    }
    const HostStage hs{h_in, d_in, in_bytes, h_out};
    return decode_impl(q, k_new, v_new, k_cache, v_cache, num_blocks, block_tables, max_blocks_per_seq, seq_lens,
                       max_seq_len, batch, num_q_heads, num_kv_heads, head_dim, block_size, k_scale, v_scale,
                       sm_scale, window, out, workspace, workspace_bytes, stream, FP8KV_ENGINE_DEFAULT, 1, nullptr,
                       nullptr, false, &hs);
}

extern "C" fp8kv_status fp8kv_debug_paged_decode_stall(const void* q, const uint8_t* k_cache,
                                                       const uint8_t* v_cache, int64_t num_blocks,
                                                       const int32_t* block_tables, int max_blocks_per_seq,
                                                       const int32_t* seq_lens, int max_seq_len, int batch,
                                                       int num_q_heads, int num_kv_heads, int head_dim,
                                                       int block_size, float k_scale, float v_scale, float sm_scale,
                                                       int window, void* out, void* workspace,
                                                       size_t workspace_bytes, void* stream, int stall_stage,
                                                       uint64_t wait_limit_ns) {
    FP8KV_TRACE("fp8kv_debug_paged_decode_stall");
    if (stall_stage < 0 || wait_limit_ns == 0 || wait_limit_ns > kWaitLimitNs) return FP8KV_ERR_INVALID_ARG;
    const StallHook dbg{stall_stage, wait_limit_ns};
    return decode_impl(q, nullptr, nullptr, k_cache, v_cache, num_blocks, block_tables, max_blocks_per_seq, seq_lens,
                       max_seq_len, batch, num_q_heads, num_kv_heads, head_dim, block_size, k_scale, v_scale,
                       sm_scale, window, out, workspace, workspace_bytes, stream, FP8KV_ENGINE_CUDA_CORES, 1, nullptr,
                       nullptr, false, nullptr, &dbg);
}

// ---------------------------------------------------------------- allocation-free variant
//
// Some callers cannot allocate device memory at the point where they decode:
// a serving engine that reserved nearly all HBM up front for its own paged-KV
// pool (so a late cudaMalloc fails or fragments that pool), host code running
// under a no-allocation rule (a fixed-budget or real-time loop, a plugin inside
// a framework that owns every device buffer), or a language binding with no
// CUDA allocator at hand.  For them the split-merge scratch lives in a
// fixed-size device array that is part of the library image itself.

namespace fp8kv {

// 8 MiB covers every workload shape exercised here: the largest, 16
// sequences of up to 32K tokens at head_dim 256 with 8 query heads per kv
// head, needs (16 units + 304 CTAs) x 8 heads x 256 dims x 4 B = 2.6 MB of
// partials.  Every device that loads the library holds this array until the
// process exits.
constexpr size_t kStaticScratchBytes = size_t(8) << 20;
static __device__ __align__(256) uint8_t g_static_scratch[kStaticScratchBytes];

// Device address of the array on the current device, looked up once per device
// (host code only sees a host-side stand-in for the symbol).
static void* static_scratch_address() {
    static std::mutex mu;
    static void* addr[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
    std::lock_guard<std::mutex> lock(mu);
    if (addr[dev] == nullptr) {
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, g_static_scratch) != cudaSuccess) return nullptr;
        addr[dev] = p;
    }
    return addr[dev];
}

}  // namespace fp8kv

extern "C" fp8kv_status fp8kv_paged_decode_noalloc(const void* q, const uint8_t* k_cache, const uint8_t* v_cache,
                                                   int64_t num_blocks, const int32_t* block_tables,
                                                   int max_blocks_per_seq, const int32_t* seq_lens, int max_seq_len,
                                                   int batch, int num_q_heads, int num_kv_heads, int head_dim,
                                                   int block_size, float k_scale, float v_scale, float sm_scale,
                                                   int window, void* out, void* stream) {
    FP8KV_TRACE("fp8kv_paged_decode_noalloc");
    if (batch < 0 || num_kv_heads < 1 || num_q_heads < 1 || num_q_heads % num_kv_heads != 0 || max_seq_len < 0)
        return FP8KV_ERR_INVALID_ARG;
    if (!supported(head_dim, block_size, num_q_heads / num_kv_heads)) return FP8KV_ERR_UNSUPPORTED;
    if (batch == 0) return FP8KV_OK;
    int sms = 0;
    if (device_sms(&sms) != 0) return FP8KV_ERR_CUDA;
    const HeadMap hm = head_map(num_q_heads, num_kv_heads, head_dim, false);  // the default engine's
    const Plan p = make_plan(batch, hm.units_per_seq, head_dim, max_seq_len, window, sms);
    const WsLayout w = ws_layout(batch, num_q_heads, hm.units_per_seq, head_dim, p);
    if (w.total > kStaticScratchBytes) return FP8KV_ERR_WORKSPACE;  // problem too large for the fixed array
    void* scratch = static_scratch_address();
    if (scratch == nullptr) return FP8KV_ERR_CUDA;
    // The array keeps the previous call's contents: the error word and the
    // split counters must start at zero.
    if (cudaMemsetAsync(scratch, 0, w.ml, static_cast<cudaStream_t>(stream)) != cudaSuccess) return FP8KV_ERR_CUDA;
    return fp8kv_paged_decode(q, k_cache, v_cache, num_blocks, block_tables, max_blocks_per_seq, seq_lens,
                              max_seq_len, batch, num_q_heads, num_kv_heads, head_dim, block_size, k_scale, v_scale,
                              sm_scale, window, out, scratch, kStaticScratchBytes, stream);
}

extern "C" fp8kv_status fp8kv_workspace_init(void* workspace, size_t workspace_bytes, void* stream) {
    FP8KV_TRACE("fp8kv_workspace_init");
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return FP8KV_ERR_INVALID_ARG;
    return cudaMemsetAsync(workspace, 0, workspace_bytes, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? FP8KV_OK
               : FP8KV_ERR_CUDA;
}

extern "C" fp8kv_status fp8kv_read_error(void* workspace, uint32_t* code, void* stream) {
    FP8KV_TRACE("fp8kv_read_error");
    if (!workspace || !code) return FP8KV_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint32_t zero = 0;
    if (cudaMemcpyAsync(code, workspace, sizeof(uint32_t), cudaMemcpyDeviceToHost, s) != cudaSuccess)
        return FP8KV_ERR_CUDA;
    if (cudaMemcpyAsync(workspace, &zero, sizeof(uint32_t), cudaMemcpyHostToDevice, s) != cudaSuccess)
        return FP8KV_ERR_CUDA;
    return cudaStreamSynchronize(s) == cudaSuccess ? FP8KV_OK : FP8KV_ERR_CUDA;
}

extern "C" const char* fp8kv_status_string(fp8kv_status status) {
    switch (status) {
        case FP8KV_OK: return "FP8KV_OK";
        case FP8KV_ERR_INVALID_ARG: return "FP8KV_ERR_INVALID_ARG";
        case FP8KV_ERR_UNSUPPORTED: return "FP8KV_ERR_UNSUPPORTED";
        case FP8KV_ERR_WORKSPACE: return "FP8KV_ERR_WORKSPACE";
        case FP8KV_ERR_CUDA: return "FP8KV_ERR_CUDA";
        case FP8KV_ERR_TIMEOUT: return "FP8KV_ERR_TIMEOUT";
        default: return "FP8KV_ERR_UNKNOWN";
    }
}
