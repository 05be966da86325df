// Chunked-prefill attention over a block-scaled E4M3 cache: one K and one V
// scale for every (page, kv head), the granularity below the per-tensor and
// per-head scales of gpusmith.com, "FP8 KV Cache Quantization: Capacity Gains
// and Accuracy Risk", "Scales and calibration".  How the scales enter the
// softmax is described at PageScales (prefill_kernels.cuh).
//
// Chunks of several query tiles at d = 64 and 128 run the two-tile kernel of
// the per-tensor call with BS = true.  Everything else -- d = 256, and chunks
// of at most 128 query rows (drafted tokens being checked, short turns) -- runs
// the one-tile kernel below.
#include "prefill_kernels.cuh"

namespace fp8kv {
namespace prefill {

// ---------------------------------------------------------------------------
// The one-tile kernel: 128 query rows of one (sequence, kv head) per CTA and
// one key range, in stages of 128 keys (64 at d = 256).
//
// A short chunk reads the whole cache for a handful of rows, so what bounds it
// is not the tensor cores but how fast a stage's pages become f16 operand
// tiles: shared memory moves them in (fp8), out to the converting threads, in
// again (f16, twice the bytes) and out to the MMAs, 224 KB per 32 KB of cache
// at d = 128, 0.85 us of shared-memory bandwidth a stage.  Hence:
//   * eight converter warps (4-11), in groups of 128 threads that each own a
//     64-key granule (one group of 256 at d = 256): copies two stages ahead
//     (one at d = 256), block ids one stage ahead of their copies, then K into
//     the K tile (once the score MMAs of the stage before have read it) and V,
//     transposed, into one of two V^T tiles;
//   * one thread of warp 12 issues the MMAs, the scores one stage ahead of the
//     values: S has two buffers in tensor memory, so the softmax of a stage runs
//     while the tensor cores compute the next stage's scores.  The MMAs of one
//     thread run in issue order, which is what lets S(s + 1) overwrite the
//     buffer that holds P(s - 1): O += P(s - 1) V was issued before it;
//   * four softmax warps (0-3), thread = row = TMEM lane, P over S in TMEM, O
//     summed by the tensor cores with the lazy rescale of the two-tile kernel.
//     A rescale waits for the value MMAs of the stage before (their commit also
//     frees the V^T tile); it is rare.
//   * REP: a chunk of at most 128 / REP rows fills the tile with REP copies of
//     its rows, copy r taking the r-th part of every stage's keys (its P is zero
//     elsewhere): each thread then runs 1 / REP of the softmax, which is what a
//     row's stage would otherwise take longest for.  The copies' (m, l, O) are
//     combined through shared memory at the end.
// Every mbarrier wait is bounded, and the first role to give up ends the
// others' waits (abort flag), as in the two-tile kernel.
namespace one {
constexpr int kConvWarp0 = 4;              // warps 4-11 convert
constexpr int kConv = 8 * 32;
constexpr int kMmaWarp = 12;
constexpr int kThreads = 13 * 32;
constexpr int kConvBar = 2;                // named barriers of the converter groups: 2, 3
}  // namespace one

template <int D>
struct OneGeo {
    static constexpr int KEYS = D == 256 ? 64 : 128;    // keys per stage
    static constexpr int PAGES = KEYS / kBS;
    static constexpr int GROUPS = KEYS / tcg::kKeys;    // converter groups: 64-key granules per stage
    static constexpr int GT = one::kConv / GROUPS;      // threads of a group
    static constexpr int GPAGES = tcg::kKeys / kBS;     // pages of a granule
    static constexpr int NB = D / 64;
    static constexpr int QTB = NB * 128 * 128;          // Q tile: 128 rows x d
    static constexpr int KAT = KEYS * 128;              // one 128-byte atom column of the K tile
    static constexpr int KTB = NB * KAT;                // K tile: KEYS x d
    static constexpr int VAT = D * 128;                 // one atom column of a V^T tile: d rows x 64 keys
    static constexpr int VTB = GROUPS * VAT;            // a V^T tile: d rows x KEYS
    static constexpr int GSLOT = 2 * tcg::kKeys * D;    // one fp8 staging granule: 64 K rows, then 64 V rows
    static constexpr int STAGES = D == 256 ? 2 : 3;     // stages in the fp8 staging ring
    static constexpr int QT = 0, KT = QTB, VT = KT + KTB, STG = VT + 2 * VTB;
    static constexpr int SMEM = STG + STAGES * GROUPS * GSLOT;   // 224 KB at d = 256 and 128, 112 KB at 64
    // TMEM: two S buffers (P written over the first half of each) at [0, KEYS)
    // and [KEYS, 2 KEYS), the FP32 output accumulator at [256, 256 + d)
    static constexpr uint32_t OC = 256, COLS = 512;
    static_assert(2 * KEYS <= 256 && OC + D <= COLS, "TMEM columns");
};

template <int D, int REP>
__global__ void __launch_bounds__(one::kThreads, 1) paged_prefill_one_kernel(const Args a) {
    using namespace one;
    using Og = OneGeo<D>;
    constexpr int KEYS = Og::KEYS, PAGES = Og::PAGES, GT = Og::GT, GPAGES = Og::GPAGES;
    constexpr int RT = 128 / REP;                  // rows of the chunk in the tile
    constexpr int KP = KEYS / REP;                 // keys of a stage that one thread weighs
    constexpr int HK = KP > 64 ? 64 : KP;          // ... of which at once
    constexpr int NH = KP / HK;
    constexpr int XS = D + 4;                      // floats per row of the copies' exchange (16-byte steps over all banks)
    static_assert(KP % 32 == 0, "whole TMEM loads");
    static_assert((REP - 1) * RT * (XS * 4 + 8) <= Og::STG - Og::KT, "the exchange fits over the operand tiles");
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t k_full, k_empty, v_full[2], v_empty[2], s_full[2], p_full[2], done_bar;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_sh;
    __shared__ float4 psc[4][PAGES];
    __shared__ float row_scale[RT];
    volatile int* abort_flag = &abort_sh;
    uint8_t* sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const uint32_t sb = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        mbar_init(&k_full, kConv);
        mbar_init(&k_empty, 1);            // tcgen05.commit
        for (int j = 0; j < 2; ++j) {
            mbar_init(&v_full[j], kConv);
            mbar_init(&v_empty[j], 1);
            mbar_init(&s_full[j], 1);
            mbar_init(&p_full[j], 128);
        }
        mbar_init(&done_bar, 1);
        abort_sh = 0;
        fence_barrier_init();
    }
    griddep_wait();                // inputs may come from the previous grid on the stream
    griddep_launch_dependents();
    const int b = blockIdx.z, hk = blockIdx.y;
    const int tile = blockIdx.x / a.splits, split = blockIdx.x % a.splits;
    Unit u;
    if (!make_unit<0>(a, b, tile, blockIdx.x == 0 && hk == 0 && tid == 0, u)) return;
    const int lg = a.log2_group;
    const int pg0 = u.kmin / kBS, np_all = u.kmax / kBS - pg0 + 1;
    const int sp0 = pg0 + static_cast<int>(static_cast<int64_t>(split) * np_all / a.splits);
    const int sp1 = pg0 + static_cast<int>(static_cast<int64_t>(split + 1) * np_all / a.splits);
    const int nst = (sp1 - sp0 + PAGES - 1) / PAGES;
    const int32_t* bt = a.block_tables + static_cast<int64_t>(b) * a.max_blocks_per_seq;

    // ---- converter group g's granule of a stage: pages [granule_page(s), ...).
    // Lane p < GPAGES holds the block of page p of the stage to be copied next.
    const int ct = tid - kConvWarp0 * 32, grp = ct / GT, gt = ct % GT;   // (warps 4-11)
    auto granule_page = [&](int s) { return sp0 + s * PAGES + grp * GPAGES; };
    // (The id as the table has it: looking at it here would wait for the read.)
    auto blocks_of = [&](int s) {
        const int pg = granule_page(s) + lane;
        return lane < GPAGES && pg < sp1 ? __ldg(bt + pg) : 0;
    };
    auto load_granule = [&](int s, int ids) {
        const int np = sp1 - granule_page(s);     // pages left (<= 0 past the range)
        if (ids < 0 || ids >= a.num_blocks) {     // block 0 is read instead
            report(a.err, FP8KV_ERR_INVALID_ARG);
            ids = 0;
        }
        const uint32_t dst = sb + Og::STG + ((s % Og::STAGES) * Og::GROUPS + grp) * Og::GSLOT;
        constexpr int CPR = D / 16, CPP = kBS * CPR;   // 16-byte chunks per row, per page
#pragma unroll
        for (int it = 0; it < GPAGES * CPP / GT; ++it) {
            const int i = gt + it * GT, p = i / CPP, ci = i % CPP;   // p is the same for a warp
            const int id = __shfl_sync(0xffffffffu, ids, p);
            if (p < np) {
                const int r = ci / CPR, c = ci % CPR, k = p * kBS + r;
                const int64_t src = (static_cast<int64_t>(id) * a.num_kv_heads + hk) * (kBS * D) + r * D + c * 16;
                cp_async16(dst + stg_k<D>(k, c), a.k_cache + src);
                cp_async16(dst + tcg::kKeys * D + stg_v<D>(k, c), a.v_cache + src);
            }
        }
        cp_async_commit();
    };

    // ---- set-up: the converters start the first stages' copies, then all
    // warps but the last build the Q tile
    const int part = (tid & 127) / RT;            // the row's copy (warps 0-3; the same for a warp)
    const int r = u.R0 + (tid & 127) % RT;
    const bool rv = warp < 4 && (tid & 127) % RT < a.rows && r < u.rows;
    int next_ids = 0;
    if (warp >= kConvWarp0 && warp < kMmaWarp) {
        int ids[Og::STAGES];
#pragma unroll
        for (int s = 0; s < Og::STAGES; ++s) ids[s] = blocks_of(s);
#pragma unroll
        for (int s = 0; s < Og::STAGES - 1; ++s) load_granule(s, ids[s]);
        next_ids = ids[Og::STAGES - 1];
    }
    if (warp < kMmaWarp) {
        // The Q tile, by warps 0-11: CL lanes share a row (a 16-byte chunk of 8
        // values each, so the loads are coalesced and all of a thread's are in
        // flight), find its largest magnitude by shuffles, and write the row as
        // f16 -- once for every copy -- scaled by a power of two so that the
        // copy of the bf16 values is exact.  A negative score scale goes into
        // Q: the row's scale is >= 0.
        constexpr int CL = D / 8, RPW = 32 / CL, NB0 = RT / (RPW * kMmaWarp) + 1;   // lanes per row, rows per warp and batch
        const float sign = a.score_scale < 0.f ? -1.f : 1.f;
        const int c = lane % CL;
        uint4 qv[NB0];
        auto row_of = [&](int i) { return (i * kMmaWarp + warp) * RPW + lane / CL; };   // row of the tile, batch i
#pragma unroll
        for (int i = 0; i < NB0; ++i) {
            const int row = row_of(i), rr = u.R0 + row;
            qv[i] = make_uint4(0, 0, 0, 0);
            if (row < RT && rr < u.rows)
                qv[i] = __ldg(reinterpret_cast<const uint4*>(
                            a.q + (static_cast<int64_t>(u.q0 + (rr >> lg)) * a.num_q_heads + (hk << lg) +
                                   (rr & ((1 << lg) - 1))) * D) + c);
        }
#pragma unroll
        for (int i = 0; i < NB0; ++i) {
            const int row = row_of(i);
            const uint32_t w4[4] = {qv[i].x, qv[i].y, qv[i].z, qv[i].w};
            float qmax = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                qmax = fmaxf(qmax, fmaxf(fabsf(bf16_to_f32(w4[e] & 0xFFFF)), fabsf(bf16_to_f32(w4[e] >> 16))));
#pragma unroll
            for (int off = CL / 2; off; off >>= 1) qmax = fmaxf(qmax, __shfl_xor_sync(0xffffffffu, qmax, off));
            int shift = 0;
            if (qmax > 0.f) {
                const int e = static_cast<int>((__float_as_uint(qmax) >> 23) & 0xFF) - 127;
                shift = max(-100, min(100, 14 - e));
            }
            const float up = sign * __uint_as_float(static_cast<uint32_t>(127 + shift) << 23);
            uint32_t f[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                f[e] = pack_f16x2(bf16_to_f32(w4[e] & 0xFFFF) * up, bf16_to_f32(w4[e] >> 16) * up);
            if (row < RT) {
#pragma unroll
                for (int o = 0; o < REP; ++o) {
                    const int t = o * RT + row;
                    *reinterpret_cast<uint4*>(sm + Og::QT + (c >> 3) * 16384 + t * 128 + (((c & 7) ^ (t & 7)) << 4)) =
                        make_uint4(f[0], f[1], f[2], f[3]);
                }
                if (c == 0)
                    row_scale[row] = fabsf(a.score_scale) * __uint_as_float(static_cast<uint32_t>(127 - shift) << 23);
            }
        }
    }
    if (warp == 0) tc::alloc(&tmem_base, Og::COLS);
    tc::fence_proxy_async_smem();  // the Q tile is read by the tensor cores
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = tmem_base;
    const uint32_t trow = tm + (static_cast<uint32_t>((warp & 3) * 32) << 16);   // this warp's TMEM lanes (warps 0-3)

    float m = -INFINITY, l = 0.f;
    if (warp < 4) {
        // ---------------------------------------------------------- softmax
        const float cs = row_scale[(tid & 127) % RT];
        const int pq = u.L - u.n + (rv ? r >> lg : 0);
        const int lq = (a.window > 0 && pq + 1 > a.window) ? pq + 1 - a.window : 0;
        // the warp's first position and its last valid row's window start: a
        // stage of keys in [wlo1, wpos0] is attended in full by every row of the warp
        const int wr0 = u.R0 + (warp * 32) % RT;
        const int wpos0 = u.L - u.n + (wr0 >> lg);
        const int wpos1 = u.L - u.n + (max(0, min(wr0 + 31, u.rows - 1)) >> lg);
        const int wlo1 = (a.window > 0 && wpos1 + 1 > a.window) ? wpos1 + 1 - a.window : 0;
        {
            float z[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) z[j] = 0.f;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) tc::st32(trow + Og::OC + 32 * c, z);
            tc::wait_st();
        }
        const bool warp_rows = wr0 < u.rows;   // a warp of no rows only keeps the handshake
        PageScales<PAGES> feed(a, bt, hk, sp0, sp1, lane);
        for (int st = 0; st < nst; ++st) {
            const int buf = st & 1;
            bool ok = wait_or_abort(&s_full[buf], (st >> 1) & 1, a.wait_ns, abort_flag);
            if (!__all_sync(0xffffffffu, ok)) break;   // warp-uniform: the TMEM loads below are collective
            if (warp_rows) {
                tc::fence_after_sync();
                const int pgs = sp0 + st * PAGES;
                const int nk = min(PAGES, sp1 - pgs) * kBS;         // the stage's keys
                const int t0 = pgs * kBS;
                const bool interior = nk == KEYS && t0 + KEYS - 1 <= wpos0 && t0 >= wlo1;
                const uint32_t scol = trow + buf * KEYS + part * KP;           // this copy's scores
                const uint32_t pcol = trow + buf * KEYS + part * (KP / 2);     // and its P, two keys a column
                feed.publish(psc[warp], pgs);
                const float4* scale = psc[warp] + part * (KP / kBS);
                auto load = [&](int h, float (&sv)[HK]) {
#pragma unroll
                    for (int c = 0; c < HK / 32; ++c)
                        tc::ld32(scol + HK * h + 32 * c, *reinterpret_cast<float(*)[32]>(sv + 32 * c));
#pragma unroll
                    for (int c = 0; c < HK / 32; ++c) tc::wait_ld(*reinterpret_cast<float(*)[32]>(sv + 32 * c));
                };
                auto key_ok = [&](int jj) {   // jj: key of the stage
                    const int key = t0 + jj;
                    return jj < nk && rv && key >= lq && key <= pq;
                };
                float mx = -INFINITY;
                auto maxima = [&](int h, const float (&sv)[HK]) {
                    // page by page: the largest raw score, scaled (cs and the
                    // K scale are >= 0), plus the V scale's logarithm
#pragma unroll
                    for (int pp = 0; pp < HK / kBS; ++pp) {
                        float mp[2] = {-INFINITY, -INFINITY};
                        if (interior) {
#pragma unroll
                            for (int i = 0; i < kBS; ++i) mp[i & 1] = fmaxf(mp[i & 1], sv[kBS * pp + i]);
                        } else {
#pragma unroll
                            for (int i = 0; i < kBS; ++i)
                                mp[i & 1] = fmaxf(mp[i & 1], key_ok(part * KP + HK * h + kBS * pp + i) ? sv[kBS * pp + i]
                                                                                                      : -INFINITY);
                        }
                        const float big = fmaxf(mp[0], mp[1]);
                        const float4 w = scale[HK / kBS * h + pp];
                        if (big != -INFINITY) mx = fmaxf(mx, fmaf(big, cs * w.x, w.y));
                    }
                };
                float sv[HK];
                if constexpr (NH == 1) {
                    load(0, sv);
                    maxima(0, sv);
                } else {   // the scores are read twice, 64 at a time
#pragma unroll 1
                    for (int h = 0; h < NH; ++h) {
                        load(h, sv);
                        maxima(h, sv);
                    }
                }
                // the reference maximum moves only by more than 8 (log2 units);
                // a row that had none (m = -inf) holds O = 0 and l = 0
                const float mn = fmaxf(m, mx);
                const bool upd = mn > m + ws::kRescaleLog2;
                const bool held = upd && m != -INFINITY;
                float alpha = 1.f;
                if (upd) {
                    alpha = fast_exp2(m - mn);
                    l *= alpha;
                    m = mn;
                }
                if (__any_sync(0xffffffffu, held)) {
                    // O = O * alpha for the warp's rows, once the value MMAs of stage st - 1 are in
                    ok = wait_or_abort(&v_empty[buf ^ 1], ((st - 1) >> 1) & 1, a.wait_ns, abort_flag);
                    if (!__all_sync(0xffffffffu, ok)) break;
                    tc::fence_after_sync();
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        float x[32];
                        tc::ld32(trow + Og::OC + 32 * c, x);
                        tc::wait_ld(x);
#pragma unroll
                        for (int j = 0; j < 32; ++j) x[j] *= alpha;
                        tc::st32(trow + Og::OC + 32 * c, x);
                    }
                }
                const float nmuse = m == -INFINITY ? 0.f : -m;
                auto weights = [&](int h) {
                    float pw[HK / 2];
#pragma unroll
                    for (int pp = 0; pp < HK / kBS; ++pp) {
                        const float4 w = scale[HK / kBS * h + pp];
                        const float c = cs * w.x, n = w.y + nmuse;
                        float ps[2] = {0.f, 0.f};
                        if (interior) {
#pragma unroll
                            for (int i = 0; i < kBS / 2; ++i) {   // key pairs in packed FP32 pairs
                                const int j = kBS / 2 * pp + i;
                                float x0, x1;
                                fma_f32x2(x0, x1, sv[2 * j], sv[2 * j + 1], c, c, n, n);
                                const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
                                add_f32x2(ps[0], ps[1], p0, p1);
                                pw[j] = __uint_as_float(pack_f16x2(p0, p1));
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < kBS / 2; ++i) {   // masked keys weigh 0 (also when cs = 0)
                                const int j = kBS / 2 * pp + i, jj = part * KP + HK * h + 2 * j;
                                const float p0 = key_ok(jj) ? fast_exp2(fmaf(sv[2 * j], c, n)) : 0.f;
                                const float p1 = key_ok(jj + 1) ? fast_exp2(fmaf(sv[2 * j + 1], c, n)) : 0.f;
                                ps[0] += p0;
                                ps[1] += p1;
                                pw[j] = __uint_as_float(pack_f16x2(p0, p1));
                            }
                        }
                        l = fmaf(ps[0] + ps[1], w.z, l);
                    }
                    if constexpr (HK == 64) tc::st32(pcol + 32 * h, *reinterpret_cast<float(*)[32]>(pw));
                    else tc::st16(pcol + 16 * h, *reinterpret_cast<float(*)[16]>(pw));
                };
                if constexpr (NH == 1) {
                    weights(0);
                } else {
#pragma unroll 1
                    for (int h = 0; h < NH; ++h) {
                        // P of half h goes to columns whose S (of half h / 2 and below) has been read
                        load(h, sv);
                        weights(h);
                    }
                }
                if constexpr (REP > 1) {   // the other copies' keys weigh 0 (their scores in this lane are not needed)
                    float z[KP / 2];
#pragma unroll
                    for (int j = 0; j < KP / 2; ++j) z[j] = 0.f;
#pragma unroll
                    for (int o = 1; o < REP; ++o) {
                        const uint32_t col = trow + buf * KEYS + ((part + o) % REP) * (KP / 2);
                        if constexpr (KP == 64) tc::st32(col, *reinterpret_cast<float(*)[32]>(z));
                        else tc::st16(col, *reinterpret_cast<float(*)[16]>(z));
                    }
                }
                tc::wait_st();
                tc::fence_before_sync();
            }
            mbar_arrive(&p_full[buf]);     // P (and the rescaled O) are in TMEM
        }
    } else if (warp < kMmaWarp) {
        // ---------------------------------------------------------- converters
        for (int st = 0; st < nst; ++st) {
            load_granule(st + Og::STAGES - 1, next_ids);   // its slot was read in iteration st - 1
            next_ids = blocks_of(st + Og::STAGES);
            cp_async_wait<Og::STAGES - 1>();               // this thread's copies of stage st have landed
            const uint8_t* stg = sm + Og::STG + ((st % Og::STAGES) * Og::GROUPS + grp) * Og::GSLOT;
            const int pg = granule_page(st);
            // the K tile is free once the score MMAs of stage st - 1 have completed
            bool ok = st == 0 || wait_or_abort(&k_empty, (st - 1) & 1, a.wait_ns, abort_flag);
            if (named_bar_or(kConvBar + grp, GT, !ok)) break;   // the group's copies landed (or all of it gives up)
            if (pg < sp1)                                       // an empty granule's keys are masked
                convert_stage_k<D, Og::KAT, GT>(stg, sm + Og::KT + grp * (tcg::kKeys * 128), gt);
            tc::fence_proxy_async_smem();                       // the tile is read by the tensor cores
            mbar_arrive(&k_full);
            // V^T tile st & 1 is free once the value MMAs of stage st - 2 have completed
            const int j = st & 1;
            ok = st < 2 || wait_or_abort(&v_empty[j], ((st >> 1) + 1) & 1, a.wait_ns, abort_flag);
            if (named_bar_or(kConvBar + grp, GT, !ok)) break;
            convert_stage_v<D, GT>(stg, sm + Og::VT + j * Og::VTB + grp * Og::VAT, gt, pg * kBS, min(GPAGES, sp1 - pg),
                                   u.kmin, u.kmax);             // zeros past the range
            tc::fence_proxy_async_smem();
            mbar_arrive(&v_full[j]);
            named_bar_sync(kConvBar + grp, GT);                 // the granule is read before it is refilled
        }
        cp_async_wait<0>();
    } else if (lane == 0) {
        // ---------------------------------------------------------- MMA issuer
        constexpr uint32_t id_s = tc::idesc_f16_f32(128, KEYS);
        constexpr uint32_t id_o = tc::idesc_f16_f32(128, D);
        const bool stall_cta = blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0;
        // S = Q K^T of stage s into its buffer
        auto issue_s = [&](int s) {
            if (!wait_or_abort(&k_full, s & 1, a.wait_ns, abort_flag)) return false;
            tc::fence_after_sync();
            if (!(s == a.stall_stage && stall_cta)) {   // test hook: this stage's S never arrives
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const uint32_t off = (ks & 3) * 32;
                    tc::mma_f16(tm + (s & 1) * KEYS, tc::desc_k_sw128(sb + Og::QT + (ks >> 2) * 16384 + off),
                                tc::desc_k_sw128(sb + Og::KT + (ks >> 2) * Og::KAT + off), id_s, ks > 0);
                }
                tc::commit(&s_full[s & 1]);
            }
            tc::commit(&k_empty);                // the K tile is free when the score MMAs complete
            return true;
        };
        bool ok = nst == 0 || issue_s(0);
        for (int st = 0; st < nst && ok; ++st) {
            if (st + 1 < nst && !issue_s(st + 1)) break;
            if (!wait_or_abort(&p_full[st & 1], (st >> 1) & 1, a.wait_ns, abort_flag) ||
                !wait_or_abort(&v_full[st & 1], (st >> 1) & 1, a.wait_ns, abort_flag))
                break;
            tc::fence_after_sync();
            // O += P V: P (128 rows x KEYS) from the first half of the stage's S columns
#pragma unroll
            for (int ks = 0; ks < KEYS / 16; ++ks)
                tc::mma_f16_ts(tm + Og::OC, tm + (st & 1) * KEYS + ks * 8,
                               tc::desc_k_sw128(sb + Og::VT + (st & 1) * Og::VTB + (ks >> 2) * Og::VAT + (ks & 3) * 32),
                               id_o, 1);
            tc::commit(&v_empty[st & 1]);        // the V^T tile is free, and O complete, when the value MMAs complete
        }
        // every MMA this thread issued completes before TMEM is released
        tc::commit(&done_bar);
        mbar_wait_bounded(&done_bar, 0, tcg::kWaitNs);
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const bool failed = *abort_flag != 0;
    if constexpr (REP > 1) {
        // copies 1 .. REP - 1 hand their rows over through shared memory (the
        // operand tiles are done with): FP32 outputs, maximum and sum
        float* xo = reinterpret_cast<float*>(sm + Og::KT);
        float2* xml = reinterpret_cast<float2*>(xo + (REP - 1) * RT * XS);
        const int row = (tid & 127) % RT;
        if (!failed && warp < 4 && part > 0) {
            const int at = (part - 1) * RT + row;
            xml[at] = make_float2(m, l);
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                float x[32];
                tc::ld32(trow + Og::OC + 32 * c, x);
                tc::wait_ld(x);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<float4*>(xo + at * XS + 32 * c + 4 * i) =
                        make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
            }
        }
        __syncthreads();
    }
    if (failed) {
        if (tid == 0) report(a.err, FP8KV_ERR_TIMEOUT);
    } else if (warp < 4 && part == 0) {
        // ---- the rows' outputs (or partials) from the TMEM accumulator; every
        // thread of the warp loads (tcgen05.ld is collective), valid rows store
        float f[REP];
        f[0] = 1.f;
        if constexpr (REP > 1) {
            const float2* xml = reinterpret_cast<const float2*>(reinterpret_cast<const float*>(sm + Og::KT) + (REP - 1) * RT * XS);
            float mm = m;
#pragma unroll
            for (int o = 1; o < REP; ++o) mm = fmaxf(mm, xml[(o - 1) * RT + tid].x);
            const float mu = mm == -INFINITY ? 0.f : mm;
            f[0] = fast_exp2(m - mu);
            l *= f[0];
#pragma unroll
            for (int o = 1; o < REP; ++o) {
                const float2 x = xml[(o - 1) * RT + tid];
                f[o] = fast_exp2(x.x - mu);
                l = fmaf(x.y, f[o], l);
            }
            m = mm;
        }
        const int64_t unit = (static_cast<int64_t>(b) * a.num_kv_heads + hk) * a.tiles + tile;
        const float so = l > 0.f ? 1.f / l : 0.f;
        uint4* orow = reinterpret_cast<uint4*>(
            a.out + (static_cast<int64_t>(u.q0 + (rv ? r >> lg : 0)) * a.num_q_heads + (hk << lg) +
                     (rv ? r & ((1 << lg) - 1) : 0)) * D);
        const int64_t slot = (unit * a.splits + split) * a.rows + tid;
        float4* po = reinterpret_cast<float4*>(a.part_o + slot * D);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
            float x[32];
            tc::ld32(trow + Og::OC + 32 * c, x);
            tc::wait_ld(x);
            if constexpr (REP > 1) {
                const float* xo = reinterpret_cast<const float*>(sm + Og::KT);
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] *= f[0];
#pragma unroll
                for (int o = 1; o < REP; ++o)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 y = *reinterpret_cast<const float4*>(xo + ((o - 1) * RT + tid) * XS + 32 * c + 4 * i);
                        x[4 * i] = fmaf(y.x, f[o], x[4 * i]);
                        x[4 * i + 1] = fmaf(y.y, f[o], x[4 * i + 1]);
                        x[4 * i + 2] = fmaf(y.z, f[o], x[4 * i + 2]);
                        x[4 * i + 3] = fmaf(y.w, f[o], x[4 * i + 3]);
                    }
            }
            if (!rv) continue;
            if (a.splits == 1) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    orow[4 * c + i] = make_uint4(pack_bf16x2(x[8 * i] * so, x[8 * i + 1] * so),
                                                 pack_bf16x2(x[8 * i + 2] * so, x[8 * i + 3] * so),
                                                 pack_bf16x2(x[8 * i + 4] * so, x[8 * i + 5] * so),
                                                 pack_bf16x2(x[8 * i + 6] * so, x[8 * i + 7] * so));
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) po[8 * c + i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
            }
        }
        if (rv && a.splits > 1) a.part_ml[slot] = make_float2(m, l);
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 0) {
        tc::fence_after_sync();
        tc::dealloc(tm, Og::COLS);
    }
}

// ---------------------------------------------------------------- launch

// Launches `kernel` with programmatic launch; raises its dynamic
// shared-memory limit on the first use on a device (`done`: a bit per device).
static cudaError_t launch_with(void (*kernel)(const Args), std::atomic<uint64_t>& done, size_t smem, dim3 grid, int threads,
                               const Args& a, cudaStream_t s) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
    if (smem > 0 && (bit == 0 || !(done.load(std::memory_order_acquire) & bit))) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
        done.fetch_or(bit, std::memory_order_release);
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int D, int REP>
static cudaError_t launch_one_rep(const Args& a, dim3 grid, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    return launch_with(paged_prefill_one_kernel<D, REP>, done, OneGeo<D>::SMEM + 1024, grid, one::kThreads, a, s);
}

// A chunk of at most 128 / REP rows runs REP copies of them (max_q_len is the
// host's bound of every sequence's chunk).
template <int D>
static cudaError_t launch_one(const Args& a, dim3 grid, cudaStream_t s) {
    const int64_t rows = static_cast<int64_t>(a.max_q_len) << a.log2_group;
    if constexpr (D < 256) {
        if (rows <= 32) return launch_one_rep<D, 4>(a, grid, s);
    }
    if (rows <= 64) return launch_one_rep<D, 2>(a, grid, s);
    return launch_one_rep<D, 1>(a, grid, s);
}

template <int D, int G>
static cudaError_t launch_block_g(int kind, const Args& a, int batch, cudaStream_t s) {
    const unsigned hkv = static_cast<unsigned>(a.num_kv_heads), bz = static_cast<unsigned>(batch);
    cudaError_t e = cudaErrorInvalidValue;
    if (kind == kKindOne) {
        e = launch_one<D>(a, dim3(static_cast<unsigned>(a.tiles * a.splits), hkv, bz), s);
    } else {
        if constexpr (D < 256) {
            static std::atomic<uint64_t> done{0};
            const int pairs = (a.tiles + ws::kTiles - 1) / ws::kTiles;
            e = launch_with(paged_prefill_ws_kernel<D, G, true>, done, static_cast<size_t>(WsGeo<D>::SMEM) + 1024,
                            dim3(static_cast<unsigned>(pairs * a.splits), hkv, bz), ws::kThreads, a, s);
        }
    }
    if (e != cudaSuccess || a.splits == 1) return e;
    static std::atomic<uint64_t> none{0};
    return launch_with(prefill_merge_kernel<D, G>, none, 0,
                       dim3(static_cast<unsigned>(a.tiles * (a.rows / 8)), hkv, bz), 256, a, s);
}

template <int D>
static cudaError_t launch_block_d(int G, int kind, const Args& a, int batch, cudaStream_t s) {
    switch (G) {
        case 1: return launch_block_g<D, 1>(kind, a, batch, s);
        case 2: return launch_block_g<D, 2>(kind, a, batch, s);
        case 4: return launch_block_g<D, 4>(kind, a, batch, s);
        case 8: return launch_block_g<D, 8>(kind, a, batch, s);
        case 16: return launch_block_g<D, 16>(kind, a, batch, s);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_block(int head_dim, int G, int kind, const Args& a, int batch, cudaStream_t s) {
    return head_dim == 64    ? launch_block_d<64>(G, kind, a, batch, s)
           : head_dim == 128 ? launch_block_d<128>(G, kind, a, batch, s)
                             : launch_block_d<256>(G, kind, a, batch, s);
}

}  // namespace prefill
}  // namespace fp8kv
