// Chunked-prefill attention over a block-scaled E4M3 cache: one K and one V
// scale for every (page, kv head), the granularity below the per-tensor and
// per-head scales of gpusmith.com, "FP8 KV Cache Quantization: Capacity Gains
// and Accuracy Risk", "Scales and calibration".
//
// Two kernels on the 5th-generation tensor cores: chunks of several query tiles
// at d = 64 and 128 run the two-tile kernel, everything else -- d = 256, and
// chunks of at most 128 query rows (drafted tokens being checked, short turns)
// -- the one-tile kernel.
//
// How the scales enter the softmax.  With c_t the codes and ks, vs the scales of
// key t's page, in log2 units:
//     score  s_t = x_t (cs ks),   x_t the raw score q . ck_t,
//     weight w_t = 2^(s_t + log2 vs - m),
//     O = sum_t w_t cv_t,   l = sum_t w_t / vs,   out = O / l.
// The V scale goes into the exponent, where it costs nothing: it is the addend
// of the FMA that applies the score multiplier, one multiplier and one addend
// per page of 16 keys.  m refers to s + log2 vs, so weights stay small however
// the scales differ, and a weight is rounded to f16 relative to the largest in
// the sum it enters.  The row sum takes each page's weights, unrounded, times
// 1 / vs, in FP32.  The exponent is one FMA of the raw score, off by up to
// 2^-23 of m: scores beyond 2^26 in size could leave f16's range.
#include <cuda_fp16.h>

#include "prefill_common.cuh"

namespace fp8kv {
namespace prefill {

// ---------------------------------------------------------------------------
// What the two kernels share.

// A range's page scales, read by one warp: lane p < PAGES holds page p of a
// stage, its scales one stage ahead and its block id two.
template <int PAGES>
struct PageScales {
    const Args& a;
    const int32_t* bt;   // the sequence's block-table row
    int hk, end, lane;   // kv head; first page past the range
    int id;              // block of the page of the stage after next, as the table has it
    float k, v;          // next stage's scales

    // The id as the table has it: looking at it here would wait for the read.
    __device__ __forceinline__ int block_of(int pg) const {
        return lane < PAGES && pg + lane < end ? ld_input(bt + pg + lane) : 0;
    }
    // The scales of the pages at pg, whose ids are held; 1 past the range.  A
    // bad id reads block 0's, as the copies do (they report it).
    __device__ __forceinline__ void fetch(int pg) {
        k = v = 1.f;
        if (lane < PAGES && pg + lane < end) {
            const int64_t b = id >= 0 && id < a.num_blocks ? id : 0;
            k = ld_input(a.k_page_scales + b * a.num_kv_heads + hk);
            v = ld_input(a.v_page_scales + b * a.num_kv_heads + hk);
        }
    }
    // Starts the reads of the stage at page pg and of the block ids after it.
    __device__ __forceinline__ PageScales(const Args& args, const int32_t* row, int head, int pg, int past, int ln)
        : a(args), bt(row), hk(head), end(past), lane(ln) {
        id = block_of(pg);
        fetch(pg);
        id = block_of(pg + PAGES);
    }
    // The stage's entries into the table.
    __device__ __forceinline__ void write(float4* table) const {
        if (lane < PAGES) table[lane] = make_float4(k, log2f(v), 1.f / v, 0.f);
    }
    // The reads move on from the stage at page pg.
    __device__ __forceinline__ void advance(int pg) {
        fetch(pg + PAGES);
        id = block_of(pg + 2 * PAGES);
    }
};


// A unit's query rows [R0, R0 + ROWS) as f16 tiles of 128 rows x d at `qt`,
// by the NW warps wi = 0 .. NW - 1: CL lanes share a row (a 16-byte chunk of 8
// values each, so the loads are coalesced and all of a thread's are in
// flight), find its largest magnitude by shuffles, and write the row -- REP
// times, ROWS apart -- scaled by a power of two so that the copy of the bf16
// values is exact.  row_scale is what takes a raw score back into log2 units.
// A negative score scale goes into Q, so row_scale is positive; at least
// 1e-30, so that a masked score of -inf stays one under a score scale of zero
// (no raw score reaches 2^40: its product with 1e-30 is zero to every sum).
template <int D, int ROWS, int REP, int NW>
__device__ __forceinline__ void build_q_tiles(const Args& a, const Unit& u, int hk, int R0, uint8_t* qt,
                                              float* row_scale, int wi, int lane) {
    constexpr int CL = D / 8, RPW = 32 / CL;                     // lanes per row, rows per warp and batch
    constexpr int NB = (ROWS + RPW * NW - 1) / (RPW * NW);       // batches
    constexpr int QTB = D / 64 * 16384;                          // bytes of a tile
    const int lg = a.log2_group, c = lane % CL;
    const float sign = a.score_scale < 0.f ? -1.f : 1.f;
    uint4 qv[NB];
    auto row_of = [&](int i) { return (i * NW + wi) * RPW + lane / CL; };
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        const int row = row_of(i), rr = R0 + row;
        qv[i] = make_uint4(0, 0, 0, 0);
        if (row < ROWS && rr < u.rows)
            qv[i] = ld_input(reinterpret_cast<const uint4*>(
                        a.q + (static_cast<int64_t>(u.q0 + (rr >> lg)) * a.num_q_heads + (hk << lg) +
                               (rr & ((1 << lg) - 1))) * D) + c);
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
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
        if (row < ROWS) {
#pragma unroll
            for (int o = 0; o < REP; ++o) {
                const int t = o * ROWS + row;
                *reinterpret_cast<uint4*>(qt + (t >> 7) * QTB + (c >> 3) * 16384 + (t & 127) * 128 +
                                          (((c & 7) ^ (t & 7)) << 4)) = make_uint4(f[0], f[1], f[2], f[3]);
            }
            if (c == 0)
                row_scale[row] =
                    fmaxf(fabsf(a.score_scale) * __uint_as_float(static_cast<uint32_t>(127 - shift) << 23), 1e-30f);
        }
    }
}

// The weights of HK keys of one row under the reference maximum m: w = 2^(s cs
// ks + log2 vs - m), as f16 pairs into the TMEM columns from pcol, their sum
// over the V scales added to ls, and the largest sum of a page's in top.
// Masked scores are -inf.  Key pairs go through packed FP32 pairs.
template <int HK>
__device__ __forceinline__ void weigh_keys(const float (&sv)[HK], const float4* scale, float cs, float m, uint32_t pcol,
                                           float& ls, float& top) {
    const float nmuse = m == -INFINITY ? 0.f : -m;
#pragma unroll
    for (int p2 = 0; p2 < HK / 32; ++p2) {   // two pages: 16 columns of P
        float pw[16];
#pragma unroll
        for (int pp = 0; pp < 2; ++pp) {
            const float4 w = scale[2 * p2 + pp];
            const float c = cs * w.x, n = w.y + nmuse;
            float ps[2] = {0.f, 0.f};
#pragma unroll
            for (int i = 0; i < kBS / 2; ++i) {
                const int j = kBS * (2 * p2 + pp) + 2 * i;
                float x0, x1;
                fma_f32x2(x0, x1, sv[j], sv[j + 1], c, c, n, n);
                const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
                add_f32x2(ps[0], ps[1], p0, p1);
                pw[8 * pp + i] = __uint_as_float(pack_f16x2(p0, p1));
            }
            const float sum = ps[0] + ps[1];
            ls = fmaf(sum, w.z, ls);
            top = fmaxf(top, sum);
        }
        tc::st16(pcol + 16 * p2, pw);
    }
}

// Scores of HK keys from position `key0` on that a row may not attend become
// -inf: it attends [lq, pq], of which the stage has keys below `end`.
template <int HK>
__device__ __forceinline__ void mask_keys(float (&sv)[HK], int key0, int lq, int pq, int end) {
    const int lo = lq - key0, hi = min(pq, end - 1) - key0;
#pragma unroll
    for (int j = 0; j < HK; ++j) sv[j] = j >= lo && j <= hi ? sv[j] : -INFINITY;
}

// Hands registers between the warpgroups of a CTA: every warp of a warpgroup
// calls it.  An increase waits until the others have given up enough.
template <int N>
__device__ __forceinline__ void more_regs() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void fewer_regs() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// A page whose weights under a row's reference sum to more than this moves the
// reference.  No weight of a smaller sum is above it, so all are f16.
constexpr float kMaxSum = 256.f;

// ---------------------------------------------------------------------------
// The one-tile kernel: 128 query rows of one (sequence, kv head) per CTA and
// one key range, in stages of 128 keys (64 at d = 256).
//
// A short chunk reads the whole cache for a handful of rows, so what bounds it
// is not the tensor cores but how fast a stage's pages become f16 operand
// tiles: shared memory moves them in (fp8), out to the converting threads, in
// again (f16, twice the bytes) and out to the MMAs, 224 KB per 32 KB of cache
// at d = 128, 0.85 us of shared-memory bandwidth a stage.  Hence:
//   * two copy warps (14 for K, 15 for V) keep a ring of three stages (two at
//     d = 256) filled with cp.async; a slot's barrier counts the copies as they
//     land.  Block ids are read a stage before their copies;
//   * eight converter warps (4-11): K into the K tile (once the score MMAs of the
//     stage before have read it) and V, transposed, into one of two V^T tiles;
//   * one thread of warp 12 issues the MMAs, the scores one stage ahead of the
//     values: S has two buffers in tensor memory, so the softmax of a stage runs
//     while the tensor cores compute the next stage's scores.  (The MMAs of one
//     thread run in issue order: S(s + 1) may overwrite S(s - 1), and the commit
//     of S(s) tells that O += P(s - 2) V is done with its P buffer.);
//   * warp 13 prepares the page scales, a stage ahead;
//   * four softmax warps (0-3), thread = row = TMEM lane; P has two buffers of
//     its own in tensor memory, and O is summed by the tensor cores, rescaled
//     when the reference maximum of a row moves.  A stage is weighed under the
//     reference the row already has, and only a page whose weights sum to more
//     than 2^8 (or a row's first keys) makes the warp look for the maximum,
//     rescale and weigh again: no maximum pass, one read of S.  A rescale waits
//     for the value MMAs of the stage before (their commit also frees the V^T
//     tile).  A load from tensor memory waits for value MMAs in flight, so a
//     stage's scores are read before the P of the stage before is handed over;
//   * REP: a chunk of at most 128 / REP rows fills the tile with REP copies of
//     its rows, copy r taking the r-th part of every stage's keys (its P is zero
//     elsewhere): each thread then runs 1 / REP of the softmax, which is what a
//     row's stage would otherwise take longest for.  The copies' (m, l, O) are
//     combined through shared memory at the end.
// Every mbarrier wait is bounded, and the first role to give up ends the
// others' waits (abort flag), as in the two-tile kernel.
//
// Measured: 8 x 20K, 32 over 8 heads, d = 128, 5 to 14 new tokens: 120 us, 330 MB
// read at 2.75 TB/s (the hand-overs and MMAs alone take 83, of which 27 are the
// three waves' first stages); 4 x 9K, up to 777 new tokens, window 512, 8 over 1 heads,
// d = 256: 42 us, 310 TFLOP/s, two waves of one CTA per SM.  With 2 splits a unit
// and one wave (128 CTAs) the first took 127.  REP by the rows a chunk may have:
// 8 x 20K, 8 tokens (32 rows): 99 us with four copies, 112 with two or one; 8 x 16K,
// d = 64, 4 tokens (32 rows): 70, 82 and 86, 8 tokens (64 rows): 83 with two, 88 with
// one; d = 256, 16 x 9K, 8 tokens (64 rows): 38 and 41.  Two copies at d = 128 win
// where a CTA has few stages and lose where it has many: 8 x 2000, 16 tokens
// (64 rows): 22.6 us and 23.1; 16 x 4000, 60 tokens, 16 over 16 heads, window 512:
// 27.8 and 29.4; 40 x 3000, 16 tokens: 107 and 105; 8 x 20K, 9 tokens: 113.1 and 112.2
// (d = 128 with two copies spills 12 bytes, d = 64 with one or two 8 to 36).
// Against the two-tile kernel, 8 x 20K: 33 tokens (two tiles) 228 us and 186 there.
namespace one {
constexpr int kConvWarp0 = 4;              // warps 4-11 convert
constexpr int kConv = 8 * 32;
constexpr int kMmaWarp = 12;
constexpr int kScaleWarp = 13;
constexpr int kCopyWarp0 = 14;             // warp 14 copies K pages, warp 15 V pages
constexpr int kThreads = 16 * 32;
// Registers a thread: launched with kRegs, then shared out by warpgroup (0-3
// softmax, 4-11 converters, 12-15); the shares add up to the launch's total.
constexpr int kRegs = 128, kSoftRegs = 184, kConvRegs = 112, kAuxRegs = 104;
static_assert(kSoftRegs + 2 * kConvRegs + kAuxRegs <= 4 * kRegs, "register shares");
}  // namespace one

template <int D>
struct OneGeo {
    static constexpr int KEYS = D == 256 ? 64 : 128;    // keys per stage
    static constexpr int PAGES = KEYS / kBS;
    static constexpr int GROUPS = KEYS / tcg::kKeys;    // converter groups: 64-key granules per stage
    static constexpr int GT = one::kConv / GROUPS;      // threads of a group
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
    // TMEM columns: two S buffers from 0, the FP32 output accumulator (d) at OC,
    // two P buffers (two keys a column) from PC
    static constexpr uint32_t OC = 256, COLS = 512;
    static constexpr uint32_t PC = D == 256 ? 2 * KEYS : OC + 128;
    static_assert(2 * KEYS <= OC && OC + D <= COLS, "TMEM columns");
    static_assert(D == 256 ? PC + KEYS <= OC : OC + D <= PC && PC + KEYS <= COLS, "TMEM columns");
};

template <int D, int REP>
__global__ void __launch_bounds__(one::kThreads, 1) paged_prefill_one_kernel(const Args a) {
    using namespace one;
    using Og = OneGeo<D>;
    constexpr int KEYS = Og::KEYS, PAGES = Og::PAGES, GT = Og::GT, STAGES = Og::STAGES;
    constexpr int RT = 128 / REP;                  // rows of the chunk in the tile
    constexpr int KP = KEYS / REP;                 // keys of a stage that one thread weighs
    constexpr int HK = KP > 64 ? 64 : KP;          // ... of which at once
    constexpr int NH = KP / HK;
    constexpr int XS = D + 4;                      // floats per row of the copies' exchange (16-byte steps over all banks)
    static_assert(KP % 32 == 0, "whole TMEM loads");
    static_assert((REP - 1) * RT * (XS * 4 + 8) <= Og::STG - Og::KT, "the exchange fits over the operand tiles");
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t f_full[STAGES], f_empty[STAGES], c_full[2], k_full, k_empty, v_full[2], v_empty[2], s_full[2],
        p_full[2], done_bar;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_sh;
    __shared__ float4 psc[2][PAGES];
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
            mbar_init(&c_full[j], 1);      // the scale warp
        }
        for (int j = 0; j < STAGES; ++j) {
            mbar_init(&f_full[j], 64);     // the copy warps' threads, as their copies land
            mbar_init(&f_empty[j], kConv);
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

    // ---- set-up: the copy warps start the first stages' copies, the softmax
    // and converter warps build the Q tile
    const int part = (tid & 127) / RT;            // the row's copy (warps 0-3; the same for a warp)
    const int r = u.R0 + (tid & 127) % RT;
    const bool rv = warp < 4 && (tid & 127) % RT < a.rows && r < u.rows;
    // Stage s's block ids, lane p holding page p's as the table has it (looking
    // at it here would wait for the read).
    auto blocks_of = [&](int s) {
        const int pg = sp0 + s * PAGES + lane;
        return lane < PAGES && pg < sp1 ? ld_input(bt + pg) : 0;
    };
    // A copy warp's half of stage s (K rows or V rows) into its ring slot; the
    // slot's barrier counts the copies as they land.
    const bool copy_v = warp == kCopyWarp0 + 1;
    auto copy_stage = [&](int s, int ids) {
        const int np = min(PAGES, sp1 - sp0 - s * PAGES);
        if (ids < 0 || ids >= a.num_blocks) {     // block 0 is read instead
            report(a.err, FP8KV_ERR_INVALID_ARG);
            ids = 0;
        }
        const uint8_t* cache = copy_v ? a.v_cache : a.k_cache;
        const uint32_t slot = sb + Og::STG + (s % STAGES) * (Og::GROUPS * Og::GSLOT) + (copy_v ? tcg::kKeys * D : 0);
        constexpr int CPR = D / 16;               // 16-byte chunks per row; a page's rows are contiguous
#pragma unroll
        for (int p = 0; p < PAGES; ++p) {
            const int id = __shfl_sync(0xffffffffu, ids, p);
            if (p < np) {
                const uint8_t* src = cache + (static_cast<int64_t>(id) * a.num_kv_heads + hk) * (kBS * D) + lane * 16;
                const uint32_t dst = slot + (p / 4) * Og::GSLOT;
#pragma unroll
                for (int i = 0; i < kBS * CPR / 32; ++i) {
                    const int ci = lane + 32 * i, k = (p % 4) * kBS + ci / CPR, c = ci % CPR;
                    cp_async16(dst + (copy_v ? stg_v<D>(k, c) : stg_k<D>(k, c)), src + 512 * i);
                }
            }
        }
        cp_async_mbar_arrive(&f_full[s % STAGES]);
    };
    int next_ids = 0;
    if (warp >= kCopyWarp0) {
        int ids[STAGES + 1];
#pragma unroll
        for (int s = 0; s <= STAGES; ++s) ids[s] = blocks_of(s);
#pragma unroll
        for (int s = 0; s < STAGES; ++s)
            if (s < nst) copy_stage(s, ids[s]);
        next_ids = ids[STAGES];
    }
    if (warp < kMmaWarp) build_q_tiles<D, RT, REP, kMmaWarp>(a, u, hk, u.R0, sm + Og::QT, row_scale, warp, lane);
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
        more_regs<kSoftRegs>();
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
            // O starts at zero; so does P, of which each copy then writes its own part only
            float z[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) z[j] = 0.f;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) tc::st32(trow + Og::OC + 32 * c, z);
#pragma unroll
            for (int c = 0; c < KEYS / 32; ++c) tc::st32(trow + Og::PC + 32 * c, z);
            tc::wait_st();
        }
        const bool warp_rows = wr0 < u.rows;   // a warp of no rows only keeps the handshake
        // (the waits' results are made warp-uniform: the TMEM loads are collective)
        auto wait_s = [&](int s) {
            return __all_sync(0xffffffffu, wait_or_abort(&s_full[s & 1], (s >> 1) & 1, a.wait_ns, abort_flag));
        };
        // half h of this copy's scores of stage s (HK keys), masked
        float sv[HK];
        auto load = [&](int s, int h) {
            const uint32_t scol = trow + (s & 1) * KEYS + part * KP + HK * h;
#pragma unroll
            for (int c = 0; c < HK / 32; ++c)
                tc::ld32(scol + 32 * c, *reinterpret_cast<float(*)[32]>(sv + 32 * c));
#pragma unroll
            for (int c = 0; c < HK / 32; ++c) tc::wait_ld(*reinterpret_cast<float(*)[32]>(sv + 32 * c));
            const int t0 = (sp0 + s * PAGES) * kBS;
            if (!(t0 + KEYS <= sp1 * kBS && t0 + KEYS - 1 <= wpos0 && t0 >= wlo1))
                mask_keys<HK>(sv, t0 + part * KP + HK * h, lq, rv ? pq : -1, sp1 * kBS);
        };
        bool ok = true;
        if (NH == 1 && nst > 0) {
            ok = wait_s(0);
            if (ok && warp_rows) {
                tc::fence_after_sync();
                load(0, 0);
            }
        }
        for (int st = 0; st < nst && ok; ++st) {
            const int buf = st & 1;
            if (NH > 1 && !wait_s(st)) break;
            if (!__all_sync(0xffffffffu, wait_or_abort(&c_full[buf], (st >> 1) & 1, a.wait_ns, abort_flag))) break;
            if (warp_rows) {
                if (NH > 1) tc::fence_after_sync();
                const int t0 = (sp0 + st * PAGES) * kBS;
                const uint32_t pcol = trow + Og::PC + buf * (KEYS / 2) + part * (KP / 2);  // this copy's P, two keys a column
                const float4* scale = psc[buf] + part * (KP / kBS);
                float ls, top = 0.f;
                // First under the reference the row has, which mostly still
                // holds: the scores are read once and no maximum is looked for.
                // A row's first keys, or a page whose weights sum to more than
                // 2^8 (no weight of a smaller sum is above it, so all are f16),
                // send the warp the long way.  A look for first keys leaves the
                // other rows of the warp under their references (a window's
                // rows start in different stages), so it is followed by the
                // same question; a look at a pass's sums settles every row.
                const int k0 = t0 + part * KP, k1 = min(sp1 * kBS, k0 + KP) - 1;
                bool look = __any_sync(0xffffffffu, m == -INFINITY && rv && pq >= k0 && lq <= k1 && k0 <= k1);
                bool settled = false;
#pragma unroll 1
                while (true) {
                    if (look) {
                        // page by page (from tensor memory again, in a loop:
                        // this path is rare and should be small): the largest
                        // raw score, scaled (cs and the K scale are > 0),
                        // plus the V scale's logarithm
                        float mx = -INFINITY;
#pragma unroll 1
                        for (int pg = 0; pg < KP / kBS; ++pg) {
                            float x[16], big = -INFINITY;
                            tc::ld16(trow + buf * KEYS + part * KP + kBS * pg, x);
                            tc::wait_ld(x);
                            mask_keys<16>(x, k0 + kBS * pg, lq, rv ? pq : -1, sp1 * kBS);
#pragma unroll
                            for (int i = 0; i < kBS; ++i) big = fmaxf(big, x[i]);
                            const float4 w = scale[pg];
                            mx = fmaxf(mx, fmaf(big, cs * w.x, w.y));
                        }
                        // such a row's reference moves to its maximum; a row that
                        // had none (m = -inf) holds O = 0 and l = 0
                        const float mn = fmaxf(m, mx);
                        const bool upd = mn > m && (m == -INFINITY || top > kMaxSum);
                        const bool held = upd && m != -INFINITY;
                        float alpha = 1.f;
                        if (upd) {
                            alpha = fast_exp2(m - mn);
                            l *= alpha;
                            m = mn;
                        }
                        if (__any_sync(0xffffffffu, held)) {
                            // O = O * alpha for the warp's rows, once the value MMAs of stage st - 1 are in
                            ok = __all_sync(0xffffffffu, wait_or_abort(&v_empty[buf ^ 1], ((st - 1) >> 1) & 1, a.wait_ns,
                                                                       abort_flag));
                            if (!ok) break;
                            tc::fence_after_sync();
#pragma unroll 1
                            for (int c = 0; c < D / 16; ++c) {   // (16 at a time: the scores are in registers)
                                float x[16];
                                tc::ld16(trow + Og::OC + 16 * c, x);
                                tc::wait_ld(x);
#pragma unroll
                                for (int j = 0; j < 16; ++j) x[j] *= alpha;
                                tc::st16(trow + Og::OC + 16 * c, x);
                            }
                        }
                    }
                    ls = top = 0.f;
#pragma unroll 1
                    for (int h = 0; h < NH; ++h) {
                        if constexpr (NH > 1) load(st, h);
                        weigh_keys<HK>(sv, scale + HK / kBS * h, cs, m, pcol + HK / 2 * h, ls, top);
                    }
                    if (settled) break;
                    look = settled = __any_sync(0xffffffffu, top > kMaxSum);
                    if (!look) break;
                }
                if (!ok) break;
                l += ls;
            }
            if (NH == 1 && st + 1 < nst) {
                // the next stage's scores move to registers before P is handed
                // over: a load would wait for the value MMAs, which then run
                ok = wait_s(st + 1);
                if (!ok) break;
                if (warp_rows) {
                    tc::fence_after_sync();
                    load(st + 1, 0);
                }
            }
            if (warp_rows) {
                tc::wait_st();
                tc::fence_before_sync();
            }
            mbar_arrive(&p_full[buf]);     // P (and the rescaled O) are in TMEM
        }
    } else if (warp < kMmaWarp) {
        // ---------------------------------------------------------- converters
        fewer_regs<kConvRegs>();
        const int ct = tid - kConvWarp0 * 32, grp = ct / GT, gt = ct % GT;
        for (int st = 0; st < nst; ++st) {
            const int slot = st % STAGES;
            const uint8_t* stg = sm + Og::STG + (slot * Og::GROUPS + grp) * Og::GSLOT;
            const int pg = sp0 + st * PAGES + grp * (tcg::kKeys / kBS);
            // stage st's pages have landed; the K tile is free once the score
            // MMAs of stage st - 1 have completed
            if (!wait_or_abort(&f_full[slot], (st / STAGES) & 1, a.wait_ns, abort_flag)) break;
            if (st > 0 && !wait_or_abort(&k_empty, (st - 1) & 1, a.wait_ns, abort_flag)) break;
            if (pg < sp1)                                       // an empty granule's keys are masked
                convert_stage_k<D, Og::KAT, GT>(stg, sm + Og::KT + grp * (tcg::kKeys * 128), gt);
            tc::fence_proxy_async_smem();                       // the tile is read by the tensor cores
            mbar_arrive(&k_full);
            // V^T tile st & 1 is free once the value MMAs of stage st - 2 have completed
            const int j = st & 1;
            if (st >= 2 && !wait_or_abort(&v_empty[j], ((st >> 1) + 1) & 1, a.wait_ns, abort_flag)) break;
            convert_stage_v<D, GT>(stg, sm + Og::VT + j * Og::VTB + grp * Og::VAT, gt, pg * kBS,
                                   min(tcg::kKeys / kBS, sp1 - pg), u.kmin, u.kmax);   // zeros past the range
            tc::fence_proxy_async_smem();
            mbar_arrive(&v_full[j]);
            mbar_arrive(&f_empty[slot]);
        }
    } else {
    fewer_regs<kAuxRegs>();
    if (warp >= kCopyWarp0) {
        // ---------------------------------------------------------- copies
        for (int st = STAGES; st < nst; ++st) {
            if (!__all_sync(0xffffffffu, wait_or_abort(&f_empty[st % STAGES], (st / STAGES + 1) & 1, a.wait_ns, abort_flag)))
                break;
            copy_stage(st, next_ids);
            next_ids = blocks_of(st + 1);
        }
        cp_async_wait_all();               // no copy lands after the CTA is gone
    } else if (warp == kScaleWarp) {
        // ---------------------------------------------------------- page scales
        PageScales<PAGES> feed(a, bt, hk, sp0, sp1, lane);
        for (int st = 0; st < nst; ++st) {
            // the table was last read for stage st - 2, before its P was handed over
            if (st >= 2 &&
                !__all_sync(0xffffffffu, wait_or_abort(&p_full[st & 1], ((st >> 1) + 1) & 1, a.wait_ns, abort_flag)))
                break;
            feed.write(psc[st & 1]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&c_full[st & 1]);
            feed.advance(sp0 + st * PAGES);
        }
    } else if (lane == 0) {   // (of warp 12)
        // ---------------------------------------------------------- MMA issuer
        constexpr uint32_t id_s = tc::idesc_f16_f32(128, KEYS);
        constexpr uint32_t id_o = tc::idesc_f16_f32(128, D);
        const bool stall_cta = blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0;
        const uint64_t qd = tc::desc_k_sw128(sb + Og::QT), kd = tc::desc_k_sw128(sb + Og::KT),
                       vd0 = tc::desc_k_sw128(sb + Og::VT);
        // S = Q K^T of stage s into its buffer
        auto issue_s = [&](int s) {
            if (!wait_or_abort(&k_full, s & 1, a.wait_ns, abort_flag)) return false;
            tc::fence_after_sync();
            if (!(s == a.stall_stage && stall_cta)) {   // test hook: this stage's S never arrives
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    tc::mma_f16(tm + (s & 1) * KEYS, tc::desc_at(qd, (ks >> 2) * 16384 + (ks & 3) * 32),
                                tc::desc_at(kd, (ks >> 2) * Og::KAT + (ks & 3) * 32), id_s, ks > 0);
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
            // O += P V: P (128 rows x KEYS) from tensor memory
            const uint32_t pc = tm + Og::PC + (st & 1) * (KEYS / 2);
            const uint64_t vd = tc::desc_at(vd0, (st & 1) * Og::VTB);
#pragma unroll
            for (int ks = 0; ks < KEYS / 16; ++ks)
                tc::mma_f16_ts(tm + Og::OC, pc + ks * 8, tc::desc_at(vd, (ks >> 2) * Og::VAT + (ks & 3) * 32), id_o, 1);
            tc::commit(&v_empty[st & 1]);        // the V^T tile is free, and O complete, when the value MMAs complete
        }
        // every MMA this thread issued completes before TMEM is released
        tc::commit(&done_bar);
        mbar_wait_bounded(&done_bar, 0, tcg::kWaitNs);
    }
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

// ---------------------------------------------------------------------------
// The two-tile kernel (d = 64 and 128, chunks of at least two tiles): 256 query
// rows of one (sequence, kv head) per CTA, so that each stage's operand tiles
// serve two tiles, in stages of 128 keys.
//
// Roles, handing over through mbarriers:
//   * warps 8-11 copy and convert K, warps 12-15 V (transposed): cp.async a
//     stage ahead into a ring of their own (a barrier of the four warps tells
//     that a stage has landed and that the slot to refill has been read), block
//     ids a stage ahead of that, then the conversion into the K tile or into one
//     of two V^T tiles;
//   * one thread of warp 16 issues the MMAs, tile by tile in turn: once P of the
//     first 64 keys of stage s is in, its half of O += P V; once P of the others
//     is, their half, then S = Q K^T of stage s + 1 over the same columns (the
//     MMAs of one thread run in issue order);
//   * warp 17 prepares the page scales, a stage ahead;
//   * warps 0-3 and 4-7 (a warpgroup per tile, thread = row = TMEM lane) weigh
//     the stage in two halves of 64 keys as the one-tile kernel does -- under
//     the reference the row has, one read of S, P over S already read.
// The two tiles ping-pong: while one tile's warps weigh, the tensor cores run
// the other's MMAs.
//
// What bounds it: the round trip of a tile -- its warps weigh a stage (about
// 2600 cycles, of which each of the two reads of S waits for the MMAs in
// flight), then the tensor cores run its MMAs -- next to which they are 48%
// busy.  8 x 20K, chunks of 512 tokens (1.35 TFLOP): 1397 us back to back,
// 968 TFLOP/s (1375 when the clocks were a little higher, which the figures below
// compare with); 8 x 16K, 64 over 8 heads, d = 64, 512 tokens each (1.06 TFLOP):
// 1742 us, 607 TFLOP/s.  The MMAs and hand-overs alone take 980 us of the first,
// all but the softmax 1065.  The same with
//   * one hand-over of P a stage, not two: 1433 us;
//   * stages of 64 keys with two S buffers a tile: 1819 us when this kernel took
//     1464.  At N = 64 the score MMAs read Q from shared memory twice as often
//     for the same work.  (Scores of 128 keys as two MMAs of N = 64, the second
//     half's issued while the first half is weighed: 1700 us);
//   * 32 keys at a time, the next 32 being read meanwhile: 1590 us;
//   * two threads a row, each half of the keys (16 softmax warps, one read of S a
//     stage, at 96 registers): 1412 us when this kernel took 1433; the reads of S
//     take longer the more warps read;
//   * the units of the last, part-empty wave split over their keys and merged:
//     1431 us (8 x 20K with 512 tokens each, 3.4 waves: 1305 for 1357).
namespace two {
constexpr int kTiles = 2;
constexpr int kKWarp0 = 8, kVWarp0 = 12;   // warps 8-11 convert K, 12-15 V
constexpr int kMmaWarp = 16, kScaleWarp = 17;
constexpr int kThreads = 20 * 32;          // (warps 18 and 19 fill the last warpgroup)
// Registers a thread: launched with kRegs, then shared out by warpgroup -- the
// softmax holds 64 scores.  The shares add up to the launch's total, or less,
// so that every increase is granted.
constexpr int kRegs = 96, kSoftRegs = 136, kConvRegs = 72, kAuxRegs = 64;
static_assert(2 * kSoftRegs + 2 * kConvRegs + kAuxRegs <= 5 * kRegs, "register shares");
constexpr int kBar = 2;                    // named barriers of the converter groups: 2 (K), 3 (V)
constexpr int kStg = 2;                    // stages in a staging ring
}  // namespace two

template <int D>
struct TwoGeo {
    static constexpr int KEYS = 128, PAGES = KEYS / kBS, GRAN = KEYS / tcg::kKeys;
    static constexpr int QTB = D / 64 * 128 * 128;      // one Q tile: 128 rows x d
    static constexpr int KAT = KEYS * 128;              // one 128-byte atom column of the K tile
    static constexpr int KTB = D / 64 * KAT;            // the K tile: 128 keys x d
    static constexpr int VAT = D * 128;                 // one atom column of a V^T tile: d rows x 64 keys
    static constexpr int VTB = GRAN * VAT;              // a V^T tile: d rows x 128 keys
    static constexpr int GSLOT = tcg::kKeys * D;        // 64 staged fp8 rows
    static constexpr int SLOT = GRAN * GSLOT;           // one staging slot
    static constexpr int QT = 0, KT = QT + two::kTiles * QTB, VT = KT + KTB, STG = VT + 2 * VTB;
    static constexpr int SMEM = STG + 2 * two::kStg * SLOT;   // 224 KB at d = 128, 112 KB at 64
    // TMEM columns per tile: S (P over its first half), then O
    static constexpr uint32_t OC = KEYS, TC = 256, COLS = two::kTiles * TC;
    static_assert(OC + D <= TC, "TMEM columns");
};

template <int D>
__global__ void __launch_bounds__(two::kThreads, 1) paged_prefill_two_kernel(const Args a) {
    using namespace two;
    using Tg = TwoGeo<D>;
    constexpr int KEYS = Tg::KEYS, PAGES = Tg::PAGES, HK = KEYS / 2;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t k_full, k_empty, v_full[2], v_empty[2], c_full[2], c_empty[2];
    __shared__ uint64_t s_full[kTiles], p_half[kTiles], p_full[kTiles], h_done[kTiles], done_bar;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_sh;
    __shared__ float4 psc[2][PAGES];
    __shared__ float row_scale[kTiles * 128];
    volatile int* abort_flag = &abort_sh;
    uint8_t* sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const uint32_t sb = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        mbar_init(&k_full, 128);
        mbar_init(&k_empty, 1);            // tcgen05.commit
        for (int j = 0; j < 2; ++j) {
            mbar_init(&v_full[j], 128);
            mbar_init(&v_empty[j], 1);
            mbar_init(&c_full[j], 1);      // the scale warp
            mbar_init(&c_empty[j], 8);     // the softmax warps
        }
        for (int i = 0; i < kTiles; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_half[i], 128);
            mbar_init(&p_full[i], 128);
            mbar_init(&h_done[i], 1);
        }
        mbar_init(&done_bar, 1);
        abort_sh = 0;
        fence_barrier_init();
    }
    griddep_wait();                // inputs may come from the previous grid on the stream
    griddep_launch_dependents();
    const int b = blockIdx.z, hk = blockIdx.y;
    const int pair = blockIdx.x / a.splits, split = blockIdx.x % a.splits;
    Unit u, u1;
    if (!make_unit<0>(a, b, 2 * pair, blockIdx.x == 0 && hk == 0 && tid == 0, u)) return;
    const bool has1 = make_unit<0>(a, b, 2 * pair + 1, false, u1);
    const int lg = a.log2_group;
    // the pair's keys: the first tile's window starts first, the second tile's rows end last
    const int kmin = u.kmin, kmax = has1 ? u1.kmax : u.kmax;
    const int pg0 = kmin / kBS, np_all = kmax / kBS - pg0 + 1;
    const int sp0 = pg0 + static_cast<int>(static_cast<int64_t>(split) * np_all / a.splits);
    const int sp1 = pg0 + static_cast<int>(static_cast<int64_t>(split + 1) * np_all / a.splits);
    const int nst = (sp1 - sp0 + PAGES - 1) / PAGES;
    const int32_t* bt = a.block_tables + static_cast<int64_t>(b) * a.max_blocks_per_seq;

    // ---- set-up: the converters start the first stages' copies, then warps
    // 0-15 build the Q tiles
    const bool is_v = warp >= kVWarp0;            // (of warps 8-15)
    const int ct = tid & 127;                     // thread within its group of four warps
    // Stage s's block ids, lane p holding page p's as the table has it (looking
    // at it here would wait for the read).
    auto blocks_of = [&](int s) {
        const int pg = sp0 + s * PAGES + lane;
        return lane < PAGES && pg < sp1 ? ld_input(bt + pg) : 0;
    };
    auto copy_stage = [&](int s, int ids) {       // one commit group per stage, also an empty one
        const int np = sp1 - sp0 - s * PAGES;     // pages left (<= 0 past the range)
        if (ids < 0 || ids >= a.num_blocks) {     // block 0 is read instead
            report(a.err, FP8KV_ERR_INVALID_ARG);
            ids = 0;
        }
        const uint8_t* cache = is_v ? a.v_cache : a.k_cache;
        const uint32_t dst = sb + Tg::STG + ((is_v ? kStg : 0) + s % kStg) * Tg::SLOT;
        constexpr int CPR = D / 16, CPP = kBS * CPR;   // 16-byte chunks per row, per page
#pragma unroll
        for (int it = 0; it < PAGES * CPP / 128; ++it) {
            const int i = ct + it * 128, p = i / CPP, ci = i % CPP;   // p is the same for a warp
            const int id = __shfl_sync(0xffffffffu, ids, p);
            if (p < np) {
                const int k = (p % 4) * kBS + ci / CPR, c = ci % CPR;
                cp_async16(dst + (p / 4) * Tg::GSLOT + (is_v ? stg_v<D>(k, c) : stg_k<D>(k, c)),
                           cache + (static_cast<int64_t>(id) * a.num_kv_heads + hk) * (kBS * D) + ci * 16);
            }
        }
        cp_async_commit();
    };
    int next_ids = 0;
    if (warp >= kKWarp0 && warp < kMmaWarp) {
        const int id0 = blocks_of(0);
        next_ids = blocks_of(1);
        copy_stage(0, id0);
    }
    if (warp < kMmaWarp)
        build_q_tiles<D, kTiles * 128, 1, kMmaWarp>(a, u, hk, u.R0, sm + Tg::QT, row_scale, warp, lane);
    if (warp == 0) tc::alloc(&tmem_base, Tg::COLS);
    tc::fence_proxy_async_smem();  // the Q tiles are read by the tensor cores
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = tmem_base;

    const int ti = warp >> 2;                     // the tile of warps 0-7
    const int r = u.R0 + tid;                     // its row (the tiles' rows are consecutive)
    const bool rv = warp < 8 && r < u.rows;
    const uint32_t trow = tm + (ti & 1) * Tg::TC + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    float m = -INFINITY, l = 0.f;
    if (warp < 8) {
        // ---------------------------------------------------------- softmax of tile ti
        more_regs<kSoftRegs>();
        const float cs = row_scale[tid];
        const int pq = rv ? u.L - u.n + (r >> lg) : -1;
        const int lq = (a.window > 0 && pq + 1 > a.window) ? pq + 1 - a.window : 0;
        // the warp's first position and its last valid row's window start: a
        // stage of keys in [wlo1, wpos0] is attended in full by every row of the warp
        const int wr0 = u.R0 + warp * 32;
        const int wpos0 = u.L - u.n + (wr0 >> lg);
        const int wpos1 = u.L - u.n + (max(0, min(wr0 + 31, u.rows - 1)) >> lg);
        const int wlo1 = (a.window > 0 && wpos1 + 1 > a.window) ? wpos1 + 1 - a.window : 0;
        const bool warp_rows = wr0 < u.rows;      // a warp of no rows only keeps the handshake
        {
            float z[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) z[j] = 0.f;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) tc::st32(trow + Tg::OC + 32 * c, z);
            tc::wait_st();
        }
        float sv[HK];
        auto load = [&](int s, int hf) {          // half hf of the row's scores of stage s, masked
            tc::ld32(trow + HK * hf, *reinterpret_cast<float(*)[32]>(sv));
            tc::ld32(trow + HK * hf + 32, *reinterpret_cast<float(*)[32]>(sv + 32));
            tc::wait_ld(*reinterpret_cast<float(*)[32]>(sv));
            tc::wait_ld(*reinterpret_cast<float(*)[32]>(sv + 32));
            const int t0 = (sp0 + s * PAGES) * kBS;
            if (!(t0 + KEYS <= sp1 * kBS && t0 + KEYS - 1 <= wpos0 && t0 >= wlo1))
                mask_keys<HK>(sv, t0 + HK * hf, lq, pq, sp1 * kBS);
        };
        bool ok = true;
        for (int st = 0; st < nst && ok; ++st) {
            // S of stage st is in; its commit also covers the P V of stage
            // st - 1, so O is complete and P's columns are free.  (The waits'
            // result is made warp-uniform: the TMEM loads are collective.)
            if (!__all_sync(0xffffffffu, wait_or_abort(&s_full[ti], st & 1, a.wait_ns, abort_flag) &&
                                             wait_or_abort(&c_full[st & 1], (st >> 1) & 1, a.wait_ns, abort_flag)))
                break;
            if (warp_rows) {
                tc::fence_after_sync();
                const int t0 = (sp0 + st * PAGES) * kBS;
                float lst = 0.f;
#pragma unroll 1
                for (int hf = 0; hf < 2; ++hf) {
                    load(st, hf);
                    const float4* scale = psc[st & 1] + PAGES / 2 * hf;
                    float ls, top = 0.f;
                    // as in the one-tile kernel: under the reference the row has,
                    // or the long way for its first keys (looked for in the whole
                    // stage, at its first half) and then for a page that outgrows it
                    bool look = hf == 0 && __any_sync(0xffffffffu, m == -INFINITY && pq >= t0 &&
                                                                       lq < min(t0 + KEYS, sp1 * kBS));
                    bool settled = false;
#pragma unroll 1
                    while (true) {
                        if (look) {
                            // (keeps the search inside the branch: it was computed
                            // ahead of it, 250 cycles a half)
#pragma unroll
                            for (int j = 0; j < HK; ++j) asm volatile("" : "+f"(sv[j]));
                            float mx = -INFINITY;
                            auto page_max = [&](const float* x, const float4& w) {
                                float big = -INFINITY;
#pragma unroll
                                for (int i = 0; i < kBS; ++i) big = fmaxf(big, x[i]);
                                mx = fmaxf(mx, fmaf(big, cs * w.x, w.y));
                            };
#pragma unroll
                            for (int pg = 0; pg < PAGES / 2; ++pg) page_max(sv + kBS * pg, scale[pg]);
                            if (hf == 0) {
#pragma unroll 1
                                for (int pg = PAGES / 2; pg < PAGES; ++pg) {
                                    float x[16];
                                    tc::ld16(trow + kBS * pg, x);
                                    tc::wait_ld(x);
                                    mask_keys<16>(x, t0 + kBS * pg, lq, pq, sp1 * kBS);
                                    page_max(x, scale[pg]);
                                }
                            }
                            const float mn = fmaxf(m, mx);
                            const bool upd = mn > m && (m == -INFINITY || top > kMaxSum);
                            const bool held = upd && m != -INFINITY;
                            float alpha = 1.f;
                            if (upd) {
                                alpha = fast_exp2(m - mn);
                                l *= alpha;
                                lst *= alpha;
                                m = mn;
                            }
                            if (__any_sync(0xffffffffu, held)) {
                                // O = O * alpha for the warp's rows (16 columns at a time: the scores are in
                                // registers), once the first half's value MMAs are in
                                if (hf == 1) {
                                    ok = __all_sync(0xffffffffu, wait_or_abort(&h_done[ti], st & 1, a.wait_ns, abort_flag));
                                    if (!ok) break;
                                    tc::fence_after_sync();
                                }
#pragma unroll 1
                                for (int c = 0; c < D / 16; ++c) {
                                    float x[16];
                                    tc::ld16(trow + Tg::OC + 16 * c, x);
                                    tc::wait_ld(x);
#pragma unroll
                                    for (int j = 0; j < 16; ++j) x[j] *= alpha;
                                    tc::st16(trow + Tg::OC + 16 * c, x);
                                }
                            }
                        }
                        ls = top = 0.f;
                        weigh_keys<HK>(sv, scale, cs, m, trow + HK / 2 * hf, ls, top);
                        if (settled) break;
                        look = settled = __any_sync(0xffffffffu, top > kMaxSum);
                        if (!look) break;
                    }
                    lst += ls;
                    if (!ok) break;
                    if (hf == 0) {             // P of the first half may go
                        tc::wait_st();
                        tc::fence_before_sync();
                        mbar_arrive(&p_half[ti]);
                    }
                }
                if (!ok) break;
                l += lst;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&c_empty[st & 1]);
            if (warp_rows) {
                tc::wait_st();
                tc::fence_before_sync();
            } else {
                mbar_arrive(&p_half[ti]);
            }
            mbar_arrive(&p_full[ti]);      // P (and the rescaled O) are in TMEM
        }
    } else if (warp < kMmaWarp) {
        // ---------------------------------------------------------- converters of K or of V
        fewer_regs<kConvRegs>();
        const int bar = kBar + (is_v ? 1 : 0);
        const uint8_t* ring = sm + Tg::STG + (is_v ? kStg * Tg::SLOT : 0);
        bool ok = true;
        for (int st = 0; st < nst; ++st) {
            cp_async_wait<0>();                // this thread's copies of stage st have landed
            // everyone's have; the slot of stage st - 1 has been read (or all give up)
            if (named_bar_or(bar, 128, !ok)) break;
            copy_stage(st + 1, next_ids);
            next_ids = blocks_of(st + 2);
            const int j = st & 1;
            // the K tile is free once the score MMAs of stage st - 1 have completed,
            // V^T tile j once the value MMAs of stage st - 2 have
            if (is_v) ok = st < 2 || wait_or_abort(&v_empty[j], ((st >> 1) + 1) & 1, a.wait_ns, abort_flag);
            else ok = st < 1 || wait_or_abort(&k_empty, (st - 1) & 1, a.wait_ns, abort_flag);
            if (!ok) continue;                 // (to the barrier, where the group leaves together)
            const int pg = sp0 + st * PAGES;
            const uint8_t* slot = ring + st % kStg * Tg::SLOT;
#pragma unroll 1
            for (int g = 0; g < Tg::GRAN; ++g) {
                const int np = sp1 - pg - g * (tcg::kKeys / kBS);    // pages left
                if (is_v)   // (the conversion's V rows follow 64 K rows in its source)
                    convert_stage_v<D>(slot + g * Tg::GSLOT - tcg::kKeys * D, sm + Tg::VT + j * Tg::VTB + g * Tg::VAT, ct,
                                       (pg + g * (tcg::kKeys / kBS)) * kBS, min(tcg::kKeys / kBS, np), kmin, kmax);
                else if (np > 0)   // an empty granule's keys are masked
                    convert_stage_k<D, Tg::KAT>(slot + g * Tg::GSLOT, sm + Tg::KT + g * (tcg::kKeys * 128), ct);
            }
            tc::fence_proxy_async_smem();      // the tile is read by the tensor cores
            mbar_arrive(is_v ? &v_full[j] : &k_full);
        }
        cp_async_wait<0>();                    // no copy lands after the CTA is gone
    } else {
    fewer_regs<kAuxRegs>();
    if (warp == kScaleWarp) {
        // ---------------------------------------------------------- page scales
        PageScales<PAGES> feed(a, bt, hk, sp0, sp1, lane);
        for (int st = 0; st < nst; ++st) {
            if (st >= 2 && !__all_sync(0xffffffffu, wait_or_abort(&c_empty[st & 1], ((st >> 1) + 1) & 1, a.wait_ns,
                                                                  abort_flag)))
                break;
            feed.write(psc[st & 1]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&c_full[st & 1]);
            feed.advance(sp0 + st * PAGES);
        }
    } else if (warp == kMmaWarp && lane == 0) {
        // ---------------------------------------------------------- MMA issuer
        constexpr uint32_t id_s = tc::idesc_f16_f32(128, KEYS);
        constexpr uint32_t id_o = tc::idesc_f16_f32(128, D);
        const bool stall_cta = blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0;
        const uint64_t qd0 = tc::desc_k_sw128(sb + Tg::QT), kd = tc::desc_k_sw128(sb + Tg::KT),
                       vd0 = tc::desc_k_sw128(sb + Tg::VT);
        // S = Q K^T of stage s for tile i
        auto issue_s = [&](int i, int s) {
            if (i == 0) {
                if (!wait_or_abort(&k_full, s & 1, a.wait_ns, abort_flag)) return false;
                tc::fence_after_sync();
            }
            const uint64_t qd = tc::desc_at(qd0, i * Tg::QTB);
            if (!(s == a.stall_stage && stall_cta)) {   // test hook: this stage's S never arrives
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    tc::mma_f16(tm + i * Tg::TC, tc::desc_at(qd, (ks >> 2) * 16384 + (ks & 3) * 32),
                                tc::desc_at(kd, (ks >> 2) * Tg::KAT + (ks & 3) * 32), id_s, ks > 0);
                tc::commit(&s_full[i]);
            }
            if (i == kTiles - 1) tc::commit(&k_empty);   // the K tile is free when the score MMAs complete
            return true;
        };
        bool ok = true;
        for (int i = 0; i < kTiles && ok && nst > 0; ++i) ok = issue_s(i, 0);
        for (int st = 0; st < nst && ok; ++st)
            for (int i = 0; i < kTiles && ok; ++i) {
                const int j = st & 1;
                ok = wait_or_abort(&p_half[i], st & 1, a.wait_ns, abort_flag) &&
                     (i > 0 || wait_or_abort(&v_full[j], (st >> 1) & 1, a.wait_ns, abort_flag));
                if (!ok) break;
                tc::fence_after_sync();
                // O += P V: P (128 rows x 128 keys) from the first half of the S columns
                const uint32_t pc = tm + i * Tg::TC;
                const uint64_t vd = tc::desc_at(vd0, j * Tg::VTB);
#pragma unroll
                for (int ks = 0; ks < KEYS / 32; ++ks)
                    tc::mma_f16_ts(pc + Tg::OC, pc + ks * 8, tc::desc_at(vd, (ks >> 2) * Tg::VAT + (ks & 3) * 32), id_o, 1);
                tc::commit(&h_done[i]);
                ok = wait_or_abort(&p_full[i], st & 1, a.wait_ns, abort_flag);
                if (!ok) break;
                tc::fence_after_sync();
#pragma unroll
                for (int ks = KEYS / 32; ks < KEYS / 16; ++ks)
                    tc::mma_f16_ts(pc + Tg::OC, pc + ks * 8, tc::desc_at(vd, (ks >> 2) * Tg::VAT + (ks & 3) * 32), id_o, 1);
                // the V^T tile is free when both tiles' value MMAs complete
                if (i == kTiles - 1) tc::commit(&v_empty[j]);
                if (st + 1 < nst) ok = issue_s(i, st + 1);
            }
        // every MMA this thread issued completes before TMEM is released
        tc::commit(&done_bar);
        mbar_wait_bounded(&done_bar, 0, tcg::kWaitNs);
    }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const bool failed = *abort_flag != 0;
    if (failed) {
        if (tid == 0) report(a.err, FP8KV_ERR_TIMEOUT);
    } else if (warp < 8) {
        // ---- the rows' outputs (or partials) from the TMEM accumulator; every
        // thread of the warp loads (tcgen05.ld is collective), valid rows store
        const int64_t unit = (static_cast<int64_t>(b) * a.num_kv_heads + hk) * a.tiles + 2 * pair + ti;
        const float so = l > 0.f ? 1.f / l : 0.f;
        uint4* orow = reinterpret_cast<uint4*>(
            a.out + (static_cast<int64_t>(u.q0 + (rv ? r >> lg : 0)) * a.num_q_heads + (hk << lg) +
                     (rv ? r & ((1 << lg) - 1) : 0)) * D);
        const int64_t slot = (unit * a.splits + split) * a.rows + (tid & 127);
        float4* po = reinterpret_cast<float4*>(a.part_o + slot * D);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
            float x[32];
            tc::ld32(trow + Tg::OC + 32 * c, x);
            tc::wait_ld(x);
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
        tc::dealloc(tm, Tg::COLS);
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

// Whether a kernel is launched with the registers that its warpgroups' shares
// add up to: with fewer an increase would never be granted.  Asked until the
// answer is yes.
static bool launched_with(void (*kernel)(const Args), int regs, std::atomic<bool>& known) {
    if (known.load(std::memory_order_relaxed)) return true;
    cudaFuncAttributes at;
    if (cudaFuncGetAttributes(&at, kernel) != cudaSuccess || at.numRegs < regs) return false;
    known.store(true, std::memory_order_relaxed);
    return true;
}

template <int D, int REP>
static cudaError_t launch_one_rep(const Args& a, dim3 grid, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    static std::atomic<bool> known{false};
    if (!launched_with(paged_prefill_one_kernel<D, REP>, one::kRegs, known)) return cudaErrorInvalidConfiguration;
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
            static std::atomic<bool> known{false};
            if (!launched_with(paged_prefill_two_kernel<D>, two::kRegs, known)) return cudaErrorInvalidConfiguration;
            const int pairs = (a.tiles + two::kTiles - 1) / two::kTiles;
            e = launch_with(paged_prefill_two_kernel<D>, done, static_cast<size_t>(TwoGeo<D>::SMEM) + 1024,
                            dim3(static_cast<unsigned>(pairs * a.splits), hkv, bz), two::kThreads, a, s);
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
