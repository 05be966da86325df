// Rotary positions applied to q and k on the way into a paged cache.
//
// Two kernels over the same arithmetic:
//   * rope_append_kernel: every token's q is rotated into q_out, its k is
//     rotated and its k and v are converted (E4M3 or E5M2 codes under a
//     per-tensor or per-head scale, or bf16) and written at the token's slot.
//     With no rotation the codes are those of quant_append_kernel.
//   * rope_append_block_kernel: the newest tokens of each sequence go into an
//     E4M3 cache that keeps one scale for every (page, kv head) of K and of V
//     (the granularity below the per-tensor and per-head scales of
//     gpusmith.com, "FP8 KV Cache Quantization: Capacity Gains and Accuracy
//     Risk", "Scales and calibration").  A page whose new rows do not fit its
//     scale is requantised.
//
// Mathematics.  Frequency i of token t turns by the angle
//     a = positions[axis(i)][t] * inv_freq[i]
// (the real product of the int32 position and the fp32 frequency), and the
// pair (x, y) it owns becomes (x cos a - y sin a, y cos a + x sin a).  In
// fp32 the product of a position of 20,000 and a frequency of 1 is off by
// 1e-3; here the angle is kept in turns as a sum of two fp32 numbers and only
// its fraction is rounded (turn_sincos below).
//
// What bounds them: HBM.  q is read and written (2 bytes per element each
// way), k and v are read and their codes written; there are about 3 flops per
// byte.  Layout of the work: a thread owns an "item" of 16 elements of one
// row, chosen so that both halves of each pair are in it (two 16-byte loads);
// the cosines and sines of a CTA's at most 16 tokens are computed once into
// shared memory, in the order in which a warp's items read them (float4
// columns, free of bank conflicts), and serve all heads.
//
// Measured: rope_append_kernel, 16,000 tokens of 64 + 2 x 8 heads of 64 into bf16
// pages (328 MB): 54.7 us, 6.0 TB/s; rope_append_block_kernel, 8 x 2000 tokens of
// 32 + 2 x 8 heads of 128 (361 MB): 66.9 us, 5.4 TB/s; a decode step of 8 tokens
// 4.1 and 5.4 us, the launch and a chain of loads.  128-thread CTAs took 67 and
// 70 us, five CTAs per SM (48 registers) 80 in the second, three query items in
// flight 63 in the first.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "fp8kv.h"
#include "trace.cuh"
#include "ptx.cuh"

namespace fp8kv {

int device_sms(int* sms);  // SM count of the current device (paged_decode.cu)

namespace rope {

constexpr int kThreads = 256;
constexpr int kTok = 16;          // tokens per CTA: one page, or 16 consecutive tokens
constexpr int kBS = 16;           // tokens per page of the block-scaled cache
constexpr int kMaxAxes = 4;
constexpr size_t kWorkspace = 256;  // the error word
constexpr float kE4m3Max = 448.f;
constexpr int kExpLo = -40, kExpHi = 40;  // exponents a page's scale may take

struct Rope {
    const int32_t* positions;   // [axes][num_tokens], or null: the position in the sequence
    const float* inv_freq;      // [rotary_dim / 2]
    const uint8_t* freq_axis;   // [rotary_dim / 2], or null: axis 0
    int axes;
    int rot;                    // items of a row that turn: rotary_dim / 16
};

struct Rows {
    const uint16_t* q;          // bf16, token t at q + t * q_stride, heads contiguous; null: no queries
    const uint16_t* k;
    const uint16_t* v;
    uint16_t* q_out;            // bf16 [num_tokens][Hq][D]
    int64_t q_stride, k_stride, v_stride;
    int64_t num_tokens;
    int hq, hkv;
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// cos and sin of pos * f.  f / (2 pi) is held as th + te (1 / (2 pi) as two
// fp32 numbers, products with their fma remainders: about 2^-48 relative).
// The position is split into two integers of at most 19 and 12 bits, each
// exact in fp32, so that every product below is a rounded value plus an exact
// remainder, of which only the fractions are kept.  What is rounded is the
// final fraction of a turn in [-1/2, 1/2]: 1.5e-8 turns.  (A NaN or infinite
// f gives NaN.)
__device__ __forceinline__ float2 turn_sincos(int pos, float f) {
    constexpr float kInvHi = 0x1.45f306p-3f, kInvLo = 0x1.b9391p-28f;   // 1 / (2 pi)
    const float th = f * kInvHi;
    const float te = fmaf(f, kInvLo, fmaf(f, kInvHi, -th));
    const float ph = static_cast<float>(pos & ~4095), pl = static_cast<float>(pos & 4095);
    const float a = ph * th, b = pl * th;
    float ae = fmaf(ph, th, -a), be = fmaf(pl, th, -b);
    ae -= rintf(ae);
    const float ar = a - rintf(a), br = b - rintf(b);
    const float r = ar + br;                               // two-sum: r + re == ar + br
    const float bb = r - ar;
    const float re = (ar - (r - bb)) + (br - bb);
    float c = fmaf(ph, te, pl * te);
    c -= rintf(c);
    const float rest = ((ae + be) + re) + c;
    float turn = r - rintf(r) + rest;
    turn -= rintf(turn);
    float s, co;
    sincospif(2.f * turn, &s, &co);
    return make_float2(co, s);
}

// The table of a CTA's `cnt` tokens: entry (token, k, item j) holds cos and
// sin of frequencies 8j + 2k and 8j + 2k + 1, so that the items j of a warp
// read consecutive float4s for each k.
__device__ __forceinline__ void fill_table(float4* tab, const Rope& rp, int64_t t0, int cnt, int p0,
                                           int64_t num_tokens, int tid) {
    const int per = rp.rot * 4;    // float4 entries per token
    for (int i = tid; i < cnt * per; i += kThreads) {
        const int tok = i / per, rem = i - tok * per;
        const int k = rem / rp.rot, j = rem - k * rp.rot;
        const int f0 = 8 * j + 2 * k;
        float2 cs[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            int pos = p0 + tok;
            if (rp.positions) {
                int ax = rp.freq_axis ? rp.freq_axis[f0 + e] : 0;
                ax = ax < rp.axes ? ax : 0;                 // never past the positions array
                pos = ld_input(rp.positions + static_cast<int64_t>(ax) * num_tokens + t0 + tok);
            }
            cs[e] = turn_sincos(pos, ld_input(rp.inv_freq + f0 + e));
        }
        tab[i] = make_float4(cs[0].x, cs[0].y, cs[1].x, cs[1].y);
    }
}

// First elements of the two 8-element halves of item j of a row: a turning
// item holds both elements of each of its 8 pairs.
template <bool PAIRS>
__device__ __forceinline__ void item_place(const Rope& rp, int j, int& e0, int& e1) {
    if (!PAIRS && j < rp.rot) {
        e0 = 8 * j;
        e1 = 8 * (rp.rot + j);
    } else {
        e0 = 16 * j;
        e1 = 16 * j + 8;
    }
}

__device__ __forceinline__ void unpack(const uint4& a, const uint4& b, float (&x)[16]) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
    }
}

// Turns item j (j < rot) of a row of token `tok` of the table.
template <bool PAIRS>
__device__ __forceinline__ void turn(float (&x)[16], const float4* tab, const Rope& rp, int tok, int j) {
    const float4* e = tab + tok * 4 * rp.rot + j;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float4 cs = e[k * rp.rot];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float c = h ? cs.z : cs.x, s = h ? cs.w : cs.y;
            const int i = 2 * k + h;
            // the pair of frequency 8j + i: elements i and 8 + i of the item, or 2i and 2i + 1
            float& a = PAIRS ? x[2 * i] : x[i];
            float& b = PAIRS ? x[2 * i + 1] : x[8 + i];
            const float u = fmaf(a, c, -(b * s)), v = fmaf(b, c, a * s);
            a = u;
            b = v;
        }
    }
}

__device__ __forceinline__ void pack(const float (&x)[16], uint4& a, uint4& b) {
    a = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    b = make_uint4(pack_bf16x2(x[8], x[9]), pack_bf16x2(x[10], x[11]), pack_bf16x2(x[12], x[13]),
                   pack_bf16x2(x[14], x[15]));
}

// Item i of `heads` rows a token -> (token, row, item of the row).  The
// quotient by `heads` through a reciprocal: i / IPR < 2^20 and heads < 2^16,
// so (row + 1/2) / heads stays 2^-17 away from a whole number, and two
// roundings of a number below 16 move it by 2^-19.
template <int IPR>
__device__ __forceinline__ void item_of(int i, int heads, float inv, int& tok, int& r, int& j) {
    const int row = i / IPR;
    tok = static_cast<int>((static_cast<float>(row) + 0.5f) * inv);
    r = row - tok * heads;
    j = i % IPR;
}

// The q rows of heads [h0, h1) of `cnt` tokens from t0: read, turn, round once
// to bf16, write; two items of a thread in flight.  A thread reads its items
// before it writes them and no other thread touches them, so q_out may be q.
// The first two are read before the rotation table is waited for (`ready`).
template <int D, bool PAIRS, typename F>
__device__ __forceinline__ void q_rows(const Rows& rw, const Rope& rp, const float4* tab, int64_t t0, int cnt, int h0,
                                       int h1, int tid, F ready) {
    constexpr int IPR = D / 16;
    const int heads = h1 - h0, n = cnt * heads * IPR;
    const float inv = 1.f / static_cast<float>(heads);
    bool waited = false;
    for (int i0 = tid; i0 < n || !waited; i0 += 2 * kThreads) {
        uint4 a[2], b[2];
        int tok[2], e0[2], e1[2], j[2], h[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int i = i0 + u * kThreads;
            if (i < n) {
                item_of<IPR>(i, heads, inv, tok[u], h[u], j[u]);
                item_place<PAIRS>(rp, j[u], e0[u], e1[u]);
                const uint16_t* src = rw.q + (t0 + tok[u]) * rw.q_stride + static_cast<int64_t>(h0 + h[u]) * D;
                a[u] = *reinterpret_cast<const uint4*>(src + e0[u]);
                b[u] = *reinterpret_cast<const uint4*>(src + e1[u]);
            }
        }
        if (!waited) {
            ready();
            waited = true;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if (i0 + u * kThreads < n) {
                if (j[u] < rp.rot) {
                    float x[16];
                    unpack(a[u], b[u], x);
                    turn<PAIRS>(x, tab, rp, tok[u], j[u]);
                    pack(x, a[u], b[u]);
                }
                uint16_t* dst = rw.q_out + ((t0 + tok[u]) * rw.hq + h0 + h[u]) * D;
                *reinterpret_cast<uint4*>(dst + e0[u]) = a[u];
                *reinterpret_cast<uint4*>(dst + e1[u]) = b[u];
            }
        }
    }
}

// 16 values divided by the scale (one IEEE division each) as FP8 codes.
template <bool E5M2>
__device__ __forceinline__ void codes16(const float (&x)[16], float s, uint32_t (&o)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint16_t lo, hi;
        const float e0 = __fdiv_rn(x[4 * i], s), e1 = __fdiv_rn(x[4 * i + 1], s);
        const float e2 = __fdiv_rn(x[4 * i + 2], s), e3 = __fdiv_rn(x[4 * i + 3], s);
        if constexpr (E5M2) {
            lo = f32x2_to_e5m2x2_satfinite(e0, e1);
            hi = f32x2_to_e5m2x2_satfinite(e2, e3);
        } else {
            lo = f32x2_to_e4m3x2_satfinite(e0, e1);
            hi = f32x2_to_e4m3x2_satfinite(e2, e3);
        }
        o[i] = static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
    }
}

__device__ __forceinline__ void store_codes(uint8_t* row, int e0, int e1, const uint32_t (&o)[4]) {
    if (e1 == e0 + 8) {
        *reinterpret_cast<uint4*>(row + e0) = make_uint4(o[0], o[1], o[2], o[3]);
    } else {
        *reinterpret_cast<uint2*>(row + e0) = make_uint2(o[0], o[1]);
        *reinterpret_cast<uint2*>(row + e1) = make_uint2(o[2], o[3]);
    }
}

// ---------------------------------------------------------------- slots

struct SlotArgs {
    Rows rw;
    Rope rp;
    const int64_t* slots;       // [num_tokens]
    void* k_cache;              // [num_blocks][Hkv][block_size][D], 1 or 2 bytes per element
    void* v_cache;
    int64_t num_slots;
    int block_size;
    float k_scale, v_scale;
    const float* k_scales;      // [Hkv], or null
    const float* v_scales;
};

// FMT: fp8kv_cache_format.  grid: (blocks of kTok tokens, head splits); split
// y takes an equal run of the q heads and an equal run of the kv heads.
template <int D, int FMT, bool PAIRS>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const SlotArgs a) {
    constexpr int IPR = D / 16;   // items per row
    extern __shared__ float4 tab[];
    __shared__ int64_t row_sh[kTok];   // the token's row of cache head 0, -1: not written
    griddep_launch_dependents();
    griddep_wait();               // the inputs and the cache may be the previous grid's
    const Rows& rw = a.rw;
    const int tid = threadIdx.x;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTok;
    const int cnt = static_cast<int>(rw.num_tokens - t0 < kTok ? rw.num_tokens - t0 : kTok);
    auto ready = [&]() {          // the rotation table and the slots
        fill_table(tab, a.rp, t0, cnt, 0, rw.num_tokens, tid);
        if (tid < cnt) {
            const int64_t s = ld_input(a.slots + t0 + tid), blk = s / a.block_size;
            row_sh[tid] = s >= 0 && s < a.num_slots ? blk * rw.hkv * a.block_size + (s - blk * a.block_size) : -1;
        }
        __syncthreads();
    };
    const int64_t y = blockIdx.y, ny = gridDim.y;
    if (rw.q)
        q_rows<D, PAIRS>(rw, a.rp, tab, t0, cnt, static_cast<int>(rw.hq * y / ny), static_cast<int>(rw.hq * (y + 1) / ny),
                         tid, ready);
    else
        ready();
    const int kv0 = static_cast<int>(rw.hkv * y / ny), kv1 = static_cast<int>(rw.hkv * (y + 1) / ny);
    const int heads = kv1 - kv0;
    const float inv = 1.f / static_cast<float>(heads);
    for (int i = tid; i < cnt * heads * IPR; i += kThreads) {
        int tok, h, j;
        item_of<IPR>(i, heads, inv, tok, h, j);
        h += kv0;
        const int64_t row0 = row_sh[tok];
        if (row0 < 0) continue;
        int e0, e1;
        item_place<PAIRS>(a.rp, j, e0, e1);
        const uint16_t* ks = rw.k + (t0 + tok) * rw.k_stride + static_cast<int64_t>(h) * D;
        const uint16_t* vs = rw.v + (t0 + tok) * rw.v_stride + static_cast<int64_t>(h) * D + 16 * j;
        uint4 k0 = __ldcs(reinterpret_cast<const uint4*>(ks + e0));
        uint4 k1 = __ldcs(reinterpret_cast<const uint4*>(ks + e1));
        const uint4 v0 = __ldcs(reinterpret_cast<const uint4*>(vs));
        const uint4 v1 = __ldcs(reinterpret_cast<const uint4*>(vs + 8));
        const int64_t row = (row0 + static_cast<int64_t>(h) * a.block_size) * D;
        float x[16];
        unpack(k0, k1, x);
        if (j < a.rp.rot) turn<PAIRS>(x, tab, a.rp, tok, j);
        if constexpr (FMT == FP8KV_CACHE_BF16) {
            uint16_t* kd = static_cast<uint16_t*>(a.k_cache) + row;
            uint16_t* vd = static_cast<uint16_t*>(a.v_cache) + row + 16 * j;
            if (j < a.rp.rot) pack(x, k0, k1);
            *reinterpret_cast<uint4*>(kd + e0) = k0;
            *reinterpret_cast<uint4*>(kd + e1) = k1;
            *reinterpret_cast<uint4*>(vd) = v0;
            *reinterpret_cast<uint4*>(vd + 8) = v1;
        } else {
            constexpr bool E5M2 = FMT == FP8KV_CACHE_E5M2;
            uint32_t o[4];
            codes16<E5M2>(x, a.k_scales ? ld_input(a.k_scales + h) : a.k_scale, o);
            store_codes(static_cast<uint8_t*>(a.k_cache) + row, e0, e1, o);
            unpack(v0, v1, x);
            codes16<E5M2>(x, a.v_scales ? ld_input(a.v_scales + h) : a.v_scale, o);
            *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.v_cache) + row + 16 * j) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

// ---------------------------------------------------------------- block scales

struct BlockArgs {
    Rows rw;
    Rope rp;
    const int32_t* block_tables;  // [B][max_blocks_per_seq]
    const int32_t* seq_lens;      // [B], the new tokens included
    const int32_t* q_starts;      // [B + 1], or null: one new token per sequence
    uint8_t* k_cache;             // E4M3 [num_blocks][Hkv][16][D]
    uint8_t* v_cache;
    float* k_scales;              // [num_blocks][Hkv]
    float* v_scales;
    uint32_t* err;
    int64_t num_blocks;
    int max_blocks_per_seq;
    int max_seq_len;
    int batch;
};

// The least power of two 2^e, e in [-40, 40], with amax <= 448 * 2^e, from
// amax's bits (448 = 1.75 * 2^8; amax is finite and >= 0).  Why a power of
// two: E4M3 is a floating format, so a finer scale only moves the edge of its
// subnormals, while a power of two makes x / scale exact (a code is rounded
// once in all) and requantising a page whose scale grew exact for every code
// that stays normal.  The range keeps products and quotients of two scales
// and the score multiplier far inside fp32.
__device__ __forceinline__ float least_power(float amax) {
    const uint32_t b = __float_as_uint(amax);
    int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    e = max(kExpLo, min(kExpHi, e));
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// The largest finite magnitude of an item.  (fmaxf passes over NaN; an
// infinity sends the item round again.)
__device__ __forceinline__ float amax16(const float (&x)[16]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(x[i]));
    if (m == INFINITY) {
        m = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(x[i]) < INFINITY ? fabsf(x[i]) : 0.f);
    }
    return m;
}

// codes16 of E4M3 under a page's scale.  Most are powers of two, where the
// product with the reciprocal is the quotient, exactly, and a quarter of the
// instructions.
__device__ __forceinline__ void page_codes16(const float (&x)[16], float s, uint32_t (&o)[4]) {
    const uint32_t b = __float_as_uint(s), e = b >> 23;
    if ((b & 0x7FFFFFu) == 0 && e >= 1 && e <= 253) {
        const float r = __uint_as_float((254u - e) << 23);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] = static_cast<uint32_t>(f32x2_to_e4m3x2_satfinite(x[4 * i] * r, x[4 * i + 1] * r)) |
                   (static_cast<uint32_t>(f32x2_to_e4m3x2_satfinite(x[4 * i + 2] * r, x[4 * i + 3] * r)) << 16);
    } else {
        codes16<false>(x, s, o);
    }
}

// Codes of an older row's 16-element chunk from scale `from` to scale `to`.
__device__ __forceinline__ void requantise(uint8_t* p, float ratio) {
    const uint4 c = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t f01, f23;
        e4m3x4_to_f16x2x2(w[i], f01, f23);
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&f01));
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&f23));
        o[i] = static_cast<uint32_t>(f32x2_to_e4m3x2_satfinite(a.x * ratio, a.y * ratio)) |
               (static_cast<uint32_t>(f32x2_to_e4m3x2_satfinite(b.x * ratio, b.y * ratio)) << 16);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(o[0], o[1], o[2], o[3]);
}

// What one CTA works on: the new rows of one page of one sequence.
struct PageWork {
    int64_t t0;     // first packed token
    int cnt;        // new tokens in the page (0: nothing to do)
    int r0;         // their first row in the page; rows [0, r0) hold older tokens
    int pos;        // sequence position of the first
    int block;      // the page's block, -1: out of range (not written)
};

// CTA x -> (sequence, page) without a scan over the batch: sequence b gets the
// CTA indices from q_starts[b] / 16 + 2b on, and its n new tokens touch at
// most floor(n / 16) + 2 pages, so the runs never meet.  The sequence is found
// by a warp-wide search (32 probes a level); lengths or starts out of bounds
// are reported and the sequence is skipped.
__device__ __forceinline__ PageWork find_page(const BlockArgs& a, int lane) {
    PageWork w;
    w.cnt = 0;
    w.t0 = 0;
    w.r0 = w.pos = 0;
    w.block = -1;
    const int64_t x = blockIdx.x;
    // a sequence of n tokens from packed row q0 and length L that the documented bounds allow
    auto fits = [&](int64_t q0, int64_t n, int L) {
        return n >= 0 && L >= n && L <= a.max_seq_len && q0 >= 0 && q0 + n <= a.rw.num_tokens;
    };
    auto report = [&]() {
        if (lane == 0) atomicCAS(a.err, 0u, static_cast<uint32_t>(FP8KV_ERR_INVALID_ARG));
    };
    int b = static_cast<int>(x);
    int64_t q0 = x, n = 1, j = 0;
    if (a.q_starts) {
        // starts that fall could hide a sequence from the search, so CTA b looks
        // at sequence b whatever it finds (there are at least 2 CTAs a sequence)
        int own0 = 0, own1 = 0, own_len = 0;
        const bool own = x < a.batch;
        if (own) {
            own0 = ld_input(a.q_starts + x);
            own1 = ld_input(a.q_starts + x + 1);
            own_len = ld_input(a.seq_lens + x);
        }
        int lo = 0, cnt = a.batch;
        while (cnt > 1) {
            const int step = (cnt + 31) / 32;
            const int at = lo + lane * step;
            const bool le = lane * step < cnt &&
                            static_cast<int64_t>(ld_input(a.q_starts + at)) / kBS + 2 * static_cast<int64_t>(at) <= x;
            const int k = max(1, __popc(__ballot_sync(0xffffffffu, le)));
            const int skip = (k - 1) * step;
            lo += skip;
            cnt = min(step, cnt - skip);
        }
        b = lo;
        q0 = ld_input(a.q_starts + b);
        n = ld_input(a.q_starts + b + 1) - q0;
        j = x - (q0 / kBS + 2 * static_cast<int64_t>(b));
        if (own && own0 != own1 && !fits(own0, static_cast<int64_t>(own1) - own0, own_len)) report();
    }
    const int L = ld_input(a.seq_lens + b);
    if (!a.q_starts && L == 0) return w;    // an empty slot of a padded batch
    if (n == 0) return w;
    if (!fits(q0, n, L)) {
        report();
        return w;
    }
    const int p0 = static_cast<int>(L - n);
    const int64_t page = p0 / kBS + j;
    if (j < 0 || page > (L - 1) / kBS) return w;
    const int first = static_cast<int>(page) * kBS;
    const int start = max(p0, first);
    w.r0 = start - first;
    w.cnt = min(L - first, kBS) - w.r0;
    w.pos = start;
    w.t0 = q0 + (start - p0);
    w.block = ld_input(a.block_tables + static_cast<int64_t>(b) * a.max_blocks_per_seq + page);
    if (w.block < 0 || w.block >= a.num_blocks) {
        report();
        w.block = -1;
    }
    return w;
}

// grid: (CTA indices of pages, head splits); split y takes an equal run of
// the q heads and an equal run of the kv heads.  For K and V, D threads hold
// one head of the page (16 rows x D / 16 items), so kThreads / D heads go at a
// time: load, turn, largest magnitude over the page (shuffles, then shared
// memory, one barrier), new scale, codes.
template <int D, bool PAIRS>
__global__ void __launch_bounds__(kThreads, 4) rope_append_block_kernel(const BlockArgs a) {
    constexpr int IPR = D / 16;
    constexpr int HPI = kThreads / D;          // heads per iteration
    constexpr int WPH = D / 32;                // warps per head
    extern __shared__ float4 tab[];
    __shared__ PageWork sw;
    __shared__ float2 red[2][kThreads / 32];
    griddep_launch_dependents();
    griddep_wait();               // the inputs and the cache may be the previous grid's
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (warp == 0) {
        const PageWork w = find_page(a, lane);
        if (lane == 0) sw = w;
    }
    __syncthreads();
    const PageWork w = sw;
    if (w.cnt == 0) return;
    const Rows& rw = a.rw;
    const Rope& rp = a.rp;
    auto ready = [&]() {          // the rotation table
        fill_table(tab, rp, w.t0, w.cnt, w.pos, rw.num_tokens, tid);
        __syncthreads();
    };
    const int64_t y = blockIdx.y, ny = gridDim.y;
    if (rw.q)
        q_rows<D, PAIRS>(rw, rp, tab, w.t0, w.cnt, static_cast<int>(rw.hq * y / ny),
                         static_cast<int>(rw.hq * (y + 1) / ny), tid, ready);
    else
        ready();
    if (w.block < 0) return;
    const int kv0 = static_cast<int>(rw.hkv * y / ny), kv1 = static_cast<int>(rw.hkv * (y + 1) / ny);
    const int slot = tid / D, row = (tid % D) / IPR, j = tid % IPR;
    const bool is_new = row >= w.r0 && row < w.r0 + w.cnt;
    const int tok = row - w.r0;
    int e0, e1;
    item_place<PAIRS>(rp, j, e0, e1);
    int it = 0;
    for (int hb = kv0; hb < kv1; hb += HPI, ++it) {
        const int h = hb + slot;
        const bool live = h < kv1;
        const int64_t ph = static_cast<int64_t>(w.block) * rw.hkv + h;
        float x[16];
        uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;      // (V stays packed: half the registers)
        float mk = 0.f, mv = 0.f, old_k = 0.f, old_v = 0.f;
        if (live && w.r0 > 0) {
            old_k = __ldcg(a.k_scales + ph);   // (past L1: the heads beside it are written by other CTAs)
            old_v = __ldcg(a.v_scales + ph);
        }
        if (live && is_new) {
            const uint16_t* ks = rw.k + (w.t0 + tok) * rw.k_stride + static_cast<int64_t>(h) * D;
            const uint16_t* vs = rw.v + (w.t0 + tok) * rw.v_stride + static_cast<int64_t>(h) * D + 16 * j;
            const uint4 k0 = __ldcs(reinterpret_cast<const uint4*>(ks + e0));
            const uint4 k1 = __ldcs(reinterpret_cast<const uint4*>(ks + e1));
            v0 = __ldcs(reinterpret_cast<const uint4*>(vs));
            v1 = __ldcs(reinterpret_cast<const uint4*>(vs + 8));
            unpack(v0, v1, x);
            mv = amax16(x);
            unpack(k0, k1, x);
            if (j < rp.rot) turn<PAIRS>(x, tab, rp, tok, j);
            mk = amax16(x);
        }
#pragma unroll
        for (int off = 16; off; off >>= 1) {
            mk = fmaxf(mk, __shfl_xor_sync(0xffffffffu, mk, off));
            mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, off));
        }
        // alternating buffers: one barrier an iteration
        if (lane == 0) red[it & 1][warp] = make_float2(mk, mv);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < WPH; ++i) {
            const float2 m = red[it & 1][slot * WPH + i];
            mk = fmaxf(mk, m.x);
            mv = fmaxf(mv, m.y);
        }
        if (!live) continue;
        // a page with older rows keeps its scale while the new rows fit it
        const bool keep_k = w.r0 > 0 && mk <= kE4m3Max * old_k, keep_v = w.r0 > 0 && mv <= kE4m3Max * old_v;
        const float sk = keep_k ? old_k : fmaxf(old_k, least_power(mk));
        const float sv = keep_v ? old_v : fmaxf(old_v, least_power(mv));
        uint8_t* kp = a.k_cache + (ph * kBS + row) * D;
        uint8_t* vp = a.v_cache + (ph * kBS + row) * D;
        if (is_new) {
            uint32_t o[4];
            page_codes16(x, sk, o);
            store_codes(kp, e0, e1, o);
            unpack(v0, v1, x);
            page_codes16(x, sv, o);
            *reinterpret_cast<uint4*>(vp + 16 * j) = make_uint4(o[0], o[1], o[2], o[3]);
        } else if (row < w.r0) {
            if (!keep_k) requantise(kp + 16 * j, old_k / sk);
            if (!keep_v) requantise(vp + 16 * j, old_v / sv);
        }
        if (tid % D == 0) {
            if (!keep_k) a.k_scales[ph] = sk;
            if (!keep_v) a.v_scales[ph] = sv;
        }
    }
}

// ---------------------------------------------------------------- host side

bool a16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool a4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool good_scale(float s) { return std::isfinite(s) && s > 0.f; }

// The checks the two calls share; on success the rows and the rotation.
fp8kv_status make_rows(const void* q, int64_t q_stride, void* q_out, const void* k_new, int64_t k_stride,
                       const void* v_new, int64_t v_stride, int64_t num_tokens, int num_q_heads, int num_kv_heads,
                       int head_dim, Rows* rw) {
    if (!k_new || !v_new || !a16(k_new) || !a16(v_new)) return FP8KV_ERR_INVALID_ARG;
    if ((q == nullptr) != (q_out == nullptr) || (q && (!a16(q) || !a16(q_out)))) return FP8KV_ERR_INVALID_ARG;
    const int64_t kv_row = static_cast<int64_t>(num_kv_heads) * head_dim;
    const int64_t q_row = static_cast<int64_t>(num_q_heads) * head_dim;
    auto bad = [&](int64_t stride, int64_t row) {
        return stride % 8 != 0 || stride < row || stride > (INT64_C(1) << 60) / num_tokens;
    };
    if (bad(k_stride, kv_row) || bad(v_stride, kv_row)) return FP8KV_ERR_INVALID_ARG;
    if (q && (bad(q_stride, q_row) || (q == q_out && q_stride != q_row))) return FP8KV_ERR_INVALID_ARG;
    rw->q = static_cast<const uint16_t*>(q);
    rw->k = static_cast<const uint16_t*>(k_new);
    rw->v = static_cast<const uint16_t*>(v_new);
    rw->q_out = static_cast<uint16_t*>(q_out);
    rw->q_stride = q_stride;
    rw->k_stride = k_stride;
    rw->v_stride = v_stride;
    rw->num_tokens = num_tokens;
    rw->hq = num_q_heads;
    rw->hkv = num_kv_heads;
    return FP8KV_OK;
}

fp8kv_status make_rope(const int32_t* positions, int num_axes, const float* inv_freq, const uint8_t* freq_axis,
                       int rotary_dim, bool need_positions, Rope* rp) {
    rp->positions = positions;
    rp->inv_freq = inv_freq;
    rp->freq_axis = freq_axis;
    rp->axes = num_axes;
    rp->rot = rotary_dim / 16;
    if (rotary_dim == 0) return FP8KV_OK;
    if (!inv_freq || !a4(inv_freq) || (positions && !a4(positions))) return FP8KV_ERR_INVALID_ARG;
    if (!positions && (need_positions || num_axes != 1)) return FP8KV_ERR_INVALID_ARG;
    return FP8KV_OK;
}

fp8kv_status check_shape(int num_q_heads, int num_kv_heads, int head_dim, int rotary_dim, int rope_style,
                         int num_axes, int64_t num_tokens, int64_t num_blocks) {
    if (num_tokens < 0 || num_blocks < 1 || num_q_heads < 0 || num_q_heads > 65535 || num_kv_heads < 1 ||
        num_kv_heads > 65535)
        return FP8KV_ERR_INVALID_ARG;
    if (rope_style != FP8KV_ROPE_HALVES && rope_style != FP8KV_ROPE_PAIRS) return FP8KV_ERR_INVALID_ARG;
    if (num_axes < 1 || num_axes > kMaxAxes || rotary_dim < 0) return FP8KV_ERR_INVALID_ARG;
    if (!(head_dim == 64 || head_dim == 128 || head_dim == 256)) return FP8KV_ERR_UNSUPPORTED;
    if (rotary_dim > head_dim) return FP8KV_ERR_INVALID_ARG;
    if (rotary_dim % 16 != 0 || num_tokens >= (INT64_C(1) << 31)) return FP8KV_ERR_UNSUPPORTED;
    return FP8KV_OK;
}

// CTAs that share the heads of one block of tokens: enough for `want` CTAs in
// all, at most one for every 4 heads of a token (the rotation table is
// computed once per CTA).
int head_splits(int64_t blocks, int heads, int sms) {
    const int64_t want = static_cast<int64_t>(sms) * 4;
    int64_t y = (want + blocks - 1) / blocks;
    const int64_t most = (heads + 3) / 4;
    y = y < most ? y : most;
    return static_cast<int>(y < 1 ? 1 : y);
}

template <typename A>
cudaError_t launch(void (*kernel)(const A), const A& a, int64_t blocks, int splits, int rot, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(splits));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(kTok) * rot * 4 * sizeof(float4);   // at most 16 KB
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int FMT, bool PAIRS>
void (*slot_kernel_d(int d))(const SlotArgs) {
    return d == 64    ? rope_append_kernel<64, FMT, PAIRS>
           : d == 128 ? rope_append_kernel<128, FMT, PAIRS>
                      : rope_append_kernel<256, FMT, PAIRS>;
}

template <int FMT>
void (*slot_kernel(int d, bool pairs))(const SlotArgs) {
    return pairs ? slot_kernel_d<FMT, true>(d) : slot_kernel_d<FMT, false>(d);
}

template <bool PAIRS>
void (*block_kernel(int d))(const BlockArgs) {
    return d == 64    ? rope_append_block_kernel<64, PAIRS>
           : d == 128 ? rope_append_block_kernel<128, PAIRS>
                      : rope_append_block_kernel<256, PAIRS>;
}

}  // namespace rope
}  // namespace fp8kv

extern "C" fp8kv_status fp8kv_rope_append(const void* q, int64_t q_stride, void* q_out, const void* k_new,
                                          int64_t k_stride, const void* v_new, int64_t v_stride,
                                          const int32_t* positions, int num_axes, const float* inv_freq,
                                          const uint8_t* freq_axis, int rotary_dim, int rope_style,
                                          const int64_t* slot_mapping, int64_t num_tokens, void* k_cache, void* v_cache,
                                          int64_t num_blocks, int block_size, int num_q_heads, int num_kv_heads,
                                          int head_dim, int cache_format, float k_scale, float v_scale,
                                          const float* k_scales, const float* v_scales, void* stream) {
    FP8KV_TRACE("fp8kv_rope_append");
    using namespace fp8kv::rope;
    const fp8kv_status sh = check_shape(num_q_heads, num_kv_heads, head_dim, rotary_dim, rope_style, num_axes,
                                        num_tokens, num_blocks);
    if (sh != FP8KV_OK) return sh;
    if (block_size < 1) return FP8KV_ERR_INVALID_ARG;
    if (cache_format != FP8KV_CACHE_E4M3 && cache_format != FP8KV_CACHE_E5M2 && cache_format != FP8KV_CACHE_BF16)
        return FP8KV_ERR_INVALID_ARG;
    if (!good_scale(k_scale) || !good_scale(v_scale)) return FP8KV_ERR_INVALID_ARG;
    if ((k_scales == nullptr) != (v_scales == nullptr) || !a4(k_scales) || !a4(v_scales)) return FP8KV_ERR_INVALID_ARG;
    if (cache_format == FP8KV_CACHE_BF16 && (k_scales || k_scale != 1.f || v_scale != 1.f))
        return FP8KV_ERR_INVALID_ARG;   // a bf16 cache has no scales
    if (num_blocks > (INT64_C(1) << 60) / (static_cast<int64_t>(block_size) * num_kv_heads * head_dim))
        return FP8KV_ERR_INVALID_ARG;
    if (num_tokens == 0) return FP8KV_OK;
    if (!k_cache || !v_cache || !a16(k_cache) || !a16(v_cache) || !slot_mapping ||
        (reinterpret_cast<uintptr_t>(slot_mapping) & 7u) || (q && num_q_heads < 1))
        return FP8KV_ERR_INVALID_ARG;
    SlotArgs a;
    fp8kv_status st = make_rows(q, q_stride, q_out, k_new, k_stride, v_new, v_stride, num_tokens, num_q_heads,
                                num_kv_heads, head_dim, &a.rw);
    if (st != FP8KV_OK) return st;
    st = make_rope(positions, num_axes, inv_freq, freq_axis, rotary_dim, true, &a.rp);
    if (st != FP8KV_OK) return st;
    a.slots = slot_mapping;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.num_slots = num_blocks * block_size;
    a.block_size = block_size;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    int sms = 0;
    if (fp8kv::device_sms(&sms) != 0) return FP8KV_ERR_CUDA;
    const int64_t blocks = (num_tokens + kTok - 1) / kTok;
    const int splits = head_splits(blocks, (q ? num_q_heads : 0) + 2 * num_kv_heads, sms);
    const bool pairs = rope_style == FP8KV_ROPE_PAIRS;
    auto kernel = cache_format == FP8KV_CACHE_E4M3   ? slot_kernel<FP8KV_CACHE_E4M3>(head_dim, pairs)
                  : cache_format == FP8KV_CACHE_E5M2 ? slot_kernel<FP8KV_CACHE_E5M2>(head_dim, pairs)
                                                     : slot_kernel<FP8KV_CACHE_BF16>(head_dim, pairs);
    return launch(kernel, a, blocks, splits, a.rp.rot, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? FP8KV_OK
               : FP8KV_ERR_CUDA;
}

extern "C" fp8kv_status fp8kv_rope_append_block(const void* q, int64_t q_stride, void* q_out, const void* k_new,
                                                int64_t k_stride, const void* v_new, int64_t v_stride,
                                                int64_t num_tokens, const int32_t* positions, int num_axes,
                                                const float* inv_freq, const uint8_t* freq_axis, int rotary_dim,
                                                int rope_style, uint8_t* k_cache, uint8_t* v_cache, float* k_scales,
                                                float* v_scales, int64_t num_blocks, const int32_t* block_tables,
                                                int max_blocks_per_seq, const int32_t* seq_lens,
                                                const int32_t* q_starts, int max_seq_len, int batch, int num_q_heads,
                                                int num_kv_heads, int head_dim, int block_size, void* workspace,
                                                size_t workspace_bytes, void* stream) {
    FP8KV_TRACE("fp8kv_rope_append_block");
    using namespace fp8kv::rope;
    const fp8kv_status sh = check_shape(num_q_heads, num_kv_heads, head_dim, rotary_dim, rope_style, num_axes,
                                        num_tokens, num_blocks);
    if (sh != FP8KV_OK) return sh;
    if (batch < 0 || batch > 65535 || max_seq_len < 0 || max_blocks_per_seq < 0) return FP8KV_ERR_INVALID_ARG;
    if (block_size != kBS || num_blocks >= (INT64_C(1) << 31) || num_blocks * num_kv_heads >= (INT64_C(1) << 31))
        return FP8KV_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(max_blocks_per_seq) * block_size < max_seq_len) return FP8KV_ERR_INVALID_ARG;
    if (!q_starts && num_tokens != batch) return FP8KV_ERR_INVALID_ARG;
    if (batch == 0 || num_tokens == 0 || max_seq_len == 0) return FP8KV_OK;
    if (!k_cache || !v_cache || !a16(k_cache) || !a16(v_cache) || !k_scales || !v_scales || !a4(k_scales) ||
        !a4(v_scales) || !block_tables || !a4(block_tables) || !seq_lens || !a4(seq_lens) || !a4(q_starts) ||
        (q && num_q_heads < 1))
        return FP8KV_ERR_INVALID_ARG;
    BlockArgs a;
    fp8kv_status st = make_rows(q, q_stride, q_out, k_new, k_stride, v_new, v_stride, num_tokens, num_q_heads,
                                num_kv_heads, head_dim, &a.rw);
    if (st != FP8KV_OK) return st;
    st = make_rope(positions, num_axes, inv_freq, freq_axis, rotary_dim, false, &a.rp);
    if (st != FP8KV_OK) return st;
    if (!workspace || workspace_bytes < kWorkspace || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return FP8KV_ERR_WORKSPACE;
    a.block_tables = block_tables;
    a.seq_lens = seq_lens;
    a.q_starts = q_starts;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.err = static_cast<uint32_t*>(workspace);
    a.num_blocks = num_blocks;
    a.max_blocks_per_seq = max_blocks_per_seq;
    a.max_seq_len = max_seq_len;
    a.batch = batch;
    int sms = 0;
    if (fp8kv::device_sms(&sms) != 0) return FP8KV_ERR_CUDA;
    // sequence b's CTAs start at q_starts[b] / 16 + 2b (find_page)
    const int64_t blocks = q_starts ? num_tokens / kBS + 2 * static_cast<int64_t>(batch) : batch;
    const int64_t pages = q_starts ? (num_tokens + kBS - 1) / kBS : batch;
    const int splits = head_splits(pages, (q ? num_q_heads : 0) + 2 * num_kv_heads, sms);
    auto kernel = rope_style == FP8KV_ROPE_PAIRS ? block_kernel<true>(head_dim) : block_kernel<false>(head_dim);
    return launch(kernel, a, blocks, splits, a.rp.rot, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? FP8KV_OK
               : FP8KV_ERR_CUDA;
}
