// How the tree attention cuts its work over CTAs (plain host/device integer
// arithmetic: the kernels and the host-side checks run the same functions).
//
// A unit is (sequence, kv head, block of query rows); sequence b has
// heads * blocks_b of them, each over the same n_b pages.  The units' pages are
// laid end to end, each unit's behind kLeadPages places that hold none and stand
// for what a CTA that begins another unit spends on it; the P places in all are
// cut into C equal contiguous ranges, one per CTA (partition.cuh).  A CTA's range
// overlaps one or more units' pages, each overlap a segment.  A unit that lies in
// one range is finished by its CTA; any other leaves one partial per segment.  A
// CTA has at most two such segments, its first (of a unit begun before its range)
// and its last (of a unit begun in it), so two partial slots a CTA suffice at any
// batch.
#pragma once

#include <cstdint>

#include "partition.cuh"

#if defined(__CUDACC__)
#define FP8KV_HD __host__ __device__ __forceinline__
#else
#define FP8KV_HD inline
#endif

namespace fp8kv {
namespace tree {

// A turn to another unit takes about five stages' time.  Measured with 16, 24, 40,
// 56 and 80: 16 x 20K tokens, d 256, 8 nodes 67.1, 65.2, 59.8, 60.7 and 61.2 us; 8 x
// 20K, d 128, 16 nodes 86.6, 85.9, 84.9, 84.1 and 84.0; 5 x 9K in bf16 88.6, 89.6,
// 90.4, 93.0 and 96.0.
constexpr int kLeadPages = 40;

// CTAs that share P places: at least min_pages each, at most `most`.
FP8KV_HD int cta_count(int64_t P, int most, int min_pages) {
    const int64_t want = (P + min_pages - 1) / min_pages;
    return static_cast<int>(want < 1 ? 1 : want < most ? want : most);
}

// Pages of a sequence of L tokens, the last n of them drafted: those that any
// node attends.  The oldest key is the root's, at position L - n.
FP8KV_HD int first_key(int L, int n, int window) {
    const int64_t lo = static_cast<int64_t>(L) - n + 1 - window;
    return window > 0 && lo > 0 ? static_cast<int>(lo) : 0;
}
FP8KV_HD int unit_pages(int L, int n, int window) { return n > 0 ? (L - 1) / 16 - first_key(L, n, window) / 16 + 1 : 0; }

struct Segment {
    int b, hk, rb;     // sequence, kv head, block of query rows
    int lp0, lp1;      // pages [lp0, lp1) of the unit
    int64_t base;      // the unit's first place in the list
    int np;            // pages of the unit
};

// The place behind the unit that begins at `base`.
FP8KV_HD int64_t unit_end(const Segment& s) { return s.base + kLeadPages + s.np; }

// The segment at place `pos` of a range that ends at `end` (its pages are none
// where the range ends in the unit's lead).
// pre[b]: places of the sequences before b; blocks_of(b), pages_of(b): blocks of
// query rows of sequence b, pages of its units.  (A sequence's units have less
// than 2^31 places in all, so one 32-bit division finds the unit.)
template <typename Blocks, typename Pages>
FP8KV_HD Segment segment_at(int64_t pos, int64_t end, const int64_t* pre, int batch, const Blocks& blocks_of,
                            const Pages& pages_of) {
    int lo = 0, hi = batch - 1;   // the last b with pre[b] <= pos; it has units, since pos < pre[batch]
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (pre[mid] <= pos) lo = mid; else hi = mid - 1;
    }
    Segment s;
    s.b = lo;
    s.np = pages_of(lo);
    const uint32_t u = static_cast<uint32_t>(pos - pre[lo]) / static_cast<uint32_t>(s.np + kLeadPages);
    const uint32_t blocks = static_cast<uint32_t>(blocks_of(lo));
    s.hk = static_cast<int>(u / blocks);
    s.rb = static_cast<int>(u % blocks);
    s.base = pre[lo] + static_cast<int64_t>(u) * (s.np + kLeadPages);
    const int64_t p0 = pos - s.base - kLeadPages, p1 = end - s.base - kLeadPages;
    s.lp0 = static_cast<int>(p0 > 0 ? p0 : 0);
    s.lp1 = static_cast<int>(p1 < s.np ? p1 : s.np);
    if (s.lp1 < s.lp0) s.lp1 = s.lp0;
    return s;
}

// The slot of the partial that CTA c leaves of a unit beginning at `base`.
FP8KV_HD int64_t partial_slot(const Partition& q, int c, int64_t base) {
    return 2 * static_cast<int64_t>(c) + (base + kLeadPages >= range_start(q, c) ? 1 : 0);
}

}  // namespace tree
}  // namespace fp8kv

#undef FP8KV_HD
