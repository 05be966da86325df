// How the tree attention cuts its work over CTAs (plain host/device integer
// arithmetic: the kernels and the host-side checks run the same functions).
//
// A unit is (sequence, kv head, block of query rows); sequence b has
// heads * blocks_b of them, each over the same n_b pages.  The units' pages are
// laid end to end, P in all, and cut into C equal contiguous ranges, one per
// CTA (partition.cuh); a CTA's range overlaps one or more units, each overlap
// a segment.  A unit that lies in one range is finished by its CTA; any other
// leaves one partial per segment.  A CTA has at most two such segments, its
// first (of a unit begun before its range) and its last (of a unit begun in
// it), so two partial slots a CTA suffice at any batch.
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

// CTAs that share P pages: at least min_pages each, at most `most`.
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
    int64_t base;      // the unit's first page in the list
    int np;            // pages of the unit
};

// The segment that begins at page `pos` of a range that ends at `end`.
// pre[b]: pages of the sequences before b; units[b]: units of b.
template <typename Blocks>
FP8KV_HD Segment segment_at(int64_t pos, int64_t end, const int64_t* pre, int batch, int heads, const Blocks& blocks_of) {
    int lo = 0, hi = batch - 1;   // the last b with pre[b] <= pos; it has pages, since pos < pre[batch]
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (pre[mid] <= pos) lo = mid; else hi = mid - 1;
    }
    Segment s;
    s.b = lo;
    const int blocks = blocks_of(lo);
    s.np = static_cast<int>((pre[lo + 1] - pre[lo]) / (static_cast<int64_t>(heads) * blocks));
    const int64_t off = pos - pre[lo];
    const int u = static_cast<int>(off / s.np);
    s.hk = u / blocks;
    s.rb = u - s.hk * blocks;
    s.base = pre[lo] + static_cast<int64_t>(u) * s.np;
    s.lp0 = static_cast<int>(pos - s.base);
    s.lp1 = static_cast<int>((end - s.base < s.np ? end - s.base : s.np));
    return s;
}

// The slot of the partial that CTA c leaves of a unit beginning at `base`.
FP8KV_HD int64_t partial_slot(const Partition& q, int c, int64_t base) {
    return 2 * static_cast<int64_t>(c) + (base >= range_start(q, c) ? 1 : 0);
}

}  // namespace tree
}  // namespace fp8kv

#undef FP8KV_HD
