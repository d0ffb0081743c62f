// Attention behind shared prefixes: what its kernels share.
//
// The sequences of a group agree in their first tokens, so those are attended to
// once for the rows of all: the pass over the prefixes treats a group's query rows
// that share a key-value head as one block of rows, the pass over the rest is the one of
// gdn_attn_decode from a.skip[b] on, and a merge joins what both leave.
//
// What is shared in earnest is the prefix cut to a multiple of kShareStep and to
// less than any new token of the group sees, so the pass over the prefixes needs no
// masks, and the rest is never empty; a group of one sequence shares nothing
// (attn_share_plan_kernel).  Items of that pass are (group g, key-value head h, row block rb) with
// `setup` units and one per tile, cut into equal ranges of units like the others' (attn_common.cuh).
#pragma once

#include "attn_common.cuh"

namespace gdn {
namespace attn {

__device__ __forceinline__ void group_bounds(const ShareArgs& s, int g, int& lo, int& hi) {
    lo = 0;
    hi = s.a.B;
    if (s.cu != nullptr) {
        lo = min(max(s.cu[g], 0), s.a.B);
        hi = min(max(s.cu[g + 1], lo), s.a.B);
    }
}
// A part of an item of the pass over the prefixes, worked on by one CTA.
struct PrefixSegment {
    int tile0, tile1;  // its tiles; 0, 0: the CTA's range has ended
    int parts;         // how many CTAs' parts the item has if this is the first, else 0
    int h, seq0;       // key-value head, first sequence of the group
    int leader;        // the sequence whose pages are read
    int r0, nr;        // rows r0 .. r0 + nr of the group's
};
// Index of row r of a group's (first sequence seq0) among the [B, K, H_q] rows.
__device__ __forceinline__ int64_t prefix_row(const AttnArgs& a, int seq0, int h, int r) {
    const int b = r / a.rows;
    return row_index(a, seq0 + b, h, r - b * a.rows);
}

struct PrefixWalk {
    int64_t total, at, end;
    int c, n;  // the CTA, of how many that take part
    __device__ __forceinline__ PrefixWalk(const ShareArgs& s, int c_, int n_) : c(c_), n(n_) {
        total = s.groups[s.G].unit0;
        if (n > total) n = (int)total;
        at = c < n ? cta_begin(total, c, n) : 0;
        end = c < n ? cta_begin(total, c + 1, n) : 0;
    }
    __device__ __forceinline__ bool next(const ShareArgs& s, int tile, PrefixSegment& g) {
        while (at < end) {
            int lo = 0, hi = s.G - 1;  // the last group that starts at or before the unit
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (s.groups[mid].unit0 <= at) lo = mid; else hi = mid - 1;
            }
            const PrefixGroup grp = s.groups[lo];
            const int rows = grp.seqs * s.a.rows;
            const int units = s.setup + min(max(grp.share, 0), s.a.max_pages * s.a.page_size) / tile;
            const int64_t off = at - grp.unit0;
            const int64_t item = off / units;
            const int from = (int)(off - item * units);
            const int64_t left = end - at;
            const int upto = left < units - from ? from + (int)left : units;
            const int64_t last = at + (units - from) - 1;  // the item's
            at += upto - from;
            if (upto <= s.setup) continue;  // the range ends before the item's tiles
            g.tile0 = from > s.setup ? from - s.setup : 0;
            g.tile1 = upto - s.setup;
            g.parts = g.tile0 > 0 ? 0 : cta_of(total, last, n) - c + 1;
            g.h = grp.blocks > 0 ? (int)(item / grp.blocks) : s.a.H_kv;
            if (g.h >= s.a.H_kv) return false;  // (never in a call that keeps to the rules)
            g.seq0 = grp.seq0;
            g.leader = min(max(grp.leader, 0), s.a.B - 1);
            g.r0 = (int)(item - (int64_t)g.h * grp.blocks) * s.rows_per_block;
            g.nr = min(s.rows_per_block, rows - g.r0);
            return true;
        }
        return false;
    }
};

// pre_stat's last two words: the first CTA and how many, the row in its block.
__device__ __forceinline__ float4 prefix_stat(float m, float sum, int parts, int r) {
    return make_float4(sum == 0.f ? -INFINITY : m, sum, __int_as_float((int)blockIdx.x | parts << 16), __int_as_float(r));
}
// A CTA's slot: maxima and sums of rows_per_block rows, then their outputs.
__device__ __forceinline__ float* prefix_slot(const ShareArgs& s, int c) { return s.pre_slots + c * s.pre_slot_floats; }

}  // namespace attn
}  // namespace gdn
