// Attention behind shared prefixes: what its kernels share.
//
// The sequences of a group agree in their first tokens, so those are attended to
// once for the rows of all: a group's query rows that share a key-value head are one block
// of rows over the prefix's tiles.  What is shared in earnest is the prefix cut to a multiple of kShareStep and
// to less than any new token of the group sees, so prefixes need no masks, and what a
// sequence has of its own is never empty; a group of one sequence shares nothing
// (attn_share_plan_kernel).
//
// The work is a list of records: the groups' prefixes, then what each sequence has of its own, as
// the tiles behind its prefix.  (On CUDA cores, whose time goes by the rows, the latter is
// gdn_attn_decode's kernel from a.skip[b] on where there are few.)  Items are (record, key-value head, row block) with `setup` units and
// one per tile; all units are cut into equal ranges, one per CTA, as attn_common.cuh
// does.  A row's first part of a record goes to its place in a.part_o or s.pre_o, with how many
// CTAs' parts there are beside it, and a part that starts inside an item to the
// CTA's one slot; attn_merge_kernel puts them together.
#pragma once

#include "attn_common.cuh"

namespace gdn {
namespace attn {

// A part of an item, worked on by one CTA.
struct alignas(16) SharedSegment {
    int tile0, tile1;  // its tiles; 0, 0: the CTA's range has ended
    int parts;         // how many CTAs' parts the item has if this is the first, else 0
    int h, seq0;       // key-value head, first of the sequences whose rows these are
    int leader;        // the sequence whose pages are read
    int r0, nr;        // rows r0 .. r0 + nr of theirs
    int len;           // a sequence's own tokens: its length; a prefix, which all rows see: 0
    int pad[3];
};
// Index of row r of the sequences from seq0 on among the [B, K, H_q] rows.
__device__ __forceinline__ int64_t shared_row(const AttnArgs& a, int seq0, int h, int r) {
    const int b = r / a.rows;
    return row_index(a, seq0 + b, h, r - b * a.rows);
}

// The segments of one CTA's unit range, in order; by whole warps.
struct SharedWalk {
    int64_t total, at, end, rec_end;
    ShareRecord rec;
    int r, len;  // the record, its sequence's length (a prefix: 0)
    int c, n;    // the CTA, of how many that take part
    __device__ __forceinline__ SharedWalk(const ShareArgs& s, int c_, int n_) : rec_end(0), r(0), len(0), c(c_), n(n_) {
        // (the first step of find() needs nothing but the records: its loads go out with the total's)
        const int step = (s.records + 31) >> 5, i = (threadIdx.x & 31) * step;
        const int64_t mine = i < s.records ? s.rec[i].unit0 : INT64_MAX;
        total = s.rec[s.records].unit0;
        if (n > total) n = (int)total;
        at = c < n ? cta_begin(total, c, n) : 0;
        end = c < n ? cta_begin(total, c + 1, n) : 0;
        r = (31 - __clz(__ballot_sync(0xffffffffu, mine <= at) | 1)) * step;
        if (at < end) find(s, min(s.records, r + step));
    }
    // The last record before `hi` that starts at or before unit `at`, from record r on: 32 at a time.
    __device__ __forceinline__ void find(const ShareArgs& s, int hi) {
        const int lane = threadIdx.x & 31;
        while (hi - r > 1) {
            const int step = (hi - r + 31) >> 5, i = r + lane * step;
            const uint32_t past = __ballot_sync(0xffffffffu, i < hi && s.rec[i].unit0 <= at);
            r += (31 - __clz(past | 1)) * step;
            hi = min(hi, r + step);
        }
        rec = s.rec[r];
        rec_end = s.rec[r + 1].unit0;
        len = r < s.G ? 0 : clamped_len(s.a, r - s.G);
    }
    __device__ __forceinline__ bool next(const ShareArgs& s, SharedSegment& g) {
        while (at < end) {
            if (at >= rec_end) find(s, s.records);
            const int units = s.setup + rec.tiles;
            const int64_t off = at - rec.unit0;
            const int64_t item = off / units;
            const int from = (int)(off - item * units);
            const int64_t left = end - at;
            const int upto = left < units - from ? from + (int)left : units;
            const int64_t last = at + (units - from) - 1;  // the item's
            at += upto - from;
            if (upto <= s.setup) continue;  // the range ends before the item's tiles
            const int inside = from > s.setup ? from - s.setup : 0;
            g.parts = inside > 0 ? 0 : upto == units ? 1 : cta_of(total, last, n) - c + 1;
            g.tile0 = rec.tile0 + inside;
            g.tile1 = rec.tile0 + upto - s.setup;
            g.h = (int)(item / rec.blocks);
            g.seq0 = rec.seq0;
            g.leader = rec.leader;
            g.r0 = (int)(item - (int64_t)g.h * rec.blocks) * s.rows_per_block;
            g.nr = min(s.rows_per_block, rec.seqs * s.a.rows - g.r0);
            g.len = len;
            return true;
        }
        return false;
    }
};

// A statistic's last two words: the first CTA and how many, the row in its block.
__device__ __forceinline__ float4 part_stat(float m, float sum, int parts, int r) {
    return make_float4(sum == 0.f ? -INFINITY : m, sum, __int_as_float((int)blockIdx.x | parts << 16), __int_as_float(r));
}
// A CTA's slot: maxima and sums of rows_per_block rows, then their outputs.
__device__ __forceinline__ float* shared_slot(const ShareArgs& s, int c) { return s.slots + c * s.slot_floats; }

}  // namespace attn
}  // namespace gdn
