// Attention behind shared prefixes: what its kernels share.
//
// The sequences of a group agree in their first tokens, so those are attended to
// once for the rows of all: a group's query rows that share a key-value head are one block
// of rows over the prefix's tiles.  What is shared in earnest is the prefix cut to a multiple of kShareStep and
// to less than any new token of the group sees, so prefixes need no masks, and what a
// sequence has of its own is never empty; a group of one sequence shares nothing
// (attn_share_plan_kernel; with few groups and sequences every CTA finds that out by itself, SharedWalk::plan).
//
// The work is a list of records: the groups' prefixes, then what each sequence has of its own, as
// the tiles behind its prefix.  (On CUDA cores, whose time goes by the rows, the latter is
// gdn_attn_decode's kernel from a.skip[b] on where there are few.)  Items are (record, key-value
// head, row block) with `setup` units and one per tile; all units are cut into equal ranges, one per
// CTA, as attn_common.cuh does.  A row's first part of a record goes to its place in a.part_o or s.pre_o, with how many
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

// What a group of `count` sequences with tokens shares in earnest, of the prefix that is said: less than the first new token of
// any of them sees.
__device__ __forceinline__ int shared_tokens(const AttnArgs& a, int prefix, int count, int least) {
    const int share = count > 1 ? min(prefix, least - a.K) : 0;
    return share > 0 ? share / kShareStep * kShareStep : 0;
}
// Row blocks and units of a record of `seqs` sequences.
__device__ __forceinline__ int64_t size_record(const ShareArgs& s, ShareRecord& rec) {
    rec.blocks = (int)(((int64_t)rec.seqs * s.a.rows + s.rows_per_block - 1) / s.rows_per_block);
    return rec.tiles > 0 ? (int64_t)rec.blocks * s.a.H_kv * (s.setup + rec.tiles) : 0;
}
// The record of a group's prefix, of what sequence b has of its own; their units.
__device__ __forceinline__ int64_t prefix_record(const ShareArgs& s, ShareRecord& rec, int first, int behind, int leader,
                                                 int share) {
    rec.seq0 = first;
    rec.seqs = max(behind - first, 0);
    rec.leader = leader;
    rec.tile0 = 0;
    rec.tiles = share / s.tile;
    return size_record(s, rec);
}
__device__ __forceinline__ int64_t own_record(const ShareArgs& s, ShareRecord& rec, int b, int len, int share) {
    rec.seq0 = rec.leader = b;
    rec.seqs = 1;
    rec.tile0 = share / s.tile;
    rec.tiles = len > 0 ? (len - 1) / s.tile + 1 - rec.tile0 : 0;
    return size_record(s, rec);
}
__device__ __forceinline__ int group_begin(const ShareArgs& s, int g) {
    return s.cu != nullptr ? min(max(s.cu[g], 0), s.a.B) : g * s.a.B;
}

// The segments of one CTA's unit range, in order; by whole warps.  FEW: s.few.  (With a branch instead, the tensor-core
// kernel's other warps came out slower too: 32 sequences with 16 new tokens 152 -> 159 us.)
template <bool FEW>
struct SharedWalk {
    int64_t total, at, end, rec_end;
    ShareRecord rec;
    int r, len;  // the record, its sequence's length (a prefix: 0)
    int c, n;    // the CTA, of how many that take part
    ShareRecord its;  // few: the lane's record, its sequence's length
    int its_len;
    __device__ __forceinline__ SharedWalk(const ShareArgs& s, int c_, int n_)
        : rec_end(0), r(0), len(0), c(c_), n(n_), its_len(0) {
        if (FEW) {
            plan(s);
            if (n > total) n = (int)total;
            at = c < n ? cta_begin(total, c, n) : 0;
            end = c < n ? cta_begin(total, c + 1, n) : 0;
            if (at < end) find(s, s.records);
            return;
        }
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
    // The plan where there are few groups and sequences: lane g has group g, lane G + b sequence b.  (us a call with the
    // plan in a kernel before this one, and here: 4 sequences behind 1000 tokens 16.4, 14.3; 8 behind 262000 95.7, 92.5.
    // With three records to a lane it took as long as that kernel: 64 sequences 63.5, 63.6.)  CTA 0 tells the kernels
    // behind this one what the sequences share.
    __device__ __forceinline__ void plan(const ShareArgs& s) {
        const AttnArgs& a = s.a;
        const int lane = threadIdx.x & 31, b = lane - s.G;
        const bool seq = b >= 0 && b < a.B;
        its_len = seq ? clamped_len(a, b) : 0;
        const int begin = lane <= s.G ? group_begin(s, lane) : a.B, prefix = lane < s.G ? s.prefix[lane] : 0;
        its = {};
        int64_t units = 0;
        int share = 0;  // of the lane's sequence
#pragma unroll 1
        for (int g = 0; g < s.G; ++g) {
            const int first = __shfl_sync(0xffffffffu, begin, g), behind = __shfl_sync(0xffffffffu, begin, g + 1);
            const bool in = seq && first <= b && b < behind && its_len > 0;
            const uint32_t those = __ballot_sync(0xffffffffu, in);
            const int least = __reduce_min_sync(0xffffffffu, in ? its_len : INT32_MAX);
            const int n = shared_tokens(a, __shfl_sync(0xffffffffu, prefix, g), __popc(those), least);
            if (in) share = n;
            if (lane == g) units = prefix_record(s, its, first, behind, those != 0 ? __ffs(those) - 1 - s.G : 0, n);
        }
        if (seq) {
            if (s.records > s.G) units = own_record(s, its, b, its_len, share);
            if (blockIdx.x == 0) const_cast<int32_t*>(a.skip)[b] = share;
        }
        int64_t inc = units;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        its.unit0 = inc - units;
        total = __shfl_sync(0xffffffffu, inc, 31);
    }
    // The last record before `hi` that starts at or before unit `at`, from record r on: 32 at a time.
    __device__ __forceinline__ void find(const ShareArgs& s, int hi) {
        const int lane = threadIdx.x & 31;
        if (FEW) {
            r = 31 - __clz(__ballot_sync(0xffffffffu, lane < hi && its.unit0 <= at));  // (record 0 starts at 0)
            rec.unit0 = __shfl_sync(0xffffffffu, its.unit0, r);
            rec.seq0 = __shfl_sync(0xffffffffu, its.seq0, r);
            rec.seqs = __shfl_sync(0xffffffffu, its.seqs, r);
            rec.tile0 = __shfl_sync(0xffffffffu, its.tile0, r);
            rec.tiles = __shfl_sync(0xffffffffu, its.tiles, r);
            rec.leader = __shfl_sync(0xffffffffu, its.leader, r);
            rec.blocks = __shfl_sync(0xffffffffu, its.blocks, r);
            rec_end = __shfl_sync(0xffffffffu, its.unit0, (r + 1) & 31);
            if (r + 1 >= hi) rec_end = total;
            len = r < s.G ? 0 : __shfl_sync(0xffffffffu, its_len, r);
            return;
        }
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
