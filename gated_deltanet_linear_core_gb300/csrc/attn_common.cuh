// Work division shared by the paged-cache attention kernels (attn_ffma.cu,
// attn_tc.cu) and the kernel that joins their partial results.
//
// An item is (sequence b, key-value head h, row block rb): a block of the
// sequence's K*G query rows that share h (G = H_q / H_kv; row r is new token
// r / G, query head h*G + r % G).  An item's units are its tiles of `tile`
// cached tokens, at least one (an empty sequence still has rows to write),
// after `setup` units that stand for what starting an item costs: a CTA that
// gets several short sequences gets fewer tiles.  All units of a call, item
// after item, are cut into equal contiguous ranges, one per CTA, whatever the
// lengths are: the lengths stay on the device, so the host never waits for them
// and a captured graph follows them.  A CTA that covers an item's tiles whole
// writes its rows; otherwise it leaves the running maximum, sum and unnormalised
// output in one of its two workspace slots (its part starts inside the item's
// tiles: slot 2c; at their start: 2c + 1), and attn_join_kernel combines the
// slots in CTA order, told by the CTAs what to join (JoinTask).
#pragma once

#include <math.h>

#include "gdn_common.cuh"
#include "gdn_launch.h"

namespace gdn {
namespace attn {

__device__ __forceinline__ int clamped_len(const AttnArgs& a, int b) {
    const int64_t cap = (int64_t)a.max_pages * a.page_size;
    const int n = a.lens[b];
    return n < 0 ? 0 : (n > cap ? (int)cap : n);
}
__device__ __forceinline__ int tiles_of(int len, int tile) { return len <= tile ? 1 : (len - 1) / tile + 1; }
__device__ __forceinline__ int units_of(const AttnArgs& a, int len, int tile) { return a.setup + tiles_of(len, tile); }

// First unit of CTA c of n.
__host__ __device__ __forceinline__ int64_t cta_begin(int64_t total, int c, int n) { return total * c / n; }
// The CTA whose range holds unit u.
__device__ __forceinline__ int cta_of(int64_t total, int64_t u, int n) { return (int)(((u + 1) * n - 1) / total); }

struct Place {
    int64_t total;  // units of the whole call
    int64_t first;  // first unit of sequence b's items
    int b, len;     // the sequence that holds the unit asked for, its clamped length
};

// Units of the call and the sequence that holds the first unit of CTA c of the
// n that take part (at most one per unit), by one warp: a lane adds up a 32nd of the sequences, then the warp searches the lane's
// share that holds the unit.  (A block-wide scan saves loads but costs three
// barriers, which at the start of a call is longer.)
__device__ __forceinline__ Place find_place(const AttnArgs& a, int tile, int c, int& n) {
    const int lane = threadIdx.x & 31;
    const int64_t mult = (int64_t)a.H_kv * a.n_rb;
    const int per = (a.B + 31) / 32;
    int64_t inc = 0;
#pragma unroll 4
    for (int i = 0; i < per; ++i) {
        const int b = lane * per + i;
        if (b < a.B) inc += units_of(a, clamped_len(a, b), tile);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
    }
    Place p;
    p.total = __shfl_sync(0xffffffffu, inc, 31) * mult;
    p.first = 0;
    p.b = p.len = 0;
    if (n > p.total) n = (int)p.total;
    if (c >= n) return p;
    const int64_t want = cta_begin(p.total, c, n);
    const int owner = __ffs(__ballot_sync(0xffffffffu, want < inc * mult)) - 1;
    const int64_t before = __shfl_sync(0xffffffffu, inc, owner > 0 ? owner - 1 : 0);
    if (owner > 0) p.first = before * mult;
    const int end = min(a.B, (owner + 1) * per);
    for (int b0 = owner * per; b0 < end; b0 += 32) {
        const int b = b0 + lane;
        const int len = b < end ? clamped_len(a, b) : 0;
        int sum = b < end ? units_of(a, len, tile) : 0;  // inclusive scan: 32 sequences' units fit 31 bits
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += v;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, want < p.first + sum * mult);
        if (past != 0) {
            const int l = __ffs(past) - 1;
            const int less = __shfl_sync(0xffffffffu, sum, l > 0 ? l - 1 : 0);
            p.b = b0 + l;
            p.len = __shfl_sync(0xffffffffu, len, l);
            if (l > 0) p.first += less * mult;
            break;
        }
        p.first += __shfl_sync(0xffffffffu, sum, 31) * mult;
    }
    return p;
}

// The segments (parts of items) of one CTA's unit range, in order.
struct Segment {
    int b, h, rb, len;   // item
    int tile0, tile1;    // its tiles [tile0, tile1) of this segment
    int tiles;           // tiles of the whole item
};
struct Walk {
    int64_t at, end, item0;  // units; item0: first unit of sequence b's items
    int b, len;
    __device__ __forceinline__ Walk(const Place& p, int64_t lo, int64_t hi)
        : at(lo), end(hi), item0(p.first), b(p.b), len(p.len) {}
    __device__ __forceinline__ bool next(const AttnArgs& a, int tile, Segment& s) {
        while (at < end) {
            int units = units_of(a, len, tile);
            while (at >= item0 + (int64_t)units * a.H_kv * a.n_rb) {
                item0 += (int64_t)units * a.H_kv * a.n_rb;
                len = clamped_len(a, ++b);
                units = units_of(a, len, tile);
            }
            const int64_t off = at - item0;
            const int item = (int)(off / units);
            const int from = (int)(off - (int64_t)item * units);
            const int64_t left = end - at;
            const int upto = left < units - from ? from + (int)left : units;
            at += upto - from;
            if (upto <= a.setup) continue;  // the range ends before the item's tiles
            s.tile0 = from > a.setup ? from - a.setup : 0;
            s.tile1 = upto - a.setup;
            s.tiles = units - a.setup;
            s.h = item / a.n_rb;
            s.rb = item - s.h * a.n_rb;
            s.b = b;
            s.len = len;
            return true;
        }
        return false;
    }
};

// Rows of row block rb.
__device__ __forceinline__ int block_rows(const AttnArgs& a, int rb) { return min(a.rb_rows, a.rows - rb * a.rb_rows); }
// Cached tokens row r of a sequence of len tokens sees.
__device__ __forceinline__ int visible(const AttnArgs& a, int len, int r) { return len - (a.K - 1 - r / a.group); }
// Index of row r of (b, h) among the [B, K, H_q] rows.
__device__ __forceinline__ int64_t row_index(const AttnArgs& a, int b, int h, int r) {
    const int i = r / a.group;
    return ((int64_t)b * a.K + i) * a.H_q + h * a.group + (r - i * a.group);
}

// What to join where CTA c's range starts inside an item: the item, and the CTAs
// that worked on it.  Written by CTA c (one thread), so that the join needs
// neither the lengths nor any of the divisions here.
struct alignas(16) JoinTask {
    int n;         // CTAs that worked on the item (0: the range starts with an item of its own)
    int c0;        // the first of them: its part is in slot 2 c0 + 1, that of CTA c0 + i in slot 2 (c0 + i)
    int b, h, rb;  // the item
    int pad[3];
};
__device__ __forceinline__ JoinTask* join_task(const AttnArgs& a, int c) { return reinterpret_cast<JoinTask*>(a.ws) + c; }
// `first`: the CTA's first segment, just taken from its walk; null: it has none.
__device__ __forceinline__ void write_join_task(const AttnArgs& a, const Place& p, const Walk& walk, const Segment* first,
                                                int c, int n) {
    JoinTask t;
    t.n = 0;
    if (first != nullptr && first->tile0 > 0) {
        const Segment& s = *first;
        const int64_t u = walk.item0 + (int64_t)(s.h * a.n_rb + s.rb) * (a.setup + s.tiles) + a.setup;
        t.c0 = cta_of(p.total, u, n);
        t.n = cta_of(p.total, u + s.tiles - 1, n) - t.c0 + 1;
        t.b = s.b;
        t.h = s.h;
        t.rb = s.rb;
    }
    *join_task(a, c) = t;
}

// A workspace slot: maxima (log2 domain) and sums of its rows, then their
// unnormalised outputs; and the slot of a CTA's part of an item.
__device__ __forceinline__ float* slot_ptr(const AttnArgs& a, int slot) {
    return a.ws + kAttnMaxCtas * (sizeof(JoinTask) / 4) + (int64_t)slot * a.slot_floats;
}
__device__ __forceinline__ int part_slot(const Segment& s) { return 2 * blockIdx.x + (s.tile0 > 0 ? 0 : 1); }

constexpr float kNone = -3.0e38f;     // running maximum of a row without a score above -inf yet
constexpr float kSlack = 8.0f;        // how far (log2) scores may exceed the running maximum before it is moved
constexpr float kLn2 = 0.6931471805599453f;

// Joins C columns over the warp's lanes, halving the columns a lane holds at
// each step: v[0 .. C / 32) of lane i becomes columns (C / 32) i .. (C = 16: lane
// i has column i / 2).  A reduction per column costs several times as much.
template <int C, typename F>
__device__ __forceinline__ void join_lanes(float* v, int lane, F f) {
#pragma unroll
    for (int h = C / 2, o = 16; o >= 1; h /= 2, o /= 2) {
        if (h >= 1) {
#pragma unroll
            for (int c = 0; c < C / 2; ++c)
                if (c < h) {
                    const float send = lane & o ? v[c] : v[c + h];
                    const float keep = lane & o ? v[c + h] : v[c];
                    v[c] = f(keep, __shfl_xor_sync(0xffffffffu, send, o));
                }
        } else {
            v[0] = f(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
        }
    }
}

}  // namespace attn
}  // namespace gdn
