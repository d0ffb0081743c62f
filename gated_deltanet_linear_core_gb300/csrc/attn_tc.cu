// Attention of the newest tokens over the paged cache on tcgen05 tensor cores
// (bf16).
//
// With at most 128 query rows per key-value head the work is bound by reading
// the cache once, so the products are laid out for the cache tiles as they
// arrive: a tile is 128 tokens, and the tokens (then the head dims) are the
// M = 128 side of the MMAs, the query rows the N side:
//   S^T [128 tokens x N rows] = K Q^T        (A = K tile, B = Q; both K-major)
//   O^T [128 dims x N rows]  += V^T P^T      (A = V tile, B = P; both MN-major)
// No tile is transposed or copied, and an MMA of few rows costs what reading
// its A operand from shared memory costs (128 B/clock, five times the HBM rate
// per SM).  K and V tiles land by TMA, one box per page piece, in slots of 128
// tokens x 128 dims, so a tile of head dim 256 is four slots of a ring.
//
// Softmax: a thread owns one token (TMEM lane) and CPT rows (columns).  The
// running maximum of a row is moved only when a score exceeds it by 2^8 (P then
// stays below 2^8, harmless in f32 sums), so most tiles need one vote and no
// rescaling of O.  P is handed to the MMA as two bf16 (the value cut to 8 bits
// and the rounded rest, 16 bits in all): one bf16 alone would add an error of
// the size of the output's own rounding.  Both are columns of one MMA (2 N
// columns, joined at the end): its time is that of reading V, so the rest is
// free; two MMAs per step were bound by that (64 rows: 3.2 us per tile of head
// dim 256 where HBM takes 2.9).  Only 128 rows of head dims above 128 take two,
// which add up: O in two parts has no room in tensor memory there.
// Sums are kept per thread in f32 and joined at the end.
//
// Warps: 0 walks the CTA's range, tells the others its segments and loads K and V
// (the walk in every role cost 600 short sequences with 5 new tokens 14 us of 116),
// 1 issues the MMAs, 2 loads Q of the next segment as soon as S of the last tile
// is done, the others are the softmax.  Where a box has 16 tokens or less, warp 2
// loads V: a TMA load takes its warp some 80 clocks, and a tile of head dim 256 is
// 64 of them at 16 tokens (64 ragged sequences, pages of 8: 174 us with one warp,
// 111 with two; of 64: 103 and 105, so there one has both).  The MMA warp runs S
// of the next tile ahead of P V of this one, across segments too, so that only
// the outputs stand between two segments.  Every wait is bounded (1 s): on a
// timeout the roles run out without waiting, the copies in flight land, TMEM is
// freed and the error word is set.
#include <cuda.h>

#include "attn_common.cuh"
#include "tc_ptx.cuh"

namespace gdn {

__device__ int g_attn_error;  // bit 0: a bounded wait gave up

namespace {

using namespace attn;
using namespace tc;

constexpr int TILE = 128;
constexpr int SLAB = TILE * 128;      // bytes of 128 tokens x 64 dims
constexpr int SLOT = 2 * SLAB;        // ... x 128 dims
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr int kSmemMax = 232448;

template <int N, int NDB>
struct Layout {
    // Columns (rows of Q) per softmax thread and per TMEM access, chosen by time: 128 rows of head dim 256 took 222 us
    // with 16 warps and 267 with 8; of head dim 128, whose O has both parts of P, 84 with 16 (16 columns at a time; 138
    // with 32, most of whose registers spill) and 83 with 8; 32 rows 165 and 166.  Both forms of 128 rows spill 44 bytes.
    static constexpr int CPT = N <= 32 ? 16 : N == 64 || NDB == 2 ? 32 : 64;
    static constexpr int CH = N == 128 && NDB == 2 ? 16 : CPT < 32 ? CPT : 32;
    static constexpr int NWG = N / CPT;           // softmax warpgroups
    static constexpr int NSW = 4 * NWG;           // softmax warps
    static constexpr int NT = 96 + 32 * NSW;
    static constexpr int PBUF = N <= 64 ? 2 : 1;  // buffers of P
    // P of a tile: 128-byte rows of 64 columns.  N = 16: both buffers' [hi | lo] side by side in one
    // block; N = 32: [hi | lo] in one block per buffer; else hi and lo in blocks of their own.
    static constexpr int P_BYTES = N == 16 ? SLAB : N == 32 ? 2 * SLAB : PBUF * 2 * ((N + 63) / 64) * SLAB;
    static constexpr int Q_BYTES = 2 * NDB * N * 128;
    static constexpr int SCR = 4 * NWG * CH * 4;     // scratch: a value per lane quarter and column of one access
    static constexpr int BARS = 320, SEGS = 4;  // barriers; segments told ahead
    static constexpr int SMALL = BARS + SEGS * 32 + N * 4 * 3 + SCR;
    static constexpr int FIT = (kSmemMax - P_BYTES - Q_BYTES - SMALL) / SLOT;
    static constexpr int NS = FIT < 6 ? FIT : 6;
    // Slots are filled and used in the order K(0), K(1), V(0), K(2), V(1), .. of a segment's n tiles
    // (S of a tile runs ahead of P V of the one before): offsets from the segment's first slot.
    __device__ static __forceinline__ int k_slot(int j) { return j == 0 ? 0 : NDB * (2 * j - 1); }
    __device__ static __forceinline__ int v_slot(int j, int n) { return NDB * (j + 1 < n ? 2 * j + 2 : 2 * n - 1); }
    static constexpr int O_Q = NS * SLOT;
    static constexpr int O_P = O_Q + Q_BYTES;
    static constexpr int O_BAR = O_P + P_BYTES;
    static constexpr int O_SEG = O_BAR + BARS;
    static constexpr int O_M = O_SEG + SEGS * 32;
    static constexpr int O_VIS = O_M + N * 4;
    static constexpr int O_F = O_VIS + N * 4;
    static constexpr int O_SCR = O_F + N * 4;
    static constexpr int SMEM = O_BAR + SMALL;
    static constexpr int T_S = 0, T_O = 2 * N;
    static constexpr int PARTS = N <= 64 || NDB == 1 ? 2 : 1;  // O of P's upper and lower parts side by side, or their sum
    static constexpr int T_USED = (2 + NDB * PARTS) * N;
    static constexpr int T_COLS = T_USED <= 64 ? 64 : T_USED <= 128 ? 128 : T_USED <= 256 ? 256 : 512;
    static_assert(N * 512 <= P_BYTES, "output rows");
    static_assert(SMEM <= kSmemMax && NS >= 3, "shared memory");
    static_assert(35 * 8 <= BARS, "barriers");

    // byte offset of P's column block (16-byte chunk j of 8 columns) of token t
    __device__ static __forceinline__ uint32_t p_off(int buf, int lo, int chunk, int t) {
        uint32_t base = 0;
        int c = chunk;
        if constexpr (N == 16) c = buf * 4 + lo * 2 + chunk;
        else if constexpr (N == 32) { base = buf * SLAB; c = lo * 4 + chunk; }
        else {
            base = ((buf * 2 + lo) * ((N + 63) / 64) + (chunk >> 3)) * SLAB;
            c = chunk & 7;
        }
        return base + t * 128 + ((c ^ (t & 7)) << 4);
    }
    // start of P's operand (first token, first column) for the MMA descriptor
    __device__ static __forceinline__ uint32_t p_start(int buf, int lo) {
        if constexpr (N == 16) return buf * 64 + lo * 32;
        else if constexpr (N == 32) return buf * SLAB + lo * 64;
        else return (buf * 2 + lo) * ((N + 63) / 64) * SLAB;
    }
};

// What warp 0 tells the other roles of a segment: only it walks the range (the
// walk's code and divisions in every role cost each of them more than the note).
struct alignas(16) SegmentNote {
    Segment s;
    int more;  // 0: the range has ended
};
static_assert(sizeof(SegmentNote) == 32, "notes");

// Bounded wait; returns at once when another role has given up.
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    if (mbar_test(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
        if (mbar_test(bar, parity)) return true;
        if ((it & 31) == 0) {
            if (*abort_flag) return false;
            if (globaltimer_ns() - t0 > kWaitNs) {
                *abort_flag = 1;
                return false;
            }
        }
    }
}

// The same for a slot's position counter to reach `pos`.
__device__ __forceinline__ bool loaded_or_abort(volatile int* filled, int pos, volatile int* abort_flag) {
    if (*filled >= pos) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
        if (*filled >= pos) return true;
        if ((it & 31) == 0) {
            if (*abort_flag) return false;
            if (globaltimer_ns() - t0 > kWaitNs) {
                *abort_flag = 1;
                return false;
            }
        }
    }
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}
template <int NTHR>
__device__ __forceinline__ void softmax_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(NTHR) : "memory");
}
template <int NTHR>
__device__ __forceinline__ bool softmax_any(bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x), "n"(NTHR)
        : "memory");
    return r != 0;
}
// The same for the warpgroup that shares columns (named barriers 2 ..).
__device__ __forceinline__ void group_sync(int wg) { asm volatile("bar.sync %0, 128;" ::"r"(2 + wg) : "memory"); }
__device__ __forceinline__ bool group_any(int wg, bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x), "r"(2 + wg)
        : "memory");
    return r != 0;
}
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float* v) {
    if constexpr (N == 16) tmem_ld16(taddr, v); else tmem_ld32(taddr, v);
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
        "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
        : "memory");
}
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const float* v) {
    if constexpr (N == 16) tmem_st16(taddr, v); else tmem_st32(taddr, v);
}
__device__ __forceinline__ bool finite_bf16x8(uint4 u) {
    bool ok = true;
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) ok = ok && (w[i] & 0x7f80u) != 0x7f80u && (w[i] & 0x7f800000u) != 0x7f800000u;
    return ok;
}
__device__ __forceinline__ uint32_t zero_non_finite(uint32_t w) {
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
    return w;
}

// Operand descriptors by their low words (address and lbo in units of 16 bytes); the high word is the same for
// all (sbo 1024, version, 128-byte swizzle: sdesc_sw128).
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return (saddr >> 4) | ((lbo >> 4) << 16); }
__device__ __forceinline__ void mma_lo(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
    constexpr uint32_t hi = (1024u >> 4) | (1u << 14) | (2u << 29);
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
        "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(hi)
        : "memory");
}

template <int N, int NDB>
__global__ void __launch_bounds__(Layout<N, NDB>::NT, 1)
attn_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, AttnArgs a,
               int piece) {
    using L = Layout<N, NDB>;
    constexpr int CPT = L::CPT, NS = L::NS, NSOFT = 32 * L::NSW;
    extern __shared__ __align__(1024) uint8_t sm[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::O_BAR);
    uint64_t* full = bars;            // [6] slot landed (TMA)
    uint64_t* empty = bars + 6;       // [6] slot consumed (commit)
    uint64_t* s_full = bars + 12;     // [2] S of a tile done
    uint64_t* p_full = bars + 14;     // [2] P of a tile written, V tail mended (softmax warps)
    uint64_t* pv_done = bars + 16;    // [2] P V of a tile done
    uint64_t* q_full = bars + 18;     // a segment's Q written (Q warp)
    uint64_t* q_empty = bars + 19;    // S of a segment's last tile done
    uint64_t* seg_full = bars + 20;   // [4] a segment is told (warp 0)
    uint64_t* seg_empty = bars + 24;  // [4] ... and taken note of (MMA warp, Q warp, softmax warps)
    uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + 28);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
    volatile int* filled = reinterpret_cast<volatile int*>(bars + 30);  // [6] one more than the last position loaded into a slot
    uint64_t* drained = bars + 34;    // every MMA issued is done (abort)
    volatile int* odd_v = reinterpret_cast<volatile int*>(tslot + 2);  // a new token's value is not finite
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < 6; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
            filled[i] = 0;
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], L::NSW);
            mbar_init(&pv_done[i], 1);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        mbar_init(drained, 1);
        for (int i = 0; i < L::SEGS; ++i) {
            mbar_init(&seg_full[i], 1);
            mbar_init(&seg_empty[i], 2 + L::NSW);
        }
        *abort_flag = 0;
        *odd_v = 0;
        fence_mbar_init();
        prefetch_tmap(&kmap);
        prefetch_tmap(&vmap);
    }
    if (warp == 1) {
        tmem_alloc(tslot, L::T_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = *tslot;
    pdl_wait();
    pdl_trigger();

    Segment s;
    SegmentNote* notes = reinterpret_cast<SegmentNote*>(sm + L::O_SEG);
    int sg = 0;  // segments told or taken note of
    // The next segment, from warp 0: false at the end of the CTA's range.  `ok` turns false where the wait gave up.
    auto heard = [&](bool& ok) -> bool {
        const int e = sg % L::SEGS;
        ok = wait_or_abort(&seg_full[e], (uint32_t)((sg / L::SEGS) & 1), abort_flag);
        if (!ok) return false;
        const SegmentNote n = notes[e];
        s = n.s;
        ++sg;
        return n.more != 0;
    };
    auto took_note = [&] { mbar_arrive(&seg_empty[(sg - 1) % L::SEGS]); };  // one thread per role, after heard()
    const int nslab = (a.D + 63) / 64;  // 64-dim slabs of a cache row

    // Page pieces of a tile: lane p of a loading warp takes piece p.
    const int np = TILE / piece;
    const bool two = piece <= 16;  // V has a warp of its own
    auto look_up = [&](const Segment& g, int tile, int& y, int& z) {
        const int t = tile * TILE + lane * piece;
        z = a.n_pages;  // reads as zeros
        y = 0;
        if (lane < np && t < g.len) {
            const int pg = t / a.page_size;
            const int page = a.table[(int64_t)g.b * a.max_pages + pg];
            if (page >= 0 && page < a.n_pages) z = page;
            y = g.h * a.page_size + (t - pg * a.page_size);
        }
    };
    auto load = [&](const CUtensorMap* map, const Segment& g, int tile, int y, int z, int sl) -> bool {  // into slots sl ..
        const int left = g.len - tile * TILE;
        const int have = left >= TILE ? np : (left + piece - 1) / piece;  // pieces with tokens
        for (int db = 0; db < NDB; ++db, ++sl) {
            const int st = sl % NS;
            // the slot's last load may be the other warp's, and still to come: until then the barrier's parity
            // would speak of the load before it
            if (sl >= NS && !__all_sync(0xffffffffu, loaded_or_abort(&filled[st], sl - NS + 1, abort_flag) &&
                                                         wait_or_abort(&empty[st], (uint32_t)((sl / NS - 1) & 1), abort_flag)))
                return false;
            const int slabs = nslab - 2 * db < 2 ? nslab - 2 * db : 2;
            if (lane == 0) {
                mbar_arrive_expect_tx(&full[st], (uint32_t)(have * piece * 128 * slabs));
                filled[st] = sl + 1;
            }
            __syncwarp();
            if (lane < have) {
                const uint32_t dst = smem_u32(sm) + st * SLOT + lane * piece * 128;
                for (int i = 0; i < slabs; ++i) tma_load_3d(dst + i * SLAB, map, &full[st], (2 * db + i) * 64, y, z);
            }
        }
        return true;
    };

    if (warp == 0) {
        // ------------------------------------------------ K and V
        int n_cta = gridDim.x;
        const Place place = find_place(a, TILE, blockIdx.x, n_cta);
        const bool works = (int)blockIdx.x < n_cta;
        Walk walk(place, works ? cta_begin(place.total, blockIdx.x, n_cta) : 0,
                  works ? cta_begin(place.total, blockIdx.x + 1, n_cta) : 0);
        int sl0 = 0;  // slots before
        bool ok = true, more = true;
        while (ok && more) {
            more = walk.next(a, TILE, s);
            const int e = sg % L::SEGS;
            if (sg >= L::SEGS)
                ok = __all_sync(0xffffffffu, wait_or_abort(&seg_empty[e], (uint32_t)((sg / L::SEGS - 1) & 1), abort_flag));
            if (!ok) break;
            if (lane == 0) {
                notes[e].s = s;
                notes[e].more = more;
                mbar_arrive(&seg_full[e]);
            }
            ++sg;
            const int n = more && s.len > 0 ? s.tile1 - s.tile0 : 0;
            int yv = 0, zv = 0, yk = 0, zk = 0, yn = 0, zn = 0;  // pieces of tiles j, j + 1, and j + 2 looked up ahead
            if (n > 0) look_up(s, s.tile0, yk, zk);
            for (int j = -1; ok && n > 0 && j < n; ++j) {  // K of tile j + 1, V of tile j
                if (j + 2 < n) look_up(s, s.tile0 + j + 2, yn, zn);
                if (j + 1 < n) ok = load(&kmap, s, s.tile0 + j + 1, yk, zk, sl0 + L::k_slot(j + 1));
                if (j >= 0 && !two) ok = ok && load(&vmap, s, s.tile0 + j, yv, zv, sl0 + L::v_slot(j, n));
                yv = yk;
                zv = zk;
                yk = yn;
                zk = zn;
            }
            sl0 += 2 * NDB * n;
            if (sg == 1 && lane == 0) write_join_task(a, place, walk, more ? &s : nullptr, blockIdx.x, n_cta);
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMAs (lane 0)
        if (lane == 0) {
            const uint32_t base = smem_u32(sm);
            const int ksteps = (a.D + 15) / 16;
            int it = 0, seg = 0, sl0 = 0;  // tiles, segments and slots before
            // the issue loops are unrolled and step the descriptors by constants (their address field counts 16
            // bytes): with descriptors built per MMA, one thread's issue rate, 60 ns each, was the tile's bound
            auto slot_full = [&](int k) { return wait_or_abort(&full[k % NS], (uint32_t)((k / NS) & 1), abort_flag); };
            auto issue_s = [&](int t, int k0) -> bool {  // S of the CTA's tile t, its K from slot k0 on
                for (int db = 0; db < NDB; ++db) {
                    const int k = k0 + db;
                    if (!slot_full(k)) return false;
                    tc_fence_after();
                    const int steps = ksteps - 8 * db;
                    const uint32_t ka = desc_lo(base + (k % NS) * SLOT, 16);
                    const uint32_t qa = desc_lo(base + L::O_Q + db * 2 * (N * 128), 16);
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        if (q < steps)
                            mma_lo(tb + L::T_S + (t & 1) * N, ka + (((q >> 2) * SLAB + (q & 3) * 32) >> 4),
                                     qa + (((q >> 2) * (N * 128) + (q & 3) * 32) >> 4), idesc_bf16_f32(128, N, 0, 0),
                                     db > 0 || q > 0);
                    mma_commit(&empty[k % NS]);
                }
                mma_commit(&s_full[t & 1]);
                return true;
            };
            bool ok = true;
            while (ok && heard(ok)) {
                took_note();
                if (s.len == 0) continue;
                const int n = s.tile1 - s.tile0;
                ok = wait_or_abort(q_full, (uint32_t)(seg & 1), abort_flag);
                ++seg;
                for (int j = -1; ok && j < n; ++j) {  // S of tile j + 1, then P V of tile j
                    if (j + 1 < n && !issue_s(it + (j < 0 ? 0 : 1), sl0 + L::k_slot(j + 1))) { ok = false; break; }
                    if (j + 2 == n) mma_commit(q_empty);
                    if (j < 0) continue;
                    ok = it != a.stop_at;
                    if (!ok) break;
                    ok = wait_or_abort(&p_full[it & 1], (uint32_t)((it >> 1) & 1), abort_flag);
                    if (!ok) break;
                    const int left = s.len - (s.tile0 + j) * TILE;
                    const int pk = left >= TILE ? 8 : (left + 15) / 16;  // 16-token steps with tokens
                    const int buf = L::PBUF == 2 ? it & 1 : 0;
                    for (int db = 0; db < NDB; ++db) {
                        const int k = sl0 + L::v_slot(j, n) + db;
                        if (!slot_full(k)) { ok = false; break; }
                        tc_fence_after();
                        const uint32_t va = desc_lo(base + (k % NS) * SLOT, SLAB);
#pragma unroll
                        for (int lo = 0; lo < (L::PARTS == 2 ? 1 : 2); ++lo) {
                            const uint32_t pa = desc_lo(base + L::O_P + L::p_start(buf, lo), SLAB);
#pragma unroll
                            for (int q = 0; q < 8; ++q)
                                if (q < pk)
                                    mma_lo(tb + L::T_O + db * L::PARTS * N, va + q * (2048 >> 4), pa + q * (2048 >> 4),
                                           idesc_bf16_f32(128, L::PARTS * N, 1, 1), j > 0 || lo > 0 || q > 0);
                        }
                        mma_commit(&empty[k % NS]);
                    }
                    if (!ok) break;
                    mma_commit(&pv_done[it & 1]);
                    ++it;
                }
                sl0 += 2 * NDB * n;
            }
            if (!ok) {  // MMAs that no commit above speaks of are waited for too
                mma_commit(drained);
                mbar_wait(drained, 0, kWaitNs);
            }
        }
    } else if (warp == 2) {
        // ------------------------------------------------ Q rows (zero beyond the block's rows and the head's dims), V
        int seg = 0, sl0 = 0;  // segments and slots before
        bool ok = true;
        for (;;) {
            const bool more = heard(ok);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok || !more) break;
            if (lane == 0) took_note();
            if (s.len == 0) continue;
            const int r0 = s.rb * a.rb_rows, nr = block_rows(a, s.rb), n = s.tile1 - s.tile0;
            int y = 0, z = 0, yn = 0, zn = 0;
            if (two) look_up(s, s.tile0, y, z);
            if (seg > 0) ok = __all_sync(0xffffffffu, wait_or_abort(q_empty, (uint32_t)((seg - 1) & 1), abort_flag));
            if (!ok) break;
            const uint32_t qs = smem_u32(sm) + L::O_Q;
            // 4 NDB lanes per row, 4 pieces each; a row's new token i and query head g are stepped, not divided out
            constexpr int RS = 32 / (4 * NDB);
            const int step_i = RS / a.group, step_g = RS - step_i * a.group;
            int i0 = (r0 + lane / (4 * NDB)) / a.group, g0 = r0 + lane / (4 * NDB) - i0 * a.group;
#pragma unroll 2
            for (int r = lane / (4 * NDB); r < N; r += RS) {
                const bf16* src = static_cast<const bf16*>(a.q) +
                                  (r < nr ? (((int64_t)s.b * a.K + i0) * a.H_q + s.h * a.group + g0) * a.D : 0);
                i0 += step_i;
                g0 += step_g;
                if (g0 >= a.group) {
                    g0 -= a.group;
                    ++i0;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int ch = lane % (4 * NDB) + i * 4 * NDB;  // 8 dims
                    const bool real = r < nr && ch * 8 < a.D;
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                     qs + (ch >> 3) * (N * 128) + sw128_off((uint32_t)r, (uint32_t)(ch & 7) * 8)),
                                 "l"(real ? src + ch * 8 : src), "r"(real ? 16 : 0)
                                 : "memory");
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
            ++seg;
            for (int j = 0; two && ok && j < n; ++j) {
                if (j + 1 < n) look_up(s, s.tile0 + j + 1, yn, zn);
                ok = load(&vmap, s, s.tile0 + j, y, z, sl0 + L::v_slot(j, n));
                y = yn;
                z = zn;
            }
            sl0 += 2 * NDB * n;
        }
    } else {
        // ------------------------------------------------ softmax and outputs
        constexpr int CH = L::CH;
        const int st = tid - 96;                 // softmax thread
        const int quad = warp & 3;               // its TMEM lanes: 32 quad ..
        const int row = quad * 32 + lane;        // token of a tile, head dim of an output block
        const int wg = (warp - 3) >> 2;
        const int c0 = wg * CPT;                 // its columns: c0 ..
        const uint32_t tq = tb + ((uint32_t)(quad * 32) << 16) + c0;
        float* n_s = reinterpret_cast<float*>(sm + L::O_M);     // running maxima, negative
        int* vis_s = reinterpret_cast<int*>(sm + L::O_VIS);     // tokens a row sees
        float* f_s = reinterpret_cast<float*>(sm + L::O_F);     // factors of a rescaling, 1 / l at the end
        float* scr = reinterpret_cast<float*>(sm + L::O_SCR);   // [4 lane quarters][NWG * CH]
        int it = 0, sl0 = 0;  // tiles and slots before
        bool live = true;     // no wait gave up: outputs are written only then
        auto wait = [&](uint64_t* bar, int k) {
            live = __all_sync(0xffffffffu, live && wait_or_abort(bar, (uint32_t)(k & 1), abort_flag));
        };
        // The next segment with tokens, into s; rows of empty sequences become zeros on the way.  The warps agree
        // on a wait that gave up (they meet at barriers).
        auto next_segment = [&]() -> bool {
            for (;;) {
                bool ok;
                const bool more = heard(ok);
                if (softmax_any<NSOFT>(!ok)) {
                    live = false;
                    return false;
                }
                if (!more) return false;
                if (lane == 0) took_note();
                if (s.len > 0) return true;
                const int r0 = s.rb * a.rb_rows, nr = block_rows(a, s.rb);
                for (int e = st; e < nr * a.D; e += NSOFT) {
                    const int r = e / a.D, d = e - r * a.D;
                    const int64_t at = row_index(a, s.b, s.h, r0 + r);
                    static_cast<bf16*>(a.out)[at * a.D + d] = from_f<bf16>(0.f);
                    if (d == 0 && a.lse != nullptr) a.lse[at] = -INFINITY;
                }
            }
        };
        // Sums and outputs of a segment whose last tile is handed to the MMA warp.
        auto finish_segment = [&](const Segment& s, float (&l)[CPT]) {
            const int r0 = s.rb * a.rb_rows, nr = block_rows(a, s.rb);
            const bool whole = s.tile1 - s.tile0 == s.tiles;
            // sums over the tokens: the lanes, then the warps
            join_lanes<CPT>(l, lane, [](float x, float y) { return x + y; });
            // the output loop below has this many rounds per 128 dims; the gate's values are loaded two rounds ahead
            const int rounds = (nr * 16 + NSOFT - 1) / NSOFT;
            const bool gated = whole && a.gate != nullptr;
            // row_index of the block's row c, its new token taken from what the row sees
            auto out_row = [&](int c) -> int64_t {
                const int i = vis_s[c] - s.len + a.K - 1;
                return ((int64_t)s.b * a.K + i) * a.H_q + s.h * a.group + (r0 + c - i * a.group);
            };
            auto gate_of = [&](int i) -> uint4 {
                const int db = i >= rounds ? 1 : 0, e = st + (i - db * rounds) * NSOFT, d = db * 128 + (e & 15) * 8;
                if (!gated || e >= nr * 16 || d >= a.D) return make_uint4(0u, 0u, 0u, 0u);
                return __ldg(reinterpret_cast<const uint4*>(static_cast<const bf16*>(a.gate) + out_row(e >> 4) * a.D + d));
            };
            uint4 g0 = gate_of(0), g1 = gate_of(1);
            wait(&pv_done[(it - 1) & 1], (it - 1) >> 1);  // O is done; P's memory is free
            tc_fence_after();
            // lane i now has columns 2 i and 2 i + 1 (CPT = 64), i (32) or i / 2 (16)
            float* sum_s = CPT == CH ? scr : reinterpret_cast<float*>(sm + L::O_P);  // [4 lane quarters][N]
            float* scr_w = sum_s + quad * N + c0;
            if constexpr (CPT == 64) *reinterpret_cast<float2*>(scr_w + 2 * lane) = make_float2(l[0], l[1]);
            else if (CPT == 32 || (lane & 1) == 0) scr_w[CPT == 32 ? lane : lane >> 1] = l[0];
            softmax_sync<NSOFT>();
            float* slot = slot_ptr(a, part_slot(s));
            for (int c = st; c < nr; c += NSOFT) {
                const float sum = (sum_s[c] + sum_s[N + c]) + (sum_s[2 * N + c] + sum_s[3 * N + c]);
                const float m = -n_s[c];
                f_s[c] = sum == 0.f ? 0.f : 1.0f / sum;
                if (live) {
                    if (whole) {
                        if (a.lse != nullptr)
                            a.lse[out_row(c)] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
                    } else {
                        slot[c] = sum == 0.f ? -INFINITY : m;
                        slot[a.rb_rows + c] = sum;
                    }
                }
            }
            softmax_sync<NSOFT>();
            // outputs, 128 head dims at a time: turned into rows in P's memory, then read back 8 dims at a time
            // (one thread writing its dim of every row, unrolled, spent longer on fetching code than on the rest)
            const bool odd = *odd_v != 0;
            float* o_s = reinterpret_cast<float*>(sm + L::O_P);  // [rows][128]
#pragma unroll 1
            for (int db = 0; db < NDB; ++db) {
                if (db > 0) softmax_sync<NSOFT>();
#pragma unroll 1
                for (int c = 0; c < CPT; c += CH) {
                    float o[CH];
                    const uint32_t to = tq + L::T_O + db * L::PARTS * N + c;
                    tmem_ld<CH>(to, o);
                    if constexpr (L::PARTS == 2) {
                        float o2[CH];
                        tmem_ld<CH>(to + N, o2);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < CH; ++i) o[i] += o2[i];
                    } else {
                        tmem_wait_ld();
                    }
                    if (odd && db * 128 + row < a.D) {
                        const int t1 = min(s.len, s.tile1 * TILE);
                        for (int t = max(s.tile0 * TILE, s.len - a.K + 1); t < t1; ++t) {
                            const int page = a.table[(int64_t)s.b * a.max_pages + t / a.page_size];
                            if (page < 0 || page >= a.n_pages) continue;
                            const float v = to_f(static_cast<const bf16*>(
                                a.v_cache)[(((int64_t)page * a.H_kv + s.h) * a.page_size + t % a.page_size) * a.D + db * 128 + row]);
                            if (!isfinite(v))
#pragma unroll
                                for (int i = 0; i < CH; ++i)
                                    if (t < vis_s[c0 + c + i]) o[i] += v;
                        }
                    }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < CH; ++i) o_s[(c0 + c + i) * 128 + row] = o[i];
                }
                softmax_sync<NSOFT>();
#pragma unroll 1
                for (int i = 0; i < rounds; ++i) {
                    const uint4 gv = g0;
                    g0 = g1;
                    g1 = gate_of(db * rounds + i + 2);
                    const int e = st + i * NSOFT, r = e >> 4, dd = (e & 15) * 8, d = db * 128 + dd;
                    if (r >= nr || d >= a.D || !live) continue;
                    const float4 x0 = *reinterpret_cast<const float4*>(o_s + r * 128 + dd);
                    const float4 x1 = *reinterpret_cast<const float4*>(o_s + r * 128 + dd + 4);
                    if (whole) {
                        const int64_t at = out_row(r) * a.D + d;
                        float y[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w}, gt[8];
                        const float inv = f_s[r];
                        const bool gates = gated && inv != 0.f;  // a row that sees nothing is 0 whatever its gate holds
                        unpack16<bf16>(gv, gt);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            y[i] *= inv;
                            // the approximate exponential and quotient: far below the step of bf16
                            if (gates) y[i] *= __fdividef(1.0f, 1.0f + __expf(-gt[i]));
                        }
                        store16<bf16>(static_cast<bf16*>(a.out) + at, y);
                    } else {
                        float* p = slot + a.stat_floats + r * a.D + d;
                        *reinterpret_cast<float4*>(p) = x0;
                        *reinterpret_cast<float4*>(p + 4) = x1;
                    }
                }
            }
            tc_fence_before();
        };
        alignas(8) float l[CPT];  // this token's part of the rows' sums
        for (;;) {
            // one copy of each part: the next segment, the last one's outputs, the tiles
            const Segment before = s;
            const bool more = next_segment();
            if (it > 0) finish_segment(before, l);
            if (!more) break;
            const int r0 = s.rb * a.rb_rows, nr = block_rows(a, s.rb);
            softmax_sync<NSOFT>();  // the outputs before are out of P's memory and the arrays
            for (int c = st; c < N; c += NSOFT) {
                n_s[c] = 0.f;
                vis_s[c] = c < nr ? visible(a, s.len, r0 + c) : 0;
            }
            if (st == 0) *odd_v = 0;
            softmax_sync<NSOFT>();
#pragma unroll
            for (int c = 0; c < CPT; ++c) l[c] = 0.f;
            const int least = visible(a, s.len, r0);  // what the block's first row sees
            for (int j = s.tile0; j < s.tile1; ++j, ++it) {
                const int t0 = j * TILE;
                const bool first = j == s.tile0, tail = t0 + TILE > least;
                const int buf = L::PBUF == 2 ? it & 1 : 0;
                wait(&s_full[it & 1], it >> 1);
                tc_fence_after();
#pragma unroll
                for (int c1 = 0; c1 < CPT; c1 += CH) {  // CH columns at a time
                    const uint32_t ts = tq + L::T_S + (it & 1) * N + c1;
                    float x[CH];  // scores in the log2 domain, less the running maximum
                    tmem_ld<CH>(ts, x);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < CH; c += 4) {
                        const float4 n4 = *reinterpret_cast<const float4*>(n_s + c0 + c1 + c);
                        const float2 sc = make_float2(a.scale_log2, a.scale_log2);
                        const float2 u = __ffma2_rn(make_float2(x[c], x[c + 1]), sc, make_float2(n4.x, n4.y));
                        const float2 v = __ffma2_rn(make_float2(x[c + 2], x[c + 3]), sc, make_float2(n4.z, n4.w));
                        x[c] = u.x; x[c + 1] = u.y; x[c + 2] = v.x; x[c + 3] = v.y;
                    }
                    if (tail) {
#pragma unroll
                        for (int c = 0; c < CH; ++c)
                            if (t0 + row >= vis_s[c0 + c1 + c]) x[c] = -INFINITY;
                    }
                    float top = x[0];
#pragma unroll
                    for (int c = 1; c < CH; ++c) top = fmaxf(top, x[c]);
                    if (first || group_any(wg, top > kSlack)) {
                        // ---- new maxima; sums and outputs so far are scaled to them
                        if (!first) wait(&pv_done[(it - 1) & 1], (it - 1) >> 1);
                        tc_fence_after();
                        constexpr int W = L::NWG * CH;
                        if (!first) {
                            // the scores again: less a maximum far from them, they have lost their digits
                            uint32_t hidden = 0;
#pragma unroll
                            for (int c = 0; c < CH; ++c) hidden |= (x[c] == -INFINITY ? 1u : 0u) << c;
                            tmem_ld<CH>(ts, x);
                            tmem_wait_ld();
#pragma unroll
                            for (int c = 0; c < CH; ++c) x[c] = hidden >> c & 1 ? -INFINITY : x[c] * a.scale_log2;
                        }
                        float t[CH];
#pragma unroll
                        for (int c = 0; c < CH; ++c) t[c] = x[c];
                        join_lanes<CH>(t, lane, [](float p, float q) { return fmaxf(p, q); });
                        if (CH == 32 || (lane & 1) == 0) scr[quad * W + wg * CH + (CH == 32 ? lane : lane >> 1)] = t[0];
                        group_sync(wg);
                        if ((st & 127) < CH) {
                            const int i = wg * CH + (st & 127), c = c0 + c1 + (st & 127);
                            const float m0 = -n_s[c];
                            const float t1 = fmaxf(fmaxf(scr[i], scr[W + i]), fmaxf(scr[2 * W + i], scr[3 * W + i]));
                            // rows do not move with one another; scores of -inf only leave any later one above
                            const float m1 = first ? fmaxf(t1, kNone) : t1 > m0 + kSlack ? t1 : m0;
                            n_s[c] = -m1;
                            f_s[c] = ex2_approx(m0 - m1);
                        }
                        group_sync(wg);
#pragma unroll
                        for (int c = 0; c < CH; ++c) x[c] += n_s[c0 + c1 + c];
                        if (!first) {
#pragma unroll
                            for (int c = 0; c < CH; ++c) l[c1 + c] *= f_s[c0 + c1 + c];
#pragma unroll 1
                            for (int i = 0; i < NDB * L::PARTS; ++i) {
                                float o[CH];
                                tmem_ld<CH>(tq + L::T_O + i * N + c1, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int c = 0; c < CH; ++c) o[c] *= f_s[c0 + c1 + c];
                                tmem_st<CH>(tq + L::T_O + i * N + c1, o);
                            }
                            tmem_wait_st();
                        }
                    }
                    uint32_t hi[CH / 2], lo[CH / 2];
#pragma unroll
                    for (int i = 0; i < CH / 2; ++i) {
                        const float2 p = make_float2(ex2_approx(x[2 * i]), ex2_approx(x[2 * i + 1]));
                        float2* sum = reinterpret_cast<float2*>(l + c1 + 2 * i);
                        *sum = __fadd2_rn(*sum, p);
                        const uint32_t w0 = __float_as_uint(p.x), w1 = __float_as_uint(p.y);
                        hi[i] = __byte_perm(w0, w1, 0x7632);  // the upper halves: cut, not rounded
                        // the rest, at least p's last bit: a rest of 0 would turn an infinite value into NaN
                        const float2 rest = __fadd2_rn(
                            make_float2(__uint_as_float(w0 | 1u), __uint_as_float(w1 | 1u)),
                            make_float2(__uint_as_float((w0 & 0xffff0000u) | 0x80000000u),
                                        __uint_as_float((w1 & 0xffff0000u) | 0x80000000u)));
                        lo[i] = pack_bf16x2(rest.x, rest.y);
                    }
                    if (c1 == 0 && it >= L::PBUF) wait(&pv_done[(it - L::PBUF) & 1], (it - L::PBUF) >> 1);
#pragma unroll
                    for (int c = 0; c < CH; c += 8) {
                        *reinterpret_cast<uint4*>(sm + L::O_P + L::p_off(buf, 0, (c0 + c1 + c) >> 3, row)) =
                            make_uint4(hi[c / 2], hi[c / 2 + 1], hi[c / 2 + 2], hi[c / 2 + 3]);
                        *reinterpret_cast<uint4*>(sm + L::O_P + L::p_off(buf, 1, (c0 + c1 + c) >> 3, row)) =
                            make_uint4(lo[c / 2], lo[c / 2 + 1], lo[c / 2 + 2], lo[c / 2 + 3]);
                    }
                }
                if (tail) {
                    // V rows behind the sequence's end that the MMA's last 16-token step reads become zeros
                    // (whatever lies there times a weight of 0 could be NaN); so do non-finite values of the
                    // new tokens that not all rows see -- the rows that do get them back at the end
                    const int valid = min(TILE, s.len - t0);
                    const int from = max(0, max(0, s.len - a.K + 1) - t0), upto = (valid + 15) & ~15;
#pragma unroll 1
                    for (int db = 0; db < NDB; ++db) {
                        const int k = sl0 + L::v_slot(j - s.tile0, s.tile1 - s.tile0) + db;
                        // until the slot's load is issued its barrier's parity speaks of the load before last: in a tile
                        // that is not the segment's last, the slot may still be taking in the load before (17 to 128
                        // rows of head dims above 128)
                        live = __all_sync(0xffffffffu, live && loaded_or_abort(&filled[k % NS], k + 1, abort_flag));
                        wait(&full[k % NS], k / NS);
                        const int slabs = nslab - 2 * db < 2 ? nslab - 2 * db : 2;
                        for (int e = st; e < (upto - from) * slabs * 8; e += NSOFT) {
                            const int t = from + e / (slabs * 8), rest = e % (slabs * 8);
                            uint4* p = reinterpret_cast<uint4*>(sm + (k % NS) * SLOT + (rest >> 3) * SLAB + t * 128 + (rest & 7) * 16);
                            if (t >= valid) {
                                *p = make_uint4(0u, 0u, 0u, 0u);
                            } else {
                                const uint4 v = *p;
                                if (!finite_bf16x8(v)) {
                                    *odd_v = 1;
                                    *p = make_uint4(zero_non_finite(v.x), zero_non_finite(v.y), zero_non_finite(v.z),
                                                    zero_non_finite(v.w));
                                }
                            }
                        }
                    }
                }
                fence_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[it & 1]);
            }
            sl0 += 2 * NDB * (s.tile1 - s.tile0);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && *abort_flag) {
        for (int st = 0; st < NS; ++st)  // let the copies in flight land before the CTA exits
            if (filled[st] > 0) mbar_wait(&full[st], (uint32_t)(((filled[st] - 1) / NS) & 1), kWaitNs);
        atomicOr(&g_attn_error, 1);
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tb, L::T_COLS);
    }
}

bool encode_cache(CUtensorMap* map, const void* base, const AttnArgs& a, int piece) {
    const PFN_cuTensorMapEncodeTiled_v12000 enc = tensormap_encoder();
    if (enc == nullptr) return false;
    cuuint64_t dim[3] = {(cuuint64_t)a.D, (cuuint64_t)a.H_kv * a.page_size, (cuuint64_t)a.n_pages};
    cuuint64_t str[2] = {(cuuint64_t)a.D * 2, (cuuint64_t)a.D * 2 * a.H_kv * a.page_size};
    cuuint32_t box[3] = {64, (cuuint32_t)piece, 1};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dim, str, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int N, int NDB>
cudaError_t launch_tc(const AttnArgs& a, int n_cta, int piece, cudaStream_t s) {
    using L = Layout<N, NDB>;
    CUtensorMap km, vm;
    if (!encode_cache(&km, a.k_cache, a, piece) || !encode_cache(&vm, a.v_cache, a, piece)) return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(attn_tc_kernel<N, NDB>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM);
    if (e != cudaSuccess) return e;
    return launch_pdl(attn_tc_kernel<N, NDB>, dim3((unsigned)n_cta), dim3(L::NT), L::SMEM, s, km, vm, a, piece);
}

template <int NDB>
cudaError_t launch_rows(const AttnArgs& a, int n_cta, int piece, cudaStream_t s) {
    return a.rb_rows <= 16 ? launch_tc<16, NDB>(a, n_cta, piece, s)
         : a.rb_rows <= 32 ? launch_tc<32, NDB>(a, n_cta, piece, s)
         : a.rb_rows <= 64 ? launch_tc<64, NDB>(a, n_cta, piece, s) : launch_tc<128, NDB>(a, n_cta, piece, s);
}

// Rows of a page that one TMA box takes: the largest power of two that divides the page size, a tile at most.
int page_piece(int page_size) {
    const int p = page_size & -page_size;
    return p < TILE ? p : TILE;
}

}  // namespace

bool attn_tc_takes(const AttnArgs& a, gdn_dtype_t dt) {
    // a lane loads one piece: 32 pieces of 4 tokens make a tile
    return dt == GDN_BF16 && page_piece(a.page_size) >= TILE / 32;
}

cudaError_t launch_attn_tc(const AttnArgs& a, int n_cta, cudaStream_t s) {
    const int piece = page_piece(a.page_size);
    const cudaError_t e = a.D <= 128 ? launch_rows<1>(a, n_cta, piece, s) : launch_rows<2>(a, n_cta, piece, s);
    return e != cudaSuccess ? e : launch_attn_join(a, n_cta, GDN_BF16, s);
}

cudaError_t read_and_clear_attn_error(cudaStream_t s, int* flags) {
    int hf = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&hf, g_attn_error, sizeof(int), 0, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return e;
    *flags = hf;
    if (hf != 0) {
        const int zero = 0;
        e = cudaMemcpyToSymbolAsync(g_attn_error, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s);
        if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    }
    return e;
}

}  // namespace gdn
