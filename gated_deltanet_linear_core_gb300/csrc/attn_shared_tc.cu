// Attention behind shared prefixes on tcgen05 tensor cores (bf16): the query rows that
// share a key-value head and a page table, 128 at a time, over tiles of 128 cached tokens.
//
// With hundreds of rows per cached token the products are the bound, not the
// cache, so the query rows are the M = 128 side of the MMAs and the tokens the N side:
//   S [128 rows x 128 tokens] = Q K^T    (Q and K tile in shared memory, both K-major)
//   O [128 rows x D]         += P V      (P in tensor memory, V tile in shared memory, MN-major)
// (attn_tc.cu has the tokens on the M side, for at most 128 rows per cached token.)  What a sequence
// has of its own runs through the same loop with few real rows: its tiles are bound by their
// loads all the same, and a launch of attn_tc.cu's kernel beside it took 15 to 37 us.
//
// A softmax thread owns half a row of a tile (64 tokens), so maxima and sums need no exchange
// between lanes, and P goes back into the columns of S that it came from.  A row's running
// maximum is moved only when scores far above it make the weights' sum large, which the two
// warps that share rows vote on; O is rescaled then.  P is held as two bf16 (the value cut
// to 8 bits and the rounded rest), as in attn_tc.cu: one alone would add an error of the size
// of the output's own rounding, and without the second the call takes 7 % less.  S runs one
// tile ahead of P V (two up to head dim 128), so the weights of a tile are made beside the products of another.
//
// Measured: 32 sequences with 16 new tokens (4096 rows per head, head dim 128) behind 16384 tokens 156 us a call, 147 of them
// (cold, alone) this kernel, some 2250 clocks a tile where its MMAs take 1540 (the softmax, 1630 clocks a tile, half of them
// waits that its 8 warps spend together, and the hand-overs); 64 sequences behind 32768 tokens (512 rows, head dim 256)
// 64 us a call, 58 (cold) this kernel: 18 tiles and 1.7 segments per CTA, of which the MMAs take 28.  Tried, no faster: the warpgroups on tiles in turns (164 and 76 us per call for 152 and 65),
// waits that sleep longer or poll, no search for the maximum.
//
// Warps: 0 walks the CTA's range, tells the others its segments, and loads K and V (of
// every page piece the first 64 of 128 dims; warp 3 the others), 1 issues the MMAs,
// 4 to 11 load Q and are the softmax (2 only fills the warpgroup).  Every wait is bounded
// (1 s): on a timeout the roles run out without waiting, the copies in flight land, TMEM is
// freed and the error word is set.
#include "attn_shared.cuh"
#include "attn_tc_common.cuh"

namespace gdn {

__device__ int g_shared_error;  // bit 0: a bounded wait gave up

namespace {

using namespace attn;

constexpr int ROWS = 128;
constexpr int NT = 384;
constexpr int NSOFT = 256;
// Half a tile's weights of a row add up to more than this where its running maximum is to be moved.  (The sum is there
// anyway; looking for the largest score in each tile took a fifth of the arithmetic.)
constexpr float kLarge = 4096.0f;
// Scores of this size (log2) and beyond are a unit or more off by their own rounding, and so is a maximum of them: less it
// in one multiply-add, scores as large as it would come out anywhere.  Rows with such a maximum take their scores rounded
// as it is, at every tile.  (us before and with this: 64 sequences behind 32768 tokens 65.1, 64.4, 32 with 16 new tokens
// behind 16384 154.4, 157.0; forms with fewer instructions per tile moved the two by as much, by the compiler's schedule.)
constexpr float kHuge = 0x1p24f;

template <int NDB>
struct Layout {
    static constexpr int Q_BYTES = 2 * NDB * SLAB;     // at a segment's end 4 KB per softmax warp for turning outputs into rows
    static constexpr int SMALL = 1024 + 4 * ROWS * 4;  // barriers and notes, the rows' maxima and sums
    static constexpr int FIT = (kSmemMax - Q_BYTES - SMALL) / SLOT;
    static constexpr int NS = FIT < 6 ? FIT : 6;
    static constexpr int O_Q = NS * SLOT;
    static constexpr int O_BAR = O_Q + Q_BYTES;
    static constexpr int O_SEG = O_BAR + 512;
    static constexpr int O_M = O_BAR + 1024;
    static constexpr int O_L = O_M + 2 * ROWS * 4;
    static constexpr int SMEM = O_BAR + SMALL;
    // Tensor memory: buffers of S, then O.  S runs NB - 1 tiles ahead: with three buffers the scores of a tile wait
    // while the weights of the one before are made (two leave no room for that, but D > 128 has twice the MMAs per tile).
    static constexpr int NB = NDB == 1 ? 3 : 2, AHEAD = NB - 1;
    static constexpr int T_S = 0, T_O = 512 - 128 * NDB, T_COLS = 512;
    static constexpr int SEGS = 4;  // segments told ahead
    static_assert(SMEM <= kSmemMax && NS >= 4 && NB * TILE <= T_O && 8 * 4096 <= Q_BYTES, "memory");
};
static_assert(4 * sizeof(SharedSegment) <= 512, "notes");

// D += A B with A in tensor memory (two bf16 per column), B by its descriptor's low word.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
    constexpr uint32_t hi = (1024u >> 4) | (1u << 14) | (2u << 29);
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
        "mov.b64 db, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(hi)
        : "memory");
}
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}"
        : "=r"(r)
        :
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ bool softmax_any(bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, 256, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x)
        : "memory");
    return r != 0;
}

// The two warps that share rows (named barriers 2 to 5).
__device__ __forceinline__ void pair_sync(int quad) { asm volatile("bar.sync %0, 64;" ::"r"(2 + quad) : "memory"); }
__device__ __forceinline__ bool pair_any(int quad, bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, 64, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x), "r"(2 + quad)
        : "memory");
    return r != 0;
}

template <int NDB, bool FEW>
__global__ void __launch_bounds__(NT, 1)
attn_shared_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, ShareArgs s,
                      int piece) {
    using L = Layout<NDB>;
    constexpr int NS = L::NS;
    extern __shared__ __align__(1024) uint8_t sm[];
    const AttnArgs& a = s.a;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::O_BAR);
    uint64_t* full = bars;            // [6] slot landed (TMA), told by both loading warps
    uint64_t* empty = bars + 6;       // [6] slot consumed (commit)
    uint64_t* s_full = bars + 12;     // [3] S of a tile done
    uint64_t* p_full = bars + 15;     // [3] P of a tile written (softmax warps)
    uint64_t* pv_done = bars + 18;    // [3] P V of a tile done (where S runs two tiles ahead of P V, a softmax warp can be
                                      // two tiles past the last P V: with two barriers it would take one phase for another)
    uint64_t* q_full = bars + 21;     // a segment's Q written (softmax warps)
    uint64_t* seg_full = bars + 22;   // [4] a segment is told
    uint64_t* seg_empty = bars + 26;  // [4] ... and taken note of
    uint64_t* drained = bars + 36;    // every MMA issued is done (abort)
    uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + 37);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
    volatile int* filled = reinterpret_cast<volatile int*>(bars + 38);  // [2 loading warps][6] loads into a slot
    volatile int* odd_v = reinterpret_cast<volatile int*>(bars + 44);   // a new token's value is not finite
    SharedSegment* notes = reinterpret_cast<SharedSegment*>(sm + L::O_SEG);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < 6; ++i) {
            mbar_init(&full[i], 2);
            mbar_init(&empty[i], 1);
            filled[i] = filled[6 + i] = 0;
        }
        for (int i = 0; i < 3; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], NSOFT / 32);
            mbar_init(&pv_done[i], 1);
        }
        mbar_init(q_full, NSOFT / 32);
        mbar_init(drained, 1);
        for (int i = 0; i < L::SEGS; ++i) {
            mbar_init(&seg_full[i], 1);
            mbar_init(&seg_empty[i], 2 + NSOFT / 32);
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

    SharedSegment g;
    int sg = 0;  // segments told or taken note of
    // The next segment, from warp 0: false at the end of the CTA's range.  `ok` turns false where the wait gave up.
    auto heard = [&](bool& ok) -> bool {
        ok = wait_or_abort(&seg_full[sg % L::SEGS], (uint32_t)((sg / L::SEGS) & 1), abort_flag);
        if (!ok) return false;
        g = notes[sg % L::SEGS];
        ++sg;
        return g.tile1 > 0;
    };
    auto took_note = [&] { mbar_arrive(&seg_empty[(sg - 1) % L::SEGS]); };  // one thread per warp, after heard()
    const int nslab = (a.D + 63) / 64;  // 64-dim slabs of a cache row

    // K and V of segment g, slab 0 or 1 of every 128 dims; lane p takes page piece p.
    const int np = TILE / piece;
    auto look_up = [&](int tile, int& y, int& z) {
        z = a.n_pages;  // reads as zeros
        y = 0;
        const int t = tile * TILE + lane * piece;
        if (lane < np && (g.len == 0 || t < g.len)) {
            const int pg = t / a.page_size;
            const int page = a.table[(int64_t)g.leader * a.max_pages + pg];
            if (page >= 0 && page < a.n_pages) z = page;
            y = g.h * a.page_size + (t - pg * a.page_size);
        }
    };
    int slot_in = 0, loads = 0;  // the slot that is filled next, how often all were
    auto load = [&](const CUtensorMap* map, int which, int y, int z) -> bool {  // into the next NDB slots
#pragma unroll
        for (int db = 0; db < NDB; ++db) {
            const int st = slot_in;
            if (loads > 0 && !__all_sync(0xffffffffu, wait_or_abort(&empty[st], (uint32_t)((loads - 1) & 1), abort_flag)))
                return false;
            const int slab = 2 * db + which;
            const bool real = slab < nslab;
            if (lane == 0) {
                if (real) mbar_arrive_expect_tx(&full[st], SLAB); else mbar_arrive(&full[st]);
                filled[6 * which + st] = loads + 1;
            }
            __syncwarp();
            if (real && lane < np)
                tma_load_3d(smem_u32(sm) + st * SLOT + which * SLAB + lane * piece * 128, map, &full[st], slab * 64, y, z);
            if (++slot_in == NS) {
                slot_in = 0;
                ++loads;
            }
        }
        return true;
    };
    // K of a segment's first tiles, then K of tile j + AHEAD and V of tile j: the order in which the MMAs use them
    auto load_segment = [&](int which) -> bool {
        const int n = g.tile1 - g.tile0;
        int y[L::AHEAD + 2], z[L::AHEAD + 2];  // pieces of tiles j .. j + AHEAD, and of the next one, looked up ahead
        look_up(g.tile0, y[L::AHEAD], z[L::AHEAD]);
        bool ok = true;
        for (int j = -L::AHEAD; ok && j < n; ++j) {
            const int t = j + L::AHEAD;
            if (t + 1 < n) look_up(g.tile0 + t + 1, y[L::AHEAD + 1], z[L::AHEAD + 1]);
            if (t < n) ok = load(&kmap, which, y[L::AHEAD], z[L::AHEAD]);
            if (j >= 0) ok = ok && load(&vmap, which, y[0], z[0]);
#pragma unroll
            for (int i = 0; i <= L::AHEAD; ++i) {
                y[i] = y[i + 1];
                z[i] = z[i + 1];
            }
        }
        return ok;
    };

    if (warp == 0) {
        // ------------------------------------------------ the walk; K and V, lower slabs
        SharedWalk<FEW> walk(s, blockIdx.x, gridDim.x);
        bool ok = true, more = true;
        while (ok && more) {
            g.tile0 = g.tile1 = 0;
            more = walk.next(s, g);
            const int e = sg % L::SEGS;
            if (sg >= L::SEGS)
                ok = __all_sync(0xffffffffu, wait_or_abort(&seg_empty[e], (uint32_t)((sg / L::SEGS - 1) & 1), abort_flag));
            if (!ok) break;
            if (lane == 0) {
                notes[e] = g;
                mbar_arrive(&seg_full[e]);
            }
            ++sg;
            if (more) ok = load_segment(0);
        }
    } else if (warp == 3) {
        // ------------------------------------------------ K and V, upper slabs
        bool ok = true;
        for (;;) {
            const bool more = heard(ok);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok || !more) break;
            if (lane == 0) took_note();
            ok = load_segment(1);
            if (!ok) break;
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMAs
        // The whole warp runs the loop and one elected lane waits and issues: with addresses that are constants but for the
        // slot and the buffer (the allocation is all of tensor memory, so it starts at 0), an MMA costs few instructions,
        // which the warp has to get past two busy softmax warps of its scheduler.
        const uint32_t base = smem_u32(sm);
        const int ksteps = (a.D + 15) / 16;
        int it = 0, seg = 0;        // tiles and segments before
        int slot = 0;               // slots are used in the order they are filled
        uint32_t phase = 0;
        int sb = 0, pb = 0;         // the buffers of the next S, of the next P
        uint32_t p_phase = 0;
        auto slot_done = [&](int& sl, uint32_t& ph) {
            if (++sl == NS) {
                sl = 0;
                ph ^= 1;
            }
        };
        bool ok = true;
        for (;;) {
            const bool more = heard(ok);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok || !more) break;
            if (lane == 0) took_note();
            const int n = g.tile1 - g.tile0;
            ok = __all_sync(0xffffffffu, wait_or_abort(q_full, (uint32_t)(seg & 1), abort_flag));
            ++seg;
            for (int j = -L::AHEAD; ok && j < n; ++j) {
                // S of tile j + AHEAD, then P V of tile j (that S overwrites P of an earlier tile, whose P V has been issued
                // before it: MMAs of one thread and shape run in order)
                const bool has_s = j + L::AHEAD < n, has_pv = j >= 0;
                if (elect_one()) {
                    int sl = slot;
                    uint32_t ph = phase;
                    if (has_s) {
#pragma unroll
                        for (int db = 0; db < NDB; ++db) {
                            ok = ok && wait_or_abort(&full[sl], ph, abort_flag);
                            if (!ok) break;
                            tc_fence_after();
                            const uint32_t ka = desc_lo(base + sl * SLOT, 16), qa = desc_lo(base + L::O_Q + db * SLOT, 16);
                            const uint32_t d = L::T_S + sb * TILE;
#pragma unroll
                            for (int q = 0; q < 8; ++q)
                                if (8 * db + q < ksteps)
                                    mma_lo(d, qa + (((q >> 2) * SLAB + (q & 3) * 32) >> 4),
                                           ka + (((q >> 2) * SLAB + (q & 3) * 32) >> 4), idesc_bf16_f32(ROWS, TILE, 0, 0),
                                           db > 0 || q > 0);
                            mma_commit(&empty[sl]);
                            if (db + 1 == NDB) mma_commit(&s_full[sb]);
                            slot_done(sl, ph);
                        }
                    }
                    if (has_pv) {
                        ok = ok && it != a.stop_at && wait_or_abort(&p_full[pb], p_phase, abort_flag);
#pragma unroll
                        for (int db = 0; db < NDB; ++db) {
                            ok = ok && wait_or_abort(&full[sl], ph, abort_flag);
                            if (!ok) break;
                            tc_fence_after();
                            const uint32_t va = desc_lo(base + sl * SLOT, SLAB);
                            const uint32_t pa = L::T_S + pb * TILE;
#pragma unroll
                            for (int q = 0; q < 8; ++q)  // 16 tokens: columns 8 (q % 2) of block q / 2's upper parts, then of its rests
#pragma unroll
                                for (int lo = 0; lo < 2; ++lo)
                                    mma_ts(L::T_O + db * 128, pa + (q >> 1) * 32 + lo * 16 + (q & 1) * 8, va + q * (2048 >> 4),
                                           idesc_bf16_f32(ROWS, 128, 0, 1), j > 0 || lo > 0 || q > 0);
                            mma_commit(&empty[sl]);
                            if (db + 1 == NDB) mma_commit(&pv_done[pb]);
                            slot_done(sl, ph);
                        }
                    }
                }
                ok = __all_sync(0xffffffffu, ok);
                if (has_s) {
                    sb = sb + 1 == L::NB ? 0 : sb + 1;
#pragma unroll
                    for (int db = 0; db < NDB; ++db) slot_done(slot, phase);
                }
                if (has_pv) {
#pragma unroll
                    for (int db = 0; db < NDB; ++db) slot_done(slot, phase);
                    ++it;
                    if (++pb == L::NB) {
                        pb = 0;
                        p_phase ^= 1;
                    }
                }
            }
            if (!ok) break;
        }
        if (!ok) {  // MMAs that no commit above speaks of are waited for too
            if (elect_one()) mma_commit(drained);
            __syncwarp();
            mbar_wait(drained, 0, kWaitNs);
        }
    } else if (warp >= 4) {
        // ------------------------------------------------ Q, softmax and outputs
        const int wg = (warp - 4) >> 2, quad = warp & 3;
        const int row = quad * 32 + lane;  // TMEM lane
        const uint32_t tq = tb + ((uint32_t)(quad * 32) << 16);
        float* t_s = reinterpret_cast<float*>(sm + L::O_M);  // [2][128] the warpgroups' maxima of a tile
        float* l_s = reinterpret_cast<float*>(sm + L::O_L);  // [2][128] ... and sums
        const int st = tid - 128;  // softmax thread
        int sl0 = 0;               // slots filled for the segments before
        int sb = 0;        // buffer of the next S
        uint32_t s_phase = 0;
        int last = 0;      // the buffer of the last tile
        uint32_t last_phase = 0;
        bool live = true;  // no wait gave up: outputs are written only then
        auto wait = [&](uint64_t* bar, int k) {
            live = __all_sync(0xffffffffu, live && wait_or_abort(bar, (uint32_t)(k & 1), abort_flag));
        };
        // V rows behind the sequence's end become zeros (whatever lies there times a weight of 0 could be NaN); so do
        // non-finite values of the new tokens that not all rows see: the rows that do get them back at the end.
        auto mend_v = [&](int j, int n, int t0) {
            const int valid = min(TILE, g.len - t0), from = max(0, g.len - a.K + 1 - t0);
#pragma unroll 1
            for (int db = 0; db < NDB; ++db) {
                const int k = sl0 + (min(j + L::AHEAD + 1, n) + j) * NDB + db, slot = k % NS, nth = k / NS;
                // until a slot's load is issued its barrier's parity speaks of the load before last
                live = __all_sync(0xffffffffu, live && loaded_or_abort(&filled[slot], nth + 1, abort_flag) &&
                                                   loaded_or_abort(&filled[6 + slot], nth + 1, abort_flag));
                wait(&full[slot], nth);
                const int slabs = min(2, nslab - 2 * db);
                for (int e = st; e < (TILE - from) * slabs * 8; e += NSOFT) {
                    const int t = from + e / (slabs * 8), rest = e % (slabs * 8);
                    uint4* p = reinterpret_cast<uint4*>(sm + slot * SLOT + (rest >> 3) * SLAB + t * 128 + (rest & 7) * 16);
                    if (t >= valid) {
                        *p = make_uint4(0u, 0u, 0u, 0u);
                    } else {
                        const uint4 v = *p;
                        if (!finite_bf16x8(v)) {
                            *odd_v = 1;
                            *p = make_uint4(zero_non_finite(v.x), zero_non_finite(v.y), zero_non_finite(v.z), zero_non_finite(v.w));
                        }
                    }
                }
            }
        };
        for (;;) {
            bool ok;
            const bool more = heard(ok);
            if (softmax_any(!ok)) {  // the warps agree on a wait that gave up: they meet at barriers
                live = false;
                break;
            }
            if (!more) break;
            if (lane == 0) took_note();
            // ---- Q (zero beyond the block's rows and the head's dims): a warp copies 16 rows
            int64_t at = -1;  // a lane finds a row's elements
            if (lane < 16 && (warp - 4) * 16 + lane < g.nr)
                at = shared_row(a, g.seq0, g.h, g.r0 + (warp - 4) * 16 + lane) * a.D;
            constexpr int CH = 16 * NDB;  // pieces of 8 dims per row
#pragma unroll 4
            for (int e = lane; e < 16 * CH; e += 32) {
                const int r = e / CH, ch = e % CH;
                const int64_t from = __shfl_sync(0xffffffffu, at, r);
                const bool real = from >= 0 && ch * 8 < a.D;
                const bf16* src = static_cast<const bf16*>(a.q) + (real ? from + ch * 8 : 0);
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                 smem_u32(sm) + L::O_Q + (ch >> 3) * SLAB +
                                 sw128_off((uint32_t)((warp - 4) * 16 + r), (uint32_t)(ch & 7) * 8)),
                             "l"(src), "r"(real ? 16 : 0)
                             : "memory");
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
            const int n = g.tile1 - g.tile0;
            const bool works = quad * 32 < g.nr;  // else none of the warp's rows are real: its P and O may be anything
            // tokens that the row sees, and that the sequence's first new token does
            const int vis = g.len > 0 ? g.len - (a.K - 1 - (g.r0 + row) / a.group) : 0, least = g.len - (a.K - 1);
            float m = kNone;                      // the row's running maximum
            float2 l = make_float2(0.f, 0.f);     // the sum of this warpgroup's tokens
            bool plain = true;                    // none of the warp's rows has a huge maximum
            for (int j = 0; j < n; ++j) {
                const uint32_t ts = tq + L::T_S + sb * TILE + wg * 64;
                wait(&s_full[sb], s_phase);
                tc_fence_after();
                const int t0 = (g.tile0 + j) * TILE;
                const bool tail = g.len > 0 && t0 + TILE > least;
                if (works) {
                    float w[64];  // of every 32 tokens 16 columns of upper parts, 16 of rests
                    float2 sum;
                    for (bool fits = j > 0 && plain;;) {
                        float x[64];
                        tmem_ld64(ts, x);
                        if (tail) {
                            const int upto = vis - (t0 + wg * 64);
#pragma unroll
                            for (int i = 0; i < 64; ++i)
                                if (i >= upto) x[i] = -INFINITY;
                        }
                        const bool sure = !fits;
                        if (!fits) {
                            // ---- new maxima; sums and outputs so far are scaled to them
                            float top = x[0];
#pragma unroll
                            for (int i = 1; i < 64; ++i) top = fmaxf(top, x[i]);
                            t_s[wg * ROWS + row] = top;
                            pair_sync(quad);
                            const float t = fmaxf(top, t_s[(wg ^ 1) * ROWS + row]) * a.scale_log2;
                            const float m1 = t > m + kSlack ? t : m;  // rows do not move with one another
                            const float f = ex2_approx(m - m1);
                            m = m1;
                            l.x *= f;
                            l.y *= f;
                            plain = !__any_sync(0xffffffffu, fabsf(m) >= kHuge);  // (the same in the other warp)
                            if (!plain) {
                                l_s[wg * ROWS + row] = m;
                                if (fabsf(m) >= kHuge) {
                                    const float inv = 1.0f / a.scale_log2;
#pragma unroll
                                    for (int i = 0; i < 64; ++i) x[i] = (__fmul_rn(x[i], a.scale_log2) - m) * inv;
                                    m = 0.f;  // until the weights are made
                                }
                            }
                            if (j > 0) {
                                wait(&pv_done[last], last_phase);
                                tc_fence_after();
#pragma unroll 1
                                for (int c = wg * 64 * NDB; c < (wg + 1) * 64 * NDB; c += 32) {
                                    float o[32];
                                    tmem_ld32(tq + L::T_O + c, o);
#pragma unroll
                                    for (int i = 0; i < 32; ++i) o[i] *= f;
                                    tmem_st32(tq + L::T_O + c, o);
                                }
                            }
                            fits = true;
                        }
                        sum = make_float2(0.f, 0.f);
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float2 y = __ffma2_rn(make_float2(x[2 * i], x[2 * i + 1]),
                                                        make_float2(a.scale_log2, a.scale_log2), make_float2(-m, -m));
                            const float2 p = make_float2(ex2_approx(y.x), ex2_approx(y.y));
                            sum = __fadd2_rn(sum, p);
                            const uint32_t w0 = __float_as_uint(p.x), w1 = __float_as_uint(p.y);
                            // the upper halves: cut, not rounded
                            w[(i & 16) * 2 + (i & 15)] = __uint_as_float(__byte_perm(w0, w1, 0x7632));
                            // the rest, and p's last bit: a rest of 0 would turn an infinite value into NaN
                            const float2 rest = __ffma2_rn(p, make_float2(1.0f + 0x1p-23f, 1.0f + 0x1p-23f),
                                                           make_float2(__uint_as_float((w0 & 0xffff0000u) | 0x80000000u),
                                                                       __uint_as_float((w1 & 0xffff0000u) | 0x80000000u)));
                            w[(i & 16) * 2 + 16 + (i & 15)] = __uint_as_float(pack_bf16x2(rest.x, rest.y));
                        }
                        if (sure || !pair_any(quad, sum.x + sum.y > kLarge)) break;
                        fits = false;
                    }
                    if (!plain) m = l_s[wg * ROWS + row];
                    l = __fadd2_rn(l, sum);
                    tmem_st32(ts, w);
                    tmem_st32(ts + 32, w + 32);
                    tmem_wait_st();
                }
                if (tail) {
                    mend_v(j, n, t0);
                    fence_async_smem();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[sb]);
                last = sb;
                last_phase = s_phase;
                if (++sb == L::NB) {
                    sb = 0;
                    s_phase ^= 1;
                }
            }
            sl0 += 2 * NDB * n;
            // ---- sums and outputs of the segment
            l_s[wg * ROWS + row] = l.x + l.y;
            wait(&pv_done[last], last_phase);
            tc_fence_after();
            softmax_sync();
            const float sum = l_s[row] + l_s[ROWS + row];
            const bool odd = *odd_v != 0;
            const bool real = row < g.nr && live;
            float *po = nullptr, *slot = shared_slot(s, blockIdx.x);
            if (g.parts > 0) {
                if (real) {
                    const int64_t to = shared_row(a, g.seq0, g.h, g.r0 + row);
                    po = (g.len > 0 ? a.part_o : s.pre_o) + to * a.D;
                    if (wg == 0) (g.len > 0 ? a.part_stat : s.pre_stat)[to] = part_stat(m, sum, g.parts, row);
                }
            } else if (real) {
                po = slot + 2 * ROWS + row * a.D;
                if (wg == 0) {
                    slot[row] = sum == 0.f ? -INFINITY : m;
                    slot[ROWS + row] = sum;
                }
            }
            // outputs, 32 columns at a time, turned in Q's memory so that 8 lanes write 128 bytes of a row (a lane per
            // row touches 32 lines at each store: 13 us a segment of head dim 256)
            float4* o_s = reinterpret_cast<float4*>(sm + L::O_Q + (warp - 4) * 4096);
#pragma unroll 1
            for (int c = wg * 64 * NDB; works && c < (wg + 1) * 64 * NDB && c < a.D; c += 32) {
                float o[32];
                tmem_ld32(tq + L::T_O + c, o);
                if (odd) {
                    const int upto = min(min(g.len, g.tile1 * TILE), vis);
#pragma unroll 1
                    for (int t = max(g.tile0 * TILE, least); t < upto; ++t) {
                        const int page = a.table[(int64_t)g.leader * a.max_pages + t / a.page_size];
                        if (page < 0 || page >= a.n_pages) continue;
                        const bf16* src = static_cast<const bf16*>(a.v_cache) +
                                          (((int64_t)page * a.H_kv + g.h) * a.page_size + t % a.page_size) * a.D + c;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (c + i < a.D && !isfinite(to_f(src[i]))) o[i] += to_f(src[i]);
                    }
                    __syncwarp();
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    o_s[lane * 8 + (i ^ (lane & 7))] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r = 4 * i + (lane >> 3), d = c + (lane & 7) * 4;
                    float* to = reinterpret_cast<float*>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(po), r));
                    const float4 v = o_s[r * 8 + ((lane & 7) ^ (r & 7))];
                    if (to != nullptr && d < a.D) *reinterpret_cast<float4*>(to + d) = v;
                }
                __syncwarp();
            }
            tc_fence_before();
            softmax_sync();  // O, the sums and the flag are free
            // (every warp has read the flag; none sets it again before it has met this thread at the next segment's barrier)
            if (st == 0) *odd_v = 0;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && *abort_flag) {
        for (int st = 0; st < NS; ++st) {  // let the copies in flight land before the CTA exits
            const int n0 = filled[st], n1 = filled[6 + st];
            if (n0 != n1) mbar_arrive(&full[st]);  // for the loading warp that gave up before this load
            const int n = n0 > n1 ? n0 : n1;
            if (n > 0) mbar_wait(&full[st], (uint32_t)((n - 1) & 1), kWaitNs);
        }
        atomicOr(&g_shared_error, 1);
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tb, L::T_COLS);
    }
}

template <int NDB, bool FEW>
cudaError_t launch_ndb(const ShareArgs& s, int n_cta, int piece, cudaStream_t st) {
    using L = Layout<NDB>;
    CUtensorMap km, vm;
    if (!encode_cache(&km, s.a.k_cache, s.a, piece) || !encode_cache(&vm, s.a.v_cache, s.a, piece)) return cudaErrorInvalidValue;
    const cudaError_t e = cudaFuncSetAttribute(attn_shared_tc_kernel<NDB, FEW>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM);
    if (e != cudaSuccess) return e;
    return launch_pdl(attn_shared_tc_kernel<NDB, FEW>, dim3((unsigned)n_cta), dim3(NT), L::SMEM, st, km, vm, s, piece);
}

}  // namespace

cudaError_t launch_shared_tc(const ShareArgs& s, int n_cta, cudaStream_t st) {
    const int piece = page_piece(s.a.page_size);
    if (s.few) return s.a.D <= 128 ? launch_ndb<1, true>(s, n_cta, piece, st) : launch_ndb<2, true>(s, n_cta, piece, st);
    return s.a.D <= 128 ? launch_ndb<1, false>(s, n_cta, piece, st) : launch_ndb<2, false>(s, n_cta, piece, st);
}

cudaError_t copy_shared_error(cudaStream_t s, int* word) {
    return cudaMemcpyFromSymbolAsync(word, g_shared_error, sizeof(int), 0, cudaMemcpyDeviceToHost, s);
}
cudaError_t clear_shared_error(cudaStream_t s) {
    const int zero = 0;
    return cudaMemcpyToSymbolAsync(g_shared_error, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s);
}

}  // namespace gdn
