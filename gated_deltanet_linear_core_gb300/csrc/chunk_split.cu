// Chunked gated delta rule in two tcgen05 kernels.
//
// The result is that of the per-token rule of the cortex commit "feat(stage-8c):
// linear-attention layer (Qwen3-Next GatedDeltaNet)", "Delta rule (recurrent,
// per-token)", computed with the chunked algorithm (chunk_size=64) its
// "Performance note" names; NxD-Inference PR "Add Qwen3.6-27B hybrid
// DeltaNet/GQA contrib model and vLLM serving path": chunked context encoding,
// recurrent-state checkpoints, and its "Known limitations": the direct solve,
// with the Neumann-style product as the alternative (GDN_SOLVE_NEUMANN).
//
// Of the per-chunk work only two products depend on the state S carried from
// chunk to chunk.  With G the chunk-local cumulative decay, rq / rk the
// l2-norm factors of raw q / k rows and T' = (I + A)^-1:
//   intra (independent per chunk, all chunks of all heads in parallel):
//     D1 = [K; Q] K^T,  A = beta rk e^{G_i-G_j} rk k.k (j<i),  P = rq e^{G_i-G_j} rk q.k (j<=i)
//     W^T = (diag(beta e^G rk) K)^T T'^T,  U^T = (diag(beta) V)^T T'^T,
//     K_dec = diag(e^{G_n-G_j} rk) K
//     -> workspace: W (bf16), U, P, K_dec (fp16) and e^G rq, e^{G_n} (f32)
//   chain (sequential per sequence and value head):
//     U' = U - W S;  O = diag(e^G rq) (Q S) + P U';  S <- e^{G_n} S + K_dec^T U'
// Precision: the operands the kernels form for the products of the state
// update and of P U' -- T', K_dec, U' -- are fp16 (11 significant bits
// against bf16's 8, at the same MMA rate), and so are K and V, scaled by
// their row factors, where they meet T' in the intra kernel (re-encoded in
// shared memory); the products with the raw bf16 q (D1, [Q; W] S) stay bf16.  This keeps the state's rounding error well inside the bf16
// tolerance when decay is slow and the state carries across many chunks.
// The intra kernel can also compute the layer's conv1d + SiLU itself (cortex
// "Block": depthwise causal conv, k = 4, then SiLU): it then loads raw x tiles
// with their 3-token halo, convolves them in place in shared memory with the
// conv kernel's own arithmetic (so y is the same bit for bit), and stores the
// conv'd q tile of each key head to the workspace for the chain; y never goes
// to HBM.
// The chunks of a call are processed in segments (a range of chunk indices
// over all sequences) whose intermediates fit in the workspace and, at the
// default size, in L2; the state crosses segments through final_state (or a
// workspace carry).  Every wait is bounded (1 s); a CTA that gives up sets
// the device error word, lets its copies land, frees its TMEM and returns.
#include <cudaTypedefs.h>

#include <mutex>

#include "chunk_common.cuh"
#include "gdn_launch.h"

namespace gdn {

__device__ int g_device_error;  // bit 0: a bounded wait gave up

namespace {

using namespace tc;
typedef __half f16;

constexpr int C = 64;

// Tokens per chunk: C, or 16 or 32 (GDN_CHUNK).  The kernels' tiles stay C rows;
// a shorter chunk fills the first rows of its tile, as a partial chunk does.
__host__ __device__ __forceinline__ int chunk_len(const DeltaArgs& a) {
    return a.chunk == 16 || a.chunk == 32 ? a.chunk : C;
}
constexpr int D = 128;
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr size_t kSegBytes = 1024ull << 20;  // workspace intermediates per segment

// per (chunk, value head) unit in the workspace
constexpr size_t U_WT = 16384, U_UT = 16384, U_P = 8192, U_VEC = 1024, U_KD = 16384;
constexpr size_t UNIT_BYTES = U_WT + U_UT + U_P + U_VEC + U_KD;
// per (chunk, key head), with the conv inside the kernels: the conv'd q tile
constexpr size_t U_Q = 16384;

struct Work {
    bf16* wt;       // W, [U][64][128] (row i of W = 128 d-values)
    f16* ut;        // U, [U][64][128] (row i of U = 128 v-values), fp16
    f16* p;         // P, [U][64][64], fp16
    float* vec;     // [U][256]: e^G rq (0..63), e^{G_n-G_j} rk (64..127), e^{G_n} (128)
    f16* kd;        // K_dec, [U][64][128] (row j = e^{G_n-G_j} rk_j k_j), fp16
    int32_t* coff;  // [n_seq + 1] chunk offsets
    int32_t* order; // [n_seq] the sequences, most chunks first (null: in order)
    float* carry;   // state between segments (final_state or workspace), may be null
    bf16* q;        // conv'd q, [segc][H_k][64][128] (conv inside the kernels; else null: q from qkv)
};

// Segment size and the places of the intermediates inside one scratch area:
// chunk offsets, then the per-unit arrays (two sets when segments alternate
// between them), then the carry.
struct Layout {
    int64_t segc;    // chunks per segment
    int64_t n_seg;
    int q_heads;     // key heads of the conv'd q tiles after each set of units (0: none)
    size_t off_coff, off_order, off_units, off_units2, off_carry, carry_bytes, total;
    bool two_bufs() const { return off_units2 != off_units; }
};

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// seg_bytes bounds the per-segment intermediates; coff_slots is the number of
// chunk-offset entries reserved (at least n_seq + 1), followed by n_seq slots
// of the sequences' order when `order` is set; with two_bufs, calls of
// more than one segment get a second set of intermediates, so that the intra
// kernel of a segment can run while the chain of the previous one does.
// With q_heads > 0 each set of units is followed by the segment's conv'd q
// tiles (segc x q_heads x U_Q; not counted in seg_bytes, so the segments are
// those of the call without them).
Layout layout_for(int n_seq, int64_t T, int H_v, size_t seg_bytes, size_t coff_slots, bool carry,
                  bool two_bufs, bool order = false, int q_heads = 0) {
    Layout L;
    const int64_t max_chunks = T / C + n_seq;
    int64_t segc = (int64_t)(seg_bytes / ((size_t)H_v * UNIT_BYTES));
    if (segc < 1) segc = 1;
    if (segc > max_chunks) segc = max_chunks;
    if (segc > 65535) segc = 65535;  // grid.y of the intra kernel
    L.segc = segc;
    L.n_seg = (max_chunks + segc - 1) / segc;
    L.q_heads = q_heads;
    L.off_coff = 0;
    L.off_order = order ? 4 * coff_slots : 0;
    L.off_units = align256(4 * (coff_slots + (order ? (size_t)n_seq : 0)));
    const size_t ub = (size_t)segc * ((size_t)H_v * UNIT_BYTES + (size_t)q_heads * U_Q);
    L.off_units2 = two_bufs && L.n_seg > 1 ? L.off_units + ub : L.off_units;
    L.off_carry = L.off_units2 + ub;
    L.carry_bytes = carry && L.n_seg > 1 ? (size_t)n_seq * H_v * D * D * 4 : 0;
    L.total = L.off_carry + L.carry_bytes;
    return L;
}

Layout layout_of(int n_seq, int64_t T, int H_v, int q_heads = 0) {
    return layout_for(n_seq, T, H_v, kSegBytes, (size_t)n_seq + 1, true, true, true, q_heads);
}

// Segments of a call whose chunks hold clen tokens, with the layout's segment
// size (so the same buffers): for clen < C more of them.
int64_t segments_for(const Layout& L, int n_seq, int64_t T, int clen) {
    const int64_t max_chunks = T / clen + n_seq;
    return (max_chunks + L.segc - 1) / L.segc;
}

// The intermediates of buffer `buf` (0 or 1) of a layout.
Work work_at(uint8_t* base, const Layout& L, int H_v, int buf = 0) {
    const size_t U = (size_t)L.segc * H_v;
    uint8_t* un = base + (buf == 0 ? L.off_units : L.off_units2);
    Work w;
    w.coff = reinterpret_cast<int32_t*>(base + L.off_coff);
    w.order = L.off_order ? reinterpret_cast<int32_t*>(base + L.off_order) : nullptr;
    w.wt = reinterpret_cast<bf16*>(un);
    w.ut = reinterpret_cast<f16*>(un + U * U_WT);
    w.p = reinterpret_cast<f16*>(un + U * (U_WT + U_UT));
    w.vec = reinterpret_cast<float*>(un + U * (U_WT + U_UT + U_P));
    w.kd = reinterpret_cast<f16*>(un + U * (U_WT + U_UT + U_P + U_VEC));
    w.q = L.q_heads > 0 ? reinterpret_cast<bf16*>(un + U * UNIT_BYTES) : nullptr;
    w.carry = L.carry_bytes ? reinterpret_cast<float*>(base + L.off_carry) : nullptr;
    return w;
}

// coff[i] = number of chunks of sequences 0..i-1 (one block, any n_seq); with
// `order`, also the sequences sorted by chunk count, most first (ties in
// sequence order; up to 1024 sequences, else in order), so that the chain
// kernel starts the longest sequences' CTAs first
__global__ void __launch_bounds__(1024) chunk_offsets_kernel(const int32_t* cu, int n_seq, int64_t T, int clen,
                                                             int32_t* coff, int32_t* order) {
    pdl_wait();
    pdl_trigger();
    __shared__ int32_t wsum[32];
    __shared__ int32_t base;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        base = 0;
        coff[0] = 0;
    }
    __syncthreads();
    for (int i0 = 0; i0 < n_seq; i0 += 1024) {
        const int i = i0 + tid;
        int v = 0;
        if (i < n_seq) {
            int64_t s, e;
            seq_bounds(cu, i, T, s, e);
            v = (int)((e - s + clen - 1) / clen);
        }
        int x = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) wsum[warp] = x;
        __syncthreads();
        if (warp == 0) {
            int w = wsum[lane];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, w, o);
                if (lane >= o) w += y;
            }
            wsum[lane] = w;
        }
        __syncthreads();
        const int incl = x + (warp > 0 ? wsum[warp - 1] : 0);
        if (i < n_seq) coff[i + 1] = base + incl;
        __syncthreads();
        if (tid == 1023) base += incl;
        __syncthreads();
    }
    if (order == nullptr) return;
    __shared__ int32_t len[1024];
    if (n_seq > 1024) {
        for (int i = tid; i < n_seq; i += 1024) order[i] = i;
        return;
    }
    if (tid < n_seq) len[tid] = coff[tid + 1] - coff[tid];
    __syncthreads();
    if (tid < n_seq) {
        const int li = len[tid];
        int rank = 0;
        for (int j = 0; j < n_seq; ++j) rank += (len[j] > li) || (len[j] == li && j < tid);
        order[rank] = tid;
    }
}

// ============================================================== intra kernel
// One CTA per (chunk, value head); 256 threads, three CTAs per SM (72 KB of
// shared memory and 128 TMEM columns each), so that the latency-bound phases
// of one CTA overlap the copies and MMAs of the others.
constexpr int NT_I = 256;
constexpr int IS_KQ = 0;                          // [cb0: K | Q][cb1: K | Q]; the Q halves then hold T'
constexpr int IS_V = IS_KQ + 32768;               // V, then the W staging tile
constexpr int IS_A = IS_V + 16384;                // A, f32 [64][68]; then T' (fp16) and the U staging tile
constexpr int A_PITCH = 68;
constexpr int IS_X = IS_A + 64 * A_PITCH * 4;     // solve temporaries, f32 [32][36]
constexpr int X_PITCH = 36;
constexpr int IS_VEC = IS_X + 32 * X_PITCH * 4;   // G (log2), beta, beta e^G rk, rk, rq,
                                                  // G - log2 rk, e^{G_n-G} rk
constexpr int IS_BAR = IS_VEC + 7 * 64 * 4;
constexpr int IS_TOTAL = IS_BAR + 64;
constexpr int ISMEM = IS_TOTAL + 1024;
constexpr uint32_t TI_D1 = 0, TI_DW = 0, TI_DU = 64, TI_COLS = 128;  // D1 (128 columns) is dead before W, U

// Element (r, c) of T' = (I + A)^-1, f32, in the two Q halves of the [K | Q]
// tile (rows 0-31 in the first, 32-63 in the second); float4 groups of a row
// are XOR-swizzled by the row so that column-wise reads spread over banks.
__device__ __forceinline__ float* tp_at(uint8_t* kq, int r, int c) {
    return reinterpret_cast<float*>(kq + (r < 32 ? 8192 : 24576) + (r & 31) * 256) +
           ((((c >> 2) ^ (r & 15)) & 15) << 2) + (c & 3);
}

// v[lane] without dynamic register indexing (a tree of selects on lane's bits).
__device__ __forceinline__ float select_lane(const float (&v)[32], int lane) {
    float a[16], b[8], c[4], d[2];
#pragma unroll
    for (int k = 0; k < 16; ++k) a[k] = (lane & 16) ? v[k + 16] : v[k];
#pragma unroll
    for (int k = 0; k < 8; ++k) b[k] = (lane & 8) ? a[k + 8] : a[k];
#pragma unroll
    for (int k = 0; k < 4; ++k) c[k] = (lane & 4) ? b[k + 4] : b[k];
#pragma unroll
    for (int k = 0; k < 2; ++k) d[k] = (lane & 2) ? c[k + 2] : c[k];
    return (lane & 1) ? d[1] : d[0];
}

// qmap covers qkv (y, or the raw x with CONV); qsmap, with CONV, the
// segment's conv'd q tiles in the workspace.
template <bool NEUMANN, bool CONV>
__global__ void __launch_bounds__(NT_I, 3)
chunk_intra_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap wmap,
                   const __grid_constant__ CUtensorMap umap, const __grid_constant__ CUtensorMap qsmap,
                   DeltaArgs a, Work w, int64_t C0) {
    pdl_wait();
    pdl_trigger();
    const int h = blockIdx.x;
    const int64_t gc = C0 + blockIdx.y;
    // first token and length of chunk gc, its sequence and that sequence's
    // first and end tokens (no loads for one sequence without offsets)
    const int clen = chunk_len(a);
    int64_t t0, s0 = 0, s1 = a.T;
    int n, seq = 0;
    if (a.cu == nullptr) {
        t0 = gc * clen;
        if (t0 >= a.T) return;  // past the last chunk of the call
        n = (int)(a.T - t0 < clen ? a.T - t0 : clen);
    } else {
        if (gc >= w.coff[a.n_seq]) return;
        int lo_s = 0, hi_s = a.n_seq - 1;  // sequence of chunk gc
        while (lo_s < hi_s) {
            const int mid = (lo_s + hi_s + 1) >> 1;
            if ((int64_t)w.coff[mid] <= gc) lo_s = mid; else hi_s = mid - 1;
        }
        seq_bounds(a.cu, lo_s, a.T, s0, s1);
        seq = lo_s;
        t0 = s0 + (gc - w.coff[lo_s]) * clen;
        n = (int)(s1 - t0 < clen ? s1 - t0 : clen);
    }
    const int kh = h / (a.H_v / a.H_k);
    const int xq = kh * D, xk = a.H_k * D + kh * D, xv = 2 * a.H_k * D + h * D;
    const int64_t u = (int64_t)blockIdx.y * a.H_v + h;

    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* kq = sm + IS_KQ;
    uint8_t* vv = sm + IS_V;
    float* Am = reinterpret_cast<float*>(sm + IS_A);
    float* Xs = reinterpret_cast<float*>(sm + IS_X);
    float* Gs = reinterpret_cast<float*>(sm + IS_VEC);
    float* Bs = Gs + 64;
    float* FWs = Gs + 128;
    float* RKs = Gs + 192;
    float* RQs = Gs + 256;
    float* Ms = Gs + 320;
    float* DECs = Gs + 384;
    float* EMs = Xs;  // rk_j 2^{-G_j}, and the flag below: in the solve's scratch, free until the solve
    int* fact_flag = reinterpret_cast<int*>(Xs + 64);
    uint64_t* bar_tma = reinterpret_cast<uint64_t*>(sm + IS_BAR);
    uint64_t* bar_mma = bar_tma + 1;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(bar_tma + 2);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int quarter = warp & 3, half = warp >> 2;
    const int row = quarter * 32 + lane;
    const uint32_t lo = (uint32_t)(quarter * 32) << 16;
    constexpr float kLog2e = 1.4426950408889634f;

    if (tid == 0) {
        mbar_init(bar_tma, 1);
        mbar_init(bar_mma, 1);
        fence_mbar_init();
        mbar_arrive_expect_tx(bar_tma, 6 * 8192);
        // with CONV, tile row j holds token t0 - 3 + j (rows before token 0 read as zeros)
        const int y = CONV ? (int)t0 - 3 : (int)t0;
        tma_load_2d(kq, &qmap, bar_tma, xk, y);
        tma_load_2d(kq + 16384, &qmap, bar_tma, xk + 64, y);
        tma_load_2d(kq + 8192, &qmap, bar_tma, xq, y);
        tma_load_2d(kq + 24576, &qmap, bar_tma, xq + 64, y);
        tma_load_2d(vv, &qmap, bar_tma, xv, y);
        tma_load_2d(vv + 8192, &qmap, bar_tma, xv + 64, y);
    }
    if (warp == 0) {
        tmem_alloc(tslot, TI_COLS);
        tmem_relinquish();
    }
    // CONV: threads 0-191 each take 8 channels (16-byte column cc of 64-channel
    // block cb: K, K, Q, Q, V, V halves) of 16 rows [16 rg, 16 rg + 16); their
    // taps are fetched into L1 and, for the last row group, the 3 raw inputs
    // past the tile (tokens t0 + 61 .. t0 + 63) loaded while the tile is in flight
    const int conv_dim = 2 * a.H_k * D + a.H_v * D;
    const int rg = tid / 48, cb = (tid % 48) >> 3, cc = tid & 7;
    const bool cthr = tid < 192;
    const int cch = (cb < 2 ? xk : (cb < 4 ? xq : xv)) + (cb & 1) * 64 + cc * 8;
    uint8_t* cblk = cb < 4 ? kq + (cb & 1) * 16384 + (cb >> 1) * 8192 : vv + (cb & 1) * 8192;
    const uint4* tap_src = reinterpret_cast<const uint4*>(static_cast<const bf16*>(a.conv_w) + (int64_t)cch * 4);
    uint4 look[3];
    if constexpr (CONV) {
        if (cthr) {
            asm volatile("prefetch.global.L1 [%0];" ::"l"(tap_src));
            if (rg == 3) {
#pragma unroll
                for (int j = 0; j < 3; ++j) {
                    const int64_t t = t0 + 61 + j;
                    look[j] = t < a.T ? *reinterpret_cast<const uint4*>(static_cast<const bf16*>(a.qkv) +
                                                                        t * conv_dim + cch)
                                      : make_uint4(0u, 0u, 0u, 0u);
                }
            }
        }
    }
    if (warp == 1) {
        // beta = sigmoid(b) and g = -exp(A_log) softplus(a + dt_bias) of tokens
        // lane and lane + 32 (every load issued before any use), then the
        // chunk-local cumulative decay G in the log2 domain; zero past token n
        int64_t gi[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) gi[e] = lane + 32 * e < n ? (t0 + lane + 32 * e) * a.H_v + h : 0;
        const bool raw = a.g == nullptr;
        float gv[2], bv[2];
        if (raw) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                gv[e] = to_f(static_cast<const bf16*>(a.a)[gi[e]]);
                bv[e] = to_f(static_cast<const bf16*>(a.b)[gi[e]]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                gv[e] = a.g[gi[e]];
                bv[e] = a.beta[gi[e]];
            }
        }
        const float Al = raw ? a.A_log[h] : 0.f, dtb = raw ? a.dt_bias[h] : 0.f;
        float x[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const bool live = lane + 32 * e < n;
            const float g = raw ? gate_g(gv[e], Al, dtb) : gv[e];
            const float bt = raw ? sigmoid_f(bv[e]) : bv[e];
            x[e] = live ? g * kLog2e : 0.f;
            Bs[lane + 32 * e] = live ? bt : 0.f;
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float y0 = __shfl_up_sync(0xffffffffu, x[0], o);
            const float y1 = __shfl_up_sync(0xffffffffu, x[1], o);
            if (lane >= o) {
                x[0] += y0;
                x[1] += y1;
            }
        }
        const float G1 = x[1] + __shfl_sync(0xffffffffu, x[0], 31);
        Gs[lane] = x[0];
        Gs[lane + 32] = G1;
        // with every |G| < 100 (log2) the factors 2^{G_i} and 2^{-G_j} of A and P
        // stay normal f32 numbers, and A, P are formed from them instead of one
        // exponential per element
        float glo = fminf(x[0], G1), ghi = fmaxf(x[0], G1);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            glo = fminf(glo, __shfl_xor_sync(0xffffffffu, glo, o));
            ghi = fmaxf(ghi, __shfl_xor_sync(0xffffffffu, ghi, o));
        }
        if (lane == 0) *fact_flag = glo > -100.f && ghi < 100.f ? 1 : 0;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = *tslot;
    bool ok = __syncthreads_and(mbar_wait(bar_tma, 0, kWaitNs));
    if constexpr (CONV) {
        // y = silu(conv(x)) in place: output row r (token t0 + r) takes tile
        // rows r .. r + 3 and overwrites row r, which no later output of the
        // same thread reads; the first rows another thread overwrites are read
        // before the barrier
        if (ok && cthr && rg < 3) {
#pragma unroll
            for (int j = 0; j < 3; ++j)
                look[j] = *reinterpret_cast<const uint4*>(cblk + sw128_off(16 * rg + 16 + j, 8 * cc));
        }
        __syncthreads();
        if (ok && rg == 4 && (cb >= 4 || h % (a.H_v / a.H_k) == 0)) {
            // meanwhile threads 192-239, one per column: the conv state after the
            // sequence and the conv checkpoints in this chunk, for the CTA's V
            // channels and, in the first value head of the key head, its K and Q
            // ones -- the 3 raw inputs ending at the sequence's last token, or at
            // its token m ckpt_every - 1 ([channel][3], bit copies, as the conv
            // kernels write them; inputs before the sequence from conv_state0)
            const uint16_t* xs = static_cast<const uint16_t*>(a.qkv);
            auto write3 = [&](int64_t last, uint16_t* dst) {
                uint16_t v[24];
#pragma unroll
                for (int j = 0; j < 3; ++j) {
                    const int64_t p = last - 2 + j;
                    if (p >= s0) {
                        const uint4 r = *reinterpret_cast<const uint4*>(xs + p * conv_dim + cch);
                        const uint32_t wv[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
                        for (int q = 0; q < 8; ++q) v[3 * q + j] = (uint16_t)(wv[q >> 1] >> (16 * (q & 1)));
                    } else {
                        const uint16_t* st = static_cast<const uint16_t*>(a.conv_state0);
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            v[3 * q + j] = st != nullptr ? st[((int64_t)seq * conv_dim + cch + q) * 3 + 3 - (s0 - p)] : 0;
                    }
                }
                uint4* d4 = reinterpret_cast<uint4*>(dst);
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    d4[i] = make_uint4(v[8 * i] | (uint32_t)v[8 * i + 1] << 16, v[8 * i + 2] | (uint32_t)v[8 * i + 3] << 16,
                                       v[8 * i + 4] | (uint32_t)v[8 * i + 5] << 16, v[8 * i + 6] | (uint32_t)v[8 * i + 7] << 16);
            };
            if (a.conv_state_out != nullptr && t0 + n == s1)
                write3(s1 - 1, static_cast<uint16_t*>(a.conv_state_out) + ((int64_t)seq * conv_dim + cch) * 3);
            if (a.conv_ckpt != nullptr && a.ckpt_every > 0) {
                const int64_t N = a.ckpt_every;
                int64_t row0 = -1;
                for (int64_t m = (t0 - s0) / N + 1; s0 + m * N - 1 < t0 + n; ++m) {
                    if (s0 + m * N - 1 < t0) continue;
                    if (row0 < 0) row0 = ckpt_row0(a.cu, seq, a.T, a.ckpt_every);
                    if (row0 + m - 1 >= a.ckpt_rows) break;
                    write3(s0 + m * N - 1,
                           static_cast<uint16_t*>(a.conv_ckpt) + ((row0 + m - 1) * conv_dim + cch) * 3);
                }
            }
        }
        if (ok && cthr) {
            // two passes of 4 channels (8 bytes of each row's 16); each
            // channel's arithmetic is the conv kernel's
#pragma unroll 1
            for (int p = 0; p < 2; ++p) {
                float2 taps[2][4];
                {
                    const uint4 raw[2] = {tap_src[2 * p], tap_src[2 * p + 1]};
                    conv_taps_bf16_2(raw, taps);
                }
                auto row4 = [&](int r, float* x) {  // channels 4p .. 4p + 3 of tile row r
                    const uint2 v = *reinterpret_cast<const uint2*>(cblk + sw128_off(r, 8 * cc) + 8 * p);
                    x[0] = __uint_as_float(v.x << 16);
                    x[1] = __uint_as_float(v.x & 0xffff0000u);
                    x[2] = __uint_as_float(v.y << 16);
                    x[3] = __uint_as_float(v.y & 0xffff0000u);
                };
                float x0[4], x1[4], x2[4];
                if (rg == 0 && t0 == s0) {
                    // a sequence's first chunk: the inputs before it are its conv
                    // state ([conv_dim][3], column 0 oldest), or zeros
                    float st[12];
                    if (a.conv_state0 != nullptr) {
                        const bf16* sp = static_cast<const bf16*>(a.conv_state0) +
                                         ((int64_t)seq * conv_dim + cch + 4 * p) * 3;
#pragma unroll
                        for (int i = 0; i < 12; ++i) st[i] = to_f(sp[i]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 12; ++i) st[i] = 0.f;
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        x0[q] = st[3 * q];
                        x1[q] = st[3 * q + 1];
                        x2[q] = st[3 * q + 2];
                    }
                } else {
                    row4(16 * rg, x0);
                    row4(16 * rg + 1, x1);
                    row4(16 * rg + 2, x2);
                }
                // four rows at a time: the inputs r + 3 .. r + 6 are read before
                // the outputs r .. r + 3 are written
#pragma unroll
                for (int i0 = 0; i0 < 16; i0 += 4) {
                    float xn[4][4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int i = i0 + k;
                        if (i < 13) {
                            row4(16 * rg + i + 3, xn[k]);
                        } else {
                            const uint32_t lo = p ? look[i - 13].z : look[i - 13].x;
                            const uint32_t hi = p ? look[i - 13].w : look[i - 13].y;
                            xn[k][0] = __uint_as_float(lo << 16);
                            xn[k][1] = __uint_as_float(lo & 0xffff0000u);
                            xn[k][2] = __uint_as_float(hi << 16);
                            xn[k][3] = __uint_as_float(hi & 0xffff0000u);
                        }
                    }
                    uint2 yv[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float out[4];
                        conv4_pairs<2, bf16>(taps, x0, x1, x2, xn[k], 1, out);
                        yv[k] = make_uint2(pack_bf16x2(out[0], out[1]), pack_bf16x2(out[2], out[3]));
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            x0[q] = x1[q];
                            x1[q] = x2[q];
                            x2[q] = xn[k][q];
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        *reinterpret_cast<uint2*>(cblk + sw128_off(16 * rg + i0 + k, 8 * cc) + 8 * p) = yv[k];
                }
            }
            fence_async_smem();  // the tiles are read by the MMAs and the q store
        }
        __syncthreads();
        // the chain's q tile, once per key head
        if (ok && tid == 0 && h % (a.H_v / a.H_k) == 0) {
            const int qr = (int)(((int64_t)blockIdx.y * a.H_k + kh) * 64);
            tma_store_2d(&qsmap, kq + 8192, 0, qr);
            tma_store_2d(&qsmap, kq + 24576, 64, qr);
            bulk_commit();
        }
    }
    bool mma_pending = false;
    uint32_t mma_phase = 0;
    if (ok) {
        // D1 = [K; Q] [K; Q]^T: the k.k and q.k products of A and P, and on its
        // diagonal the squared norms of the k and q rows
        if (tid == 0) {
            tc_fence_after();
            const uint32_t akq = smem_u32(kq);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t off = (k >> 2) * 16384 + (k & 3) * 32;
                mma_bf16(tb + TI_D1, sdesc_sw128(akq + off, 16, 1024),
                         sdesc_sw128(akq + off, 16, 1024), idesc_bf16_f32(128, 128, 0, 0), k > 0);
            }
            mma_commit(bar_mma);
        }
        mma_pending = true;
        ok = __syncthreads_and(mbar_wait(bar_mma, mma_phase, kWaitNs));
    }
    if (ok) {
        mma_phase ^= 1;
        mma_pending = false;
        tc_fence_after();
        const bool isk = row < 64;
        const int i = row & 63, j0 = 32 * half;
        float d1[32];
        const uint32_t t1 = tb + lo + TI_D1 + 32 * half;
        // the warp whose 32 columns hold its rows' diagonal: l2-norm factors,
        // the row factors of W and the workspace vectors
        if (isk ? quarter == half : quarter - 2 == half) {
            float ss;
            if (isk) {
                tmem_ld32(t1, d1);
                ss = select_lane(d1, lane);
            } else {
                float dq[32];
                tmem_ld32_twice(t1, d1, t1 + 64, dq);
                ss = select_lane(dq, lane);
            }
            float f = isk ? 1.f : a.scale;
            if (a.l2norm) f = f / sqrtf(ss + 1e-6f);
            const float Gn = Gs[n - 1];
            const float eg = exp2f(Gs[i]);
            float* vec = w.vec + u * (U_VEC / 4);
            if (isk) {
                RKs[i] = f;
                FWs[i] = Bs[i] * eg * f;
                Ms[i] = Gs[i] - lg2_approx(f);
                EMs[i] = f * ex2_approx(-Gs[i]);
                const float dec = i < n ? exp2f(Gn - Gs[i]) * f : 0.f;
                vec[64 + i] = dec;
                DECs[i] = dec;
                if (i == 0) vec[128] = exp2f(Gn);
            } else {
                RQs[i] = f;
                vec[i] = eg * f;
            }
        } else {
            tmem_ld32(t1, d1);
        }
        __syncthreads();
        {   // A (k rows -> shared, f32) and P (q rows -> workspace, fp16):
            //   A_ij = beta_i rk_i rk_j e^{G_i-G_j} k_i.k_j (j<i), P_ij = rq_i rk_j e^{G_i-G_j} q_i.k_j (j<=i)
            // with the row and column factors folded into the exponent:
            //   f_i rk_j 2^{G_i-G_j} = 2^{(G_i + log2 f_i) - (G_j - log2 rk_j)}
            if (j0 <= (i | 31)) {  // else every (i, j) of this warp has j > i
                float fi = i < n ? (isk ? Bs[i] * RKs[i] : RQs[i]) : 0.f;
                const int jmax = isk ? i - 1 : i;
                if (*fact_flag) {
                    // (f_i 2^{G_i}) (rk_j 2^{-G_j}) d_ij: one exponential per row and per column
                    const float Ei = fi * ex2_approx(Gs[i]);
#pragma unroll
                    for (int g4 = 0; g4 < 8; ++g4) {
                        const float4 F4 = *reinterpret_cast<const float4*>(EMs + j0 + 4 * g4);
                        const float2 a01 = __fmul2_rn(make_float2(d1[4 * g4], d1[4 * g4 + 1]), make_float2(Ei, Ei));
                        const float2 a23 = __fmul2_rn(make_float2(d1[4 * g4 + 2], d1[4 * g4 + 3]), make_float2(Ei, Ei));
                        const float2 p01 = __fmul2_rn(a01, make_float2(F4.x, F4.y));
                        const float2 p23 = __fmul2_rn(a23, make_float2(F4.z, F4.w));
                        const int j = j0 + 4 * g4;
                        d1[4 * g4 + 0] = j + 0 <= jmax ? p01.x : 0.f;
                        d1[4 * g4 + 1] = j + 1 <= jmax ? p01.y : 0.f;
                        d1[4 * g4 + 2] = j + 2 <= jmax ? p23.x : 0.f;
                        d1[4 * g4 + 3] = j + 3 <= jmax ? p23.y : 0.f;
                    }
                } else {
                    if (fi < 0.f) {  // a negative q scale (or beta): its sign stays outside the exponent
                        fi = -fi;
#pragma unroll
                        for (int q = 0; q < 32; ++q) d1[q] = -d1[q];
                    }
                    const float Li = Gs[i] + lg2_approx(fi);  // -inf when f_i = 0
#pragma unroll
                    for (int g4 = 0; g4 < 8; ++g4) {
                        const float4 M4 = *reinterpret_cast<const float4*>(Ms + j0 + 4 * g4);
                        const float2 x01 = __fadd2_rn(make_float2(Li, Li), make_float2(-M4.x, -M4.y));
                        const float2 x23 = __fadd2_rn(make_float2(Li, Li), make_float2(-M4.z, -M4.w));
                        const float2 p01 = __fmul2_rn(make_float2(d1[4 * g4], d1[4 * g4 + 1]),
                                                      make_float2(ex2_approx(x01.x), ex2_approx(x01.y)));
                        const float2 p23 = __fmul2_rn(make_float2(d1[4 * g4 + 2], d1[4 * g4 + 3]),
                                                      make_float2(ex2_approx(x23.x), ex2_approx(x23.y)));
                        const int j = j0 + 4 * g4;
                        d1[4 * g4 + 0] = j + 0 <= jmax ? p01.x : 0.f;
                        d1[4 * g4 + 1] = j + 1 <= jmax ? p01.y : 0.f;
                        d1[4 * g4 + 2] = j + 2 <= jmax ? p23.x : 0.f;
                        d1[4 * g4 + 3] = j + 3 <= jmax ? p23.y : 0.f;
                    }
                }
            } else {
#pragma unroll
                for (int q = 0; q < 32; ++q) d1[q] = 0.f;
            }
            if (isk) {
#pragma unroll
                for (int g4 = 0; g4 < 8; ++g4)
                    *reinterpret_cast<float4*>(&Am[i * A_PITCH + j0 + 4 * g4]) =
                        make_float4(d1[4 * g4], d1[4 * g4 + 1], d1[4 * g4 + 2], d1[4 * g4 + 3]);
            } else {
                f16* pp = w.p + u * (U_P / 2) + i * 64 + j0;
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    *reinterpret_cast<uint4*>(pp + 8 * g) =
                        make_uint4(pack_h2(d1[8 * g], d1[8 * g + 1]), pack_h2(d1[8 * g + 2], d1[8 * g + 3]),
                                   pack_h2(d1[8 * g + 4], d1[8 * g + 5]), pack_h2(d1[8 * g + 6], d1[8 * g + 7]));
            }
        }
        if (CONV && tid == 0) bulk_wait_read_all();  // the q store has read the Q halves that T' takes
        __syncthreads();
        // D1 has read K: K and V are re-encoded in place as the fp16 operands
        // of the W and U products with their row factors, diag(beta e^G rk) K
        // and diag(beta) V (so that both products take T' itself), and
        // K_dec = diag(e^{G_n-G_j} rk) K goes to the workspace (fp16, rows of
        // 128 d) -- by the threads the solve's first step leaves free
        auto convert_kv = [&](int t, int nt) {
            f16* kd = w.kd + u * (U_KD / 2);
            for (int e = t; e < 1024; e += nt) {
                const int blk = e >> 9, r = (e >> 3) & 63, pc = e & 7;
                uint4* src = reinterpret_cast<uint4*>(kq + blk * 16384 + (e & 511) * 16);
                float x[8];
                unpack16<bf16>(*src, x);
                const float dc = DECs[r], fw = FWs[r];
                *src = make_uint4(pack_h2(x[0] * fw, x[1] * fw), pack_h2(x[2] * fw, x[3] * fw),
                                  pack_h2(x[4] * fw, x[5] * fw), pack_h2(x[6] * fw, x[7] * fw));
                *reinterpret_cast<uint4*>(kd + r * 128 + blk * 64 + ((pc ^ (r & 7)) << 3)) =
                    make_uint4(pack_h2(x[0] * dc, x[1] * dc), pack_h2(x[2] * dc, x[3] * dc),
                               pack_h2(x[4] * dc, x[5] * dc), pack_h2(x[6] * dc, x[7] * dc));
            }
            for (int e = t; e < 1024; e += nt) {
                const int r = (e >> 3) & 63;
                uint4* src = reinterpret_cast<uint4*>(vv + (e >> 9) * 8192 + (e & 511) * 16);
                float x[8];
                unpack16<bf16>(*src, x);
                const float bt = Bs[r];
                *src = make_uint4(pack_h2(x[0] * bt, x[1] * bt), pack_h2(x[2] * bt, x[3] * bt),
                                  pack_h2(x[4] * bt, x[5] * bt), pack_h2(x[6] * bt, x[7] * bt));
            }
        };
        if constexpr (!NEUMANN) {
            // T' = (I + A)^-1 (unit lower triangular): the four diagonal 16-blocks
            // by forward substitution (f32), then the off-diagonal blocks by
            // doubling on warp-level tf32 MMAs (T' is rounded to fp16 right after),
            //   T'_{10} = -D_1 A_{10} D_0 (and T'_{32}),  T'_{[23][01]} = -T'_{[23][23]} A_{[23][01]} T'_{[01][01]}
            if (tid < 64) {
                const int r0 = (tid >> 4) * 16, cl = tid & 15;
                float x[16];
    #pragma unroll
                for (int r = 0; r < 16; ++r) x[r] = r == cl ? 1.f : 0.f;
    #pragma unroll
                for (int q = 0; q < 15; ++q)
    #pragma unroll
                    for (int r = q + 1; r < 16; ++r) x[r] = fmaf(-Am[(r0 + r) * A_PITCH + r0 + q], x[q], x[r]);
    #pragma unroll
                for (int r = 0; r < 16; ++r) *tp_at(kq, r0 + r, r0 + cl) = x[r];
            } else {
                // meanwhile the other threads zero T' above its diagonal blocks
                // (blocks (0,1) (0,2) (0,3) (1,2) (1,3) (2,3)), 2 float4 each,
                // and re-encode K and V
    #pragma unroll
                for (int e = tid - 64; e < 384; e += NT_I - 64) {
                    const int blk = e >> 6, br = blk < 3 ? 0 : (blk < 5 ? 1 : 2);
                    const int bc = blk < 3 ? blk + 1 : (blk < 5 ? blk - 1 : 3);
                    *reinterpret_cast<float4*>(tp_at(kq, 16 * br + ((e >> 2) & 15), 16 * bc + (e & 3) * 4)) =
                        make_float4(0.f, 0.f, 0.f, 0.f);
                }
                convert_kv(tid - 64, NT_I - 64);
            }
            __syncthreads();
            const int fg = lane >> 2, ft = lane & 3;  // MMA fragment row group, thread in group
            if (warp < 4) {  // level 1, X = A_{b+1,b} D_b for b = 0, 2; warp = (block pair, 8 columns)
                const int blk = warp >> 1, c0 = 32 * blk + 8 * (warp & 1), r0 = 32 * blk + 16;
                float c[4] = {0.f, 0.f, 0.f, 0.f};
    #pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    const int k0 = 32 * blk + 8 * ks;
                    const float af[4] = {Am[(r0 + fg) * A_PITCH + k0 + ft], Am[(r0 + fg + 8) * A_PITCH + k0 + ft],
                                         Am[(r0 + fg) * A_PITCH + k0 + ft + 4], Am[(r0 + fg + 8) * A_PITCH + k0 + ft + 4]};
                    const float bfr[2] = {*tp_at(kq, k0 + ft, c0 + fg), *tp_at(kq, k0 + ft + 4, c0 + fg)};
                    mma_tf32_16x8x8(c, af, bfr);
                }
                float* xr = Xs + (16 * blk + fg) * X_PITCH + 8 * (warp & 1) + 2 * ft;
                *reinterpret_cast<float2*>(xr) = make_float2(c[0], c[1]);
                *reinterpret_cast<float2*>(xr + 8 * X_PITCH) = make_float2(c[2], c[3]);
            }
            __syncthreads();
            if (warp < 4) {  // T'_{b+1,b} = -D_{b+1} X
                const int blk = warp >> 1, n0 = 8 * (warp & 1), r0 = 32 * blk + 16;
                float c[4] = {0.f, 0.f, 0.f, 0.f};
    #pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    const int k0 = 8 * ks;
                    const float af[4] = {*tp_at(kq, r0 + fg, r0 + k0 + ft), *tp_at(kq, r0 + fg + 8, r0 + k0 + ft),
                                         *tp_at(kq, r0 + fg, r0 + k0 + ft + 4), *tp_at(kq, r0 + fg + 8, r0 + k0 + ft + 4)};
                    const float bfr[2] = {Xs[(16 * blk + k0 + ft) * X_PITCH + n0 + fg],
                                          Xs[(16 * blk + k0 + ft + 4) * X_PITCH + n0 + fg]};
                    mma_tf32_16x8x8(c, af, bfr);
                }
                const int cc = 32 * blk + n0 + 2 * ft;
                *reinterpret_cast<float2*>(tp_at(kq, r0 + fg, cc)) = make_float2(-c[0], -c[1]);
                *reinterpret_cast<float2*>(tp_at(kq, r0 + fg + 8, cc)) = make_float2(-c[2], -c[3]);
            }
            __syncthreads();
            {   // level 2, X = A_{[23][01]} T'_{[01][01]} (32 x 32); warp = (16 rows, 8 columns)
                const int mt = warp >> 2, nt = warp & 3, r0 = 32 + 16 * mt;
                float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {  // T'(k, c) = 0 for k < c
                    if (ks < nt) continue;
                    const int k0 = 8 * ks;
                    const float af[4] = {Am[(r0 + fg) * A_PITCH + k0 + ft], Am[(r0 + fg + 8) * A_PITCH + k0 + ft],
                                         Am[(r0 + fg) * A_PITCH + k0 + ft + 4], Am[(r0 + fg + 8) * A_PITCH + k0 + ft + 4]};
                    const float bfr[2] = {*tp_at(kq, k0 + ft, 8 * nt + fg), *tp_at(kq, k0 + ft + 4, 8 * nt + fg)};
                    mma_tf32_16x8x8(c, af, bfr);
                }
                float* xr = Xs + (16 * mt + fg) * X_PITCH + 8 * nt + 2 * ft;
                *reinterpret_cast<float2*>(xr) = make_float2(c[0], c[1]);
                *reinterpret_cast<float2*>(xr + 8 * X_PITCH) = make_float2(c[2], c[3]);
            }
            __syncthreads();
            {   // T'_{[23][01]} = -T'_{[23][23]} X
                const int mt = warp >> 2, nt = warp & 3, r0 = 32 + 16 * mt;
                float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {  // T'(r, 32 + k) = 0 for k > r - 32
                    if (ks >= 2 * mt + 2) break;
                    const int k0 = 8 * ks;
                    const float af[4] = {*tp_at(kq, r0 + fg, 32 + k0 + ft), *tp_at(kq, r0 + fg + 8, 32 + k0 + ft),
                                         *tp_at(kq, r0 + fg, 32 + k0 + ft + 4),
                                         *tp_at(kq, r0 + fg + 8, 32 + k0 + ft + 4)};
                    const float bfr[2] = {Xs[(k0 + ft) * X_PITCH + 8 * nt + fg], Xs[(k0 + ft + 4) * X_PITCH + 8 * nt + fg]};
                    mma_tf32_16x8x8(c, af, bfr);
                }
                *reinterpret_cast<float2*>(tp_at(kq, r0 + fg, 8 * nt + 2 * ft)) = make_float2(-c[0], -c[1]);
                *reinterpret_cast<float2*>(tp_at(kq, r0 + fg + 8, 8 * nt + 2 * ft)) = make_float2(-c[2], -c[3]);
            }
            __syncthreads();
        } else {
            // T' = (I + A)^-1 as the Neumann-style product (I + N)(I + N^2)...(I + N^32),
            // N = -A (nilpotent, so six factors are exact for 64 rows): P = N,
            // T' = I + N, then five times P <- P P and T' <- T' + T' P.  Each
            // product is a full 64 x 64 x 64 tf32 MMA, a 16 x 32 tile per warp,
            // accumulated in registers and written back in place after a barrier.
            convert_kv(tid, NT_I);
            for (int e = tid; e < 64 * 64; e += NT_I) {
                const int r = e >> 6, c = e & 63;
                const float nv = c < r ? -Am[r * A_PITCH + c] : 0.f;
                Am[r * A_PITCH + c] = nv;
                *tp_at(kq, r, c) = r == c ? 1.f : nv;
            }
            __syncthreads();
            const int fg = lane >> 2, ft = lane & 3;
            const int r0 = 16 * (warp & 3), n0 = 32 * (warp >> 2);
            for (int lev = 0; lev < 5; ++lev) {
                float c[4][4];
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) c[nt][0] = c[nt][1] = c[nt][2] = c[nt][3] = 0.f;
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) {  // P P
                    const int k0 = 8 * ks;
                    const float af[4] = {Am[(r0 + fg) * A_PITCH + k0 + ft], Am[(r0 + fg + 8) * A_PITCH + k0 + ft],
                                         Am[(r0 + fg) * A_PITCH + k0 + ft + 4],
                                         Am[(r0 + fg + 8) * A_PITCH + k0 + ft + 4]};
#pragma unroll
                    for (int nt = 0; nt < 4; ++nt) {
                        const float bfr[2] = {Am[(k0 + ft) * A_PITCH + n0 + 8 * nt + fg],
                                              Am[(k0 + ft + 4) * A_PITCH + n0 + 8 * nt + fg]};
                        mma_tf32_16x8x8(c[nt], af, bfr);
                    }
                }
                __syncthreads();
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
                    float* pr = Am + (r0 + fg) * A_PITCH + n0 + 8 * nt + 2 * ft;
                    pr[0] = c[nt][0];
                    pr[1] = c[nt][1];
                    pr[8 * A_PITCH] = c[nt][2];
                    pr[8 * A_PITCH + 1] = c[nt][3];
                }
                __syncthreads();
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) c[nt][0] = c[nt][1] = c[nt][2] = c[nt][3] = 0.f;
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) {  // T' P
                    const int k0 = 8 * ks;
                    const float af[4] = {*tp_at(kq, r0 + fg, k0 + ft), *tp_at(kq, r0 + fg + 8, k0 + ft),
                                         *tp_at(kq, r0 + fg, k0 + ft + 4), *tp_at(kq, r0 + fg + 8, k0 + ft + 4)};
#pragma unroll
                    for (int nt = 0; nt < 4; ++nt) {
                        const float bfr[2] = {Am[(k0 + ft) * A_PITCH + n0 + 8 * nt + fg],
                                              Am[(k0 + ft + 4) * A_PITCH + n0 + 8 * nt + fg]};
                        mma_tf32_16x8x8(c[nt], af, bfr);
                    }
                }
                __syncthreads();
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
                    const int cc = n0 + 8 * nt + 2 * ft;
                    *tp_at(kq, r0 + fg, cc) += c[nt][0];
                    *tp_at(kq, r0 + fg, cc + 1) += c[nt][1];
                    *tp_at(kq, r0 + fg + 8, cc) += c[nt][2];
                    *tp_at(kq, r0 + fg + 8, cc + 1) += c[nt][3];
                }
                __syncthreads();
            }
        }
        {   // T' (fp16) into the A region: the B operand of both products
            const int i = tid >> 2, c0 = (tid & 3) * 16;
            float vals[16];  // T' is zero above its diagonal (all of it is written)
#pragma unroll
            for (int g4 = 0; g4 < 4; ++g4) {
                const float4 t4 = *reinterpret_cast<const float4*>(tp_at(kq, i, c0 + 4 * g4));
                vals[4 * g4 + 0] = t4.x;
                vals[4 * g4 + 1] = t4.y;
                vals[4 * g4 + 2] = t4.z;
                vals[4 * g4 + 3] = t4.w;
            }
            store_row_h(sm + IS_A, i, c0, vals, 16);
        }
        fence_async_smem();
        tc_fence_before();
        __syncthreads();
        // W^T = (diag(beta e^G rk) K)^T T'^T,  U^T = (diag(beta) V)^T T'^T  (M = d, N = i, K = j)
        if (tid == 0) {
            tc_fence_after();
            const uint32_t akq = smem_u32(kq), av = smem_u32(vv);
            const uint32_t bt = smem_u32(sm + IS_A);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                mma_bf16(tb + TI_DW, sdesc_sw128(akq + k * 2048, 16384, 1024),
                         sdesc_sw128(bt + k * 32, 16, 1024), idesc_f16_f32(128, 64, 1, 0), k > 0);
                mma_bf16(tb + TI_DU, sdesc_sw128(av + k * 2048, 8192, 1024),
                         sdesc_sw128(bt + k * 32, 16, 1024), idesc_f16_f32(128, 64, 1, 0), k > 0);
            }
            mma_commit(bar_mma);
        }
        mma_pending = true;
        ok = __syncthreads_and(mbar_wait(bar_mma, mma_phase, kWaitNs));
    }
    if (ok) {
        mma_pending = false;
        tc_fence_after();
        // W (bf16) and U (fp16) as row-major tiles for TMA stores: the accumulators
        // (lanes = d, columns = i) are read in the 16x256b shape, whose
        // fragments stmatrix.trans writes transposed -- 16 bytes of a row at a
        // time -- into 128-byte-swizzled staging tiles (W in the consumed V
        // tile, U in the consumed A region).  Warp (quarter, half):
        // d in [32 quarter, +32), i in [32 half, +32).
        const int mk = lane >> 3, mr = lane & 7;  // this thread's row address: matrix mk, row mr
#pragma unroll
        for (int acc = 0; acc < 2; ++acc) {
            uint8_t* stg = acc == 0 ? vv : sm + IS_A;
            const uint32_t col = (acc == 0 ? TI_DW : TI_DU) + 32 * half;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int d0 = 32 * quarter + 16 * (q & 1), i0 = 32 * half + 16 * (q >> 1);
                uint32_t r[8], p[4];
                tmem_ld16x256b_x2(tb + ((uint32_t)d0 << 16) + col + 16 * (q >> 1), r);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    p[k] = acc == 0 ? pack_bf16x2(__uint_as_float(r[2 * k]), __uint_as_float(r[2 * k + 1]))
                                    : pack_h2(__uint_as_float(r[2 * k]), __uint_as_float(r[2 * k + 1]));
                // matrices: 0 (d0.., i0..), 1 (d0+8.., i0..), 2 (d0.., i0+8..), 3 (d0+8.., i0+8..)
                const int ri = i0 + 8 * (mk >> 1) + mr, rd = d0 + 8 * (mk & 1);
                stmatrix_x4_trans(stg + (rd >> 6) * 8192 + sw128_off(ri, rd & 63), p);
            }
        }
        fence_async_smem();
    } else if (tid == 0) {
        atomicOr(&g_device_error, 1);
        if (mma_pending) mbar_wait(bar_mma, mma_phase, kWaitNs);
        mbar_wait(bar_tma, 0, kWaitNs);
        if (CONV) bulk_wait_read_all();
    }
    tc_fence_before();
    __syncthreads();
    if (ok && tid == 0) {
        tma_store_2d(&wmap, vv, 0, (int)(u * 64));
        tma_store_2d(&wmap, vv + 8192, 64, (int)(u * 64));
        tma_store_2d(&umap, sm + IS_A, 0, (int)(u * 64));
        tma_store_2d(&umap, sm + IS_A + 8192, 64, (int)(u * 64));
        bulk_commit();
        bulk_wait_read_all();  // the staging tiles must outlive the copies' reads
    }
    if (warp == 0) tmem_dealloc(tb, TI_COLS);
}

// ============================================================== chain kernel
// One CTA per (sequence, value head, slice of VS value columns).  The columns
// of the state are independent under the delta rule, so a head's state can be
// split across CTAs when there are few (sequence, head) pairs.  Per chunk,
// with the chunk's rows on TMEM lanes and the slice's columns as the MMA N:
//   MMA1  [Q S; W S]      M = 128 (q rows | w rows), N = VS, K = d   (A = [Q; W], B = S, MN-major; bf16)
//   U' = U - W S          (w-row lanes; fp16 operand U')
//   MMA2  dS = K_dec^T U' M = d, N = VS, K = j (fp16)
//   S <- e^{G_n} S + dS   (f32 in registers; bf16 operand for the next MMA1)
//   MMA3  P U'            M = 128 (P and 64 rows of padding), N = VS, K = j (fp16)
//   O = (Q S) diag(e^G rq) + P U'  (q-row lanes, stored straight to global)
// Warp roles: 16 compute warps, one warp that issues the MMAs, one that
// issues the TMA loads and one that stores each chunk's O tile; they hand work
// to each other through mbarriers, so the copies, the O epilogue and the P U'
// product run off the state's critical path (MMA1 -> U' -> MMA2 -> S update ->
// next MMA1).
constexpr int NT_COMP = 512;
constexpr int NT_C = NT_COMP + 96;
constexpr int W_MMA = NT_COMP / 32, W_TMA = W_MMA + 1, W_ST = W_MMA + 2;

template <int VS>
struct ChainLayout {
    static constexpr int NB = VS / 64;                  // 64-column blocks of the slice
    static constexpr int SG_QW = 0;                     // per 64-wide d block: Q rows | W rows (16 KB)
    static constexpr int SG_P = 32768;                  // P; K_dec follows, as the padded P operand's rows 64-127
    static constexpr int SG_K = SG_P + 8192;
    static constexpr int SG_UT = SG_K + 16384;          // U rows of the slice, NB blocks of [64][64]
    static constexpr int STAGE = SG_UT + VS * 128;
    static constexpr int NST = VS == 64 ? 3 : 2;        // stages in the ring
    static constexpr int VEC = 528;                     // bytes of a chunk's vectors copied (129 floats used)
    static constexpr int CS_S = 0;                      // S [d][v] bf16, NB blocks of 16 KB
    static constexpr int CS_STAGE = CS_S + NB * 16384;
    static constexpr int CS_UP = CS_STAGE + NST * STAGE;  // U' [j][v] fp16, NB blocks of 8 KB
    static constexpr int CS_VEC = CS_UP + NB * 8192;    // the stages' vectors, NST x VEC
    static constexpr int CS_BAR = CS_VEC + NST * VEC;
    static constexpr int SMEM = CS_BAR + 192 + 1024;    // 18 barrier / flag words
    // TMEM: two buffers of [Q S; W S], dS, and OPB buffers of P U' (two when they
    // fit: the next chunk's P U' then needs no wait for this chunk's O epilogue)
    static constexpr int OPB = 5 * VS <= 512 ? 2 : 1;
    static constexpr uint32_t T_QW = 0, T_DS = 2 * VS, T_OP = 3 * VS;
    static constexpr uint32_t T_COLS = (3 + OPB) * VS <= 256 ? 256 : 512;
    static_assert(SMEM <= 232448, "chain kernel shared memory");
};

template <int N>
__device__ __forceinline__ void tmem_ldn(uint32_t taddr, float* v) {
    if constexpr (N == 16) tmem_ld16(taddr, v); else tmem_ld32(taddr, v);
}

// Bounded wait that also gives up once another role has given up (the clock
// and the flag are read every 32 polls).
__device__ __forceinline__ bool mbar_wait_or_abort(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
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
// every lane of the warp waits; the warp proceeds only if all lanes saw the phase
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    return __all_sync(0xffffffffu, mbar_wait_or_abort(bar, parity, abort_flag));
}
// after the warp's shared-memory writes and TMEM reads: one arrival per warp
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}

// CL: tokens per chunk (C, or 16 / 32), fixed at compile time so that the
// per-chunk arithmetic of C-token chunks stays constant-folded
template <int VS, int CL>
__global__ void __launch_bounds__(NT_C, 1)
chunk_chain_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap wmap,
                   const __grid_constant__ CUtensorMap utmap, const __grid_constant__ CUtensorMap pmap,
                   const __grid_constant__ CUtensorMap omap, const __grid_constant__ CUtensorMap kdmap, DeltaArgs a,
                   Work w, int64_t C0, int64_t segc) {
    // the next kernel's CTAs are placed only once this grid is done with its
    // work (pdl_trigger at the end): placed earlier, their waiting CTAs slowed
    // the chain's last CTAs
    pdl_wait();
    using Ly = ChainLayout<VS>;
    constexpr int NV = D / VS, CV = VS / 4;
    const int vp = blockIdx.x % NV;
    const int h = (blockIdx.x / NV) % a.H_v;
    const int seq_rank = blockIdx.x / (NV * a.H_v);  // CTAs start in this order: longest sequences first
    const int seq = a.cu != nullptr && w.order != nullptr ? w.order[seq_rank] : seq_rank;
    const int v0 = vp * VS;
    // chunk offsets of the sequence (one sequence without offsets: [0, ceil(T / CL)))
    constexpr int clen = CL;
    const int64_t cs = a.cu == nullptr ? 0 : w.coff[seq];
    const int64_t ce = a.cu == nullptr ? (a.T + clen - 1) / clen : w.coff[seq + 1];
    const int64_t c_lo = cs > C0 ? cs : C0, c_hi = ce < C0 + segc ? ce : C0 + segc;
    const int64_t sbase = ((int64_t)seq * a.H_v + h) * D * D;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (c_lo >= c_hi) {
        // no chunk of this sequence in this segment; an empty sequence's final
        // state is its initial state (written once, by the first segment)
        if (cs == ce && C0 == 0 && a.S_final != nullptr && a.S_final != a.S0)
            for (int e = tid; e < D * VS; e += NT_C) {
                const int64_t off = sbase + (int64_t)(e / VS) * D + v0 + e % VS;
                a.S_final[off] = a.S0 != nullptr ? a.S0[off] : 0.f;
            }
        // with the conv inside the kernels, so is its conv state: its V
        // channels and (first value head of the key head) its K and Q ones
        if (cs == ce && C0 == 0 && a.conv_state_out != nullptr && vp == 0) {
            const int r = a.H_v / a.H_k, kh = h / r;
            const int64_t cd = 2 * a.H_k * D + a.H_v * D;
            const uint16_t* src = static_cast<const uint16_t*>(a.conv_state0);
            uint16_t* dst = static_cast<uint16_t*>(a.conv_state_out);
            for (int e = tid; e < 3 * 3 * D; e += NT_C) {
                const int part = e / (3 * D), i = e % (3 * D);  // V, K, Q channel blocks
                if (part > 0 && h % r != 0) break;
                const int64_t ch = part == 0 ? 2 * a.H_k * D + h * D : (part == 1 ? a.H_k * D : 0) + kh * D;
                const int64_t off = ((int64_t)seq * cd + ch) * 3 + i;
                dst[off] = src != nullptr ? src[off] : 0;
            }
        }
        return;
    }
    const int kh = h / (a.H_v / a.H_k);
    const int xq = kh * D;
    int64_t s0, s1;
    seq_bounds(a.cu, seq, a.T, s0, s1);
    const int64_t L = s1 - s0;
    const int nch = (int)(c_hi - c_lo);

    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    constexpr int NST = Ly::NST;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Ly::CS_BAR);
    uint64_t* full = bars;        // [NST] stage landed (TMA)
    uint64_t* empty = bars + 3;   // [NST] stage consumed: tcgen05.commit after P U', and the O store has read it
    uint64_t* m1 = bars + 6;      // [Q S; W S] done
    uint64_t* m2 = bars + 7;      // dS done
    uint64_t* m3 = bars + 8;      // P U' done
    uint64_t* s_rdy = bars + 9;   // S operand written (16 compute warps)
    uint64_t* u_rdy = bars + 10;  // U' operands written, stage reads done (16 compute warps)
    uint64_t* o_done = bars + 11; // [2] O epilogue's TMEM reads of a P U' buffer done (8 q-row warps)
    uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + 13);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 14);
    uint64_t* o_staged = bars + 15;  // [NST] the stage's O tile staged (8 q-row warps)
    auto stage_of = [&](int k) { return sm + Ly::CS_STAGE + (k % NST) * Ly::STAGE; };
    auto vec_of = [&](int k) { return sm + Ly::CS_VEC + (k % NST) * Ly::VEC; };

    if (tid == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 2);
        }
        for (int i = 6; i < 9; ++i) mbar_init(&bars[i], 1);
        mbar_init(s_rdy, NT_COMP / 32);
        mbar_init(u_rdy, NT_COMP / 32);
        mbar_init(&o_done[0], NT_COMP / 64);
        mbar_init(&o_done[1], NT_COMP / 64);
        for (int i = 0; i < NST; ++i) mbar_init(&o_staged[i], NT_COMP / 64);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(tslot, Ly::T_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = *tslot;

    if (warp == W_TMA) {
        // ------------------------------------------------ TMA producer (lane 0)
        if (lane == 0) {
            int issued = 0;  // stages issued
            for (int k = 0; k < nch; ++k) {
                const int b = k % NST;
                if (k >= NST && !mbar_wait_or_abort(&empty[b], (uint32_t)((k / NST - 1) & 1), abort_flag)) break;
                const int64_t gcc = c_lo + k;
                uint8_t* st = stage_of(k);
                const int64_t uu = (gcc - C0) * a.H_v + h;
                // q from qkv, or the intra kernel's conv'd q tile of (chunk, key head)
                const int qx = w.q != nullptr ? 0 : xq;
                const int qy = w.q != nullptr ? (int)(((gcc - C0) * a.H_k + kh) * 64) : (int)(s0 + (gcc - cs) * clen);
                mbar_arrive_expect_tx(&full[b], Ly::STAGE + Ly::VEC);
                tma_load_2d(st + Ly::SG_QW, &qmap, &full[b], qx, qy);
                tma_load_2d(st + Ly::SG_QW + 8192, &wmap, &full[b], 0, (int)(uu * 64));
                tma_load_2d(st + Ly::SG_QW + 16384, &qmap, &full[b], qx + 64, qy);
                tma_load_2d(st + Ly::SG_QW + 24576, &wmap, &full[b], 64, (int)(uu * 64));
                tma_load_2d(st + Ly::SG_P, &pmap, &full[b], 0, (int)(uu * 64));
                tma_load_2d(st + Ly::SG_K, &kdmap, &full[b], 0, (int)(uu * 64));
                tma_load_2d(st + Ly::SG_K + 8192, &kdmap, &full[b], 64, (int)(uu * 64));
#pragma unroll
                for (int nb = 0; nb < Ly::NB; ++nb)
                    tma_load_2d(st + Ly::SG_UT + nb * 8192, &utmap, &full[b], v0 + 64 * nb, (int)(uu * 64));
                bulk_load(vec_of(k), w.vec + uu * (int64_t)(U_VEC / 4), (uint32_t)Ly::VEC, &full[b]);
                issued = k + 1;
            }
            // on abort: let the copies in flight land before the CTA exits
            if (*abort_flag)
                for (int k = issued - NST > 0 ? issued - NST : 0; k < issued; ++k)
                    mbar_wait(&full[k % NST], (uint32_t)((k / NST) & 1), kWaitNs);
        }
    } else if (warp == W_ST) {
        // ------------------------------------------------ O stores (lane 0)
        // once the 8 q-row warps have staged a full chunk's O tile, store it
        // by TMA; the stage is released when the store has read it
        if (lane == 0) {
            for (int k = 0; k < nch; ++k) {
                if (!mbar_wait_or_abort(&o_staged[k % NST], (uint32_t)((k / NST) & 1), abort_flag)) break;
                const int64_t lc = c_lo + k - cs;
                if (clen == C && L - lc * C >= C) {  // a full tile of C rows
                    uint8_t* otile = stage_of(k) + Ly::SG_P;
#pragma unroll
                    for (int nb = 0; nb < Ly::NB; ++nb)
                        tma_store_2d(&omap, otile + nb * 8192, h * D + v0 + 64 * nb, (int)(s0 + lc * C));
                    bulk_commit();
                    bulk_wait_read_all();
                }
                mbar_arrive(&empty[k % NST]);
            }
            bulk_wait_all();  // O stores complete before the CTA exits
        }
    } else if (warp == W_MMA) {
        // ------------------------------------------------ MMA issuer (lane 0)
        if (lane == 0) {
            const uint32_t bs = smem_u32(sm + Ly::CS_S);
            const uint32_t bup = smem_u32(sm + Ly::CS_UP);
            uint64_t* last = nullptr;  // the last commit, for the drain on abort
            uint32_t last_parity = 0;
            for (int k = 0; k < nch; ++k) {
                const int b = k & 1;  // TMEM buffers
                const uint32_t par = (uint32_t)(k & 1);
                const uint32_t st = smem_u32(stage_of(k));
                if (!mbar_wait_or_abort(&full[k % NST], (uint32_t)((k / NST) & 1), abort_flag)) break;
                if (!mbar_wait_or_abort(s_rdy, par, abort_flag)) break;
                tc_fence_after();
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    mma_bf16(tb + Ly::T_QW + VS * b,
                             sdesc_sw128(st + Ly::SG_QW + (q >> 2) * 16384 + (q & 3) * 32, 16, 1024),
                             sdesc_sw128(bs + q * 2048, 16384, 1024), idesc_bf16_f32(128, VS, 0, 1), q > 0);
                mma_commit(m1);
                last = m1;
                last_parity = par;
                if (!mbar_wait_or_abort(u_rdy, par, abort_flag)) break;
                tc_fence_after();
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    mma_bf16(tb + Ly::T_DS, sdesc_sw128(st + Ly::SG_K + q * 2048, 8192, 1024),
                             sdesc_sw128(bup + q * 2048, 8192, 1024), idesc_f16_f32(128, VS, 1, 1), q > 0);
                mma_commit(m2);
                last = m2;
                // P U' into buffer ob once the O epilogue of its previous use is done
                const int ob = Ly::OPB == 2 ? b : 0;
                if (k >= Ly::OPB &&
                    !mbar_wait_or_abort(&o_done[ob], (uint32_t)(((k / Ly::OPB) - 1) & 1), abort_flag))
                    break;
                tc_fence_after();
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    mma_bf16(tb + Ly::T_OP + VS * ob, sdesc_sw128(st + Ly::SG_P + q * 32, 16, 1024),
                             sdesc_sw128(bup + q * 2048, 8192, 1024), idesc_f16_f32(128, VS, 0, 1), q > 0);
                mma_commit(m3);
                mma_commit(&empty[k % NST]);
                last = m3;
            }
            if (*abort_flag && last != nullptr) mbar_wait(last, last_parity, kWaitNs);
        }
    } else {
        // ------------------------------------------------ compute warps
        // warp (quarter, cg): TMEM lanes 32 quarter + lane -- q rows 0-63, w rows
        // 64-127, state rows d -- and the slice's columns [c0, c0 + CV)
        const int quarter = warp & 3, cg = warp >> 2;
        const int lrow = quarter * 32 + lane;
        const int c0 = cg * CV;
        const uint32_t lo = (uint32_t)(quarter * 32) << 16;
        const bool qrow = quarter < 2;
        uint8_t* s_op = sm + Ly::CS_S + (c0 >> 6) * 16384;    // this thread's block of the S operand
        uint8_t* up_op = sm + Ly::CS_UP + (c0 >> 6) * 8192;   // ... of U' (fp16)
        const int cb = c0 & 63;
        int64_t ck_row0 = 0;
        if (a.ckpt_every > 0 && a.ckpt != nullptr) ck_row0 = ckpt_row0(a.cu, seq, a.T, a.ckpt_every);

        // initial state of this segment: the sequence's initial state at its
        // first chunk, else what the previous segment left in the carry.
        // Thread (lrow = d, cg) holds S[d][v0 + c0 .. v0 + c0 + CV).
        float sv[CV];
        {
            const float* src = (c_lo == cs) ? a.S0 : w.carry;
            const float* p = src != nullptr ? src + sbase + (int64_t)lrow * D + v0 + c0 : nullptr;
#pragma unroll
            for (int q = 0; q < CV; q += 4) {
                const float4 f = p != nullptr ? *reinterpret_cast<const float4*>(p + q) : make_float4(0.f, 0.f, 0.f, 0.f);
                sv[q] = f.x;
                sv[q + 1] = f.y;
                sv[q + 2] = f.z;
                sv[q + 3] = f.w;
            }
            store_row_bf16(s_op, lrow, cb, sv, CV);
            fence_async_smem();
            warp_arrive(s_rdy, lane);
        }

        for (int k = 0; k < nch; ++k) {
            const int b = k & 1;  // TMEM buffers
            const uint32_t par = (uint32_t)(k & 1);
            uint8_t* st = stage_of(k);
            const float* vs = reinterpret_cast<const float*>(vec_of(k));
            const int64_t gcc = c_lo + k;
            const int64_t lc = gcc - cs;
            const int64_t t0 = s0 + lc * clen;
            const int n = (int)(L - lc * clen < clen ? L - lc * clen : clen);

            if (!warp_wait(&full[k % NST], (uint32_t)((k / NST) & 1), abort_flag)) break;
            if (!warp_wait(m1, par, abort_flag)) break;
            tc_fence_after();
            // everything this chunk needs from its stage is read before u_rdy:
            // the stage is reloaded once P U' has completed
            const float eGn = vs[128];
            float erq = 0.f;
            if (!qrow) {
                // U' = U - W S for w row j (fp16 operand of MMA2 and MMA3)
                const int j = lrow - 64;
                const uint8_t* ut = st + Ly::SG_UT + (c0 >> 6) * 8192;
#pragma unroll
                for (int h16 = 0; h16 < CV; h16 += 16) {
                    float ws[16], up[16];
                    unpack8_h(*reinterpret_cast<const uint4*>(ut + sw128_off(j, cb + h16)), up);
                    unpack8_h(*reinterpret_cast<const uint4*>(ut + sw128_off(j, cb + h16 + 8)), up + 8);
                    tmem_ld16(tb + lo + Ly::T_QW + VS * b + c0 + h16, ws);
#pragma unroll
                    for (int q = 0; q < 16; ++q) up[q] -= ws[q];
                    store_row_h(up_op, j, cb + h16, up, 16);
                }
                fence_async_smem();
            } else {
                erq = vs[lrow];  // e^{G_i} rq_i of q row i
            }
            warp_arrive(u_rdy, lane);

            // S <- e^{G_n} S + dS -> bf16 S operand (and checkpoint)
            if (!warp_wait(m2, par, abort_flag)) break;
            tc_fence_after();
            {
                const int64_t done = lc * clen + n;
                float* ck = nullptr;
                if (a.ckpt_every > 0 && a.ckpt != nullptr && done % a.ckpt_every == 0) {
                    const int64_t crow = ck_row0 + done / a.ckpt_every - 1;
                    if (crow < a.ckpt_rows)
                        ck = a.ckpt + (crow * a.H_v + h) * D * D + (int64_t)lrow * D + v0 + c0;
                }
                float ds[CV];
                tmem_ldn<CV>(tb + lo + Ly::T_DS + c0, ds);
#pragma unroll
                for (int q = 0; q < CV; ++q) sv[q] = fmaf(eGn, sv[q], ds[q]);
                store_row_bf16(s_op, lrow, cb, sv, CV);
                fence_async_smem();
                if (ck != nullptr)
#pragma unroll
                    for (int q = 0; q < CV; q += 4)
                        *reinterpret_cast<float4*>(ck + q) = make_float4(sv[q], sv[q + 1], sv[q + 2], sv[q + 3]);
            }
            warp_arrive(s_rdy, lane);

            // O = (Q S) diag(e^G rq) + P U' of this chunk (q-row lanes), while
            // the next chunk's MMA1 runs.  A full chunk's O tile is staged in
            // the stage's consumed P | K region and written by TMA stores;
            // the last, partial chunk of a sequence is stored row by row.
            if (qrow) {
                if (!warp_wait(m3, par, abort_flag)) break;
                tc_fence_after();
                uint8_t* ostg = st + Ly::SG_P + (c0 >> 6) * 8192;
                bf16* o = static_cast<bf16*>(a.o) + ((t0 + lrow) * a.H_v + h) * D + v0 + c0;
#pragma unroll
                for (int h16 = 0; h16 < CV; h16 += 16) {
                    float qs[16], po[16];
                    tmem_ld16_twice(tb + lo + Ly::T_QW + VS * b + c0 + h16, qs,
                                    tb + lo + Ly::T_OP + VS * (Ly::OPB == 2 ? b : 0) + c0 + h16, po);
#pragma unroll
                    for (int q = 0; q < 16; ++q) po[q] = fmaf(erq, qs[q], po[q]);
                    if (n == C) {
                        store_row_bf16(ostg, lrow, cb + h16, po, 16);
                    } else if (lrow < n) {
                        store16(o + h16, po);
                        store16(o + h16 + 8, po + 8);
                    }
                }
                fence_async_smem();
                const int ob = Ly::OPB == 2 ? b : 0;
                warp_arrive(&o_done[ob], lane);
                if (lane == 0) mbar_arrive(&o_staged[k % NST]);
            }
        }
        if (!*abort_flag) {
            float* dst = a.S_final != nullptr ? a.S_final : w.carry;
            if (dst != nullptr) {
                float* p = dst + sbase + (int64_t)lrow * D + v0 + c0;
#pragma unroll
                for (int q = 0; q < CV; q += 4)
                    *reinterpret_cast<float4*>(p + q) = make_float4(sv[q], sv[q + 1], sv[q + 2], sv[q + 3]);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    pdl_trigger();
    if (tid == 0 && *abort_flag) atomicOr(&g_device_error, 1);
    if (warp == 0) tmem_dealloc(tb, Ly::T_COLS);
}

}  // namespace


PFN_cuTensorMapEncodeTiled_v12000 tensormap_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

unsigned long long current_context_id() {
    using GetCurrent = CUresult (*)(CUcontext*);
    using GetId = CUresult (*)(CUcontext, unsigned long long*);
    static GetCurrent get_current = nullptr;
    static GetId get_id = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            get_current = reinterpret_cast<GetCurrent>(p);
        p = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuCtxGetId", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            get_id = reinterpret_cast<GetId>(p);
    });
    CUcontext c = nullptr;
    unsigned long long id = 0;
    if (get_current == nullptr || get_id == nullptr || get_current(&c) != CUDA_SUCCESS || c == nullptr ||
        get_id(c, &id) != CUDA_SUCCESS)
        return 0;
    return id;
}

namespace {

bool encode2d(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows, uint32_t box_cols,
              uint32_t box_rows, CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16) {
    const PFN_cuTensorMapEncodeTiled_v12000 enc = tensormap_encoder();
    if (enc == nullptr) return false;
    cuuint64_t gdim[2] = {cols, rows};
    cuuint64_t gstr[1] = {cols * 2};
    cuuint32_t box[2] = {box_cols, box_rows};
    cuuint32_t es[2] = {1, 1};
    return enc(map, type, 2, const_cast<void*>(base), gdim, gstr, box,
               es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int sm_count() {
    static int count[128];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return 1;
    if (count[dev] == 0) {
        int c = 0;
        if (cudaDeviceGetAttribute(&c, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || c < 1) c = 1;
        count[dev] = c;
    }
    return count[dev];
}

// Chunk offsets, then per segment: intra, chain.  The chain splits each
// head's state into two 64-column slices when that still leaves at most one
// CTA per SM.  With a second stream s_pre and an event (one segment only), the
// offsets and intra kernels run on s_pre and the chain on s after the event,
// so the caller can overlap them with other work.  With two sets of
// intermediates (w[0], w[1]) and more than one segment, the intra kernels run
// on a stream of this call, each as soon as the chain two segments earlier is
// done with its buffer, so that a segment's intra kernel runs on the SMs the
// previous segment's chain leaves free; events order the two streams.
cudaError_t run_segments(const DeltaArgs& a, const Work* w, int nbuf, const Layout& Ly, cudaStream_t s,
                         cudaStream_t s_pre = nullptr, cudaEvent_t ev_pre = nullptr) {
    const uint64_t conv_dim = 2ull * a.H_k * D + (uint64_t)a.H_v * D;
    const uint64_t U = (uint64_t)Ly.segc * a.H_v;
    const bool split = (int64_t)a.n_seq * a.H_v * 2 <= sm_count();
    constexpr CUtensorMapDataType F16 = CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const bool conv = a.conv_w != nullptr;
    if (conv != (w[0].q != nullptr)) return cudaErrorInvalidValue;
    // qmap: qkv (x with the conv inside); cq[i]: where the chain reads q from
    CUtensorMap qmap, omap, wtmap[2], utmap[2], pmap[2], kdmap[2], cq[2];
    if (!encode2d(&qmap, a.qkv, conv_dim, (uint64_t)a.T, 64, 64) ||
        !encode2d(&omap, a.o, (uint64_t)a.H_v * D, (uint64_t)a.T, 64, 64))
        return cudaErrorInvalidValue;
    for (int i = 0; i < nbuf; ++i) {
        if (!encode2d(&wtmap[i], w[i].wt, 128, U * 64, 64, 64) || !encode2d(&utmap[i], w[i].ut, 128, U * 64, 64, 64, F16) ||
            !encode2d(&pmap[i], w[i].p, 64, U * 64, 64, 64, F16) || !encode2d(&kdmap[i], w[i].kd, 128, U * 64, 64, 64, F16))
            return cudaErrorInvalidValue;
        cq[i] = qmap;
        if (conv && !encode2d(&cq[i], w[i].q, 128, (uint64_t)Ly.segc * a.H_k * 64, 64, 64))
            return cudaErrorInvalidValue;
    }
    cudaError_t e = cudaSuccess;
    for (const void* k : {(const void*)chunk_intra_kernel<false, false>, (const void*)chunk_intra_kernel<true, false>,
                          (const void*)chunk_intra_kernel<false, true>, (const void*)chunk_intra_kernel<true, true>})
        if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, ISMEM);
    // the chain kernel for this call's chunk length
    const int clen = chunk_len(a);
    auto chain64 = clen == 16 ? chunk_chain_kernel<64, 16> : clen == 32 ? chunk_chain_kernel<64, 32>
                                                                        : chunk_chain_kernel<64, C>;
    auto chain128 = clen == 16 ? chunk_chain_kernel<128, 16> : clen == 32 ? chunk_chain_kernel<128, 32>
                                                                          : chunk_chain_kernel<128, C>;
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(chain64, cudaFuncAttributeMaxDynamicSharedMemorySize, ChainLayout<64>::SMEM);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(chain128, cudaFuncAttributeMaxDynamicSharedMemorySize, ChainLayout<128>::SMEM);
    if (e != cudaSuccess) return e;

    const bool two = ev_pre != nullptr && Ly.n_seg == 1;
    const bool overlap = ev_pre == nullptr && nbuf == 2 && Ly.n_seg > 1;
    if (ev_pre != nullptr && !two) {
        // more than one segment: everything in order on s, after s_pre's work
        if ((e = cudaEventRecord(ev_pre, s_pre)) != cudaSuccess || (e = cudaStreamWaitEvent(s, ev_pre, 0)) != cudaSuccess)
            return e;
    }
    // the overlapped schedule's stream and events, released (once their work
    // is done) when the call returns
    cudaStream_t aux = nullptr;
    cudaEvent_t ev_go = nullptr, ev_i[2] = {nullptr, nullptr}, ev_c[2] = {nullptr, nullptr};
    auto release = [&]() {
        for (cudaEvent_t ev : {ev_go, ev_i[0], ev_i[1], ev_c[0], ev_c[1]})
            if (ev != nullptr) cudaEventDestroy(ev);
        if (aux != nullptr) cudaStreamDestroy(aux);
    };
    if (overlap) {
        e = cudaStreamCreateWithFlags(&aux, cudaStreamNonBlocking);
        for (cudaEvent_t* ev : {&ev_go, &ev_i[0], &ev_i[1], &ev_c[0], &ev_c[1]})
            if (e == cudaSuccess) e = cudaEventCreateWithFlags(ev, cudaEventDisableTiming);
        if (e != cudaSuccess) {
            release();
            return e;
        }
    }
    cudaStream_t si = two ? s_pre : s;
    if (a.cu != nullptr && (e = launch_pdl(chunk_offsets_kernel, dim3(1), dim3(1024), 0, si, a.cu, a.n_seq, a.T, chunk_len(a),
                                           w[0].coff, w[0].order)) != cudaSuccess) {
        release();
        return e;
    }
    if (overlap) {
        // the intra kernels start after everything queued on s so far
        if ((e = cudaEventRecord(ev_go, s)) != cudaSuccess || (e = cudaStreamWaitEvent(aux, ev_go, 0)) != cudaSuccess) {
            release();
            return e;
        }
        si = aux;
    }
    for (int64_t seg = 0; seg < Ly.n_seg && e == cudaSuccess; ++seg) {
        const int64_t C0 = seg * Ly.segc;
        const int b = overlap ? (int)(seg & 1) : 0;
        // buffer b was last read by the chain of segment seg - 2
        if (overlap && seg >= 2 && (e = cudaStreamWaitEvent(aux, ev_c[b], 0)) != cudaSuccess) break;
        const dim3 ig((unsigned)a.H_v, (unsigned)Ly.segc);
        if (conv)
            e = a.neumann ? launch_pdl(chunk_intra_kernel<true, true>, ig, dim3(NT_I), ISMEM, si, qmap, wtmap[b],
                                       utmap[b], cq[b], a, w[b], C0)
                          : launch_pdl(chunk_intra_kernel<false, true>, ig, dim3(NT_I), ISMEM, si, qmap, wtmap[b],
                                       utmap[b], cq[b], a, w[b], C0);
        else
            e = a.neumann ? launch_pdl(chunk_intra_kernel<true, false>, ig, dim3(NT_I), ISMEM, si, qmap, wtmap[b],
                                       utmap[b], cq[b], a, w[b], C0)
                          : launch_pdl(chunk_intra_kernel<false, false>, ig, dim3(NT_I), ISMEM, si, qmap, wtmap[b],
                                       utmap[b], cq[b], a, w[b], C0);
        if (e != cudaSuccess) break;
        if (two || overlap) {
            cudaEvent_t ev = two ? ev_pre : ev_i[b];
            if ((e = cudaGetLastError()) != cudaSuccess || (e = cudaEventRecord(ev, si)) != cudaSuccess ||
                (e = cudaStreamWaitEvent(s, ev, 0)) != cudaSuccess)
                break;
        }
        if (split)
            e = launch_pdl(chain64, dim3((unsigned)(a.n_seq * a.H_v * 2)), dim3(NT_C),
                           ChainLayout<64>::SMEM, s, cq[b], wtmap[b], utmap[b], pmap[b], omap, kdmap[b], a, w[b], C0,
                           Ly.segc);
        else
            e = launch_pdl(chain128, dim3((unsigned)(a.n_seq * a.H_v)), dim3(NT_C),
                           ChainLayout<128>::SMEM, s, cq[b], wtmap[b], utmap[b], pmap[b], omap, kdmap[b], a, w[b], C0,
                           Ly.segc);
        if (e != cudaSuccess) break;
        if (overlap && (e = cudaEventRecord(ev_c[b], s)) != cudaSuccess) break;
    }
    release();
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

size_t chunk_split_workspace_bytes(int n_seq, int64_t T, int H_v) {
    return layout_of(n_seq, T, H_v).total;
}

size_t chunk_split_conv_workspace_bytes(int n_seq, int64_t T, int H_k, int H_v) {
    return layout_of(n_seq, T, H_v, H_k).total;
}

int chunk_split_launches(int n_seq, int64_t T, int H_v, bool has_cu, int chunk) {
    const int clen = chunk == 16 || chunk == 32 ? chunk : C;
    return (has_cu ? 1 : 0) + 2 * (int)segments_for(layout_of(n_seq, T, H_v), n_seq, T, clen);
}

cudaError_t launch_chunk_split(const DeltaArgs& a, void* workspace, size_t ws_bytes, cudaStream_t s) {
    Layout Ly = layout_of(a.n_seq, a.T, a.H_v, a.conv_w != nullptr ? a.H_k : 0);
    if (workspace == nullptr || ws_bytes < Ly.total) return cudaErrorInvalidValue;
    Work w[2];
    const int nbuf = Ly.two_bufs() ? 2 : 1;
    for (int i = 0; i < nbuf; ++i) {
        w[i] = work_at(static_cast<uint8_t*>(workspace), Ly, a.H_v, i);
        if (a.S_final != nullptr) w[i].carry = a.S_final;
    }
    // shorter chunks: the same buffers over more segments, the state carried
    // between them through final_state when the layout has no carry of its own
    Ly.n_seg = segments_for(Ly, a.n_seq, a.T, chunk_len(a));
    if (Ly.n_seg > 1 && w[0].carry == nullptr) return cudaErrorInvalidValue;
    return run_segments(a, w, nbuf, Ly, s);
}

cudaError_t launch_chunk_split_two(const DeltaArgs& a, void* workspace, size_t ws_bytes, cudaStream_t s_pre,
                                   cudaStream_t s_chain, cudaEvent_t ev_pre) {
    const Layout Ly = layout_of(a.n_seq, a.T, a.H_v);
    if (workspace == nullptr || ws_bytes < Ly.total || ev_pre == nullptr || a.conv_w != nullptr)
        return cudaErrorInvalidValue;
    Work w = work_at(static_cast<uint8_t*>(workspace), Ly, a.H_v);
    if (a.S_final != nullptr) w.carry = a.S_final;
    return run_segments(a, &w, 1, Ly, s_chain, s_pre, ev_pre);
}

namespace {
// One bounded wait that runs out: nothing arrives at the barrier.
__global__ void bounded_wait_selftest_kernel(uint64_t limit_ns) {
    __shared__ alignas(8) uint64_t bar;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        fence_mbar_init();
        if (!mbar_wait(&bar, 0, limit_ns)) atomicOr(&g_device_error, 1);
    }
}
}  // namespace

cudaError_t launch_bounded_wait_selftest(uint64_t limit_ns, cudaStream_t s) {
    bounded_wait_selftest_kernel<<<1, 32, 0, s>>>(limit_ns);
    return cudaGetLastError();
}

cudaError_t copy_device_error(cudaStream_t s, int* word) {
    return cudaMemcpyFromSymbolAsync(word, g_device_error, sizeof(int), 0, cudaMemcpyDeviceToHost, s);
}
cudaError_t clear_device_error(cudaStream_t s) {
    const int zero = 0;
    return cudaMemcpyToSymbolAsync(g_device_error, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s);
}

}  // namespace gdn

// ===================================================================== no-allocation variant
// gdn_chunk_prefill_noalloc runs the same two kernels with their scratch in a
// fixed array that is part of the library image, for callers that cannot
// allocate device memory.  Smaller segments than the workspace variant (the
// array is 24 MiB) mean more launches; the arithmetic is the same.
namespace gdn {

namespace {

constexpr size_t kStaticScratchBytes = 24ull << 20;
constexpr int kStaticMaxSeq = 16384;

static __device__ __align__(256) uint8_t g_prefill_scratch[kStaticScratchBytes];

std::mutex g_scratch_mu;
void* g_scratch_ptr[128];                // device address of g_prefill_scratch, per device ordinal
unsigned long long g_scratch_ctx[128];   // ... valid in the context with this id

Layout static_layout(int n_seq, int64_t T, int H_v) {
    return layout_for(n_seq, T, H_v, kStaticScratchBytes - align256(4 * ((size_t)kStaticMaxSeq + 1)) - 256,
                      (size_t)kStaticMaxSeq + 1, false, false);
}

}  // namespace

bool chunk_split_static_fits(int n_seq, int H_v) {
    if (n_seq < 1 || n_seq > kStaticMaxSeq) return false;
    // one chunk per segment must fit
    const Layout L = layout_for(n_seq, 0, H_v, 0, (size_t)kStaticMaxSeq + 1, false, false);
    return L.off_units + (size_t)H_v * UNIT_BYTES <= kStaticScratchBytes;
}

cudaError_t launch_chunk_split_static(const DeltaArgs& a, cudaStream_t s) {
    if (!chunk_split_static_fits(a.n_seq, a.H_v) || a.S_final == nullptr || a.conv_w != nullptr)
        return cudaErrorInvalidValue;
    // set-up once per device (per context of that device: a device reset
    // creates a new context, in which the array may sit elsewhere), with that
    // device current: the host-side name of the array is not a device address
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 128) return cudaErrorInvalidDevice;
    uint8_t* base = nullptr;
    {
        std::lock_guard<std::mutex> lock(g_scratch_mu);
        const unsigned long long ctx = current_context_id();
        if (g_scratch_ptr[dev] == nullptr || ctx == 0 || ctx != g_scratch_ctx[dev]) {
            void* p = nullptr;
            e = cudaGetSymbolAddress(&p, g_prefill_scratch);
            if (e != cudaSuccess) return e;
            g_scratch_ptr[dev] = p;
            g_scratch_ctx[dev] = current_context_id();  // the lookup made the device's context current
        }
        base = static_cast<uint8_t*>(g_scratch_ptr[dev]);
    }
    // layout inside the fixed array: chunk offsets, chunk metadata, then as
    // many chunks per segment as fit; final_state carries the state between
    // segments
    const Layout Ly = static_layout(a.n_seq, a.T, a.H_v);
    if (Ly.total > kStaticScratchBytes) return cudaErrorInvalidValue;
    Work w = work_at(base, Ly, a.H_v);
    w.carry = a.S_final;
    return run_segments(a, &w, 1, Ly, s);
}

}  // namespace gdn
