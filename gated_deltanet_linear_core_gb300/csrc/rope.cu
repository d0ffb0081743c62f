// gdn_rope and gdn_rope_kv_append: head norm and rotary positions of queries and
// keys, and the new tokens' keys and values into the pages of the cache.
//
// With f_j the frequency of pair j and p the token's position on the pair's axis,
//   x <- x / sqrt(mean x^2 + eps) w,   (a, b) <- mscale (a cos p f_j - b sin p f_j, b cos p f_j + a sin p f_j)
// A copy with some arithmetic on the way; HBM-bound.  Every warp works on its own, without barriers: it takes
// a few tokens (or a share of one's rows), looks up where they go in the cache (a lane each), makes their cosines and
// sines (a pair per lane, once for all heads), and copies their rows.  A lane holds both sides of
// its pairs, so a rotation needs no exchange, and its cosines stay in registers over the
// heads.  Rows come through shared memory, kStages steps ahead and across tokens (cp.async; a lane reads back what
// it copied itself): with loads into registers, four rows at a time, 32768 prompt tokens into the cache took
// 163 us, in blocks with barriers as well.
//
// Measured: those 121 us (691 MB, 84 % of the copy bandwidth; 76 M warp instructions; 131 with batches of tokens dealt to the
// warps in turns, of which some got one more); 32760 patches of 16 heads of 80 out of a fused projection 35 us (168 MB,
// 71 %; issue 52 %, 19 warps per SM that wait 2.1 of their 9.1 clocks an instruction for loads, positions among them, and 1.2 for
// shared memory: none of the three is full; 18 M warp instructions, 25 M and 37 us with the cache's part in the same code).
//
// The angle of a far position keeps no digits in f32: p f is held in turns, as a 64-bit
// fraction of one turn (f / 2 pi in f64, times 2^64), whose product with the integer p drops whole
// turns by itself.  It is off by at most |p f| 2^-52 + |p| 2^-62 rad.  As a signed number its value goes to f32,
// so that small angles keep their digits too (its upper 32 bits alone: 1.5e-9 rad, the sine of frequency 1e-7 at
// position 1 off by half a percent), and to sincospif.  For f32 outputs what that rounding leaves is made good to
// first order (5003 tokens of 7 heads of 72, 36 dims rotated: 2.9e-8 rel-L2 from 64 bits, 3.9e-8 without; bf16
// rounds 2^16 times as coarsely).
#include "gdn_common.cuh"
#include "gdn_launch.h"

namespace gdn {

namespace {

constexpr int NT = 128;
constexpr int NW = NT / 32;
constexpr int kStages = 4;
constexpr int kTokens = 4;  // of a warp at once (one by one, looking up and the cosines took two thirds of the time)

template <int BYTES> struct RawOf;
template <> struct RawOf<16> { using type = uint4; };
template <> struct RawOf<8> { using type = uint2; };
template <> struct RawOf<4> { using type = uint32_t; };
template <> struct RawOf<2> { using type = uint16_t; };

// V elements as they lie in memory, and as f32.
template <typename E, int V>
struct Vec {
    using Raw = typename RawOf<V * (int)sizeof(E)>::type;
    union {
        Raw raw;
        E e[V];
        uint32_t w[V * sizeof(E) >= 4 ? V * sizeof(E) / 4 : 1];
    };
    __device__ __forceinline__ Vec() {}
    // copies to shared memory, there after the next wait (two bytes: at once)
    __device__ __forceinline__ static void fetch(Raw* to, const E* p) {
        if constexpr (sizeof(Raw) == 2) {
            *to = *reinterpret_cast<const Raw*>(p);
        } else {
            const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(to));
            if constexpr (sizeof(Raw) == 16)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(p) : "memory");
            else
                asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(p), "n"(sizeof(Raw)) : "memory");
        }
    }
    __device__ __forceinline__ void store(E* p) const { *reinterpret_cast<Raw*>(p) = raw; }
};

// The 2 V elements of two vectors as V pairs of f32 (V = 1: one of each), and back.
template <typename E, int V>
__device__ __forceinline__ void widen(const Vec<E, V>& a, const Vec<E, V>& b, float2 (&z)[V]) {
    if constexpr (V == 1) {
        z[0] = make_float2(to_f(a.e[0]), to_f(b.e[0]));
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const Vec<E, V>& x = k < V / 2 ? a : b;
            const int at = k % (V / 2);
            if constexpr (sizeof(E) == 2) {
                const uint32_t w = x.w[at];
                z[k] = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
            } else {
                z[k] = make_float2(x.e[2 * at], x.e[2 * at + 1]);
            }
        }
    }
}
template <typename E, int V>
__device__ __forceinline__ void narrow(const float2 (&z)[V], Vec<E, V>& a, Vec<E, V>& b) {
    if constexpr (V == 1) {
        a.e[0] = from_f<E>(z[0].x);
        b.e[0] = from_f<E>(z[0].y);
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            Vec<E, V>& x = k < V / 2 ? a : b;
            const int at = k % (V / 2);
            if constexpr (sizeof(E) == 2) {
                x.w[at] = pack_bf16x2(z[k].x, z[k].y);
            } else {
                x.e[2 * at] = z[k].x;
                x.e[2 * at + 1] = z[k].y;
            }
        }
    }
}

// Where a token goes: sequence and place; false for a token outside every sequence.
__device__ __forceinline__ bool find_token(const RopeArgs& a, int64_t t, int& b, int64_t& pos) {
    int64_t end;
    if (a.cu == nullptr) {
        const uint32_t per = (uint32_t)a.T / (uint32_t)a.B;  // T < 2^31
        b = (int)((uint32_t)t / per);
        end = (int64_t)(b + 1) * per;
    } else {
        int64_t start;
        b = seq_of_token(a.cu, a.B, t);
        seq_bounds(a.cu, b, a.T, start, end);
        if (t < start || t >= end) return false;
    }
    pos = (int64_t)a.lens[b] - (end - t);
    return true;
}

// V pairs per item, IT items per lane; NEIGHBOURS: pairs (2j, 2j + 1), else (j, j + R / 2).
// `lg` lanes take a row (a power of two where a norm adds up over them), a warp `tb` tokens at once or one of `parts`
// shares of a token's rows: those of its query heads, key heads and value heads.  (One loop for the three, whose sources
// and places are picked per row: with a loop for each, a small call waited for its code, 320 tokens 17.8 us.)
// CTAs per SM: as many as the registers allow without spills (norm, no cache, 33000 tokens of 8 heads of 128, us with 4
// and 5: f32 53.7, 52.0, 16-byte bf16 accesses 30.9, 40.8).
constexpr int rope_ctas(int V, bool norm, bool cache) { return norm && (cache || V == 8) ? 4 : 5; }
template <typename E, int V, int IT, bool NEIGHBOURS, bool NORM, bool CACHE>
__global__ void __launch_bounds__(NT, rope_ctas(V, NORM, CACHE)) rope_kernel(RopeArgs a, int lg, int tb, int parts) {
    extern __shared__ __align__(16) float sm[];
    const int half = a.R >> 1, tid = threadIdx.x, warp = tid >> 5;
    uint64_t* turn_s = reinterpret_cast<uint64_t*>(sm);  // [half] frequencies, 2^-64 turns per position
    float* odd_s = sm + 2 * half;                        // [half] 0, NaN where the frequency is not finite
    int* axis_s = reinterpret_cast<int*>(sm + 3 * half); // [half] axes, -1: none
    float* w_s = sm + ((4 * half + 3) & ~3);             // [2][D] norm weights of queries and keys
    using Raw = typename Vec<E, V>::Raw;
    // the warp's stages [kStages][IT][a, b][32], of which a lane fills and reads its own
    Raw* stage_s = reinterpret_cast<Raw*>(w_s + 2 * a.D) + warp * (kStages * IT * 64) + (tid & 31);
    float* cos_s = reinterpret_cast<float*>(reinterpret_cast<Raw*>(w_s + 2 * a.D) + NW * (kStages * IT * 64)) +
                   warp * (2 * tb * half);               // [tb][half] of the warp's tokens
    float* sin_s = cos_s + tb * half;
    pdl_wait();
    pdl_trigger();
    if (tid < half) {  // (half is at most NT)
        double c = (double)a.inv_freq[tid] * 0.15915494309189533577;  // turns per position
        odd_s[tid] = (float)(c - c);
        const double part = fabs(c) - floor(fabs(c));
        const uint64_t turn = isfinite(c) ? (uint64_t)__double2ull_rn(part * 18446744073709551616.0) : 0;
        turn_s[tid] = c < 0 ? 0 - turn : turn;
        const int ax = a.axes != nullptr ? a.axes[tid] : 0;
        axis_s[tid] = ax >= 0 && ax < a.n_axes ? ax : -1;
    }
    for (int d = tid; NORM && d < a.D; d += NT) {
        if (a.q_w != nullptr) w_s[d] = a.q_w[d];
        if (a.k_w != nullptr) w_s[a.D + d] = a.k_w[d];
    }
    __syncthreads();

    const int wl = tid & 31, rw = 32 / lg, grp = wl / lg, lane = wl - grp * lg;  // rows of a warp at once
    const int items = (a.D >> 1) / V;
    int off_a[IT], off_b[IT], pair[IT];
    bool has[IT], turns[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int it = lane + i * lg, p = it * V;
        has[i] = it < items && grp < rw;
        turns[i] = has[i] && p < half;
        pair[i] = p;
        if (NEIGHBOURS) {
            off_a[i] = 2 * p;
            off_b[i] = 2 * p + V;
        } else if (p < half) {
            off_a[i] = p;
            off_b[i] = p + half;
        } else {  // dims that are not rotated, in two halves too
            off_a[i] = p + half;
            off_b[i] = p + (a.D >> 1);
        }
    }
    const int64_t cache_head = (int64_t)a.page_size * a.D;
    const int step = parts * rw;
    constexpr int kinds = CACHE ? 3 : 1;
    // the warp's items, shares of tokens: equal ranges, so that all warps end together
    const uint32_t all = (uint32_t)(a.T * parts), warps = gridDim.x * NW, nth = blockIdx.x * NW + warp;  // T < 2^31
    const uint32_t each = all / warps, more = all - each * warps;  // (several parts: few tokens)
    const int64_t item0 = (int64_t)nth * each + min(nth, more), item1 = item0 + each + (nth < more ? 1 : 0);
    auto split = [&](int64_t item, int64_t& token, int& h) {  // an item's token and this lane's first head
        token = parts == 1 ? item : (uint32_t)item / (uint32_t)parts;  // several parts: few tokens
        h = (int)(item - token * parts) * rw + grp;
    };
    auto batch = [&](int64_t item) { return parts == 1 ? (int)min((int64_t)tb, item1 - item) : 1; };  // tokens at once
    // the rows, those of an item's queries, keys and values after one another, kStages ahead
    struct {
        int64_t item, token, skip;  // an item, its token, elements between a lane's rows
        const E* x;
        int h0, h, heads, kind, stage;
    } in;
    in.item = item0;
    in.stage = 0;
    auto enter = [&](int kind) {  // the token's rows of a kind
        in.kind = kind;
        in.h = in.h0;
        if (!CACHE) kind = 0;
        in.heads = kind == 0 ? a.H_q : a.H_kv;
        const int64_t tok = kind == 0 ? a.q_tok : kind == 1 ? a.k_tok : a.v_tok;
        const int64_t head = kind == 0 ? a.q_head : kind == 1 ? a.k_head : a.v_head;
        in.x = static_cast<const E*>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) + in.token * tok + in.h * head;
        in.skip = step * head;
    };
    auto begin = [&] {
        if (in.item >= item1) return;
        split(in.item, in.token, in.h0);
        enter(0);
    };
    begin();
    auto fetch = [&] {
        if (in.item < item1) {
            if (in.h < in.heads)
#pragma unroll
                for (int i = 0; i < IT; ++i)
                    if (has[i]) {
                        Vec<E, V>::fetch(stage_s + (in.stage * IT + i) * 64, in.x + off_a[i]);
                        Vec<E, V>::fetch(stage_s + (in.stage * IT + i) * 64 + 32, in.x + off_b[i]);
                    }
            in.h += step;
            in.x += in.skip;
            if (in.h - grp >= in.heads) {  // (the lanes of a warp go on together)
                // (a share of a token's heads that has no key head has no rows of the later kinds: no stage, as below)
                if (CACHE && in.kind + 1 < kinds && in.h0 - grp < a.H_kv) {
                    enter(in.kind + 1);
                } else {
                    ++in.item;
                    begin();
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        in.stage = (in.stage + 1) % kStages;
    };
#pragma unroll 1
    for (int i = 0; i < kStages; ++i) fetch();
    int stage = 0;
    const float inv_d = 1.0f / (float)a.D;
    const uint32_t per_half = (65536 + half - 1) / half;  // e / half = e per_half / 65536 for e < 65536 / half
    float2 wt[IT][V];  // the norm's weights of a lane's dims
    auto weights = [&](int kind) {
        const float* wr = w_s + (kind == 0 ? 0 : a.D);
#pragma unroll
        for (int i = 0; i < IT; ++i)
            if (has[i])
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const float* wa = wr + (V == 1 ? off_a[i] : k < V / 2 ? off_a[i] + 2 * k : off_b[i] + 2 * k - V);
                    wt[i][k] = V == 1 ? make_float2(wa[0], wr[off_b[i]]) : *reinterpret_cast<const float2*>(wa);
                }
    };
    if (NORM && !CACHE) weights(0);
    for (int64_t item = item0; item < item1;) {
        int64_t first;
        int h0;
        split(item, first, h0);
        const int n = batch(item);
        item += n;
        // lane i: token i's place in its sequence, and its row (page, head 0, position in page), -1: nowhere
        int64_t its_row = -1, its_pos = 0;
        bool its_member = true;
        if (CACHE && wl < n) {
            int b;
            its_member = find_token(a, first + wl, b, its_pos);
            if (its_member && its_pos >= 0 && its_pos < (int64_t)a.max_pages * a.page_size) {
                const int pg = (int)((uint32_t)its_pos / (uint32_t)a.page_size);
                const int page = a.table[(int64_t)b * a.max_pages + pg];
                if (page >= 0 && page < a.n_pages)
                    its_row = (int64_t)page * a.H_kv * a.page_size + (its_pos - (int64_t)pg * a.page_size);
            }
        }
        __syncwarp();  // the cosines before are read
        for (int e0 = 0; e0 < n * half; e0 += 32) {
            const int e = e0 + wl, t = min((int)((uint32_t)e * per_half >> 16), n - 1), j = e - t * half;
            int64_t p = CACHE ? __shfl_sync(0xffffffffu, its_pos, t) : 0;
            if (e < n * half) {
                const int ax = axis_s[j];
                if (a.positions != nullptr) p = ax >= 0 ? a.positions[ax * a.T + first + t] : 0;
                const int64_t f = ax >= 0 ? (int64_t)((uint64_t)p * turn_s[j]) : 0;  // 2^-63 half turns
                const float odd = ax >= 0 ? odd_s[j] : 0.f;
                float s, c;
                if constexpr (sizeof(E) == 2) {
                    sincospif((float)f * 0x1p-63f + odd, &s, &c);
                } else {
                    // the nearest multiple of 2^-24 half turns, which f32 holds (one half turn and minus one are the
                    // same), and the rest
                    const int32_t top = (int32_t)((int64_t)((uint64_t)f + (1ull << 38)) >> 39);
                    const float rest = (float)(int64_t)((uint64_t)f - ((uint64_t)(int64_t)top << 39)) * (0x1p-63f * 3.14159265358979f);
                    float s0, c0;
                    sincospif((float)top * 0x1p-24f + odd, &s0, &c0);
                    s = fmaf(c0, rest, s0);
                    c = fmaf(-s0, rest, c0);
                }
                cos_s[e] = c * a.mscale;
                sin_s[e] = s * a.mscale;
            }
        }
        __syncwarp();
#pragma unroll 1
        for (int t = 0; t < n; ++t) {
        const int64_t token = first + t, row = CACHE ? __shfl_sync(0xffffffffu, its_row, t) : -1;
        const bool member = !CACHE || __shfl_sync(0xffffffffu, (int)its_member, t) != 0;
        float co[IT][V], si[IT][V];
#pragma unroll
        for (int i = 0; i < IT; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int at = turns[i] ? t * half + pair[i] + v : 0;
                co[i][v] = cos_s[at];
                si[i][v] = sin_s[at];
            }
#pragma unroll 1
        for (int kind = 0; kind < kinds; ++kind) {
            const int heads = kind == 0 ? a.H_q : a.H_kv;
            const int64_t head = kind == 0 ? a.o_head : cache_head;
            E* to = kind == 0 ? static_cast<E*>(a.q_out) + token * a.o_tok
                              : static_cast<E*>(kind == 1 ? a.k_cache : a.v_cache) + row * a.D;
            to += h0 * head;
            const int64_t skip = step * head;
            const bool there = member && grp < rw && (kind == 0 || row >= 0);
            const bool norm = (kind == 0 ? a.q_w : kind == 1 ? a.k_w : nullptr) != nullptr;
            if (NORM && CACHE && norm) weights(kind);
#pragma unroll 1
            for (int h = h0; h - grp < heads; h += step, to += skip) {
                Vec<E, V> xa[IT], xb[IT];
                asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
#pragma unroll
                for (int i = 0; i < IT; ++i) {
                    xa[i].raw = stage_s[(stage * IT + i) * 64];
                    xb[i].raw = stage_s[(stage * IT + i) * 64 + 32];
                }
                stage = (stage + 1) % kStages;
                fetch();
                if (kind < 2) {  // values are copied
                    float2 z[IT][V];
#pragma unroll
                    for (int i = 0; i < IT; ++i) widen<E, V>(xa[i], xb[i], z[i]);
                    if (NORM && norm) {
                        float2 sq = make_float2(0.f, 0.f);
#pragma unroll
                        for (int i = 0; i < IT; ++i)
                            if (has[i])
#pragma unroll
                                for (int k = 0; k < V; ++k) sq = __ffma2_rn(z[i][k], z[i][k], sq);
                        float sum = h < heads ? sq.x + sq.y : 0.f;
                        for (int o = lg >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                        const float scale = rsqrtf(fmaf(sum, inv_d, a.eps));
#pragma unroll
                        for (int i = 0; i < IT; ++i) {
                            if (!has[i]) continue;
#pragma unroll
                            for (int k = 0; k < V; ++k) z[i][k] = __fmul2_rn(__fmul2_rn(z[i][k], make_float2(scale, scale)), wt[i][k]);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < IT; ++i) {
                        if (turns[i]) {
                            if constexpr (NEIGHBOURS || V == 1) {
#pragma unroll
                                for (int k = 0; k < V; ++k)
                                    z[i][k] = __ffma2_rn(z[i][k], make_float2(co[i][k], co[i][k]),
                                                         __fmul2_rn(make_float2(z[i][k].y, z[i][k].x),
                                                                    make_float2(-si[i][k], si[i][k])));
                            } else {
#pragma unroll
                                for (int k = 0; k < V / 2; ++k) {
                                    const float2 p = z[i][k], q = z[i][V / 2 + k];
                                    const float2 c = make_float2(co[i][2 * k], co[i][2 * k + 1]);
                                    const float2 sn = make_float2(si[i][2 * k], si[i][2 * k + 1]);
                                    z[i][k] = __ffma2_rn(p, c, __fmul2_rn(q, make_float2(-sn.x, -sn.y)));
                                    z[i][V / 2 + k] = __ffma2_rn(q, c, __fmul2_rn(p, sn));
                                }
                            }
                        }
                        if ((NORM && norm) || turns[i]) narrow<E, V>(z[i], xa[i], xb[i]);  // what is neither passes bit for bit
                    }
                }
                if (there && h < heads)
#pragma unroll
                    for (int i = 0; i < IT; ++i)
                        if (has[i]) {
                            xa[i].store(to + off_a[i]);
                            xb[i].store(to + off_b[i]);
                        }
            }
        }
        }
    }
}

template <typename E, int V, bool NEIGHBOURS>
cudaError_t launch_v(const RopeArgs& a, cudaStream_t s) {
    constexpr int IT = V >= 4 ? 1 : 4 / V;  // 128 pairs at most
    const int items = (a.D >> 1) / V, half = a.R >> 1;
    int lg = items;
    if (a.q_w != nullptr || a.k_w != nullptr || items > 32) {
        lg = 1;
        while (lg < 32 && lg < items) lg *= 2;
    }
    const int rw = 32 / lg;
    // few tokens: several warps share one's rows
    const int most = (a.H_q + rw - 1) / rw;
    int64_t parts = 152 * 4 * NW / a.T;  // all warps at once
    parts = parts < 1 ? 1 : (parts > most ? most : parts);
    const bool norm = a.q_w != nullptr || a.k_w != nullptr;
    const int ctas = 152 * rope_ctas(V, norm, a.k_cache != nullptr);  // resident at once
    const int64_t each = (a.T + ctas * NW - 1) / (ctas * NW);  // tokens of a warp
    const int tb = (int)(each < kTokens ? each : kTokens);
    int64_t blocks = (a.T * parts + NW - 1) / NW;
    blocks = blocks > ctas ? ctas : blocks;
    const size_t smem = sizeof(float) * (((4 * half + 3) & ~3) + 2 * a.D + NW * 2 * tb * half) +
                        (size_t)NW * kStages * IT * 64 * V * sizeof(E);
    const auto kernel = a.k_cache != nullptr
                            ? (norm ? rope_kernel<E, V, IT, NEIGHBOURS, true, true> : rope_kernel<E, V, IT, NEIGHBOURS, false, true>)
                            : (norm ? rope_kernel<E, V, IT, NEIGHBOURS, true, false> : rope_kernel<E, V, IT, NEIGHBOURS, false, false>);
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3((unsigned)blocks), dim3(NT), smem, s, a, lg, tb, (int)parts);
}

template <typename E, bool NEIGHBOURS>
cudaError_t launch_e(const RopeArgs& a, cudaStream_t s) {
    // the widest access that the halves of the rotated dims and of the others allow
    const int both = (a.R >> 1) | (a.D >> 1);
    if (sizeof(E) == 2 && both % 8 == 0) return launch_v<E, sizeof(E) == 2 ? 8 : 4, NEIGHBOURS>(a, s);
    if (both % 4 == 0) return launch_v<E, 4, NEIGHBOURS>(a, s);
    if (both % 2 == 0) return launch_v<E, 2, NEIGHBOURS>(a, s);
    return launch_v<E, 1, NEIGHBOURS>(a, s);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, gdn_dtype_t dt, cudaStream_t s) {
    if (a.T == 0) return cudaSuccess;
    if (dt == GDN_BF16) return a.neighbours ? launch_e<bf16, true>(a, s) : launch_e<bf16, false>(a, s);
    return a.neighbours ? launch_e<float, true>(a, s) : launch_e<float, false>(a, s);
}

}  // namespace gdn
