// Attention of the newest tokens over the paged cache on CUDA cores (f32, and
// the bf16 shapes the tensor-core kernel does not take), and the kernel that
// joins the partial results of either.
//
// The pages name these layers without defining them beyond their head layout
// and output gate (NxD-Inference PR "Add Qwen3-Coder-Next ... contrib model":
// GQA softmax attention, head_dim 256, attn_output_gate); the arithmetic is
// plain softmax attention: with n = len - (K - 1 - i) for new token i,
//   s_t = scale q . k_t,  out = sum_{t<n} e^{s_t} v_t / sum_{t<n} e^{s_t}
//   [* sigmoid(gate)],    lse = log sum_{t<n} e^{s_t}
// one pass over the tokens with the running maximum m, sum l and output O:
//   m' = max(m, max s),  l <- l 2^(m-m') + sum 2^(s-m'),  O <- O 2^(m-m') + P V
// (scores in the log2 domain, all statistics in f32; m is moved only when a
// score exceeds it by 2^8, so O is rarely rescaled).  2^x is the hardware's
// approximate form throughout, for weights and for the joins' factors, in f32
// too: within 2^-22, some steps of f32, and 0 below 2^-126.
//
// Reading the cache is the bound of few rows (64 ragged sequences of 512 to 8192
// tokens in f32, 4 rows of head dim 128: 168 us, 6.5 TB/s; 8 rows are bound by
// the instructions of the products: 227 us), so every warp works on its own,
// without barriers between tokens: a lane holds 4 (or 8) dims of the rows' Q and
// O, a warp takes T tokens at a time, and a lane copies its dims of the next T (or
// 2 T) tokens' K and V into shared memory, where it alone reads them (cp.async; with
// loads straight into registers, which overlap with no arithmetic of the warp,
// 211 and 298 us).  The T R partial dot products are joined over the lanes by
// halving, which leaves each lane a score, and the weights go back through a few
// words of shared memory.
// Blocks have at most kAttnFfmaRows rows: 16 in one pass (registers for 8 warps
// only) took longer than two passes of 8, of which the second reads from L2.
// The warps' results are joined at the end of a segment.
#include "attn_common.cuh"

#include "tc_ptx.cuh"

namespace gdn {

namespace {

using namespace attn;

constexpr int TT = 64;  // tokens of a unit

// Copies 16 (or 8) bytes to shared memory, or zeros.
__device__ __forceinline__ void copy_async(float4* dst, const void* src, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(dst)), "l"(src), "r"(real ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy_async(uint2* dst, const void* src, bool real) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(tc::smem_u32(dst)), "l"(src), "r"(real ? 8 : 0)
                 : "memory");
}
// four consecutive elements, and as f32
template <typename E> struct Four { using type = float4; };
template <> struct Four<bf16> { using type = uint2; };
__device__ __forceinline__ float4 as_f32(float4 u) { return u; }
__device__ __forceinline__ float4 as_f32(uint2 u) {
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ float4 ld4(const float* p) { return __ldcs(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ float4 ld4(const bf16* p) { return as_f32(__ldcs(reinterpret_cast<const uint2*>(p))); }

__device__ __forceinline__ void store4(float* p, float4 y) { *reinterpret_cast<float4*>(p) = y; }
__device__ __forceinline__ void store4(bf16* p, float4 y) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
}

// R rows per block (of which block_rows are real), NV x 4 dims per lane, T tokens at a time, NW warps, ST stages.
template <typename E, int R, int NV>
struct Ffma {
    static constexpr int T = R == 4 ? 8 : 4;
    // As many warps as registers allow, stages of 192 KB in all in f32 (4 rows of head dim 128: 8 warps with 3 stages
    // 194 us, 12 with 2 168; 8 rows of head dim 256: 12 warps spill).  bf16 has room for more, but is bound by issue: more
    // stages of it only cost at the start (4 rows: 16 warps with 2 stages 150 us, with 3 160, 12 with 4 184).
    static constexpr int NW = R == 4 && sizeof(E) == 4 ? 12 / NV : 16 / NV;
    static constexpr int ST = R == 4 ? 2 : 3;
    static constexpr int STAGE = 2 * T * NV * 32;             // fours of a warp's stage: K, then V
    static constexpr int NT = NW * 32;
    static constexpr int C = T * R;       // scores of T tokens
    static constexpr int S = C / 32;      // scores per lane
    static constexpr int PER = R / S;     // lanes per token
    // floats of all warps' stages, a warp's at least those of its outputs (R rows of NV x 128)
    static constexpr int STAGE_FLOATS = NW * ST * STAGE * (int)sizeof(typename Four<E>::type) / 4;
    static_assert(C % 32 == 0 && PER * T == 32, "a lane holds whole scores");
    static_assert(STAGE_FLOATS / NW >= R * NV * 128, "outputs fit the stages");
};

template <typename E, int R, int NV>
__global__ void __launch_bounds__(Ffma<E, R, NV>::NT, 1) attn_ffma_kernel(AttnArgs a) {
    using G = Ffma<E, R, NV>;
    constexpr int T = G::T, NW = G::NW, S = G::S, PER = G::PER;
    using F = typename Four<E>::type;
    extern __shared__ __align__(16) float sm[];
    float* p_s = sm + G::STAGE_FLOATS;  // [NW][T][R] weights
    float* m_s = p_s + NW * G::C;               // [NW][R]
    float* l_s = m_s + NW * R;                  // [NW][R]
    int* vis_s = reinterpret_cast<int*>(l_s + NW * R);  // [R] tokens a row sees
    const int D = a.D, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // the warp's stages [ST][K, V][T][NV][32], of which a lane fills and reads its own; at the end its outputs [R][D]
    F* stages = reinterpret_cast<F*>(sm) + warp * G::ST * G::STAGE + lane;
    constexpr int O_STEP = G::STAGE_FLOATS / NW;
    float* o_w = sm + warp * O_STEP;

    pdl_wait();
    pdl_trigger();
    int n_cta = gridDim.x;
    const Place place = find_place(a, TT, blockIdx.x, n_cta);
    const int64_t u0 = (int)blockIdx.x < n_cta ? cta_begin(place.total, blockIdx.x, n_cta) : 0;
    const int64_t u1 = (int)blockIdx.x < n_cta ? cta_begin(place.total, blockIdx.x + 1, n_cta) : 0;
    Walk walk(place, u0, u1);
    const E* kc = static_cast<const E*>(a.k_cache);
    const E* vc = static_cast<const E*>(a.v_cache);
    const bool has[2] = {lane * 4 < D, NV > 1 && (lane + 32) * 4 < D};
    float* p_w = p_s + warp * G::C;
    const int my_t = lane / PER, my_r = lane % PER * S;  // token of the lane's scores, first row

    Segment s;
    bool more = walk.next(a, TT, s);
    if (tid == G::NT - 32) write_join_task(a, place, walk, more ? &s : nullptr, blockIdx.x, n_cta);
    for (; more; more = walk.next(a, TT, s)) {
        const int r0 = s.rb * a.rb_rows, nr = block_rows(a, s.rb);
        const int end = min(s.len, s.tile1 * TT);
        const int32_t* table = a.table + (int64_t)s.b * a.max_pages;
        auto place_of = [&](int t) -> int64_t {  // element offset of token t's row, -1: no such token
            if (t >= end) return -1;
            const int pg = t / a.page_size, page = table[pg];
            if (page < 0 || page >= a.n_pages) return -1;
            return (((int64_t)page * a.H_kv + s.h) * a.page_size + (t - pg * a.page_size)) * D;
        };
        auto issue = [&](int stage, int64_t off) {  // lane i: token i of the T
            F* to = stages + stage * G::STAGE;
#pragma unroll
            for (int t = 0; t < T; ++t) {
                const int64_t at = __shfl_sync(0xffffffffu, off, t);
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    const bool real = at >= 0 && has[v];
                    const int64_t from = real ? at + (lane + 32 * v) * 4 : 0;
                    copy_async(to + (t * NV + v) * 32, kc + from, real);
                    copy_async(to + ((T + t) * NV + v) * 32, vc + from, real);
                }
            }
        };
        int t0 = s.tile0 * TT + warp * T;
        int64_t next = place_of(t0 + lane % T);
#pragma unroll 1
        for (int i = 0; i < G::ST; ++i) {
            const int64_t off = next;
            next = place_of(t0 + (i + 1) * NW * T + lane % T);
            issue(i, off);
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
        int stage = 0;
        if (tid < R) vis_s[tid] = tid < nr ? visible(a, s.len, r0 + tid) : 0;
        float4 q[R][NV], o[R][NV];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                o[r][v] = make_float4(0.f, 0.f, 0.f, 0.f);
                q[r][v] = o[r][v];
                if (r < nr && has[v])
                    q[r][v] = ld4(static_cast<const E*>(a.q) + row_index(a, s.b, s.h, r0 + r) * D + (lane + 32 * v) * 4);
            }
        __syncthreads();
        float m[S], l[S];
        int vis[S];
#pragma unroll
        for (int i = 0; i < S; ++i) {
            m[i] = kNone;
            l[i] = 0.f;
            vis[i] = vis_s[my_r + i];
        }
        const int least = vis_s[0];
        for (; t0 < end; t0 += NW * T) {
            asm volatile("cp.async.wait_group %0;" ::"n"(G::ST - 1) : "memory");
            const F* k_s = stages + stage * G::STAGE;
            const F* v_s = k_s + T * NV * 32;
            // ---- scores: partial dot products, joined over the lanes
            float x[G::C];
#pragma unroll
            for (int t = 0; t < T; ++t) {
                float4 kv[NV];
#pragma unroll
                for (int v = 0; v < NV; ++v) kv[v] = as_f32(k_s[(t * NV + v) * 32]);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    float2 d = __fmul2_rn(make_float2(kv[0].x, kv[0].y), make_float2(q[r][0].x, q[r][0].y));
                    d = __ffma2_rn(make_float2(kv[0].z, kv[0].w), make_float2(q[r][0].z, q[r][0].w), d);
                    if constexpr (NV > 1) {
                        d = __ffma2_rn(make_float2(kv[NV - 1].x, kv[NV - 1].y),
                                       make_float2(q[r][NV - 1].x, q[r][NV - 1].y), d);
                        d = __ffma2_rn(make_float2(kv[NV - 1].z, kv[NV - 1].w),
                                       make_float2(q[r][NV - 1].z, q[r][NV - 1].w), d);
                    }
                    x[t * R + r] = d.x + d.y;
                }
            }
            join_lanes<G::C>(x, lane, [](float u, float w) { return u + w; });
            const bool tail = t0 + T > least || t0 + T > end;
            bool over = false;
#pragma unroll
            for (int i = 0; i < S; ++i) {
                x[i] *= a.scale_log2;
                if (tail && (t0 + my_t >= vis[i] || t0 + my_t >= end)) x[i] = -INFINITY;
                over = over || x[i] - m[i] > kSlack;
            }
            if (__any_sync(0xffffffffu, over)) {  // new maxima; sums and outputs so far are scaled to them
                float f[S];
#pragma unroll
                for (int i = 0; i < S; ++i) {
                    float top = x[i];
#pragma unroll
                    for (int w = PER; w < 32; w *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
                    if (!(top > m[i] + kSlack)) top = m[i];  // rows do not move with one another
                    f[i] = tc::ex2_approx(m[i] - top);
                    m[i] = top;
                    l[i] *= f[i];
                }
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float g = __shfl_sync(0xffffffffu, f[r % S], r / S);
#pragma unroll
                    for (int v = 0; v < NV; ++v) {
                        o[r][v].x *= g; o[r][v].y *= g; o[r][v].z *= g; o[r][v].w *= g;
                    }
                }
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < S; ++i) {
                const float p = tc::ex2_approx(x[i] - m[i]);
                l[i] += p;
                p_w[lane * S + i] = p;  // [token][row]
            }
            __syncwarp();
            // ---- O += P V
#pragma unroll
            for (int t = 0; t < T; ++t) {
                float p[R];
#pragma unroll
                for (int r = 0; r < R; r += 4) {
                    const float4 w = *reinterpret_cast<const float4*>(p_w + t * R + r);
                    p[r] = w.x; p[r + 1] = w.y; p[r + 2] = w.z; p[r + 3] = w.w;
                }
                float4 vv[NV];
#pragma unroll
                for (int v = 0; v < NV; ++v) vv[v] = as_f32(v_s[(t * NV + v) * 32]);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    // a hidden value may be anything: a weight of 0 must not meet it
                    if (tail && t0 + t >= vis_s[r]) continue;
                    const float2 pp = make_float2(p[r], p[r]);
#pragma unroll
                    for (int v = 0; v < NV; ++v) {
                        float2* acc = reinterpret_cast<float2*>(&o[r][v]);
                        acc[0] = __ffma2_rn(pp, make_float2(vv[v].x, vv[v].y), acc[0]);
                        acc[1] = __ffma2_rn(pp, make_float2(vv[v].z, vv[v].w), acc[1]);
                    }
                }
            }
            __syncwarp();  // the reads of this stage come first
            const int64_t off = next;
            next = place_of(t0 + (G::ST + 1) * NW * T + lane % T);
            issue(stage, off);
            asm volatile("cp.async.commit_group;" ::: "memory");
            stage = stage + 1 < G::ST ? stage + 1 : 0;
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
        // ---- the warps' parts, then the rows (or this segment's part of them)
#pragma unroll
        for (int i = 0; i < S; ++i) {
#pragma unroll
            for (int w = PER; w < 32; w *= 2) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
            if (my_t == 0) {
                m_s[warp * R + my_r + i] = m[i];
                l_s[warp * R + my_r + i] = l[i];
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int v = 0; v < NV; ++v)
                if (has[v]) *reinterpret_cast<float4*>(o_w + r * D + (lane + 32 * v) * 4) = o[r][v];
        __syncthreads();
        const bool whole = s.tile1 - s.tile0 == s.tiles;
        float* slot = slot_ptr(a, part_slot(s));
        for (int e = tid; e < nr * (D / 4); e += G::NT) {
            const int r = e / (D / 4), d = (e - r * (D / 4)) * 4;
            float top = kNone, sum = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) top = fmaxf(top, m_s[w * R + r]);
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int w = 0; w < NW; ++w) {
                const float f = tc::ex2_approx(m_s[w * R + r] - top);
                const float4 x = *reinterpret_cast<const float4*>(sm + w * O_STEP + r * D + d);
                sum = fmaf(f, l_s[w * R + r], sum);
                y.x = fmaf(f, x.x, y.x); y.y = fmaf(f, x.y, y.y); y.z = fmaf(f, x.z, y.z); y.w = fmaf(f, x.w, y.w);
            }
            if (whole) {
                const int64_t row = row_index(a, s.b, s.h, r0 + r);
                const float inv = sum == 0.f ? 0.f : 1.0f / sum;
                y.x *= inv; y.y *= inv; y.z *= inv; y.w *= inv;
                if (a.gate != nullptr && sum != 0.f) {  // a row that sees nothing is 0 whatever its gate holds
                    const float4 g = ld4(static_cast<const E*>(a.gate) + row * D + d);
                    y.x *= sigmoid_f(g.x); y.y *= sigmoid_f(g.y); y.z *= sigmoid_f(g.z); y.w *= sigmoid_f(g.w);
                }
                store4(static_cast<E*>(a.out) + row * D + d, y);
                if (d == 0 && a.lse != nullptr) a.lse[row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
            } else {
                *reinterpret_cast<float4*>(slot + a.stat_floats + r * D + d) = y;
                if (d == 0) {
                    slot[r] = top == kNone ? -INFINITY : top;
                    slot[a.rb_rows + r] = sum;
                }
            }
        }
        __syncthreads();
    }
}

// Joins the parts of every item that more than one CTA worked on.  The CTAs
// whose ranges start inside an item (blockIdx.x + 1) share its rows, gridDim.y
// blocks each.  A group of threads (blockDim.x, 4 columns each) takes a row, or a
// quarter of one, and runs through the parts in CTA order (more than kSerial of
// them are shared out to several groups), keeping the running maximum, sum and
// output as the tiles do; the order is fixed, so results do not depend on timing.
// A block runs its code once, so fetching instructions is what it waits for: block
// shapes are powers of two in place of divisions, and bf16 takes the approximate
// exponential and quotient, far below the step of its rounding (16 sequences with
// 16 new tokens 83 -> 79 us; one of 201 tokens 12.2 -> 10.2).
constexpr int JT = 256;
constexpr int kSerial = 8;
struct Running {
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    template <int U>
    __device__ __forceinline__ void add(const float (&m1)[U], const float (&l1)[U], const float4 (&x)[U]) {
        float top = m;
#pragma unroll
        for (int k = 0; k < U; ++k) top = fmaxf(top, m1[k]);
        const float ref = top == -INFINITY ? 0.f : top;
        const float f = tc::ex2_approx(m - ref);
        m = top;
        l *= f;
        o.x *= f; o.y *= f; o.z *= f; o.w *= f;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const float w = tc::ex2_approx(m1[k] - ref);
            l = fmaf(l1[k], w, l);
            o.x = fmaf(x[k].x, w, o.x); o.y = fmaf(x[k].y, w, o.y);
            o.z = fmaf(x[k].z, w, o.z); o.w = fmaf(x[k].w, w, o.w);
        }
    }
};
template <typename T>
__device__ __forceinline__ float gate_of(float g) {
    return sizeof(T) == 2 ? __fdividef(1.0f, 1.0f + __expf(-g)) : sigmoid_f(g);
}
template <typename T>
__device__ __forceinline__ float inverse(float x) {
    return x == 0.f ? 0.f : sizeof(T) == 2 ? __fdividef(1.0f, x) : 1.0f / x;
}
// log_groups: log2 of blockDim.y; log_split: 2 where a group takes a quarter row, else 0.
template <typename T>
__global__ void __launch_bounds__(JT) attn_join_kernel(AttnArgs a, int log_groups, int log_split) {
    using Raw = typename Four<T>::type;
    constexpr int U = 4;  // parts at once
    __shared__ float4 o_s[JT];
    __shared__ float2 ml_s[JT];
    const int c = blockIdx.x + 1, ng = blockDim.x, g = threadIdx.y, tid = g * ng + threadIdx.x;
    pdl_wait();
    pdl_trigger();
    const JoinTask task = *join_task(a, c);
    // (the bounds hold for every task of this call's; they keep calls that share a workspace against the rules
    // from writing out of bounds)
    if (task.n < 2 || (unsigned)task.b >= (unsigned)a.B || (unsigned)task.h >= (unsigned)a.H_kv ||
        (unsigned)task.rb >= (unsigned)a.n_rb || (unsigned)task.c0 >= kAttnMaxCtas || task.c0 + task.n > kAttnMaxCtas)
        return;
    const int n = task.n;
    const int sf = (int)a.slot_floats;  // 2 kAttnMaxCtas of them fit 31 bits
    const float* slots = slot_ptr(a, 2 * task.c0);
    const int r0 = task.rb * a.rb_rows, nr = block_rows(a, task.rb);
    // 2^log_share groups on one row: about 4 parts each where there are many
    const int log_share = n > kSerial ? min(log_groups, 32 - __clz((n - 1) >> 2)) : 0;
    const int sub = g & ((1 << log_share) - 1), at_once = 1 << (log_groups - log_share);
    const int step = (n - 1) * gridDim.y * at_once;
    for (int first = ((c - task.c0 - 1) * gridDim.y + blockIdx.y) * at_once; first < nr << log_split; first += step) {
        const int rq = first + (g >> log_share), r = rq >> log_split;
        const int d = ((rq - (r << log_split)) * ng + threadIdx.x) * 4;
        const bool mine = r < nr, writes = mine && sub == 0;
        const int64_t row = writes ? row_index(a, task.b, task.h, r0 + r) : 0, at = row * a.D + d;
        Raw gate{};
        if (writes && a.gate != nullptr) gate = *reinterpret_cast<const Raw*>(static_cast<const T*>(a.gate) + at);
        Running run;
        if (mine) {
#pragma unroll 1
            for (int i = sub; i < n; i += U << log_share) {
                float m[U], l[U];
                float4 x[U];
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const int part = i + (k << log_share);
                    m[k] = -INFINITY;
                    l[k] = 0.f;
                    x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (part < n) {
                        const float* slot = slots + (part == 0 ? 1 : 2 * part) * sf;
                        m[k] = slot[r];
                        l[k] = slot[a.rb_rows + r];
                        x[k] = *reinterpret_cast<const float4*>(slot + a.stat_floats + r * a.D + d);
                    }
                }
                run.add(m, l, x);
            }
        }
        if (log_share > 0) {
            o_s[tid] = run.o;
            ml_s[tid] = make_float2(run.m, run.l);
            __syncthreads();
            if (writes)
#pragma unroll 1
                for (int i = 1; i < 1 << log_share; ++i) {
                    const float m[1] = {ml_s[tid + i * ng].x}, l[1] = {ml_s[tid + i * ng].y};
                    const float4 x[1] = {o_s[tid + i * ng]};
                    run.add(m, l, x);
                }
            __syncthreads();
        }
        if (writes) {
            const float inv = inverse<T>(run.l);
            float4 y = make_float4(run.o.x * inv, run.o.y * inv, run.o.z * inv, run.o.w * inv);
            if (a.gate != nullptr && run.l != 0.f) {
                const float4 gt = as_f32(gate);
                y.x *= gate_of<T>(gt.x); y.y *= gate_of<T>(gt.y); y.z *= gate_of<T>(gt.z); y.w *= gate_of<T>(gt.w);
            }
            store4(static_cast<T*>(a.out) + at, y);
            if (d == 0 && a.lse != nullptr) a.lse[row] = run.l == 0.f ? -INFINITY : (run.m + log2f(run.l)) * kLn2;
        }
    }
}

template <typename E, int R, int NV>
cudaError_t launch_ffma(const AttnArgs& a, int n_cta, cudaStream_t s) {
    using G = Ffma<E, R, NV>;
    const size_t smem = sizeof(float) * (G::STAGE_FLOATS + G::NW * (G::C + 2 * R) + R);
    const cudaError_t e = cudaFuncSetAttribute(attn_ffma_kernel<E, R, NV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(attn_ffma_kernel<E, R, NV>, dim3((unsigned)n_cta), dim3(G::NT), smem, s, a);
}

template <typename E>
cudaError_t launch_ffma_rows(const AttnArgs& a, int n_cta, cudaStream_t s) {
    if (a.D > 128) return a.rb_rows <= 4 ? launch_ffma<E, 4, 2>(a, n_cta, s) : launch_ffma<E, 8, 2>(a, n_cta, s);
    return a.rb_rows <= 4 ? launch_ffma<E, 4, 1>(a, n_cta, s) : launch_ffma<E, 8, 1>(a, n_cta, s);
}

}  // namespace

cudaError_t launch_attn_join(const AttnArgs& a, int n_cta, gdn_dtype_t dt, cudaStream_t s) {
    if (n_cta <= 1) return cudaSuccess;
    // fewer items than a quarter of the CTAs: many parts each
    const int log_split = a.D % 16 == 0 && (int64_t)a.B * a.H_kv * a.n_rb * 4 < n_cta ? 2 : 0;
    const int ng = (a.D / 4) >> log_split;
    int log_groups = 0;
    while ((2 << log_groups) * ng <= JT) ++log_groups;
    // enough blocks that an item of two parts takes one pass (5 new tokens, 40 rows: 114 us with a block per 16 rows,
    // 110 so; one of 201 tokens 11.1 and 10.2)
    const int y = ((a.rb_rows << log_split) + (1 << log_groups) - 1) >> log_groups;
    const dim3 grid((unsigned)(n_cta - 1), (unsigned)y), block((unsigned)ng, 1u << log_groups);
    return dt == GDN_BF16 ? launch_pdl(attn_join_kernel<bf16>, grid, block, 0, s, a, log_groups, log_split)
                          : launch_pdl(attn_join_kernel<float>, grid, block, 0, s, a, log_groups, log_split);
}

cudaError_t launch_attn_ffma(const AttnArgs& a, int n_cta, gdn_dtype_t dt, cudaStream_t s) {
    const cudaError_t e = dt == GDN_BF16 ? launch_ffma_rows<bf16>(a, n_cta, s) : launch_ffma_rows<float>(a, n_cta, s);
    return e != cudaSuccess ? e : launch_attn_join(a, n_cta, dt, s);
}

}  // namespace gdn
