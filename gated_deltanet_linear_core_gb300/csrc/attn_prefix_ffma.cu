// Attention behind shared prefixes on CUDA cores: f32, and bf16 with page sizes that the
// tensor-core kernel's loads do not take.  The prefixes, and where a sequence has more rows per
// key-value head than attn_ffma.cu takes at once what each has of its own too.
//
// 64 query rows of a group that share a key-value head against tiles of 64 cached
// tokens in shared memory; a thread holds 4 x 4 scores, then 4 rows of D / 16 outputs, a warp 8 rows (none of them
// real: it computes nothing).  V of a tile lands beside its scores, K of the next one beside its
// outputs.  Bound by latency: two warps per scheduler issue in 34 to 39 % of the clocks, 5 to 6 clocks a warp and
// instruction, of which 1.5 are the pipes', 0.6 to 1.0 barriers, 0.7 reads of shared memory (whose path is 34 to 54 %
// busy).  9 sequences of 15 rows per head in 2 groups behind 100 to 5000 tokens 39 us a call (the kernel 33 of
// them before a tile's products had sums of their own, and 46 with the copies between the products and all rows computed).
#include "attn_shared.cuh"
#include "tc_ptx.cuh"

namespace gdn {

namespace {

using namespace attn;

constexpr int ROWS = kPrefixFfmaRows;
constexpr int TT = 64;
constexpr int NT = 256;
constexpr int PS = 68;  // floats per token of P

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 ld4(const bf16* p) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ float2 ld2(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ float2 ld2(const bf16* p) {
    const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

// NC blocks of 32 head dims.
template <typename E, int NC>
struct Tiles {
    static constexpr int QS = NC * 32 + 4;                     // floats per row of Q: rows 16 bytes apart in the banks
    static constexpr int KS = NC * 32 + 16 / (int)sizeof(E);   // elements per row of K and V
    static constexpr int BYTES = 4 * (ROWS * QS + TT * PS) + 2 * TT * KS * (int)sizeof(E);
};

template <typename E, int NC, bool FEW>
__global__ void __launch_bounds__(NT, 1) attn_prefix_ffma_kernel(ShareArgs s) {
    using T = Tiles<E, NC>;
    constexpr int QS = T::QS, KS = T::KS;
    extern __shared__ __align__(16) float sm[];
    __shared__ int64_t off_s[2][TT];
    float* q_s = sm;
    float* p_s = q_s + ROWS * QS;  // [token][row]
    E* k_s = reinterpret_cast<E*>(p_s + TT * PS);
    E* v_s = k_s + TT * KS;
    const AttnArgs& a = s.a;
    const int D = a.D, tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    pdl_wait();
    pdl_trigger();
    SharedWalk<FEW> walk(s, blockIdx.x, gridDim.x);
    SharedSegment g;
    const int fours = D / 4, chunks = D * (int)sizeof(E) / 16;
    for (int i = tid; i < T::BYTES / 4; i += NT) sm[i] = 0.f;  // dims from D on stay zero
    auto place = [&](int j) {  // where the tokens of tile j lie
        if (tid < TT) {
            const int t = j * TT + tid, pg = t / a.page_size;
            int64_t at = -1;
            if (g.len == 0 || t < g.len) {
                const int page = a.table[(int64_t)g.leader * a.max_pages + pg];
                if (page >= 0 && page < a.n_pages) at = (((int64_t)page * a.H_kv + g.h) * a.page_size + (t - pg * a.page_size)) * D;
            }
            off_s[j & 1][tid] = at;
        }
    };
    auto copy = [&](E* to, const void* from, int j) {  // a tile's rows, zeros where there is no page
        for (int e = tid; e < TT * chunks; e += NT) {
            const int t = e / chunks, c = e - t * chunks;
            const int64_t at = off_s[j & 1][t];
            const E* src = static_cast<const E*>(from) + (at >= 0 ? at + c * (16 / (int)sizeof(E)) : 0);
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                             tc::smem_u32(to + t * KS + c * (16 / (int)sizeof(E)))),
                         "l"(src), "r"(at >= 0 ? 16 : 0)
                         : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    while (walk.next(s, g)) {
        __syncthreads();
        place(g.tile0);
        for (int e = tid; e < ROWS * fours; e += NT) {
            const int r = e / fours, d = (e - r * fours) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < g.nr) x = ld4(static_cast<const E*>(a.q) + shared_row(a, g.seq0, g.h, g.r0 + r) * D + d);
            *reinterpret_cast<float4*>(q_s + r * QS + d) = x;
        }
        __syncthreads();
        copy(k_s, a.k_cache, g.tile0);
        const bool works = (tid >> 5) * 8 < g.nr;  // the warp has real rows
        // tokens that the rows see, and that the sequence's first new token does
        const int least = g.len - (a.K - 1);
        int vis[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) vis[i] = g.len - (a.K - 1 - (g.r0 + 4 * ty + i) / a.group);
        float m[4], l[4];
        float2 o[4][NC];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m[i] = kNone;
            l[i] = 0.f;
#pragma unroll
            for (int c = 0; c < NC; ++c) o[i][c] = make_float2(0.f, 0.f);
        }
        for (int j = g.tile0; j < g.tile1; ++j) {
            copy(v_s, a.v_cache, j);
            if (j + 1 < g.tile1) place(j + 1);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncthreads();
            const bool tail = g.len > 0 && j * TT + TT > least;
            // ---- scores of rows 4 ty .., tokens tx + 16 ..
            if (works) {
                float2 acc[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k) acc[i][k] = make_float2(0.f, 0.f);
#pragma unroll 2
                for (int d = 0; d < D; d += 4) {
                    float4 q[4], k[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        q[i] = ld4(q_s + (4 * ty + i) * QS + d);
                        k[i] = ld4(k_s + (tx + 16 * i) * KS + d);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            acc[i][t] = __ffma2_rn(make_float2(q[i].x, q[i].y), make_float2(k[t].x, k[t].y), acc[i][t]);
                            acc[i][t] = __ffma2_rn(make_float2(q[i].z, q[i].w), make_float2(k[t].z, k[t].w), acc[i][t]);
                        }
                }
                // ---- weights
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float x[4], top = -INFINITY;
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        x[t] = (acc[i][t].x + acc[i][t].y) * a.scale_log2;
                        if (tail && j * TT + tx + 16 * t >= vis[i]) x[t] = -INFINITY;
                        top = fmaxf(top, x[t]);
                    }
                    if (__any_sync(0xffffffffu, top > m[i] + kSlack)) {
#pragma unroll
                        for (int w = 1; w < 16; w *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
                        if (top > m[i] + kSlack) {  // (the 16 threads of a row agree)
                            const float f = tc::ex2_approx(m[i] - top);
                            m[i] = top;
                            l[i] *= f;
#pragma unroll
                            for (int c = 0; c < NC; ++c) o[i][c] = __fmul2_rn(o[i][c], make_float2(f, f));
                        }
                    }
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const float p = tc::ex2_approx(x[t] - m[i]);
                        l[i] += p;
                        p_s[(tx + 16 * t) * PS + 4 * ty + i] = p;
                    }
                }
            }
            __syncthreads();
            if (j + 1 < g.tile1) copy(k_s, a.k_cache, j + 1);
            else asm volatile("cp.async.commit_group;" ::: "memory");
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncthreads();
            // ---- O += P V: rows 4 ty .., dims 2 tx + 32 ..
            // A tile's products are added up by themselves: one sum over the thousands of tokens that a CTA takes of a long
            // prefix was 1.3e-6 off (rms; 8 key-value heads of 16 behind 105570 tokens), three times as far as a
            // library's product in 32 bits (9 sequences in 2 groups 38.5 -> 38.9 us).
            float2 sum[4][NC];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < NC; ++c) sum[i][c] = make_float2(0.f, 0.f);
            auto outputs = [&](int t, bool tails) {
                const float4 p = ld4(p_s + t * PS + 4 * ty);
                const float w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const float2 v = ld2(v_s + t * KS + 32 * c + 2 * tx);
#pragma unroll
                    for (int i = 0; i < 4; ++i)  // a hidden value may be anything: a weight of 0 must not meet it
                        if (!tails || j * TT + t < vis[i]) sum[i][c] = __ffma2_rn(make_float2(w[i], w[i]), v, sum[i][c]);
                }
            };
            if (works && tail) {
#pragma unroll 1
                for (int t = 0; t < min(TT, g.len - j * TT); ++t) outputs(t, true);
            } else if (works) {
#pragma unroll 4
                for (int t = 0; t < TT; ++t) outputs(t, false);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < NC; ++c) o[i][c] = __fadd2_rn(o[i][c], sum[i][c]);
            __syncthreads();
        }
        // ---- the rows' part
        float* slot = shared_slot(s, blockIdx.x);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float sum = l[i];
#pragma unroll
            for (int w = 1; w < 16; w *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, w);
            const int r = 4 * ty + i;
            if (r >= g.nr) continue;
            float* po;
            if (g.parts > 0) {
                const int64_t at = shared_row(a, g.seq0, g.h, g.r0 + r);
                po = (g.len > 0 ? a.part_o : s.pre_o) + at * D;
                if (tx == 0) (g.len > 0 ? a.part_stat : s.pre_stat)[at] = part_stat(m[i], sum, g.parts, r);
            } else {
                po = slot + 2 * ROWS + r * D;
                if (tx == 0) {
                    slot[r] = sum == 0.f ? -INFINITY : m[i];
                    slot[ROWS + r] = sum;
                }
            }
#pragma unroll
            for (int c = 0; c < NC; ++c)
                if (32 * c + 2 * tx < D) *reinterpret_cast<float2*>(po + 32 * c + 2 * tx) = o[i][c];
        }
    }
}

template <typename E, int NC, bool FEW>
cudaError_t launch_nc(const ShareArgs& s, int n_cta, cudaStream_t st) {
    constexpr int smem = Tiles<E, NC>::BYTES;
    const cudaError_t e = cudaFuncSetAttribute(attn_prefix_ffma_kernel<E, NC, FEW>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(attn_prefix_ffma_kernel<E, NC, FEW>, dim3((unsigned)n_cta), dim3(NT), smem, st, s);
}
template <typename E, bool FEW>
cudaError_t launch_e(const ShareArgs& s, int n_cta, cudaStream_t st) {
    const int D = s.a.D;
    if (D <= 64) return launch_nc<E, 2, FEW>(s, n_cta, st);
    if (D <= 96) return launch_nc<E, 3, FEW>(s, n_cta, st);
    if (D <= 128) return launch_nc<E, 4, FEW>(s, n_cta, st);
    return D <= 192 ? launch_nc<E, 6, FEW>(s, n_cta, st) : launch_nc<E, 8, FEW>(s, n_cta, st);
}

}  // namespace

cudaError_t launch_prefix_ffma(const ShareArgs& s, int n_cta, gdn_dtype_t dt, cudaStream_t st) {
    if (s.few) return dt == GDN_BF16 ? launch_e<bf16, true>(s, n_cta, st) : launch_e<float, true>(s, n_cta, st);
    return dt == GDN_BF16 ? launch_e<bf16, false>(s, n_cta, st) : launch_e<float, false>(s, n_cta, st);
}

}  // namespace gdn
