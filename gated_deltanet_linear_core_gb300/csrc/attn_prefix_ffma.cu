// The pass over shared prefixes on CUDA cores: f32, and bf16 with page sizes that
// the tensor-core kernel's loads do not take.
//
// 64 query rows of a group that share a key-value head against tiles of 64 cached
// tokens, all in shared memory as f32; a thread holds 4 x 4 scores, then 4 rows of D / 16
// outputs.  Bound by the products (f32 fused multiply-adds).
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

// NC blocks of 64 head dims.
template <typename E, int NC>
struct Tiles {
    static constexpr int QS = NC * 64 + 4;  // floats per row: rows 16 bytes apart in the banks
    static constexpr int FLOATS = 3 * 64 * QS + TT * PS;
};

template <typename E, int NC>
__global__ void __launch_bounds__(NT, 1) attn_prefix_ffma_kernel(ShareArgs s) {
    using T = Tiles<E, NC>;
    constexpr int QS = T::QS;
    extern __shared__ __align__(16) float sm[];
    __shared__ int64_t off_s[TT];
    float* q_s = sm;
    float* k_s = q_s + 64 * QS;
    float* v_s = k_s + 64 * QS;
    float* p_s = v_s + 64 * QS;  // [token][row]
    const AttnArgs& a = s.a;
    const int D = a.D, tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    pdl_wait();
    pdl_trigger();
    SharedWalk walk(s, blockIdx.x, gridDim.x);
    SharedSegment g;
    const int fours = D / 4;
    for (int i = tid; i < 3 * 64 * QS; i += NT) sm[i] = 0.f;  // dims from D on stay zero
    while (walk.next(s, g)) {
        __syncthreads();
        for (int e = tid; e < ROWS * fours; e += NT) {
            const int r = e / fours, d = (e - r * fours) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < g.nr) x = ld4(static_cast<const E*>(a.q) + shared_row(a, g.seq0, g.h, g.r0 + r) * D + d);
            *reinterpret_cast<float4*>(q_s + r * QS + d) = x;
        }
        float m[4], l[4], o[4][4 * NC];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m[i] = kNone;
            l[i] = 0.f;
#pragma unroll
            for (int c = 0; c < 4 * NC; ++c) o[i][c] = 0.f;
        }
        for (int j = g.tile0; j < g.tile1; ++j) {
            if (tid < TT) {
                const int t = j * TT + tid, pg = t / a.page_size;
                const int page = a.table[(int64_t)g.leader * a.max_pages + pg];
                off_s[tid] = page < 0 || page >= a.n_pages
                                 ? -1
                                 : (((int64_t)page * a.H_kv + g.h) * a.page_size + (t - pg * a.page_size)) * D;
            }
            __syncthreads();
            for (int e = tid; e < TT * fours; e += NT) {
                const int t = e / fours, d = (e - t * fours) * 4;
                const int64_t at = off_s[t];
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
                if (at >= 0) {
                    x = ld4(static_cast<const E*>(a.k_cache) + at + d);
                    y = ld4(static_cast<const E*>(a.v_cache) + at + d);
                }
                *reinterpret_cast<float4*>(k_s + t * QS + d) = x;
                *reinterpret_cast<float4*>(v_s + t * QS + d) = y;
            }
            __syncthreads();
            // ---- scores of rows 4 ty .., tokens tx + 16 ..
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
                    q[i] = *reinterpret_cast<const float4*>(q_s + (4 * ty + i) * QS + d);
                    k[i] = *reinterpret_cast<const float4*>(k_s + (tx + 16 * i) * QS + d);
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
                    top = fmaxf(top, x[t]);
                }
#pragma unroll
                for (int w = 1; w < 16; w *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
                if (top > m[i] + kSlack) {  // (the 16 threads of a row agree)
                    const float f = tc::ex2_approx(m[i] - top);
                    m[i] = top;
                    l[i] *= f;
#pragma unroll
                    for (int c = 0; c < 4 * NC; ++c) o[i][c] *= f;
                }
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const float p = tc::ex2_approx(x[t] - m[i]);
                    l[i] += p;
                    p_s[(tx + 16 * t) * PS + 4 * ty + i] = p;
                }
            }
            __syncwarp();  // a row's weights are written and read by one warp
            // ---- O += P V: rows 4 ty .., dims 4 tx + 64 ..
#pragma unroll 2
            for (int t = 0; t < TT; ++t) {
                const float4 p = *reinterpret_cast<const float4*>(p_s + t * PS + 4 * ty);
                const float w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const float4 v = *reinterpret_cast<const float4*>(v_s + t * QS + 64 * c + 4 * tx);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float2* y = reinterpret_cast<float2*>(&o[i][4 * c]);
                        y[0] = __ffma2_rn(make_float2(w[i], w[i]), make_float2(v.x, v.y), y[0]);
                        y[1] = __ffma2_rn(make_float2(w[i], w[i]), make_float2(v.z, v.w), y[1]);
                    }
                }
            }
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
                po = s.pre_o + at * D;
                if (tx == 0) s.pre_stat[at] = part_stat(m[i], sum, g.parts, r);
            } else {
                po = slot + 2 * ROWS + r * D;
                if (tx == 0) {
                    slot[r] = sum == 0.f ? -INFINITY : m[i];
                    slot[ROWS + r] = sum;
                }
            }
#pragma unroll
            for (int c = 0; c < NC; ++c)
                if (64 * c + 4 * tx < D)
                    *reinterpret_cast<float4*>(po + 64 * c + 4 * tx) =
                        make_float4(o[i][4 * c], o[i][4 * c + 1], o[i][4 * c + 2], o[i][4 * c + 3]);
        }
    }
}

template <typename E, int NC>
cudaError_t launch_nc(const ShareArgs& s, int n_cta, cudaStream_t st) {
    constexpr int smem = Tiles<E, NC>::FLOATS * (int)sizeof(float);
    const cudaError_t e = cudaFuncSetAttribute(attn_prefix_ffma_kernel<E, NC>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(attn_prefix_ffma_kernel<E, NC>, dim3((unsigned)n_cta), dim3(NT), smem, st, s);
}
template <typename E>
cudaError_t launch_e(const ShareArgs& s, int n_cta, cudaStream_t st) {
    if (s.a.D <= 64) return launch_nc<E, 1>(s, n_cta, st);
    return s.a.D <= 128 ? launch_nc<E, 2>(s, n_cta, st) : launch_nc<E, 4>(s, n_cta, st);
}

}  // namespace

cudaError_t launch_prefix_ffma(const ShareArgs& s, int n_cta, gdn_dtype_t dt, cudaStream_t st) {
    return dt == GDN_BF16 ? launch_e<bf16>(s, n_cta, st) : launch_e<float>(s, n_cta, st);
}

}  // namespace gdn
