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
// one pass over the tiles with the running maximum m, sum l and output O:
//   m' = max(m, max s),  l <- l 2^(m-m') + sum 2^(s-m'),  O <- O 2^(m-m') + P V
// (scores in the log2 domain, all statistics in f32).
#include "attn_common.cuh"

namespace gdn {

namespace {

using namespace attn;

constexpr int NT = 256;   // threads
constexpr int DQ = 8;     // lanes that share a token's dot product

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// four consecutive elements of shared memory as f32
__device__ __forceinline__ float4 lds4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 lds4(const bf16* p) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xffff0000u));
}

template <typename T, int R, int TT>
struct FfmaSmem {
    int64_t rowoff[3][TT];  // element offset of the tile's rows in the caches, -1: no such token
    float s[R][TT];         // scores, then weights
    float m[R], l[R], f[R];
};

// R rows (of which block_rows are real), tiles of TT tokens, NST stages of K and V rows.
template <typename T, int R, int TT>
__global__ void __launch_bounds__(NT, 1) attn_ffma_kernel(AttnArgs a) {
    constexpr int NST = 3;
    constexpr int TPT = TT * DQ / NT;  // tokens per thread in Q K^T
    using Sm = FfmaSmem<T, R, TT>;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Sm& sm = *reinterpret_cast<Sm*>(smem_raw);
    const int D = a.D;
    float* q_s = reinterpret_cast<float*>(smem_raw + ((sizeof(Sm) + 15) & ~size_t(15)));  // [R][D]
    T* stage = reinterpret_cast<T*>(q_s + R * D);                                          // [NST][K, V][TT][D]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    pdl_wait();
    pdl_trigger();
    int n_cta = gridDim.x;
    const Place place = find_place(a, TT, blockIdx.x, n_cta);
    if ((int)blockIdx.x >= n_cta) return;
    Walk walk(place, cta_begin(place.total, blockIdx.x, n_cta), cta_begin(place.total, blockIdx.x + 1, n_cta));

    const T* kc = static_cast<const T*>(a.k_cache);
    const T* vc = static_cast<const T*>(a.v_cache);
    const int ng = D / 4;             // groups of 4 output columns
    const int nsplit = NT / ng;       // token splits of P V
    const int grp = tid % ng, split = tid / ng;
    const int chunks = D * (int)sizeof(T) / 16;  // 16-byte pieces of a row

    Segment s;
    while (walk.next(a, TT, s)) {
        const int r0 = s.rb * a.rb_rows, nr = block_rows(a, s.rb);
        const int nt = s.tile1 - s.tile0;
        // the query rows, scaled into the log2 domain
        for (int e = tid; e < R * D; e += NT) {
            const int r = e / D, d = e - r * D;
            float x = 0.f;
            if (r < nr) x = to_f(static_cast<const T*>(a.q)[row_index(a, s.b, s.h, r0 + r) * D + d]);
            q_s[e] = x;
        }
        if (tid < R) {
            sm.m[tid] = -INFINITY;
            sm.l[tid] = 0.f;
        }
        const int32_t* table = a.table + (int64_t)s.b * a.max_pages;
        auto place_rows = [&](int j) {  // where the rows of the segment's tile j are
            if (tid >= TT) return;
            const int t = (s.tile0 + j) * TT + tid;
            int64_t off = -1;
            if (j < nt && t < s.len) {
                const int pg = t / a.page_size, page = table[pg];
                if (page >= 0 && page < a.n_pages)
                    off = (((int64_t)page * a.H_kv + s.h) * a.page_size + (t - pg * a.page_size)) * D;
            }
            sm.rowoff[j % 3][tid] = off;
        };
        auto load = [&](int j) {
            if (j < nt) {
                T* kd = stage + (int64_t)(j % NST) * 2 * TT * D;
                for (int e = tid; e < TT * chunks; e += NT) {
                    const int t = e / chunks, c = e - t * chunks;
                    const int64_t off = sm.rowoff[j % 3][t];
                    const int64_t src = (off < 0 ? 0 : off) + c * (16 / (int)sizeof(T));
                    T* dst = kd + t * D + c * (16 / (int)sizeof(T));
                    const int bytes = off < 0 ? 0 : 16;
                    cp_async16((uint32_t)__cvta_generic_to_shared(dst), kc + src, bytes);
                    cp_async16((uint32_t)__cvta_generic_to_shared(dst + TT * D), vc + src, bytes);
                }
            }
            cp_async_commit();
        };
        place_rows(0);
        place_rows(1);
        place_rows(2);
        __syncthreads();
        load(0);
        load(1);
        float acc[R][4];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[r][c] = 0.f;

        for (int j = 0; j < nt; ++j) {
            cp_async_wait<1>();
            __syncthreads();  // tile j landed; everyone is done with tile j - 1
            load(j + 2);
            const T* ks = stage + (int64_t)(j % NST) * 2 * TT * D;
            const T* vs = ks + TT * D;
            const int t0 = (s.tile0 + j) * TT;
            // ---- scores: DQ lanes per token, each every 8th group of 4 dims
            {
                const int dq = tid % DQ, tk = tid / DQ;
                float sc[TPT][R];
#pragma unroll
                for (int i = 0; i < TPT; ++i)
#pragma unroll
                    for (int r = 0; r < R; ++r) sc[i][r] = 0.f;
                for (int d = dq * 4; d < D; d += DQ * 4) {
                    float4 kv[TPT];
#pragma unroll
                    for (int i = 0; i < TPT; ++i) kv[i] = lds4(ks + (tk + i * (NT / DQ)) * D + d);
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const float4 qv = lds4(q_s + r * D + d);
#pragma unroll
                        for (int i = 0; i < TPT; ++i) {
                            sc[i][r] = fmaf(kv[i].x, qv.x, sc[i][r]);
                            sc[i][r] = fmaf(kv[i].y, qv.y, sc[i][r]);
                            sc[i][r] = fmaf(kv[i].z, qv.z, sc[i][r]);
                            sc[i][r] = fmaf(kv[i].w, qv.w, sc[i][r]);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < TPT; ++i)
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        float x = sc[i][r];
#pragma unroll
                        for (int o = DQ / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                        if (dq == r % DQ) sm.s[r][tk + i * (NT / DQ)] = x * a.scale_log2;
                    }
            }
            __syncthreads();
            // ---- running maximum and sum, one warp per row
            for (int r = warp; r < R; r += NT / 32) {
                const int vis = r < nr ? visible(a, s.len, r0 + r) - t0 : 0;
                float x[TT / 32], top = -INFINITY;
#pragma unroll
                for (int i = 0; i < TT / 32; ++i) {
                    x[i] = lane + 32 * i < vis ? sm.s[r][lane + 32 * i] : -INFINITY;
                    top = fmaxf(top, x[i]);
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                const float m0 = sm.m[r], m1 = fmaxf(m0, top);
                const float ref = m1 == -INFINITY ? 0.f : m1;
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < TT / 32; ++i) {
                    const float p = exp2f(x[i] - ref);
                    sm.s[r][lane + 32 * i] = p;
                    sum += p;
                }
                sum = warp_sum(sum);
                __syncwarp();
                if (lane == 0) {
                    const float f = exp2f(m0 - ref);
                    sm.f[r] = f;
                    sm.l[r] = sm.l[r] * f + sum;
                    sm.m[r] = m1;
                }
            }
            place_rows(j + 3);
            __syncthreads();
            // ---- O = O f + P V: 4 columns per thread, groups of 4 tokens over the splits
            if (split < nsplit) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float f = sm.f[r];
#pragma unroll
                    for (int c = 0; c < 4; ++c) acc[r][c] *= f;
                }
                // some rows see less than others at the end: a weight of zero must not meet their
                // hidden values, which may be anything
                const bool ragged = t0 + TT > visible(a, s.len, r0);
                for (int tg = split * 4; tg < TT; tg += nsplit * 4) {
                    float4 v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = lds4(vs + (tg + i) * D + grp * 4);
                    if (!ragged) {
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            const float4 p = lds4(&sm.s[r][tg]);
                            const float pp[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                acc[r][0] = fmaf(pp[i], v[i].x, acc[r][0]);
                                acc[r][1] = fmaf(pp[i], v[i].y, acc[r][1]);
                                acc[r][2] = fmaf(pp[i], v[i].z, acc[r][2]);
                                acc[r][3] = fmaf(pp[i], v[i].w, acc[r][3]);
                            }
                        }
                    } else {
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            const int vis = r < nr ? visible(a, s.len, r0 + r) - t0 - tg : 0;
                            const float4 p = lds4(&sm.s[r][tg]);
                            const float pp[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (i < vis) {
                                    acc[r][0] = fmaf(pp[i], v[i].x, acc[r][0]);
                                    acc[r][1] = fmaf(pp[i], v[i].y, acc[r][1]);
                                    acc[r][2] = fmaf(pp[i], v[i].z, acc[r][2]);
                                    acc[r][3] = fmaf(pp[i], v[i].w, acc[r][3]);
                                }
                        }
                    }
                }
            }
        }
        // ---- the splits' sums, then the rows (or this segment's part of them)
        cp_async_wait<0>();
        __syncthreads();
        float* red = reinterpret_cast<float*>(stage);  // [nsplit][R][D]
        if (split < nsplit)
#pragma unroll
            for (int r = 0; r < R; ++r)
                *reinterpret_cast<float4*>(red + ((int64_t)split * R + r) * D + grp * 4) =
                    make_float4(acc[r][0], acc[r][1], acc[r][2], acc[r][3]);
        __syncthreads();
        const bool whole = nt == s.tiles;
        float* slot = slot_ptr(a, 2 * blockIdx.x + (s.first ? 0 : 1));
        for (int e = tid; e < nr * D; e += NT) {
            const int r = e / D, d = e - r * D;
            float o = 0.f;
            for (int sp = 0; sp < nsplit; ++sp) o += red[((int64_t)sp * R + r) * D + d];
            if (whole) {
                const int64_t row = row_index(a, s.b, s.h, r0 + r);
                const float l = sm.l[r];
                o = l > 0.f ? o / l : (l == 0.f ? 0.f : o);
                if (a.gate != nullptr) o *= sigmoid_f(to_f(static_cast<const T*>(a.gate)[row * D + d]));
                static_cast<T*>(a.out)[row * D + d] = from_f<T>(o);
                if (d == 0 && a.lse != nullptr)
                    a.lse[row] = l == 0.f ? -INFINITY : (sm.m[r] + log2f(l)) * kLn2;
            } else {
                slot[a.stat_floats + r * D + d] = o;
                if (d == 0) {
                    slot[r] = sm.m[r];
                    slot[a.rb_rows + r] = sm.l[r];
                }
            }
        }
        __syncthreads();
    }
}

// Joins the parts of every item that more than one CTA worked on.  The CTAs
// whose ranges start inside an item (blockIdx.x + 1) share its rows, gridDim.y
// blocks each.  A group of D / 4 threads takes a row, 4 columns per thread, and
// runs through the parts in CTA order (more than kSerial of them are
// shared out to several groups), keeping the running maximum, sum
// and output as the tiles do; the order is fixed, so results do not depend on
// timing.  Where the item lies is worked out before the wait for the kernel
// that wrote the parts: the lengths are older than that kernel.
constexpr int JT = 256;
constexpr int kSerial = 8;
struct Running {
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    __device__ __forceinline__ void add(float m1, float l1, float4 x) {
        const float top = fmaxf(m, m1);
        const float ref = top == -INFINITY ? 0.f : top;
        const float f = exp2f(m - ref), w = exp2f(m1 - ref);
        m = top;
        l = l * f + l1 * w;
        o.x = o.x * f + x.x * w; o.y = o.y * f + x.y * w; o.z = o.z * f + x.z * w; o.w = o.w * f + x.w * w;
    }
};
template <typename T>
__global__ void __launch_bounds__(JT) attn_join_kernel(AttnArgs a, int n_cta, int tile) {
    __shared__ float4 o_s[JT];
    __shared__ float2 ml_s[JT];
    const int tid = threadIdx.x, c = blockIdx.x + 1;
    const Place p = find_place(a, tile, c, n_cta);
    if (c >= n_cta) return;
    Walk walk(p, cta_begin(p.total, c, n_cta), cta_begin(p.total, c + 1, n_cta));
    Segment s;
    const int64_t u = walk.at;
    if (!walk.next(a, tile, s) || s.tile0 == 0) return;  // the range starts with an item of its own
    const int64_t u0 = u - s.tile0, u1 = u0 + s.tiles;
    const int c0 = cta_of(p.total, u0, n_cta), c1 = cta_of(p.total, u1 - 1, n_cta);
    const int first_slot = cta_begin(p.total, c0, n_cta) == u0 ? 2 * c0 : 2 * c0 + 1;
    const int n = c1 - c0 + 1;
    // many parts: groups share a row's parts, about 4 each; where a block has too few groups for that, a worker
    // takes a quarter of a row
    const int need = n > kSerial ? (n + 3) / 4 : 1;
    const int split = JT / (a.D / 4) < need && a.D % 16 == 0 ? 4 : 1;
    const int ng = a.D / 4 / split, groups = JT / ng, grp = tid % ng, g = tid / ng;
    const int r0 = s.rb * a.rb_rows, nr = block_rows(a, s.rb);
    const int workers = (n - 1) * gridDim.y, worker = (c - c0 - 1) * gridDim.y + blockIdx.y;
    const int share = need < groups ? need : groups;  // groups on one row
    const int at_once = groups / share, sub = g % share;
    pdl_wait();
    pdl_trigger();
    for (int first = worker * at_once; first < nr * split; first += workers * at_once) {
        const int rq = first + g / share, r = rq / split, d = ((rq - r * split) * ng + grp) * 4;
        const bool mine = g < at_once * share && rq < nr * split;  // whole shares only
        Running run;
        if (mine) {
            constexpr int U = 4;
            for (int i = sub; i < n; i += U * share) {
                float m[U], l[U];
                float4 x[U];
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const int part = i + k * share;
                    if (part < n) {
                        const float* slot = slot_ptr(a, part == 0 ? first_slot : 2 * (c0 + part));
                        m[k] = slot[r];
                        l[k] = slot[a.rb_rows + r];
                        x[k] = *reinterpret_cast<const float4*>(slot + a.stat_floats + r * a.D + d);
                    }
                }
#pragma unroll
                for (int k = 0; k < U; ++k)
                    if (i + k * share < n) run.add(m[k], l[k], x[k]);
            }
        }
        if (share > 1) {
            o_s[tid] = run.o;
            ml_s[tid] = make_float2(run.m, run.l);
            __syncthreads();
            if (mine && sub == 0)
                for (int i = 1; i < share; ++i) run.add(ml_s[tid + i * ng].x, ml_s[tid + i * ng].y, o_s[tid + i * ng]);
            __syncthreads();
        }
        if (mine && sub == 0) {
            const int64_t row = row_index(a, s.b, s.h, r0 + r);
            const int64_t at = row * a.D + d;
            const float inv = run.l == 0.f ? 0.f : 1.0f / run.l;
            float y[4] = {run.o.x * inv, run.o.y * inv, run.o.z * inv, run.o.w * inv};
            if (a.gate != nullptr) {
                float gt[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) gt[k] = to_f(static_cast<const T*>(a.gate)[at + k]);
#pragma unroll
                for (int k = 0; k < 4; ++k) y[k] *= sigmoid_f(gt[k]);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) static_cast<T*>(a.out)[at + k] = from_f<T>(y[k]);
            if (d == 0 && a.lse != nullptr) a.lse[row] = run.l == 0.f ? -INFINITY : (run.m + log2f(run.l)) * kLn2;
        }
    }
}

template <typename T, int R, int TT>
cudaError_t launch_ffma(const AttnArgs& a, int n_cta, cudaStream_t s) {
    // the stages' memory also holds the splits' sums at the end of a segment: at most NT * 4 columns
    const size_t stages = (size_t)3 * 2 * TT * a.D * sizeof(T), sums = (size_t)NT * 4 * R * 4;
    const size_t smem = ((sizeof(FfmaSmem<T, R, TT>) + 15) & ~size_t(15)) + (size_t)R * a.D * 4 +
                        (stages > sums ? stages : sums);
    cudaError_t e = cudaFuncSetAttribute(attn_ffma_kernel<T, R, TT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(attn_ffma_kernel<T, R, TT>, dim3((unsigned)n_cta), dim3(NT), smem, s, a);
}

template <typename T, int TT>
cudaError_t launch_ffma_rows(const AttnArgs& a, int n_cta, cudaStream_t s) {
    return a.rb_rows <= 4 ? launch_ffma<T, 4, TT>(a, n_cta, s)
         : a.rb_rows <= 8 ? launch_ffma<T, 8, TT>(a, n_cta, s) : launch_ffma<T, 16, TT>(a, n_cta, s);
}

}  // namespace

cudaError_t launch_attn_join(const AttnArgs& a, int n_cta, int tile, gdn_dtype_t dt, cudaStream_t s) {
    if (n_cta <= 1) return cudaSuccess;
    const dim3 grid((unsigned)(n_cta - 1), (unsigned)((a.rb_rows + 15) / 16));
    return dt == GDN_BF16 ? launch_pdl(attn_join_kernel<bf16>, grid, dim3(JT), 0, s, a, n_cta, tile)
                          : launch_pdl(attn_join_kernel<float>, grid, dim3(JT), 0, s, a, n_cta, tile);
}

cudaError_t launch_attn_ffma(const AttnArgs& a, int n_cta, gdn_dtype_t dt, cudaStream_t s) {
    const bool small = a.D <= 128;
    const int tile = small ? 64 : 32;
    cudaError_t e;
    if (dt == GDN_BF16)
        e = small ? launch_ffma_rows<bf16, 64>(a, n_cta, s) : launch_ffma_rows<bf16, 32>(a, n_cta, s);
    else
        e = small ? launch_ffma_rows<float, 64>(a, n_cta, s) : launch_ffma_rows<float, 32>(a, n_cta, s);
    return e != cudaSuccess ? e : launch_attn_join(a, n_cta, tile, dt, s);
}

}  // namespace gdn
