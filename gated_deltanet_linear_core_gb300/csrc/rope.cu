// gdn_rope and gdn_rope_kv_append: head norm and rotary positions of queries and
// keys, and the new tokens' keys and values into the pages of the cache.
//
// With f_j the frequency of pair j and p the token's position on the pair's axis,
//   x <- x / sqrt(mean x^2 + eps) w,   (a, b) <- mscale (a cos p f_j - b sin p f_j, b cos p f_j + a sin p f_j)
// A copy with some arithmetic on the way; HBM-bound.  A block takes TB tokens.  It first
// makes their cosines and sines (once per token, whatever the number of heads) and looks up
// where each goes in the cache; then groups of lanes take a (token, share of the heads)
// each.  A lane holds both sides of its pairs, so a rotation needs no exchange, and its
// cosines stay in registers over the heads.
//
// The angle of a far position keeps no digits in f32: p f is held in turns, as a 64-bit
// fraction of one turn (f / 2 pi in f64, times 2^64), whose product with the integer p drops whole
// turns by itself.  The fraction is off by at most |p f| 2^-52 / 2 pi turns; its upper 32
// bits go to f32 and sincospif.
#include "gdn_common.cuh"
#include "gdn_launch.h"

namespace gdn {

namespace {

constexpr int NT = 256;
constexpr int kMaxTB = 16;

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
    };
    __device__ __forceinline__ Vec() {}
    __device__ __forceinline__ void load(const E* p) { raw = __ldcs(reinterpret_cast<const Raw*>(p)); }
    __device__ __forceinline__ void store(E* p) const { *reinterpret_cast<Raw*>(p) = raw; }
};

template <typename E, int V>
__device__ __forceinline__ void widen(const Vec<E, V>& v, float (&x)[V]) {
    if constexpr (V * sizeof(E) == 16) {
        unpack16<E>(v.raw, x);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = to_f(v.e[i]);
    }
}
template <typename E, int V>
__device__ __forceinline__ void narrow(const float (&x)[V], Vec<E, V>& v) {
    if constexpr (sizeof(E) == 2 && V >= 2) {
        uint32_t w[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
        memcpy(&v.raw, w, sizeof(v.raw));
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v.e[i] = from_f<E>(x[i]);
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

// V pairs per item, IT items per lane; NEIGHBOURS: pairs (2j, 2j + 1), else (j, j + R / 2).  2^log_lg lanes take a row,
// `parts` groups of them share a token's rows: those of its query heads, key heads and value heads.  (One loop for the
// three, whose sources, places and weights are picked per row: with a loop for each, a small call waited for its code,
// 320 tokens 17.8 us.)
template <typename E, int V, int IT, bool NEIGHBOURS>
__global__ void __launch_bounds__(NT, IT == 1 ? 3 : 2) rope_kernel(RopeArgs a, int tb, int log_lg, int parts) {
    constexpr int U = IT > 1 ? 1 : 2;  // rows in flight per lane
    extern __shared__ __align__(16) float sm[];
    __shared__ int64_t row_s[kMaxTB];   // row of (page, head 0, position in page), -1: nowhere
    __shared__ int64_t pos_s[kMaxTB];   // place in the sequence
    __shared__ int in_s[kMaxTB];        // the token belongs to a sequence
    const int half = a.R >> 1, tid = threadIdx.x;
    uint64_t* turn_s = reinterpret_cast<uint64_t*>(sm);  // [half] frequencies, 2^-64 turns per position
    float* odd_s = sm + 2 * half;                        // [half] 0, NaN where the frequency is not finite
    float* w_s = sm + ((3 * half + 3) & ~3);             // [2][D] norm weights of queries and keys
    float* cos_s = w_s + 2 * a.D;                        // [tb][half]
    float* sin_s = cos_s + ((tb * half + 3) & ~3);
    pdl_wait();
    pdl_trigger();
    const int64_t t0 = (int64_t)blockIdx.x * tb;
    const int n = (int)min((int64_t)tb, a.T - t0);
    if (tid >= NT - kMaxTB) {
        const int i = tid - (NT - kMaxTB);
        if (i < n) {
            int64_t row = -1, pos = 0;
            bool in = true;
            if (a.k_cache != nullptr) {
                int b;
                in = find_token(a, t0 + i, b, pos);
                if (in && pos >= 0 && pos < (int64_t)a.max_pages * a.page_size) {
                    const int pg = (int)(pos / a.page_size);
                    const int page = a.table[(int64_t)b * a.max_pages + pg];
                    if (page >= 0 && page < a.n_pages)
                        row = (int64_t)page * a.H_kv * a.page_size + (pos - (int64_t)pg * a.page_size);
                }
            }
            row_s[i] = row;
            pos_s[i] = pos;
            in_s[i] = in;
        }
    }
    if (tid < half) {
        double c = (double)a.inv_freq[tid] * 0.15915494309189533577;  // turns per position
        odd_s[tid] = (float)(c - c);
        const double part = fabs(c) - floor(fabs(c));
        const uint64_t turn = isfinite(c) ? (uint64_t)__double2ull_rn(part * 18446744073709551616.0) : 0;
        turn_s[tid] = c < 0 ? 0 - turn : turn;
    }
    if (tid < a.D) {
        if (a.q_w != nullptr) w_s[tid] = a.q_w[tid];
        if (a.k_w != nullptr) w_s[a.D + tid] = a.k_w[tid];
    }
    __syncthreads();
    for (int e = tid; e < n * half; e += NT) {
        const int t = e / half, j = e - t * half;
        const int ax = a.axes != nullptr ? a.axes[j] : 0;
        const bool known = ax >= 0 && ax < a.n_axes;
        int64_t p = 0;
        if (known) p = a.positions == nullptr ? pos_s[t] : a.positions[ax * a.T + t0 + t];
        const int32_t f = (int32_t)(((uint64_t)p * turn_s[j]) >> 32);
        float s, c;
        sincospif((float)f * 4.656612873077392578125e-10f + (known ? odd_s[j] : 0.f), &s, &c);  // 2^-31: half turns
        cos_s[e] = c * a.mscale;
        sin_s[e] = s * a.mscale;
    }
    __syncthreads();

    const int lg = 1 << log_lg, lane = tid & (lg - 1), ng = NT >> log_lg;
    const int items = (a.D >> 1) / V;
    int off_a[IT], off_b[IT], pair[IT];
    bool has[IT], turns[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int it = lane + i * lg, p = it * V;
        has[i] = it < items;
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
    for (int g0 = 0; g0 < n * parts; g0 += ng) {  // the lanes of a warp stay together (they share the norm's sums)
        const int gi = g0 + (tid >> log_lg), t = gi < n * parts ? gi / parts : 0, part = gi - t * parts;
        const bool active = gi < n * parts && in_s[t];
        const int64_t token = t0 + t;
        float co[IT][V], si[IT][V];
#pragma unroll
        for (int i = 0; i < IT; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int at = turns[i] ? t * half + pair[i] + v : 0;
                co[i][v] = cos_s[at];
                si[i][v] = sin_s[at];
            }
        const int64_t row = row_s[t], cache_head = (int64_t)a.page_size * a.D;
        const int n_rows = a.H_q + (a.k_cache != nullptr ? 2 * a.H_kv : 0);
#pragma unroll 1
        for (int r0 = part; r0 - part < n_rows; r0 += U * parts) {
            Vec<E, V> xa[U][IT], xb[U][IT];
            E* to[U];
            const float* w[U];
            bool turn[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = r0 + u * parts, kind = r < a.H_q ? 0 : r < a.H_q + a.H_kv ? 1 : 2;
                const int h = kind == 0 ? r : kind == 1 ? r - a.H_q : r - a.H_q - a.H_kv;
                const E* x = kind == 0 ? static_cast<const E*>(a.q) + token * a.q_tok + h * a.q_head
                           : kind == 1 ? static_cast<const E*>(a.k) + token * a.k_tok + h * a.k_head
                                       : static_cast<const E*>(a.v) + token * a.v_tok + h * a.v_head;
                const int64_t place = row * a.D + h * cache_head;
                to[u] = kind == 0 ? static_cast<E*>(a.q_out) + token * a.o_tok + h * a.o_head
                      : kind == 1 ? static_cast<E*>(a.k_cache) + place : static_cast<E*>(a.v_cache) + place;
                w[u] = kind == 0 ? a.q_w : kind == 1 ? a.k_w : nullptr;
                turn[u] = kind < 2;
                if (!active || r >= n_rows || (kind > 0 && row < 0)) to[u] = nullptr;
#pragma unroll
                for (int i = 0; i < IT; ++i) {
                    xa[u][i].raw = {};
                    xb[u][i].raw = {};
                    if (to[u] != nullptr && has[i]) {
                        xa[u][i].load(x + off_a[i]);
                        xb[u][i].load(x + off_b[i]);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const bool norm = w[u] != nullptr;
                float y[IT][2 * V], scale = 1.f;
#pragma unroll
                for (int i = 0; i < IT; ++i) {
                    float ya[V], yb[V];
                    widen<E, V>(xa[u][i], ya);
                    widen<E, V>(xb[u][i], yb);
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        y[i][v] = ya[v];
                        y[i][V + v] = yb[v];
                    }
                }
                if (__any_sync(0xffffffffu, norm)) {
                    float sum = 0.f;
#pragma unroll
                    for (int i = 0; i < IT; ++i)
#pragma unroll
                        for (int v = 0; v < 2 * V; ++v) sum = fmaf(y[i][v], y[i][v], sum);
                    for (int o = lg >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    scale = rsqrtf(sum / (float)a.D + a.eps);
                }
#pragma unroll
                for (int i = 0; i < IT; ++i) {
                    if (!has[i] || to[u] == nullptr) continue;
                    if (norm) {
                        const float* wr = w_s + (w[u] == a.q_w ? 0 : a.D);
                        float wt[2 * V];
                        if constexpr (V % 4 == 0) {
#pragma unroll
                            for (int v = 0; v < V; v += 4) {
                                const float4 fa = *reinterpret_cast<const float4*>(wr + off_a[i] + v);
                                const float4 fb = *reinterpret_cast<const float4*>(wr + off_b[i] + v);
                                wt[v] = fa.x; wt[v + 1] = fa.y; wt[v + 2] = fa.z; wt[v + 3] = fa.w;
                                wt[V + v] = fb.x; wt[V + v + 1] = fb.y; wt[V + v + 2] = fb.z; wt[V + v + 3] = fb.w;
                            }
                        } else {
#pragma unroll
                            for (int v = 0; v < V; ++v) {
                                wt[v] = wr[off_a[i] + v];
                                wt[V + v] = wr[off_b[i] + v];
                            }
                        }
#pragma unroll
                        for (int v = 0; v < 2 * V; ++v) y[i][v] *= scale * wt[v];
                    }
                    const bool turned = turn[u] && turns[i];
                    if (turned) {
#pragma unroll
                        for (int v = 0; v < V; ++v) {
                            float& p = y[i][NEIGHBOURS ? 2 * v : v];
                            float& q = y[i][NEIGHBOURS ? 2 * v + 1 : V + v];
                            const float p1 = p * co[i][v] - q * si[i][v], q1 = q * co[i][v] + p * si[i][v];
                            p = p1;
                            q = q1;
                        }
                    }
                    if (norm || turned) {  // what is neither passes through bit for bit
                        float ya[V], yb[V];
#pragma unroll
                        for (int v = 0; v < V; ++v) {
                            ya[v] = y[i][v];
                            yb[v] = y[i][V + v];
                        }
                        narrow<E, V>(ya, xa[u][i]);
                        narrow<E, V>(yb, xb[u][i]);
                    }
                    xa[u][i].store(to[u] + off_a[i]);
                    xb[u][i].store(to[u] + off_b[i]);
                }
            }
        }
    }
}

template <typename E, int V, bool NEIGHBOURS>
cudaError_t launch_v(const RopeArgs& a, cudaStream_t s) {
    constexpr int IT = V >= 4 ? 1 : 4 / V;  // 128 pairs at most
    const int items = (a.D >> 1) / V, half = a.R >> 1;
    int log_lg = 0;
    while (log_lg < 5 && (1 << log_lg) < items) ++log_lg;
    const int ng = NT >> log_lg;
    // small blocks, so that lookups and cosines overlap copies; a group of lanes a token where there are many
    int64_t tb = a.T / (152 * 16);
    tb = tb < 1 ? 1 : (tb > kMaxTB ? kMaxTB : tb);
    const int rows = a.H_q + 2 * a.H_kv;
    int parts = (int)(ng / tb);
    parts = parts < 1 ? 1 : (parts > rows ? rows : parts);
    const size_t smem = sizeof(float) * (((3 * half + 3) & ~3) + 2 * a.D + 2 * (((size_t)tb * half + 3) & ~(size_t)3));
    return launch_pdl(rope_kernel<E, V, IT, NEIGHBOURS>, dim3((unsigned)((a.T + tb - 1) / tb)), dim3(NT), smem, s, a, (int)tb,
                      log_lg, parts);
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
