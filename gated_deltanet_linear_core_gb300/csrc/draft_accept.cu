// gdn_draft_accept: which drafted tokens hold under the target's probabilities
// p and the draft's q, and the token after them, from given uniforms.
//
//   draft t holds if u_t q_t(d_t) < p_t(d_t) and every draft before it holds
//   n = drafts that hold;  r = (p_n - q_n)+ if draft n failed, else p_n
//   next token = the first v with r(v) > 0 and sum_{w<=v} r(w) > u_K sum_w r(w)
// (with q null the draft's distribution is 1 at the drafted token).  The
// emitted tokens are then distributed as the target's own samples.
//
// Borders are decided exactly: u q and p - q are formed without rounding and
// the sums carry their rounding errors, so the pick does not depend on how the
// row is split.  Only row n is read (and q's when a draft failed): one cluster
// of kCluster CTAs per sequence, the row cut into segments of SEG values whose
// sums stay in shared memory; the CTAs exchange their totals through
// distributed shared memory, and the warp that owns the segment with the
// border reads that one again.
#include <cooperative_groups.h>

#include "gdn_common.cuh"
#include "gdn_launch.h"

namespace gdn {

namespace {

namespace cg = cooperative_groups;

constexpr int NT = 512;
constexpr int kCluster = 8;
constexpr int SEG = 1024;          // values per segment
constexpr int PER = SEG / 32;      // per lane when a segment is searched

template <typename T>
__device__ __forceinline__ float ldg_f(const T* p) { return to_f(__ldg(p)); }
template <>
__device__ __forceinline__ float ldg_f<bf16>(const bf16* p) {
    return __uint_as_float((uint32_t)__ldg(reinterpret_cast<const unsigned short*>(p)) << 16);
}

// A row r(v) = (p(v) - q(v))+, q: a row, or `hot` at one index, or nothing.
template <typename T>
struct Row {
    const T *p, *q;
    int hot;  // index where 1 is taken off, -1: none
};

// sum + err = sum of the values added so far, to about twice f32's precision
struct Sum2 {
    float s = 0.f, c = 0.f;
    __device__ __forceinline__ void add(float d, float e) {
        const float t = s + d;
        const float b = t - s;
        c += ((s - (t - b)) + (d - b)) + e;
        s = t;
    }
    __device__ __forceinline__ double total() const { return (double)s + (double)c; }
};
// adds (p - q)+ without rounding the difference
__device__ __forceinline__ void add_diff(Sum2& a, float p, float q) {
    const float d = p - q;
    const float b = d - p;
    const float e = (p - (d - b)) - (q + b);
    if (p > q) a.add(d, e);
}
__device__ __forceinline__ double diff_of(float p, float q) { return p > q ? (double)p - (double)q : 0.0; }

// Sum of the segment's values [v0, v1) by one warp.
// Reads 16 bytes at a time where VEC.
template <typename T, bool VEC>
__device__ __forceinline__ double segment_sum(const Row<T>& r, int v0, int v1, int lane) {
    Sum2 acc;
    constexpr int N = VEC ? Vec16<T>::N : 1;
    constexpr int U = VEC ? (SEG / 32 / N < 8 ? SEG / 32 / N : 8) : 8;  // loads in flight
    for (int v = v0 + lane * N; v < v1; v += 32 * N * U) {
        float p[U][N], q[U][N];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int at = v + i * 32 * N;
            if constexpr (VEC) {
                if (at < v1) {
                    unpack16<T>(__ldg(reinterpret_cast<const uint4*>(r.p + at)), p[i]);
                    if (r.q != nullptr) unpack16<T>(__ldg(reinterpret_cast<const uint4*>(r.q + at)), q[i]);
                }
            } else {
                if (at < v1) {
                    p[i][0] = ldg_f(r.p + at);
                    if (r.q != nullptr) q[i][0] = ldg_f(r.q + at);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int at = v + i * 32 * N + j;
                if (v + i * 32 * N >= v1) break;
                add_diff(acc, p[i][j], r.q != nullptr ? q[i][j] : (at == r.hot ? 1.f : 0.f));
            }
    }
    double t = acc.total();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    return t;
}

__device__ __forceinline__ double warp_scan(double x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

template <typename T, bool VEC>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(NT) draft_accept_kernel(DraftAcceptArgs a) {
    extern __shared__ double seg_s[];  // sums of this CTA's segments
    __shared__ double total_s;         // their sum
    __shared__ int n_s, drafts_s;
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int b = blockIdx.x / kCluster, rank = blockIdx.x % kCluster;
    const int K = a.K, V = a.V;
    const T* p = static_cast<const T*>(a.p) + (int64_t)b * (K + 1) * V;
    const T* q = a.q == nullptr ? nullptr : static_cast<const T*>(a.q) + (int64_t)b * K * V;
    pdl_wait();
    pdl_trigger();

    if (warp == 0) {
        int drafts = K;
        if (a.n_draft != nullptr) {
            drafts = a.n_draft[b];
            drafts = drafts < 0 ? 0 : (drafts > K ? K : drafts);
        }
        bool holds = false;
        if (lane < drafts) {
            const int d = a.draft[(int64_t)b * K + lane];
            if (d >= 0 && d < V) {
                const double pd = to_f(p[(int64_t)lane * V + d]);
                const double qd = q == nullptr ? 1.0 : (double)to_f(q[(int64_t)lane * V + d]);
                holds = (double)a.u[(int64_t)b * (K + 1) + lane] * qd < pd;
            }
        }
        const uint32_t held = __ballot_sync(0xffffffffu, holds);
        if (lane == 0) {
            n_s = __ffs(~held) - 1;
            drafts_s = drafts;
        }
    }
    __syncthreads();
    const int n = n_s;
    const bool failed = n < drafts_s;
    Row<T> row{p + (int64_t)n * V, nullptr, -1};
    if (failed) {
        if (q != nullptr) row.q = q + (int64_t)n * V;
        else row.hot = a.draft[(int64_t)b * K + n];
    }
    const int nseg = (V + SEG - 1) / SEG;
    const int g0 = (int)((int64_t)nseg * rank / kCluster), g1 = (int)((int64_t)nseg * (rank + 1) / kCluster);

    // a row without a positive value falls back to p alone
    bool picked = false;
    for (int pass = 0; pass < 2; ++pass) {
        for (int g = g0 + warp; g < g1; g += NT / 32) {
            const double t = segment_sum<T, VEC>(row, g * SEG, min(V, (g + 1) * SEG), lane);
            if (lane == 0) seg_s[g - g0] = t;
        }
        __syncthreads();
        if (warp == 0) {  // running sums of the segments
            double carry = 0.0;
            for (int g = 0; g < g1 - g0; g += 32) {
                double x = g + lane < g1 - g0 ? seg_s[g + lane] : 0.0;
                x = carry + warp_scan(x, lane);
                if (g + lane < g1 - g0) seg_s[g + lane] = x;
                carry = __shfl_sync(0xffffffffu, x, 31);
            }
            if (lane == 0) total_s = carry;
        }
        cluster.sync();
        double before = 0.0, sum = 0.0;
        for (int i = 0; i < kCluster; ++i) {
            if (i == rank) before = sum;
            sum += *cluster.map_shared_rank(&total_s, i);
        }
        const double after = before + total_s;
        if (sum > 0.0 && isfinite(sum)) {
            const double border =
                fmin(fmax((double)a.u[(int64_t)b * (K + 1) + K] * sum, 0.0), sum * (1.0 - 0x1p-52));
            if (warp == 0 && border >= before && border < after) {
                int g = 0;  // the first segment whose running sum passes the border
                for (;; g += 32) {
                    const bool past = g + lane < g1 - g0 && before + seg_s[g + lane] > border;
                    const uint32_t m = __ballot_sync(0xffffffffu, past);
                    if (m != 0) {
                        g += __ffs(m) - 1;
                        break;
                    }
                    if (g + 32 >= g1 - g0) {
                        g = g1 - g0 - 1;
                        break;
                    }
                }
                const double base = g == 0 ? before : before + seg_s[g - 1];
                // PER consecutive values per lane, then one lane walks its own
                const int v0 = (g0 + g) * SEG + lane * PER, v1 = min(min(V, (g0 + g + 1) * SEG), v0 + PER);
                double mine = 0.0;
                float pv[PER], qv[PER];
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    pv[j] = qv[j] = 0.f;
                    if (v0 + j < v1) {
                        pv[j] = ldg_f(row.p + v0 + j);
                        qv[j] = row.q != nullptr ? ldg_f(row.q + v0 + j) : (v0 + j == row.hot ? 1.f : 0.f);
                    }
                }
                Sum2 s2;
                int last = -1;
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    add_diff(s2, pv[j], qv[j]);
                    if (pv[j] > qv[j]) last = v0 + j;
                }
                mine = s2.total();
                const double upto = base + warp_scan(mine, lane);
                double run = __shfl_up_sync(0xffffffffu, upto, 1);
                if (lane == 0) run = base;
                const uint32_t m = __ballot_sync(0xffffffffu, last >= 0 && upto > border);
                const uint32_t any = __ballot_sync(0xffffffffu, last >= 0);
                // rounding may leave the border at the very end of the segment: its last positive value
                const int at = m != 0 ? __ffs(m) - 1 : 31 - __clz(any);
                int token = last;
                if (m != 0 && lane == at) {
#pragma unroll
                    for (int j = 0; j < PER; ++j) {
                        const double d = diff_of(pv[j], qv[j]);
                        run += d;
                        if (d > 0.0 && run > border) {
                            token = v0 + j;
                            break;
                        }
                    }
                }
                token = __shfl_sync(0xffffffffu, token, at & 31);
                if (lane == 0) a.tokens[(int64_t)b * (K + 1) + n] = token < 0 ? 0 : token;
            }
            picked = true;
        }
        cluster.sync();  // the totals have been read
        if (picked) break;
        row.q = nullptr;
        row.hot = -1;
    }
    if (rank == 0) {
        if (tid == 0) {
            a.n_accept[b] = n;
            if (!picked) a.tokens[(int64_t)b * (K + 1) + n] = 0;
            if (a.next_slot != nullptr) a.next_slot[b] = a.slots[(int64_t)b * (K + 2) + n + 1];
        }
        if (tid <= K && tid != n) a.tokens[(int64_t)b * (K + 1) + tid] = tid < n ? a.draft[(int64_t)b * K + tid] : -1;
    }
}

template <typename T>
cudaError_t launch_t(const DraftAcceptArgs& a, cudaStream_t s) {
    const int nseg = (a.V + SEG - 1) / SEG;
    const size_t smem = (size_t)((nseg + kCluster - 1) / kCluster) * sizeof(double);
    const dim3 grid((unsigned)(a.B * kCluster));
    // whole 16-byte pieces only when every row starts on one
    const bool vec = (size_t)a.V * sizeof(T) % 16 == 0;
    return vec ? launch_pdl(draft_accept_kernel<T, true>, grid, dim3(NT), smem, s, a)
               : launch_pdl(draft_accept_kernel<T, false>, grid, dim3(NT), smem, s, a);
}

}  // namespace

cudaError_t launch_draft_accept(const DraftAcceptArgs& a, gdn_dtype_t dt, cudaStream_t s) {
    if (a.B == 0) return cudaSuccess;
    return dt == GDN_BF16 ? launch_t<bf16>(a, s) : launch_t<float>(a, s);
}

}  // namespace gdn
