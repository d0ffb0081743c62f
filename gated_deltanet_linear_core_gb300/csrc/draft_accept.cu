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
// the sums carry their rounding errors (two f32 per sum; f64 adds would take
// longer than reading the row), so the pick does not depend on how the row is
// split.
//
// Only row n is read (and q's when a draft failed), so a batch is bound by HBM
// and a single sequence by latency: one cluster of kCluster CTAs per sequence,
// the row cut into segments of SEG values whose sums stay in shared memory; each
// CTA writes its total into the shared memory of all, and the warp that owns the
// segment with the border reads that one again.  A warp takes 16 bytes per lane
// and load, several loads in flight; rows that do not start on 16 bytes are
// read value by value in the same order.
#include <cooperative_groups.h>

#include "gdn_common.cuh"
#include "gdn_launch.h"

namespace gdn {

namespace {

namespace cg = cooperative_groups;

constexpr int NT = 256;
constexpr int kCluster = 8;
constexpr int SEG = 1024;  // values per segment

// A row r(v) = (p(v) - q(v))+, q: a row, or 1 at `hot`, or nothing.
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

// The 16 bytes of values at `at` on, those from V on 0.
template <typename T, bool VEC>
__device__ __forceinline__ void load_row(const T* p, int at, int V, float (&x)[Vec16<T>::N]) {
    constexpr int N = Vec16<T>::N;
    if constexpr (VEC) {
        if (at < V) {  // V is a multiple of N
            unpack16<T>(__ldg(reinterpret_cast<const uint4*>(p + at)), x);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) x[j] = 0.f;
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = at + j < V ? to_f(p[at + j]) : 0.f;
    }
}
template <typename T, bool VEC>
__device__ __forceinline__ void load_pq(const Row<T>& r, int at, int V, float (&p)[Vec16<T>::N],
                                        float (&q)[Vec16<T>::N]) {
    load_row<T, VEC>(r.p, at, V, p);
    if (r.q != nullptr) {
        load_row<T, VEC>(r.q, at, V, q);
    } else {
#pragma unroll
        for (int j = 0; j < Vec16<T>::N; ++j) q[j] = at + j == r.hot ? 1.f : 0.f;
    }
}

__device__ __forceinline__ double warp_total(double t) {
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

// Sum of the segment from v0 on, by one warp.
template <typename T, bool VEC>
__device__ __forceinline__ double segment_sum(const Row<T>& r, int v0, int V, int lane) {
    constexpr int N = Vec16<T>::N, IT = SEG / 32 / N, U = N == 4 ? 4 : 2;
    Sum2 acc;
#pragma unroll 1
    for (int i = 0; i < IT; i += U) {
        float p[U][N], q[U][N];
#pragma unroll
        for (int k = 0; k < U; ++k) load_pq<T, VEC>(r, v0 + ((i + k) * 32 + lane) * N, V, p[k], q[k]);
#pragma unroll
        for (int k = 0; k < U; ++k)
#pragma unroll
            for (int j = 0; j < N; ++j) add_diff(acc, p[k][j], q[k][j]);
    }
    return warp_total(acc.total());
}

// The first value of the segment from v0 on at which the running sum, `run`
// before the segment, passes the border (by one warp).
template <typename T, bool VEC>
__device__ __forceinline__ int pick(const Row<T>& r, int v0, int V, double run, double border, int lane) {
    constexpr int N = Vec16<T>::N, IT = SEG / 32 / N;
    double part[IT];
    int last = -1;  // this lane's last value with weight
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        float p[N], q[N];
        const int at = v0 + (i * 32 + lane) * N;
        load_pq<T, VEC>(r, at, V, p, q);
        Sum2 acc;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            add_diff(acc, p[j], q[j]);
            if (p[j] > q[j]) last = at + j;
        }
        part[i] = acc.total();
    }
    int it = -1;
    double mine = 0.0;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const double t = warp_total(part[i]);
        if (it < 0) {
            if (run + t > border) {
                it = i;
                mine = part[i];
            } else {
                run += t;
            }
        }
    }
    if (it >= 0) {
        const double upto = run + warp_scan(mine, lane);
        const uint32_t past = __ballot_sync(0xffffffffu, upto > border);
        double before = __shfl_up_sync(0xffffffffu, upto, 1);
        if (lane == 0) before = run;
        int token = -1;
        if (past != 0 && lane == __ffs(past) - 1) {
            float p[N], q[N];
            const int at = v0 + (it * 32 + lane) * N;
            load_pq<T, VEC>(r, at, V, p, q);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                if (p[j] > q[j] && !(token >= 0 && before > border)) {
                    before += (double)p[j] - (double)q[j];
                    token = at + j;
                }
            }
        }
        if (past != 0) return __shfl_sync(0xffffffffu, token, __ffs(past) - 1);
    }
    // rounding left the border at the segment's very end: its last value with weight
    return __reduce_max_sync(0xffffffffu, last);
}

template <typename T, bool VEC>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(NT, 4) draft_accept_kernel(DraftAcceptArgs a) {
    extern __shared__ double seg_s[];         // running sums of this CTA's segments
    __shared__ double total_s[2][kCluster];   // the CTAs' sums, one set per pass
    __shared__ int n_s, drafts_s;
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int b = blockIdx.x / kCluster, rank = blockIdx.x % kCluster;
    const int K = a.K, V = a.V;
    const T* p = static_cast<const T*>(a.p) + (int64_t)b * (K + 1) * V;
    const T* q = a.q == nullptr ? nullptr : static_cast<const T*>(a.q) + (int64_t)b * K * V;
    cluster.barrier_arrive();  // waited for before the first write into another CTA's shared memory
    pdl_wait();
    pdl_trigger();
    const double u = a.u[(int64_t)b * (K + 1) + K];

    if (warp == 0) {
        int drafts = a.n_draft == nullptr ? K : a.n_draft[b];
        drafts = drafts < 0 ? 0 : (drafts > K ? K : drafts);
        bool holds = false;
        if (lane < K) {
            const int d = a.draft[(int64_t)b * K + lane];
            const double ut = a.u[(int64_t)b * (K + 1) + lane];
            if (d >= 0 && d < V) {
                const double pd = to_f(p[(int64_t)lane * V + d]);
                const double qd = q == nullptr ? 1.0 : (double)to_f(q[(int64_t)lane * V + d]);
                holds = lane < drafts && ut * qd < pd;
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
    Row<T> row{p + (int64_t)n * V, nullptr, -1};
    if (n < drafts_s) {
        if (q != nullptr) row.q = q + (int64_t)n * V;
        else row.hot = a.draft[(int64_t)b * K + n];
    }
    const int nseg = (V + SEG - 1) / SEG;
    const int g0 = (int)((int64_t)nseg * rank / kCluster), g1 = (int)((int64_t)nseg * (rank + 1) / kCluster);

    // a row without a positive value falls back to p alone
    bool picked = false;
    for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
        for (int g = g0 + warp; g < g1; g += NT / 32) {
            const double t = segment_sum<T, VEC>(row, g * SEG, V, lane);
            if (lane == 0) seg_s[g - g0] = t;
        }
        __syncthreads();
        if (pass == 0) cluster.barrier_wait();
        if (warp == 0) {
            double carry = 0.0;
            for (int g = 0; g < g1 - g0; g += 32) {
                double x = g + lane < g1 - g0 ? seg_s[g + lane] : 0.0;
                x = carry + warp_scan(x, lane);
                if (g + lane < g1 - g0) seg_s[g + lane] = x;
                carry = __shfl_sync(0xffffffffu, x, 31);
            }
            if (lane < kCluster) *cluster.map_shared_rank(&total_s[pass][rank], lane) = carry;
        }
        cluster.sync();
        double before = 0.0, after = 0.0, sum = 0.0;
#pragma unroll
        for (int i = 0; i < kCluster; ++i) {
            if (i == rank) before = sum;
            sum += total_s[pass][i];
            if (i == rank) after = sum;
        }
        if (sum > 0.0 && isfinite(sum)) {
            const double border = fmin(fmax(u * sum, 0.0), sum * (1.0 - 0x1p-52));
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
                const int token =
                    pick<T, VEC>(row, (g0 + g) * SEG, V, g == 0 ? before : before + seg_s[g - 1], border, lane);
                if (lane == 0) a.tokens[(int64_t)b * (K + 1) + n] = token < 0 ? 0 : token;
            }
            picked = true;
            break;
        }
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
