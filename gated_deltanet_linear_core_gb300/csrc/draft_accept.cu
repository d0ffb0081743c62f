// gdn_draft_accept: which drafted tokens hold under the target's probabilities
// p and the draft's q, and the token after them, from given uniforms.
//
//   draft t holds if u_t q_t(d_t) < p_t(d_t) and every draft before it holds
//   n = drafts that hold;  r = (p_n - q_n)+ if draft n failed, else p_n
//   next token = the first v with r(v) > 0 and sum_{w<=v} r(w) > u_K sum_w r(w)
// (with q null the draft's distribution is 1 at the drafted token).  The
// emitted tokens are then distributed as the target's own samples.
//
// Borders are decided as good as exactly: u q and p - q are formed without
// rounding, and every sum is a pair of f32, the sum and its rounding error
// (46 bits and more), so the pick does not depend on how the row is split.
// f64 sums would cost more: at 2 adds per clock and SM the scans alone took as
// long as reading the rows.
//
// Only row n is read (and q's when a draft failed), so a batch is bound by HBM
// and a single sequence by latency: one cluster of kCluster CTAs per sequence,
// the row cut into segments of SEG values whose sums stay in shared memory; each
// CTA writes its total into the shared memory of all, and the first warp of the
// CTA that has the border finds its segment and reads that one again.  A warp takes 16 bytes per lane
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
constexpr int SEG = 512;  // values per segment

// A row r(v) = (p(v) - q(v))+, q: a row, or 1 at `hot`, or nothing.
template <typename T>
struct Row {
    const T *p, *q;
    int hot;  // index where 1 is taken off, -1: none
};

// A sum and what rounding left out of it.
struct Sum2 {
    float s = 0.f, c = 0.f;
    __device__ __forceinline__ void add(float d, float e) {  // the value d + e, |e| small beside d
        const float t = s + d;
        const float b = t - s;
        c += ((s - (t - b)) + (d - b)) + e;
        s = t;
    }
    __device__ __forceinline__ Sum2 folded() const {  // |c| at most half a step of s
        Sum2 r;
        r.s = s + c;
        r.c = c - (r.s - s);
        return r;
    }
};
__device__ __forceinline__ Sum2 operator+(Sum2 a, Sum2 b) {
    a.add(b.s, b.c);
    return a.folded();
}
__device__ __forceinline__ bool operator>(Sum2 a, Sum2 b) { return (a.s - b.s) + (a.c - b.c) > 0.f; }
// Rounded down: sums of subnormal values are multiples of the smallest step, and a border between two
// of them must not end on the upper one (a sum above it would not pass it, nor the whole sum).
__device__ __forceinline__ Sum2 operator*(float u, Sum2 a) {
    Sum2 r;
    r.s = __fmul_rd(u, a.s);
    r.c = __fmaf_rd(u, a.c, __fmaf_rd(u, a.s, -r.s));
    return r.folded();
}
__device__ __forceinline__ Sum2 shfl(Sum2 x, int lane) {
    x.s = __shfl_sync(0xffffffffu, x.s, lane);
    x.c = __shfl_sync(0xffffffffu, x.c, lane);
    return x;
}
// Adds (p - q)+ without rounding the difference: min(p, q) takes q's place, so
// that there is nothing to add where q is the larger.
__device__ __forceinline__ void add_diff(Sum2& a, float p, float q) {
    q = fminf(p, q);
    const float d = p - q;
    const float b = d - p;
    a.add(d, (p - (d - b)) - (q + b));
}
// Two sums at once in packed arithmetic (half the instructions; a row's sums
// are bound by them as much as by HBM).
struct Sum2x2 {
    float2 s = make_float2(0.f, 0.f), c = make_float2(0.f, 0.f);
    __device__ static __forceinline__ float2 sub(float2 x, float2 y) {
        return __ffma2_rn(y, make_float2(-1.f, -1.f), x);
    }
    __device__ __forceinline__ void add_diff(float2 p, float2 q) {
        q = make_float2(fminf(p.x, q.x), fminf(p.y, q.y));
        const float2 d = sub(p, q), bv = sub(d, p);
        const float2 e = sub(sub(p, sub(d, bv)), __fadd2_rn(q, bv));
        const float2 t = __fadd2_rn(s, d), b = sub(t, s);
        c = __fadd2_rn(c, __fadd2_rn(__fadd2_rn(sub(s, sub(t, b)), sub(d, b)), e));
        s = t;
    }
    __device__ __forceinline__ Sum2 total() const {
        Sum2 x, y;
        x.s = s.x; x.c = c.x;
        y.s = s.y; y.c = c.y;
        return x.folded() + y.folded();
    }
};

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
        for (int j = 0; j < Vec16<T>::N; ++j) q[j] = 0.f;
        if ((unsigned)(r.hot - at) < (unsigned)Vec16<T>::N)
#pragma unroll
            for (int j = 0; j < Vec16<T>::N; ++j)
                if (at + j == r.hot) q[j] = 1.f;
    }
}

// Inclusive sum over the lanes.  Not inlined, like the loops below not unrolled:
// a cluster runs most of this code once, and fetching it costs more than
// running it (unrolled and inlined, the search took 6 us of a call's 13).
__device__ __noinline__ Sum2 warp_scan(Sum2 x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        Sum2 y;
        y.s = __shfl_up_sync(0xffffffffu, x.s, o);
        y.c = __shfl_up_sync(0xffffffffu, x.c, o);
        if (lane >= o) x = y + x;
    }
    return x;
}

// Sum of the segment from v0 on, by one warp.
template <typename T, bool VEC>
__device__ __forceinline__ Sum2 segment_sum(const Row<T>& r, int v0, int V, int lane) {
    constexpr int N = Vec16<T>::N, IT = SEG / 32 / N, U = 2;
    Sum2x2 acc;
#pragma unroll 1
    for (int i = 0; i < IT; i += U) {
        float p[U][N], q[U][N];
#pragma unroll
        for (int k = 0; k < U; ++k) load_pq<T, VEC>(r, v0 + ((i + k) * 32 + lane) * N, V, p[k], q[k]);
#pragma unroll
        for (int k = 0; k < U; ++k)
#pragma unroll
            for (int j = 0; j < N; j += 2)
                acc.add_diff(make_float2(p[k][j], p[k][j + 1]), make_float2(q[k][j], q[k][j + 1]));
    }
    return shfl(warp_scan(acc.total()), 31);
}

// The first value of the segment from v0 on at which the running sum, `run`
// before the segment, passes the border (by one warp).
template <typename T, bool VEC>
__device__ __forceinline__ int pick(const Row<T>& r, int v0, int V, Sum2 run, Sum2 border, int lane) {
    constexpr int N = Vec16<T>::N;
    int last = -1;  // this lane's last value with weight
#pragma unroll 1
    for (int v = v0; v < v0 + SEG && v < V; v += 32 * N) {
        float p[N], q[N];
        const int at = v + lane * N;
        load_pq<T, VEC>(r, at, V, p, q);
        Sum2 acc;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            add_diff(acc, p[j], q[j]);
            if (p[j] > q[j]) last = at + j;
        }
        const Sum2 upto = run + warp_scan(acc.folded());
        const uint32_t past = __ballot_sync(0xffffffffu, acc.s > 0.f && upto > border);
        if (past != 0) {  // the lane that passes it walks its own values
            Sum2 before = shfl(upto, lane > 0 ? lane - 1 : 0);
            if (lane == 0) before = run;
            int token = -1;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                if (p[j] > q[j] && !(token >= 0 && before > border)) {
                    add_diff(before, p[j], q[j]);
                    before = before.folded();
                    token = at + j;
                }
            }
            return __shfl_sync(0xffffffffu, token, __ffs(past) - 1);
        }
        run = shfl(upto, 31);
    }
    // rounding left the border at the segment's very end: its last value with weight
    return __reduce_max_sync(0xffffffffu, last);
}

template <typename T, bool VEC>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(NT, 4) draft_accept_kernel(DraftAcceptArgs a) {
    extern __shared__ Sum2 seg_s[];         // running sums of this CTA's segments
    uint8_t* some_s = reinterpret_cast<uint8_t*>(seg_s + (a.V + SEG * kCluster - 1) / (SEG * kCluster));  // segment has weight
    __shared__ Sum2 total_s[2][kCluster];   // the CTAs' sums, one set per pass
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
    const float u = a.u[(int64_t)b * (K + 1) + K];

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
            const Sum2 t = segment_sum<T, VEC>(row, g * SEG, V, lane);
            if (lane == 0) seg_s[g - g0] = t;
        }
        __syncthreads();
        if (pass == 0) cluster.barrier_wait();
        if (warp == 0) {
            Sum2 carry;
            for (int g = 0; g < g1 - g0; g += 32) {
                Sum2 x;
                if (g + lane < g1 - g0) x = seg_s[g + lane];
                const bool some = x.s > 0.f;
                x = carry + warp_scan(x);
                if (g + lane < g1 - g0) {
                    seg_s[g + lane] = x;
                    some_s[g + lane] = some;
                }
                carry = shfl(x, 31);
            }
            if (lane < kCluster) *cluster.map_shared_rank(&total_s[pass][rank], lane) = carry;
        }
        cluster.sync();
        // the CTAs' ranges: one after the other, so that a CTA without weight has an empty one
        Sum2 before, after, sum;
#pragma unroll 1
        for (int i = 0; i < kCluster; ++i) {
            if (i == rank) before = sum;
            sum = sum + total_s[pass][i];
            if (i == rank) after = sum;
        }
        if (sum.s > 0.f && isfinite(sum.s + sum.c)) {
            // u below 1 leaves a border below the sum; anything else is brought there
            Sum2 border = (u > 0.f ? u : 0.f) * sum;
            if (!(sum > border)) border = (1.f - 0x1p-24f) * sum;
            if (warp == 0 && !(before > border) && after > border) {
                int g = -1;  // the first segment with weight whose running sum passes the border, else the last
                for (int i = 0; i < g1 - g0; i += 32) {
                    const bool some = i + lane < g1 - g0 && some_s[i + lane] != 0;
                    const uint32_t past = __ballot_sync(0xffffffffu, some && before + seg_s[i + lane] > border);
                    const uint32_t any = __ballot_sync(0xffffffffu, some);
                    if (past != 0) {
                        g = i + __ffs(past) - 1;
                        break;
                    }
                    if (any != 0) g = i + 31 - __clz(any);
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
    const int nseg = (a.V + SEG - 1) / SEG;  // at most 4096 per CTA: V <= 2^24
    const size_t smem = (size_t)((nseg + kCluster - 1) / kCluster) * (sizeof(Sum2) + 1);
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
