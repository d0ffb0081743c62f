// gdn_attn_decode_shared: how a call is cut up, its plan and merge kernels.
#include "attn_shared.cuh"
#include "tc_ptx.cuh"

namespace gdn {

namespace {

using namespace attn;

constexpr int kPlanThreads = 1024, kPlanFew = 128;  // threads of the plan; where there are at most 128 sequences and groups
constexpr int MT = 256;  // threads of a merge block that takes several rows

// Sum of x over the block's threads before this one, and `total` over all.
template <int PT>
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t& total) {
    __shared__ int64_t sums_s[PT / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
    }
    if (lane == 31) sums_s[warp] = inc;
    __syncthreads();
    int64_t w = lane < PT / 32 ? sums_s[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += v;
    }
    total = __shfl_sync(0xffffffffu, w, 31);
    const int64_t before = __shfl_sync(0xffffffffu, w, (warp - 1) & 31);
    __syncthreads();
    return inc - x + (warp > 0 ? before : 0);
}

// What every group shares in earnest, and the records, by one block.  Groups' least lengths, first
// sequences and counts are gathered in shared memory, of many groups in the workspace.
constexpr int kPlanGroups = 1024;  // groups in shared memory
constexpr int kFewGroups = 8;  // groups that SharedWalk looks at one after another
template <int PT>
__global__ void __launch_bounds__(PT) attn_share_plan_kernel(ShareArgs s) {
    __shared__ int first_s[kPlanGroups + 1], least_s[kPlanGroups], leader_s[kPlanGroups], count_s[kPlanGroups];
    const AttnArgs& a = s.a;
    const int tid = threadIdx.x, lane = tid & 31;
    const bool few = s.G <= kPlanGroups;
    int* least = few ? least_s : s.gather;
    int* leader = few ? leader_s : s.gather + s.G;
    int* count = few ? count_s : s.gather + 2 * (int64_t)s.G;
    const int B = a.B;
    pdl_wait();
    pdl_trigger();
    int len0 = tid < B ? clamped_len(a, tid) : 0;  // of the first sequence of the thread
    const int prefix0 = tid < s.G ? s.prefix[tid] : 0;
    for (int g = tid; g <= s.G; g += PT) {
        if (g < s.G) {
            least[g] = leader[g] = INT32_MAX;
            count[g] = 0;
        }
        if (few) first_s[g] = group_begin(s, g);
    }
    __syncthreads();
    auto first = [&](int g) -> int { return few ? first_s[g] : group_begin(s, g); };
    auto group_of = [&](int b) -> int {  // -1: none
        int lo = 0, hi = s.G - 1;        // the last group that starts at or before the sequence
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (first(mid) <= b) lo = mid; else hi = mid - 1;
        }
        return first(lo) <= b && b < first(lo + 1) ? lo : -1;
    };
    int group0 = -1;
    for (int b0 = 0; b0 < B; b0 += PT) {
        const int b = b0 + tid, n = b0 == 0 ? len0 : b < B ? clamped_len(a, b) : 0;
        const int g = b < B ? group_of(b) : -1;
        if (b0 == 0) group0 = g;
        // sequences without a token see nothing and do not count
        const bool counts = g >= 0 && n > 0;
        const int g1 = __shfl_sync(0xffffffffu, g, 0);
        if (__all_sync(0xffffffffu, !counts || g == g1)) {  // a warp's sequences are mostly of one group
            const int n1 = __reduce_min_sync(0xffffffffu, counts ? n : INT32_MAX);
            const int b1 = __reduce_min_sync(0xffffffffu, counts ? b : INT32_MAX);
            const int c1 = __popc(__ballot_sync(0xffffffffu, counts));
            if (lane == 0 && c1 > 0) {
                atomicMin(&least[g1], n1);
                atomicMin(&leader[g1], b1);
                atomicAdd(&count[g1], c1);
            }
        } else if (counts) {
            atomicMin(&least[g], n);
            atomicMin(&leader[g], b);
            atomicAdd(&count[g], 1);
        }
    }
    __syncthreads();
    int64_t before = 0, total;  // units of the records before
    for (int g0 = 0; g0 < s.G; g0 += PT) {
        const int g = g0 + tid;
        ShareRecord rec = {};
        int64_t units = 0;
        if (g < s.G) {
            const int share = shared_tokens(a, g0 == 0 ? prefix0 : s.prefix[g], count[g], least[g]);
            units = prefix_record(s, rec, first(g), first(g + 1), count[g] > 0 ? leader[g] : 0, share);
            least[g] = share;  // from here on
        }
        rec.unit0 = before + block_scan<PT>(units, total);
        before += total;
        if (g < s.G) s.rec[g] = rec;
    }
    int32_t* skip = const_cast<int32_t*>(a.skip);
    for (int b0 = 0; b0 < B; b0 += PT) {
        const int b = b0 + tid;
        const int n = b0 == 0 ? len0 : b < B ? clamped_len(a, b) : 0, g = b0 == 0 ? group0 : b < B ? group_of(b) : -1;
        const int share = g >= 0 && n > 0 ? least[g] : 0;
        if (b < B) skip[b] = share;
        if (s.records == s.G) continue;
        ShareRecord rec = {};
        const int64_t units = own_record(s, rec, b, n, share);
        rec.unit0 = before + block_scan<PT>(units, total);
        before += total;
        if (b < B) s.rec[s.G + b] = rec;
    }
    if (tid == 0) s.rec[s.records].unit0 = before;
}

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 ld4(const bf16* p) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ void store4(float* p, float4 y) { *reinterpret_cast<float4*>(p) = y; }
__device__ __forceinline__ void store4(bf16* p, float4 y) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
}

// Puts a row's parts together: the running maximum, sum and output over the parts in a fixed
// order.  A group of threads (blockDim.x, 4 columns each) takes a row, or where rows have many
// parts (WIDE) the groups of a block take one row together.
template <typename T, bool WIDE>
__global__ void __launch_bounds__(WIDE ? 1024 : MT) attn_merge_kernel(ShareArgs s) {
    constexpr int U = 4;  // parts at once
    extern __shared__ __align__(16) float4 o_s[];  // WIDE: the groups' outputs, then their maxima and sums
    const AttnArgs& a = s.a;
    const int ng = blockDim.x, groups = blockDim.y, g = threadIdx.y, d = threadIdx.x * 4;
    pdl_wait();
    pdl_trigger();
    const int64_t rows = (int64_t)a.B * a.K * a.H_q, row = WIDE ? blockIdx.x : (int64_t)blockIdx.x * groups + g;
    if (row >= rows) return;
    const int b = (int)(row / (a.K * a.H_q)), rest = (int)(row - (int64_t)b * a.K * a.H_q);
    const int i = rest / a.H_q;
    const float4 own_stat = a.part_stat[row];
    const float4 pre_stat = s.pre_stat[row];  // (of no meaning where nothing is shared)
    const int len = clamped_len(a, b), shared = a.skip[b];
    const int64_t at = row * a.D + d;
    float4 gt = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.gate != nullptr && (!WIDE || g == 0)) gt = ld4(static_cast<const T*>(a.gate) + at);
    // the row's parts: those of its own tokens (of the CTAs c_own ..), then the prefix's
    const bool one_kind = s.records > s.G;  // own tokens are records too, in the same slots
    const int own_rows = one_kind ? s.rows_per_block : a.rb_rows;
    const int c_own = __float_as_int(own_stat.z) & 0xffff, r_own = __float_as_int(own_stat.w);
    const int c_pre = __float_as_int(pre_stat.z) & 0xffff, r_pre = __float_as_int(pre_stat.w);
    int n_own = __float_as_int(own_stat.z) >> 16, n_pre = shared > 0 ? __float_as_int(pre_stat.z) >> 16 : 0;
    if (len - (a.K - 1 - i) <= 0) n_own = n_pre = 0;  // sees nothing
    // (the bounds hold for every call that keeps to the rules; they keep others' reads in bounds)
    if (n_own < 0 || c_own + n_own > kAttnMaxCtas || (unsigned)r_own >= (unsigned)own_rows) n_own = 0;
    if (n_pre < 0 || c_pre + n_pre > kAttnMaxCtas || (unsigned)r_pre >= (unsigned)s.rows_per_block) n_pre = 0;
    const int n = n_own + n_pre;
    Running run;
#pragma unroll 1
    for (int k0 = WIDE ? g : 0; k0 < n; k0 += WIDE ? U * groups : U) {
        float m[U], l[U];
        float4 x[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int part = k0 + k * (WIDE ? groups : 1);
            m[k] = -INFINITY;
            l[k] = 0.f;
            x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (part >= n) continue;
            const bool own = part < n_own;
            const int nth = own ? part : part - n_own;
            if (nth == 0) {
                m[k] = own ? own_stat.x : pre_stat.x;
                l[k] = own ? own_stat.y : pre_stat.y;
                x[k] = ld4((own ? a.part_o : s.pre_o) + at);
            } else {
                const float* slot = own && !one_kind ? slot_ptr(a, c_own + nth) : shared_slot(s, (own ? c_own : c_pre) + nth);
                const int r = own ? r_own : r_pre, per = own ? own_rows : s.rows_per_block;
                m[k] = slot[r];
                l[k] = slot[per + r];
                x[k] = ld4(slot + (own && !one_kind ? a.stat_floats : 2 * per) + r * a.D + d);
            }
        }
        run.add(m, l, x);
    }
    if (WIDE) {
        float2* ml_s = reinterpret_cast<float2*>(o_s + ng * groups);
        o_s[g * ng + threadIdx.x] = run.o;
        if (threadIdx.x == 0) ml_s[g] = make_float2(run.m, run.l);
        __syncthreads();
        if (g > 0) return;
#pragma unroll 4
        for (int k = 1; k < groups; ++k) {
            const float m[1] = {ml_s[k].x}, l[1] = {ml_s[k].y};
            const float4 x[1] = {o_s[k * ng + threadIdx.x]};
            run.add(m, l, x);
        }
    }
    const float inv = run.l == 0.f ? 0.f : 1.0f / run.l;
    float4 y = make_float4(run.o.x * inv, run.o.y * inv, run.o.z * inv, run.o.w * inv);
    if (a.gate != nullptr && run.l != 0.f) {  // a row that sees nothing is 0 whatever its gate holds
        y.x *= sigmoid_f(gt.x); y.y *= sigmoid_f(gt.y); y.z *= sigmoid_f(gt.z); y.w *= sigmoid_f(gt.w);
    }
    store4(static_cast<T*>(a.out) + at, y);
    if (d == 0 && a.lse != nullptr) a.lse[row] = run.l == 0.f ? -INFINITY : (run.m + log2f(run.l)) * kLn2;
}

template <typename T>
cudaError_t launch_merge(const ShareArgs& s, int n_cta, cudaStream_t st) {
    const AttnArgs& a = s.a;
    const int ng = a.D / 4;
    const int64_t rows = (int64_t)a.B * a.K * a.H_q;
    // parts that a row has if all sequences are one group, about; more groups have fewer
    const int64_t items = a.H_kv * (((int64_t)a.B * a.rows + s.rows_per_block - 1) / s.rows_per_block);
    const int64_t parts = 1 + (n_cta + items - 1) / items;
    int groups = 1;
    if (parts > 8) {
        // more groups where there are few rows (us with 1, 2, 4, 8, 16: 1024 rows of 20 parts 67.9, 65.0, 65.6, 70.0, 79.2;
        // 128 rows of 77 parts 124, 110, 103, 99, 98)
        while (groups * 4 < parts && groups * 2 * ng <= 1024 && groups * 2 * ng * rows <= n_cta * 1024) groups *= 2;
        const size_t smem = groups * (ng * sizeof(float4) + sizeof(float2));
        return launch_pdl(attn_merge_kernel<T, true>, dim3((unsigned)rows), dim3((unsigned)ng, (unsigned)groups), smem, st, s);
    }
    groups = MT / ng;
    return launch_pdl(attn_merge_kernel<T, false>, dim3((unsigned)((rows + groups - 1) / groups)),
                      dim3((unsigned)ng, (unsigned)groups), 0, st, s);
}

size_t up(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace

size_t attn_share_plan(ShareArgs& s, gdn_dtype_t dt, void* ws) {
    AttnArgs& a = s.a;
    attn_plan(a, dt);
    const bool tc = attn_tc_takes(a, dt);
    // On CUDA cores what sequences with few rows have of their own is gdn_attn_decode's kernel's, which spreads a tile's
    // tokens over all warps (us with records, with that kernel: 5 sequences of up to 900 tokens, 48 rows, head dim 16 21.8,
    // 53.7; 9 of 15 rows, head dim 80, 41, 49; 13 of 10 rows, head dim 256, 63, 54; bf16 in pages of 18: 9 of 8 rows, head dim
    // 128, 50, 48, of 24 rows 43, 50; 48 of 8 rows, head dim 256, 134, 105; 13 of 32 rows 74, 91).
    const bool own = tc || a.rows > (a.D <= 128 ? kAttnFfmaRows : 2 * kAttnFfmaRows);
    s.records = s.G + (own ? a.B : 0);
    s.few = a.B + s.G <= 32 && s.G <= kFewGroups;
    s.rows_per_block = tc ? 128 : kPrefixFfmaRows;
    s.tile = tc ? 128 : 64;
    // What starting an item costs, in tiles (of half the MMAs up to head dim 128): its first scores and weights and its
    // outputs overlap with nothing.  us with 1, 2, 3, 4, 6 and 8: 64 sequences behind 32768 tokens (head dim 256) 85, 75,
    // 70, 71, 74, 77; 32 with 16 new tokens behind 16384 (head dim 128) 279, 218, 181, 160, 158, 163.
    s.setup = !tc ? 1 : a.D <= 128 ? 5 : 3;
    s.slot_floats = 2 * s.rows_per_block + (int64_t)s.rows_per_block * a.D;
    const size_t rows = (size_t)a.B * a.K * a.H_q;
    char* base = reinterpret_cast<char*>(up(reinterpret_cast<size_t>(ws)));
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char* p = base + at;
        at += up(bytes);
        return p;
    };
    if (!tc)  // (used or not, so that more rows never need less)
        a.ws = reinterpret_cast<float*>(take(kAttnMaxCtas * (sizeof(JoinTask) + (size_t)a.slot_floats * sizeof(float))));
    s.slots = reinterpret_cast<float*>(take(kAttnMaxCtas * (size_t)s.slot_floats * sizeof(float)));
    a.part_o = reinterpret_cast<float*>(take(rows * a.D * sizeof(float)));
    s.pre_o = reinterpret_cast<float*>(take(rows * a.D * sizeof(float)));
    a.part_stat = reinterpret_cast<float4*>(take(rows * sizeof(float4)));
    s.pre_stat = reinterpret_cast<float4*>(take(rows * sizeof(float4)));
    s.rec = reinterpret_cast<ShareRecord*>(take(((size_t)s.records + 1) * sizeof(ShareRecord)));
    s.gather = reinterpret_cast<int*>(take(s.G > kPlanGroups ? 3 * (size_t)s.G * sizeof(int) : 0));
    a.skip = reinterpret_cast<int32_t*>(take((size_t)a.B * sizeof(int32_t)));
    return at + 256;
}

cudaError_t launch_attn_shared(const ShareArgs& s, gdn_dtype_t dt, cudaStream_t st) {
    const AttnArgs& a = s.a;
    if (a.B == 0 || a.K == 0) return cudaSuccess;
    const int n_cta = attn_ctas();
    const bool tc = attn_tc_takes(a, dt);
    // (a small block starts and scans sooner: 1 us)
    cudaError_t e = s.few ? cudaSuccess
                    : a.B <= kPlanFew && s.G <= kPlanFew
                        ? launch_pdl(attn_share_plan_kernel<kPlanFew>, dim3(1), dim3(kPlanFew), 0, st, s)
                        : launch_pdl(attn_share_plan_kernel<kPlanThreads>, dim3(1), dim3(kPlanThreads), 0, st, s);
    if (e == cudaSuccess) e = tc ? launch_shared_tc(s, n_cta, st) : launch_prefix_ffma(s, n_cta, dt, st);
    if (e == cudaSuccess && s.records == s.G) e = launch_attn_ffma(a, n_cta, dt, st);
    if (e != cudaSuccess) return e;
    return dt == GDN_BF16 ? launch_merge<bf16>(s, n_cta, st) : launch_merge<float>(s, n_cta, st);
}

}  // namespace gdn
