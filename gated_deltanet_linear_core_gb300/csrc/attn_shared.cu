// gdn_attn_decode_shared: how a call is cut up, its plan and merge kernels.
#include "attn_shared.cuh"
#include "tc_ptx.cuh"

namespace gdn {

namespace {

using namespace attn;

constexpr int PT = 1024;  // threads of the plan
constexpr int MT = 256;   // threads of a merge block that takes several rows

// What every group shares in earnest, by one block: a warp (or, where there are few groups, several)
// looks at a group's lengths.
__global__ void __launch_bounds__(PT) attn_share_plan_kernel(ShareArgs s) {
    __shared__ int least_s[32], first_s[32], count_s[32], share_s[32];
    __shared__ int64_t sums_s[32], before_s;
    const AttnArgs& a = s.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int32_t* skip = const_cast<int32_t*>(a.skip);
    pdl_wait();
    pdl_trigger();
    for (int b = tid; b < a.B; b += PT) skip[b] = 0;  // of sequences in no group
    __syncthreads();
    const int per = s.G >= 32 ? 1 : 32 / s.G, at_once = 32 / per;  // warps per group, groups at once
    int64_t before = 0;  // units of the groups before (warp 0)
    for (int g0 = 0; g0 < s.G; g0 += at_once) {
        const int mine = warp / per, g = g0 + mine;
        const bool works = mine < at_once && g < s.G;
        int lo = 0, hi = 0, least = INT32_MAX, first = INT32_MAX, count = 0;
        if (works) {
            group_bounds(s, g, lo, hi);
#pragma unroll 4
            for (int b = lo + (warp - mine * per) * 32 + lane; b < hi; b += per * 32) {
                const int n = clamped_len(a, b);
                if (n > 0) {  // sequences without a token see nothing and do not count
                    least = min(least, n);
                    first = min(first, b);
                    ++count;
                }
            }
        }
        least = __reduce_min_sync(0xffffffffu, least);
        first = __reduce_min_sync(0xffffffffu, first);
        count = __reduce_add_sync(0xffffffffu, count);
        if (lane == 0) {
            least_s[warp] = least;
            first_s[warp] = first;
            count_s[warp] = count;
        }
        __syncthreads();
        if (warp == 0) {  // lane i: group g0 + i
            const int gi = g0 + lane;
            int64_t units = 0;
            ShareRecord grp = {};
            if (lane < at_once && gi < s.G) {
                least = first = INT32_MAX;
                count = 0;
                for (int w = lane * per; w < (lane + 1) * per; ++w) {
                    least = min(least, least_s[w]);
                    first = min(first, first_s[w]);
                    count += count_s[w];
                }
                // less than the first new token of any sequence sees
                int share = count > 1 ? min(s.prefix[gi], least - a.K) : 0;
                share = share > 0 ? share / kShareStep * kShareStep : 0;
                int seq1;
                group_bounds(s, gi, grp.seq0, seq1);
                grp.seqs = seq1 - grp.seq0;
                grp.blocks = (int)(((int64_t)grp.seqs * a.rows + s.rows_per_block - 1) / s.rows_per_block);
                share_s[lane] = share;
                grp.tiles = share / s.tile;
                grp.leader = first == INT32_MAX ? 0 : first;
                if (share > 0) units = (int64_t)grp.blocks * a.H_kv * (s.setup + grp.tiles);
            }
            int64_t inc = units;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += v;
            }
            grp.unit0 = before + inc - units;
            if (lane < at_once && gi < s.G) s.rec[gi] = grp;
            before += __shfl_sync(0xffffffffu, inc, 31);
        }
        __syncthreads();
        if (works) {
            const int share = share_s[mine];
            if (share > 0)
                for (int b = lo + (warp - mine * per) * 32 + lane; b < hi; b += per * 32)
                    if (clamped_len(a, b) > 0) skip[b] = share;
        }
        __syncthreads();
    }
    // what the sequences have of their own
    if (tid == 0) before_s = before;
    __syncthreads();
    const int blocks = (a.rows + s.rows_per_block - 1) / s.rows_per_block;
    for (int b0 = 0; s.G + b0 < s.records; b0 += PT) {
        const int b = b0 + tid;
        ShareRecord own = {};
        int64_t units = 0;
        if (b < a.B) {
            const int n = clamped_len(a, b);
            own.seq0 = own.leader = b;
            own.seqs = 1;
            own.blocks = blocks;
            own.tile0 = skip[b] / s.tile;
            own.tiles = n > 0 ? (n - 1) / s.tile + 1 - own.tile0 : 0;
            if (n > 0) units = (int64_t)blocks * a.H_kv * (s.setup + own.tiles);
        }
        int64_t inc = units;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) sums_s[warp] = inc;
        __syncthreads();
        int64_t start = before_s;
        for (int w = 0; w < warp; ++w) start += sums_s[w];
        own.unit0 = start + inc - units;
        if (b < a.B) s.rec[s.G + b] = own;
        __syncthreads();
        if (tid == PT - 1) before_s = start + inc;
        __syncthreads();
    }
    if (tid == 0) s.rec[s.records].unit0 = before_s;
}

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
        while (groups * 4 < parts && groups * 2 * ng <= 1024) groups *= 2;
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
    s.records = s.G + (tc ? a.B : 0);
    s.rows_per_block = tc ? 128 : kPrefixFfmaRows;
    s.tile = tc ? 128 : 64;
    s.setup = 1;
    s.slot_floats = 2 * s.rows_per_block + (int64_t)s.rows_per_block * a.D;
    const size_t rows = (size_t)a.B * a.K * a.H_q;
    char* base = reinterpret_cast<char*>(up(reinterpret_cast<size_t>(ws)));
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char* p = base + at;
        at += up(bytes);
        return p;
    };
    if (!tc) a.ws = reinterpret_cast<float*>(take(kAttnMaxCtas * (sizeof(JoinTask) + (size_t)a.slot_floats * sizeof(float))));
    s.slots = reinterpret_cast<float*>(take(kAttnMaxCtas * (size_t)s.slot_floats * sizeof(float)));
    a.part_o = reinterpret_cast<float*>(take(rows * a.D * sizeof(float)));
    s.pre_o = reinterpret_cast<float*>(take(rows * a.D * sizeof(float)));
    a.part_stat = reinterpret_cast<float4*>(take(rows * sizeof(float4)));
    s.pre_stat = reinterpret_cast<float4*>(take(rows * sizeof(float4)));
    s.rec = reinterpret_cast<ShareRecord*>(take(((size_t)s.records + 1) * sizeof(ShareRecord)));
    a.skip = reinterpret_cast<int32_t*>(take((size_t)a.B * sizeof(int32_t)));
    return at + 256;
}

cudaError_t launch_attn_shared(const ShareArgs& s, gdn_dtype_t dt, cudaStream_t st) {
    const AttnArgs& a = s.a;
    if (a.B == 0 || a.K == 0) return cudaSuccess;
    const int n_cta = attn_ctas();
    const bool tc = attn_tc_takes(a, dt);
    cudaError_t e = launch_pdl(attn_share_plan_kernel, dim3(1), dim3(PT), 0, st, s);
    if (e == cudaSuccess) e = tc ? launch_shared_tc(s, n_cta, st) : launch_prefix_ffma(s, n_cta, dt, st);
    if (e == cudaSuccess && !tc) e = launch_attn_ffma(a, n_cta, dt, st);
    if (e != cudaSuccess) return e;
    return dt == GDN_BF16 ? launch_merge<bf16>(s, n_cta, st) : launch_merge<float>(s, n_cta, st);
}

}  // namespace gdn
