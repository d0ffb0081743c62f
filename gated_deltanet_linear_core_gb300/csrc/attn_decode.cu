// gdn_attn_decode: how a call is cut up, and which kernel runs it.
#include "attn_common.cuh"

namespace gdn {

namespace {
constexpr int kTcRows = 128;  // rows of a block, at most
}  // namespace

int attn_ctas() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 1;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 1;
    return n < kAttnMaxCtas ? n : kAttnMaxCtas;
}

size_t attn_plan(AttnArgs& a, gdn_dtype_t dt) {
    const int most = attn_tc_takes(a, dt) ? kTcRows : kAttnFfmaRows;
    a.group = a.H_q / a.H_kv;
    a.rows = a.K * a.group;
    a.n_rb = (a.rows + most - 1) / most;
    a.rb_rows = (a.rows + a.n_rb - 1) / a.n_rb;
    // about the tiles that HBM delivers while an item starts and ends, twice as many where they are half as large (us with
    // 0, without the doubling, and so: 16 ragged sequences with 16 new tokens 87.5, 79.2, 79.9; 8 in f32 27.3, 24.6, 23.4;
    // 64 with 5 new tokens, head dim 256, 119.1 and 109.3)
    a.setup = (!attn_tc_takes(a, dt) ? 2 : a.rb_rows <= 32 ? 1 : a.rb_rows <= 64 ? 2 : 3) * (a.D <= 128 ? 2 : 1);
    a.stat_floats = (2 * a.rb_rows + 3) & ~3;
    a.slot_floats = a.stat_floats + (int64_t)a.rb_rows * a.D;
    return kAttnMaxCtas * (sizeof(attn::JoinTask) + 2 * (size_t)a.slot_floats * sizeof(float));
}

cudaError_t launch_attn_decode(const AttnArgs& a, gdn_dtype_t dt, cudaStream_t s) {
    if (a.B == 0 || a.K == 0) return cudaSuccess;
    return attn_tc_takes(a, dt) ? launch_attn_tc(a, attn_ctas(), s) : launch_attn_ffma(a, attn_ctas(), dt, s);
}

}  // namespace gdn
