// gdn_kv_append: the new tokens' keys and values into the pages of the cache.
//
// A copy; HBM-bound.  A block takes TB consecutive tokens: its first threads
// look up where each goes (sequence, position, page), then all threads copy
// their 16-byte pieces, K and V together.
#include "gdn_common.cuh"
#include "gdn_launch.h"

namespace gdn {

namespace {

constexpr int NT = 256;
constexpr int kMaxTB = 64;
constexpr int U = 4;  // pieces of K and of V in flight per thread

__global__ void __launch_bounds__(NT) kv_append_kernel(KvAppendArgs a, int tb) {
    __shared__ int64_t row_s[kMaxTB];  // row of (page, head 0, position in page), -1: nowhere
    pdl_wait();
    pdl_trigger();
    const int64_t t0 = (int64_t)blockIdx.x * tb;
    const int n = (int)min((int64_t)tb, a.T - t0);
    if ((int)threadIdx.x < n) {
        const int64_t t = t0 + threadIdx.x;
        int b;
        int64_t end;
        bool in;
        if (a.cu == nullptr) {
            const int64_t per = a.T / a.B;
            b = (int)(t / per);
            end = (b + 1) * per;
            in = true;
        } else {
            int64_t start;
            b = seq_of_token(a.cu, a.B, t);
            seq_bounds(a.cu, b, a.T, start, end);
            in = t >= start && t < end;
        }
        const int64_t pos = (int64_t)a.lens[b] - (end - t);
        int64_t row = -1;
        if (in && pos >= 0 && pos < (int64_t)a.max_pages * a.page_size) {
            const int pg = (int)(pos / a.page_size);
            const int page = a.table[(int64_t)b * a.max_pages + pg];
            if (page >= 0 && page < a.n_pages)
                row = (int64_t)page * a.H_kv * a.page_size + (pos - (int64_t)pg * a.page_size);
        }
        row_s[threadIdx.x] = row;
    }
    __syncthreads();
    const int chunks = a.row_bytes >> 4;        // 16-byte pieces of a (token, head) row
    const int per_token = a.H_kv * chunks;
    const int all = n * per_token;
    const uint4* k = static_cast<const uint4*>(a.k) + t0 * per_token;
    const uint4* v = static_cast<const uint4*>(a.v) + t0 * per_token;
    uint4* kc = static_cast<uint4*>(a.k_cache);
    uint4* vc = static_cast<uint4*>(a.v_cache);
    for (int e0 = threadIdx.x; e0 < all; e0 += U * NT) {
        uint4 x[U], y[U];
        int64_t dst[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int e = e0 + i * NT;
            dst[i] = -1;
            if (e < all) {
                const int t = e / per_token, hc = e - t * per_token;
                const int h = hc / chunks, c = hc - h * chunks;
                if (row_s[t] >= 0) dst[i] = (row_s[t] + (int64_t)h * a.page_size) * chunks + c;
                x[i] = __ldcs(k + e);
                y[i] = __ldcs(v + e);
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (dst[i] >= 0) {
                kc[dst[i]] = x[i];
                vc[dst[i]] = y[i];
            }
    }
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& a, cudaStream_t s) {
    if (a.T == 0) return cudaSuccess;
    // many small blocks, so that lookups overlap copies (32768 prompt tokens: 26.6 us, with 4 blocks per SM 29.4)
    int64_t tb = a.T / (152 * 16);
    tb = tb < 1 ? 1 : (tb > kMaxTB ? kMaxTB : tb);
    return launch_pdl(kv_append_kernel, dim3((unsigned)((a.T + tb - 1) / tb)), dim3(NT), 0, s, a, (int)tb);
}

}  // namespace gdn
