// C ABI of the GDN layer core: argument validation and dispatch.
//
// Every entry point validates all of its arguments on the host before it
// launches anything; no device memory is read here (except in
// gdn_check_cu_seqlens, which says so).  No exception crosses the ABI.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <atomic>
#include <vector>

#include "gdn.h"
#include "gdn_launch.h"

namespace {

thread_local int g_last_cuda_error = 0;

bool aligned16(const void* p) { return p == nullptr || (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned_n(const void* p, size_t n) {
    return p == nullptr || (reinterpret_cast<uintptr_t>(p) % n) == 0;
}
size_t elem_size(gdn_dtype_t dt) { return dt == GDN_BF16 ? 2 : 4; }

gdn_status_t check_dims(const gdn_dims_t& d, gdn_dtype_t dt) {
    if (dt != GDN_F32 && dt != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (d.H_k <= 0 || d.H_v <= 0 || d.d_k <= 0 || d.d_v <= 0 || d.conv_k <= 0)
        return GDN_ERR_INVALID_ARG;
    if (d.H_v % d.H_k != 0) return GDN_ERR_INVALID_ARG;
    if (d.conv_k != 4) return GDN_ERR_UNSUPPORTED;
    if (d.d_k != d.d_v) return GDN_ERR_UNSUPPORTED;
    if (d.d_k != 16 && d.d_k != 128) return GDN_ERR_UNSUPPORTED;
    if ((int64_t)d.H_v * d.d_v > (1 << 24) || (int64_t)d.H_k * d.d_k > (1 << 24))
        return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

int64_t conv_dim_of(const gdn_dims_t& d) { return 2LL * d.H_k * d.d_k + (int64_t)d.H_v * d.d_v; }

gdn_status_t cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return GDN_OK;
    g_last_cuda_error = (int)e;
    return GDN_ERR_CUDA;
}

gdn_status_t check_ckpt(int32_t every, const void* ckpt, int64_t rows) {
    if (every < 0) return GDN_ERR_INVALID_ARG;
    if (every > 0) {
        if (every % 64 != 0) return GDN_ERR_INVALID_ARG;
        // a buffer is needed only when rows are allocated (a call whose sequences are
        // all shorter than the cadence has none)
        if (rows < 0 || (ckpt == nullptr && rows > 0)) return GDN_ERR_INVALID_ARG;
    }
    return GDN_OK;
}

gdn_status_t check_seqs(const int32_t* cu, int32_t n_seq, int64_t T) {
    if (T < 0 || T > (int64_t)INT32_MAX) return GDN_ERR_INVALID_ARG;
    if (cu == nullptr) return n_seq == 1 ? GDN_OK : GDN_ERR_INVALID_ARG;
    if (n_seq < 1 || n_seq > (1 << 24)) return GDN_ERR_INVALID_ARG;
    if (!aligned_n(cu, 4)) return GDN_ERR_ALIGN;
    return GDN_OK;
}

// gates: either (a, b, A_log, dt_bias) or (g, beta)
gdn_status_t check_gates(const void* a, const void* b, const float* A_log, const float* dt_bias,
                         const float* g, const float* beta, gdn_dtype_t dt) {
    const bool raw = a && b && A_log && dt_bias;
    const bool pre = g && beta;
    if (!raw && !pre) return GDN_ERR_INVALID_ARG;
    if (!aligned_n(a, elem_size(dt)) || !aligned_n(b, elem_size(dt)) || !aligned_n(A_log, 4) ||
        !aligned_n(dt_bias, 4) || !aligned_n(g, 4) || !aligned_n(beta, 4))
        return GDN_ERR_ALIGN;
    return GDN_OK;
}

// Page-locked words that gdn_sync_status copies the error words into, four a call: such copies wait for nothing, so the
// call waits once (into ordinary memory each copy waits by itself: 42 us a call for 17).  As many as calls run at once, up to
// 16, are kept.
std::atomic<int*> g_words[16];
cudaError_t take_status_words(int** words) {
    for (auto& slot : g_words)
        if ((*words = slot.exchange(nullptr)) != nullptr) return cudaSuccess;
    return cudaHostAlloc(reinterpret_cast<void**>(words), 4 * sizeof(int), cudaHostAllocPortable);
}
void give_status_words(int* words) {
    for (auto& slot : g_words) {
        int* none = nullptr;
        if (slot.compare_exchange_strong(none, words)) return;
    }
    cudaFreeHost(words);
}

}  // namespace

extern "C" {

const char* gdn_status_string(gdn_status_t s) {
    switch (s) {
        case GDN_OK: return "ok";
        case GDN_ERR_INVALID_ARG: return "invalid argument";
        case GDN_ERR_ALIGN: return "device pointer not 16-byte aligned";
        case GDN_ERR_UNSUPPORTED: return "unsupported dimensions";
        case GDN_ERR_WORKSPACE: return "workspace missing or too small";
        case GDN_ERR_CUDA: return "CUDA error";
        case GDN_ERR_TIMEOUT: return "device-side wait timed out";
    }
    return "unknown status";
}

int gdn_last_cuda_error(void) { return g_last_cuda_error; }

int gdn_version(void) { return (1 << 16) | 3; }

int64_t gdn_ckpt_count(const int32_t* cu, int32_t n_seq, int32_t every) {
    if (cu == nullptr || n_seq < 1 || every < 0) return -1;
    if (every == 0) return 0;
    int64_t r = 0;
    for (int32_t i = 0; i < n_seq; ++i) {
        if (cu[i + 1] < cu[i]) return -1;
        r += (int64_t)(cu[i + 1] - cu[i]) / every;
    }
    return r;
}

gdn_status_t gdn_check_cu_seqlens(const int32_t* cu, int32_t n_seq, int64_t T, void* stream) {
    if (cu == nullptr || n_seq < 1 || T < 0) return GDN_ERR_INVALID_ARG;
    std::vector<int32_t> h((size_t)n_seq + 1);
    cudaError_t e = cudaMemcpyAsync(h.data(), cu, sizeof(int32_t) * h.size(),
                                    cudaMemcpyDeviceToHost, (cudaStream_t)stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize((cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_status(e);
    if (h[0] != 0 || h[(size_t)n_seq] != T) return GDN_ERR_INVALID_ARG;
    for (int32_t i = 0; i < n_seq; ++i)
        if (h[(size_t)i + 1] < h[(size_t)i]) return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

gdn_status_t gdn_sync_status(void* stream) {
    const cudaStream_t st = (cudaStream_t)stream;
    int* words = nullptr;
    cudaError_t e = take_status_words(&words);
    if (e != cudaSuccess) return cuda_status(e);
    e = gdn::copy_device_error(st, words);
    if (e == cudaSuccess) e = gdn::copy_conv_error(st, words + 1);
    if (e == cudaSuccess) e = gdn::copy_attn_error(st, words + 2);
    if (e == cudaSuccess) e = gdn::copy_shared_error(st, words + 3);
    const cudaError_t done = cudaStreamSynchronize(st);  // (whatever was copied has landed when the words are given back)
    if (e == cudaSuccess) e = done;
    int flags[4] = {0, 0, 0, 0};
    if (e == cudaSuccess) memcpy(flags, words, sizeof(flags));
    give_status_words(words);
    if (e == cudaSuccess && flags[0] != 0) e = gdn::clear_device_error(st);
    if (e == cudaSuccess && flags[1] != 0) e = gdn::clear_conv_error(st);
    if (e == cudaSuccess && flags[2] != 0) e = gdn::clear_attn_error(st);
    if (e == cudaSuccess && flags[3] != 0) e = gdn::clear_shared_error(st);
    const int any = flags[0] | flags[1] | flags[2] | flags[3];
    if (e == cudaSuccess && any != 0) e = cudaStreamSynchronize(st);
    if (e != cudaSuccess) return cuda_status(e);
    return (any & 1) ? GDN_ERR_TIMEOUT : GDN_OK;
}

size_t gdn_layer_prefill_host_workspace_size(int64_t T, gdn_dims_t dims, gdn_dtype_t dtype) {
    if (check_dims(dims, dtype) != GDN_OK || T <= 0 || T > (int64_t)INT32_MAX) return 0;
    return gdn::layer_prefill_host_workspace_bytes(T, dims.H_k, dims.H_v, dims.d_k, (int)elem_size(dtype),
                                                   dtype == GDN_BF16 && dims.d_k == 128);
}

int64_t gdn_layer_prefill_host_piece(int64_t T, gdn_dims_t dims, gdn_dtype_t dtype) {
    if (check_dims(dims, dtype) != GDN_OK || T <= 0 || T > (int64_t)INT32_MAX) return 0;
    return gdn::layer_prefill_host_piece(T, dims.H_k, dims.H_v, dims.d_k, (int)elem_size(dtype),
                                         dtype == GDN_BF16 && dims.d_k == 128);
}

int64_t gdn_layer_prefill_host_pieces(int64_t T, gdn_dims_t dims, gdn_dtype_t dtype) {
    if (check_dims(dims, dtype) != GDN_OK || T <= 0 || T > (int64_t)INT32_MAX) return 0;
    return gdn::layer_prefill_host_pieces(T, dims.H_k, dims.H_v, dims.d_k, (int)elem_size(dtype),
                                          dtype == GDN_BF16 && dims.d_k == 128);
}

namespace {
bool page_locked(const void* p) {
    cudaPointerAttributes at;
    if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    return at.type == cudaMemoryTypeHost;
}
}  // namespace

gdn_status_t gdn_layer_prefill_host(const void* h_qkv, const void* h_z, const void* h_a,
                                    const void* h_b, const void* conv_w, const float* A_log,
                                    const float* dt_bias, const void* norm_w, int64_t T,
                                    const float* initial_state, float* final_state,
                                    const void* conv_state_in, void* conv_state_out, float scale,
                                    uint32_t flags, float norm_eps, void* h_out, void* workspace,
                                    size_t ws_bytes, gdn_dims_t dims, gdn_dtype_t dtype,
                                    void* stream) {
    gdn_status_t st = check_dims(dims, dtype);
    if (st != GDN_OK) return st;
    if (T < 0 || T > (int64_t)INT32_MAX) return GDN_ERR_INVALID_ARG;
    if (flags & ~GDN_QK_L2NORM) return GDN_ERR_INVALID_ARG;
    if (!isfinite(scale) || !isfinite(norm_eps) || norm_eps <= 0.f) return GDN_ERR_INVALID_ARG;
    if (conv_w == nullptr || A_log == nullptr || dt_bias == nullptr || norm_w == nullptr ||
        final_state == nullptr || conv_state_out == nullptr)
        return GDN_ERR_INVALID_ARG;
    if (T > 0 && (h_qkv == nullptr || h_z == nullptr || h_a == nullptr || h_b == nullptr || h_out == nullptr))
        return GDN_ERR_INVALID_ARG;
    if (!aligned16(conv_w) || !aligned16(norm_w) || !aligned_n(A_log, 4) || !aligned_n(dt_bias, 4) ||
        !aligned16(initial_state) || !aligned16(final_state) || !aligned16(conv_state_in) ||
        !aligned16(conv_state_out) || !aligned16(workspace))
        return GDN_ERR_ALIGN;
    if (T > 0 && !(page_locked(h_qkv) && page_locked(h_z) && page_locked(h_a) && page_locked(h_b) &&
                   page_locked(h_out)))
        return GDN_ERR_INVALID_ARG;
    const size_t need = gdn_layer_prefill_host_workspace_size(T, dims, dtype);
    if (need > 0 && (workspace == nullptr || ws_bytes < need)) return GDN_ERR_WORKSPACE;
    cudaStream_t s = (cudaStream_t)stream;
    if (T == 0) {
        // no tokens: the states pass through (conv state pass, then the empty prefill)
        gdn::ConvArgs c;
        memset(&c, 0, sizeof(c));
        c.w = conv_w; c.n_seq = 1; c.C = (int)conv_dim_of(dims);
        c.state_in = conv_state_in; c.state_out = conv_state_out; c.silu = 1;
        cudaError_t e = gdn::launch_conv1d_fwd(c, dtype, s);
        if (e != cudaSuccess) return cuda_status(e);
        gdn::DeltaArgs d;
        memset(&d, 0, sizeof(d));
        d.A_log = A_log; d.dt_bias = dt_bias; d.n_seq = 1;
        d.H_k = dims.H_k; d.H_v = dims.H_v; d.D = dims.d_k;
        d.S0 = initial_state; d.S_final = final_state; d.scale = 1.f;
        return cuda_status(gdn::launch_chunk_ffma(d, dtype, s));
    }
    gdn::HostLayerArgs h;
    h.h_qkv = h_qkv; h.h_z = h_z; h.h_a = h_a; h.h_b = h_b;
    h.conv_w = conv_w; h.A_log = A_log; h.dt_bias = dt_bias; h.norm_w = norm_w;
    h.T = T; h.H_k = dims.H_k; h.H_v = dims.H_v; h.D = dims.d_k;
    h.initial_state = initial_state; h.final_state = final_state;
    h.conv_state_in = conv_state_in; h.conv_state_out = conv_state_out;
    h.scale = scale == 0.f ? 1.0f / sqrtf((float)dims.d_k) : scale;
    h.eps = norm_eps;
    h.l2norm = (flags & GDN_QK_L2NORM) != 0;
    h.h_out = h_out;
    return cuda_status(gdn::launch_layer_prefill_host(h, dtype, workspace, s));
}

gdn_status_t gdn_decode_step(const void* x, const void* conv_w, void* conv_state, const void* z,
                             const void* a, const void* b, const float* A_log,
                             const float* dt_bias, float* state, const void* norm_w,
                             float norm_eps, const int32_t* slots, int32_t B, float scale,
                             uint32_t flags, void* out, gdn_dims_t dims, gdn_dtype_t dtype,
                             void* stream) {
    gdn_status_t st = check_dims(dims, dtype);
    if (st != GDN_OK) return st;
    if (B < 0 || (int64_t)B * dims.H_v > INT32_MAX) return GDN_ERR_INVALID_ARG;
    if (dims.H_v / dims.H_k > 8) return GDN_ERR_UNSUPPORTED;
    if (flags & ~GDN_QK_L2NORM) return GDN_ERR_INVALID_ARG;
    if (!isfinite(scale) || !isfinite(norm_eps) || norm_eps <= 0.f) return GDN_ERR_INVALID_ARG;
    if (B > 0 && (x == nullptr || conv_w == nullptr || conv_state == nullptr || z == nullptr ||
                  a == nullptr || b == nullptr || A_log == nullptr || dt_bias == nullptr ||
                  state == nullptr || norm_w == nullptr || out == nullptr))
        return GDN_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(conv_w) || !aligned16(conv_state) || !aligned16(z) ||
        !aligned_n(a, elem_size(dtype)) || !aligned_n(b, elem_size(dtype)) || !aligned_n(A_log, 4) ||
        !aligned_n(dt_bias, 4) || !aligned16(state) || !aligned16(norm_w) || !aligned_n(slots, 4) ||
        !aligned16(out))
        return GDN_ERR_ALIGN;
    gdn::DecodeStepArgs d;
    memset(&d, 0, sizeof(d));
    d.x = x; d.conv_w = conv_w; d.conv_state = conv_state; d.z = z; d.a = a; d.b = b;
    d.A_log = A_log; d.dt_bias = dt_bias; d.state = state; d.norm_w = norm_w; d.slots = slots;
    d.B = B; d.H_k = dims.H_k; d.H_v = dims.H_v; d.D = dims.d_k;
    d.scale = scale == 0.f ? 1.0f / sqrtf((float)dims.d_k) : scale;
    d.eps = norm_eps;
    d.l2norm = (flags & GDN_QK_L2NORM) != 0;
    d.out = out;
    return cuda_status(gdn::launch_decode_step(d, dtype, (cudaStream_t)stream));
}

gdn_status_t gdn_decode_verify(const void* x, const void* conv_w, void* conv_state, const void* z,
                               const void* a, const void* b, const float* A_log,
                               const float* dt_bias, float* state, const void* norm_w,
                               float norm_eps, const int32_t* slots, int32_t B, int32_t K,
                               float scale, uint32_t flags, void* out, gdn_dims_t dims,
                               gdn_dtype_t dtype, void* stream) {
    gdn_status_t st = check_dims(dims, dtype);
    if (st != GDN_OK) return st;
    if (B < 0 || K < 0 || K > gdn::kVerifyMaxK || (int64_t)B * K * dims.H_v > INT32_MAX)
        return GDN_ERR_INVALID_ARG;
    if (dims.H_v / dims.H_k > 8) return GDN_ERR_UNSUPPORTED;
    if (flags & ~GDN_QK_L2NORM) return GDN_ERR_INVALID_ARG;
    if (!isfinite(scale) || !isfinite(norm_eps) || norm_eps <= 0.f) return GDN_ERR_INVALID_ARG;
    if (B > 0 && K > 0 &&
        (x == nullptr || conv_w == nullptr || conv_state == nullptr || z == nullptr || a == nullptr ||
         b == nullptr || A_log == nullptr || dt_bias == nullptr || state == nullptr ||
         norm_w == nullptr || slots == nullptr || out == nullptr))
        return GDN_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(conv_w) || !aligned16(conv_state) || !aligned16(z) ||
        !aligned_n(a, elem_size(dtype)) || !aligned_n(b, elem_size(dtype)) || !aligned_n(A_log, 4) ||
        !aligned_n(dt_bias, 4) || !aligned16(state) || !aligned16(norm_w) || !aligned_n(slots, 4) ||
        !aligned16(out))
        return GDN_ERR_ALIGN;
    gdn::DecodeVerifyArgs d;
    memset(&d, 0, sizeof(d));
    d.x = x; d.conv_w = conv_w; d.conv_state = conv_state; d.z = z; d.a = a; d.b = b;
    d.A_log = A_log; d.dt_bias = dt_bias; d.state = state; d.norm_w = norm_w; d.slots = slots;
    d.B = B; d.K = K; d.H_k = dims.H_k; d.H_v = dims.H_v; d.D = dims.d_k;
    d.scale = scale == 0.f ? 1.0f / sqrtf((float)dims.d_k) : scale;
    d.eps = norm_eps;
    d.l2norm = (flags & GDN_QK_L2NORM) != 0;
    d.out = out;
    return cuda_status(gdn::launch_decode_verify(d, dtype, (cudaStream_t)stream));
}

gdn_status_t gdn_selftest_bounded_wait(int64_t limit_ns, void* stream) {
    if (limit_ns < 1000) limit_ns = 1000;
    if (limit_ns > 1000000000) limit_ns = 1000000000;
    return cuda_status(gdn::launch_bounded_wait_selftest((uint64_t)limit_ns, (cudaStream_t)stream));
}

gdn_status_t gdn_conv1d_fwd(const void* x, const void* w, const int32_t* cu_seqlens, int32_t n_seq,
                            int64_t T_tot, const void* conv_state_in, void* conv_state_out,
                            int32_t ckpt_every, void* conv_ckpt_out, int64_t ckpt_rows,
                            int32_t apply_silu, void* y, gdn_dims_t dims, gdn_dtype_t dtype,
                            void* stream) {
    gdn_status_t st = check_dims(dims, dtype);
    if (st != GDN_OK) return st;
    if ((st = check_seqs(cu_seqlens, n_seq, T_tot)) != GDN_OK) return st;
    if ((st = check_ckpt(ckpt_every, conv_ckpt_out, ckpt_rows)) != GDN_OK) return st;
    if (w == nullptr || (T_tot > 0 && (x == nullptr || y == nullptr))) return GDN_ERR_INVALID_ARG;
    if (x != nullptr && x == y) return GDN_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(w) || !aligned16(y) || !aligned16(conv_state_in) ||
        !aligned16(conv_state_out) || !aligned16(conv_ckpt_out))
        return GDN_ERR_ALIGN;
    gdn::ConvArgs a;
    a.x = x; a.w = w; a.cu = cu_seqlens; a.n_seq = n_seq; a.T = T_tot;
    a.C = (int)conv_dim_of(dims);
    a.state_in = conv_state_in; a.state_out = conv_state_out;
    a.ckpt_every = ckpt_every; a.ckpt = ckpt_every > 0 ? conv_ckpt_out : nullptr;
    a.ckpt_rows = ckpt_rows; a.silu = apply_silu != 0; a.y = y;
    return cuda_status(gdn::launch_conv1d_fwd(a, dtype, (cudaStream_t)stream));
}

gdn_status_t gdn_conv1d_update(const void* x, const void* w, void* conv_state, int32_t B,
                               int32_t apply_silu, void* y, gdn_dims_t dims, gdn_dtype_t dtype,
                               void* stream) {
    gdn_status_t st = check_dims(dims, dtype);
    if (st != GDN_OK) return st;
    if (B < 0 || B > INT32_MAX / 2) return GDN_ERR_INVALID_ARG;
    if (B > 0 && (x == nullptr || w == nullptr || conv_state == nullptr || y == nullptr))
        return GDN_ERR_INVALID_ARG;
    if (x != nullptr && x == y) return GDN_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(w) || !aligned16(conv_state) || !aligned16(y))
        return GDN_ERR_ALIGN;
    return cuda_status(gdn::launch_conv1d_update(x, w, conv_state, B, (int)conv_dim_of(dims),
                                                 apply_silu != 0, y, dtype, (cudaStream_t)stream));
}

size_t gdn_chunk_prefill_workspace_size(int32_t n_seq, int64_t T_tot, gdn_dims_t dims,
                                        gdn_dtype_t dtype) {
    if (check_dims(dims, dtype) != GDN_OK || n_seq < 1 || T_tot <= 0) return 0;
    if (dtype != GDN_BF16 || dims.d_k != 128) return 0;  // the CUDA-core path needs none
    return gdn::chunk_split_workspace_bytes(n_seq, T_tot, dims.H_v);
}

int32_t gdn_chunk_prefill_launches(int32_t n_seq, int64_t T_tot, int32_t has_cu_seqlens, gdn_dims_t dims,
                                   gdn_dtype_t dtype, uint32_t flags) {
    if (check_dims(dims, dtype) != GDN_OK || n_seq < 1 || T_tot <= 0) return 0;
    if (dtype != GDN_BF16 || dims.d_k != 128) return 1;  // the CUDA-core path: one kernel
    return gdn::chunk_split_launches(n_seq, T_tot, dims.H_v, has_cu_seqlens != 0, (int)((flags >> 8) & 0xffu));
}

namespace {
// gdn_chunk_prefill, and with norm_out set (== o) the same followed by
// RMSNormGated(o, norm_z) in place over norm_out.
gdn_status_t chunk_prefill_impl(const void* qkv, const void* a, const void* b, const float* A_log,
                                const float* dt_bias, const float* g, const float* beta,
                                const int32_t* cu_seqlens, int32_t n_seq, int64_t T_tot,
                                const float* initial_state, float* final_state, int32_t ckpt_every,
                                float* state_ckpt_out, int64_t ckpt_rows, float scale, uint32_t flags, void* o,
                                void* workspace, size_t ws_bytes, gdn_dims_t dims, gdn_dtype_t dtype,
                                void* stream, const void* norm_z, const void* norm_w, float norm_eps,
                                void* norm_out) {
    gdn_status_t st = check_dims(dims, dtype);
    if (st != GDN_OK) return st;
    if ((st = check_seqs(cu_seqlens, n_seq, T_tot)) != GDN_OK) return st;
    if ((st = check_ckpt(ckpt_every, state_ckpt_out, ckpt_rows)) != GDN_OK) return st;
    if (T_tot > 0 && (st = check_gates(a, b, A_log, dt_bias, g, beta, dtype)) != GDN_OK) return st;
    if (flags & ~(GDN_QK_L2NORM | GDN_SOLVE_NEUMANN | GDN_CHUNK(0xff))) return GDN_ERR_INVALID_ARG;
    const int chunk = ((flags >> 8) & 0xffu) == 0 ? 64 : (int)((flags >> 8) & 0xffu);
    if (chunk != 16 && chunk != 32 && chunk != 64) return GDN_ERR_INVALID_ARG;
    const bool tensor_core = dtype == GDN_BF16 && dims.d_k == 128;
    if ((flags & GDN_SOLVE_NEUMANN) && !tensor_core) return GDN_ERR_UNSUPPORTED;
    // shorter chunks on the tensor-core path run in more workspace segments,
    // between which the state crosses through final_state
    if (chunk != 64 && tensor_core && T_tot > 0 && final_state == nullptr) return GDN_ERR_UNSUPPORTED;
    if (!isfinite(scale)) return GDN_ERR_INVALID_ARG;
    if (T_tot > 0 && (qkv == nullptr || o == nullptr)) return GDN_ERR_INVALID_ARG;
    if (!aligned16(qkv) || !aligned16(o) || !aligned16(initial_state) || !aligned16(final_state) ||
        !aligned16(state_ckpt_out))
        return GDN_ERR_ALIGN;
    const size_t need = gdn_chunk_prefill_workspace_size(n_seq, T_tot, dims, dtype);
    if (need > 0 && (workspace == nullptr || ws_bytes < need)) return GDN_ERR_WORKSPACE;
    if ((int64_t)n_seq * dims.H_v * 8 > INT32_MAX) return GDN_ERR_UNSUPPORTED;

    gdn::DeltaArgs d;
    memset(&d, 0, sizeof(d));
    d.qkv = qkv; d.a = a; d.b = b; d.A_log = A_log; d.dt_bias = dt_bias;
    const bool pre = g && beta;
    d.g = pre ? g : nullptr; d.beta = pre ? beta : nullptr;
    d.cu = cu_seqlens; d.n_seq = n_seq; d.T = T_tot;
    d.H_k = dims.H_k; d.H_v = dims.H_v; d.D = dims.d_k;
    d.S0 = initial_state; d.S_final = final_state;
    d.ckpt_every = ckpt_every; d.ckpt = ckpt_every > 0 ? state_ckpt_out : nullptr;
    d.ckpt_rows = ckpt_rows;
    d.scale = scale == 0.f ? 1.0f / sqrtf((float)dims.d_k) : scale;
    d.l2norm = (flags & GDN_QK_L2NORM) != 0;
    d.neumann = (flags & GDN_SOLVE_NEUMANN) != 0;
    d.chunk = chunk;
    d.o = o;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e = need > 0 ? gdn::launch_chunk_split(d, workspace, ws_bytes, s) : gdn::launch_chunk_ffma(d, dtype, s);
    if (e == cudaSuccess && norm_out != nullptr)
        e = gdn::launch_rmsnorm_gated(o, norm_z, norm_w, norm_eps, T_tot, dims.H_v, dims.d_v, norm_out, dtype, s);
    return cuda_status(e);
}
}  // namespace

gdn_status_t gdn_chunk_prefill(const void* qkv, const void* a, const void* b, const float* A_log,
                               const float* dt_bias, const float* g, const float* beta,
                               const int32_t* cu_seqlens, int32_t n_seq, int64_t T_tot,
                               const float* initial_state, float* final_state, int32_t ckpt_every,
                               float* state_ckpt_out, int64_t ckpt_rows, float scale,
                               uint32_t flags, void* o, void* workspace, size_t ws_bytes,
                               gdn_dims_t dims, gdn_dtype_t dtype, void* stream) {
    return chunk_prefill_impl(qkv, a, b, A_log, dt_bias, g, beta, cu_seqlens, n_seq, T_tot, initial_state,
                              final_state, ckpt_every, state_ckpt_out, ckpt_rows, scale, flags, o, workspace,
                              ws_bytes, dims, dtype, stream, nullptr, nullptr, 0.f, nullptr);
}

gdn_status_t gdn_chunk_prefill_norm(const void* qkv, const void* a, const void* b, const float* A_log,
                                    const float* dt_bias, const float* g, const float* beta,
                                    const int32_t* cu_seqlens, int32_t n_seq, int64_t T_tot,
                                    const float* initial_state, float* final_state, int32_t ckpt_every,
                                    float* state_ckpt_out, int64_t ckpt_rows, float scale, uint32_t flags,
                                    const void* z, const void* norm_w, float norm_eps, void* out,
                                    void* workspace, size_t ws_bytes, gdn_dims_t dims, gdn_dtype_t dtype,
                                    void* stream) {
    if (!isfinite(norm_eps) || norm_eps <= 0.f || norm_w == nullptr) return GDN_ERR_INVALID_ARG;
    if (T_tot > 0 && z == nullptr) return GDN_ERR_INVALID_ARG;
    if (!aligned16(z) || !aligned16(norm_w)) return GDN_ERR_ALIGN;
    return chunk_prefill_impl(qkv, a, b, A_log, dt_bias, g, beta, cu_seqlens, n_seq, T_tot, initial_state,
                              final_state, ckpt_every, state_ckpt_out, ckpt_rows, scale, flags, out, workspace,
                              ws_bytes, dims, dtype, stream, z, norm_w, norm_eps, T_tot > 0 ? out : nullptr);
}

size_t gdn_layer_prefill_workspace_size(int32_t n_seq, int64_t T_tot, gdn_dims_t dims, gdn_dtype_t dtype) {
    if (check_dims(dims, dtype) != GDN_OK || n_seq < 1 || T_tot <= 0 || T_tot > (int64_t)INT32_MAX) return 0;
    // tensor-core path: the conv runs inside the chunk kernels (no y buffer)
    if (dtype == GDN_BF16 && dims.d_k == 128) return gdn::chunk_split_conv_workspace_bytes(n_seq, T_tot, dims.H_k, dims.H_v);
    return ((size_t)T_tot * (size_t)conv_dim_of(dims) * elem_size(dtype) + 255) & ~(size_t)255;
}

int32_t gdn_layer_prefill_launches(int32_t n_seq, int64_t T_tot, int32_t has_cu_seqlens, gdn_dims_t dims,
                                   gdn_dtype_t dtype, uint32_t flags) {
    if (check_dims(dims, dtype) != GDN_OK || n_seq < 1 || T_tot <= 0) return 0;
    // the chunked rule and the norm, and the conv (on the tensor-core path it
    // runs in the chunk kernels, which with conv_state_out not conv_state_in
    // also write the conv state)
    const bool tc = dtype == GDN_BF16 && dims.d_k == 128;
    return (tc ? 1 : 2) + gdn_chunk_prefill_launches(n_seq, T_tot, has_cu_seqlens, dims, dtype, flags);
}

gdn_status_t gdn_layer_prefill(const void* x, const void* z, const void* a, const void* b, const void* conv_w,
                               const float* A_log, const float* dt_bias, const void* norm_w, float norm_eps,
                               const int32_t* cu_seqlens, int32_t n_seq, int64_t T_tot,
                               const float* initial_state, float* final_state, const void* conv_state_in,
                               void* conv_state_out, int32_t ckpt_every, float* state_ckpt_out,
                               void* conv_ckpt_out, int64_t ckpt_rows, float scale, uint32_t flags, void* out,
                               void* workspace, size_t ws_bytes, gdn_dims_t dims, gdn_dtype_t dtype,
                               void* stream) {
    gdn_status_t st = check_dims(dims, dtype);
    if (st != GDN_OK) return st;
    if ((st = check_seqs(cu_seqlens, n_seq, T_tot)) != GDN_OK) return st;
    if ((st = check_ckpt(ckpt_every, state_ckpt_out, ckpt_rows)) != GDN_OK) return st;
    if ((st = check_ckpt(ckpt_every, conv_ckpt_out, ckpt_rows)) != GDN_OK) return st;
    if (!isfinite(norm_eps) || norm_eps <= 0.f) return GDN_ERR_INVALID_ARG;
    if (conv_w == nullptr || norm_w == nullptr || A_log == nullptr || dt_bias == nullptr) return GDN_ERR_INVALID_ARG;
    if (T_tot > 0 && (x == nullptr || z == nullptr || a == nullptr || b == nullptr || out == nullptr))
        return GDN_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(z) || !aligned16(norm_w) || !aligned16(out) || !aligned16(workspace))
        return GDN_ERR_ALIGN;
    const size_t need = gdn_layer_prefill_workspace_size(n_seq, T_tot, dims, dtype);
    if (need > 0 && (workspace == nullptr || ws_bytes < need)) return GDN_ERR_WORKSPACE;
    if (T_tot > 0 && dtype == GDN_BF16 && dims.d_k == 128) {
        // tensor-core path: conv1d + SiLU, the conv state and the conv
        // checkpoints inside the chunk kernels (the state in place: by a pass
        // after them), then RMSNormGated
        if ((st = check_gates(a, b, A_log, dt_bias, nullptr, nullptr, dtype)) != GDN_OK) return st;
        if (flags & ~(GDN_QK_L2NORM | GDN_SOLVE_NEUMANN | GDN_CHUNK(0xff))) return GDN_ERR_INVALID_ARG;
        const uint32_t c = (flags >> 8) & 0xffu;
        if (c != 0 && c != 16 && c != 32 && c != 64) return GDN_ERR_INVALID_ARG;
        // shorter chunks: more segments, the state crossing them through final_state
        if (c == 16 || c == 32) {
            if (final_state == nullptr) return GDN_ERR_UNSUPPORTED;
        }
        if (!isfinite(scale)) return GDN_ERR_INVALID_ARG;
        if (!aligned16(conv_w) || !aligned16(conv_state_in) || !aligned16(conv_state_out) ||
            !aligned16(conv_ckpt_out) || !aligned16(initial_state) || !aligned16(final_state) ||
            !aligned16(state_ckpt_out))
            return GDN_ERR_ALIGN;
        if ((int64_t)n_seq * dims.H_v * 8 > INT32_MAX) return GDN_ERR_UNSUPPORTED;
        gdn::DeltaArgs d;
        memset(&d, 0, sizeof(d));
        d.qkv = x; d.a = a; d.b = b; d.A_log = A_log; d.dt_bias = dt_bias;
        d.cu = cu_seqlens; d.n_seq = n_seq; d.T = T_tot;
        d.H_k = dims.H_k; d.H_v = dims.H_v; d.D = dims.d_k;
        d.S0 = initial_state; d.S_final = final_state;
        d.ckpt_every = ckpt_every; d.ckpt = ckpt_every > 0 ? state_ckpt_out : nullptr;
        d.ckpt_rows = ckpt_rows;
        d.scale = scale == 0.f ? 1.0f / sqrtf((float)dims.d_k) : scale;
        d.l2norm = (flags & GDN_QK_L2NORM) != 0;
        d.neumann = (flags & GDN_SOLVE_NEUMANN) != 0;
        d.chunk = c == 0 ? 64 : (int)c;
        d.o = out;
        d.conv_w = conv_w;
        d.conv_state0 = conv_state_in;
        // the kernels write the conv state and checkpoints unless the state is
        // updated in place (the kernels of other chunks still read it)
        const bool in_place = conv_state_out != nullptr && conv_state_out == conv_state_in;
        if (!in_place) {
            d.conv_state_out = conv_state_out;
            d.conv_ckpt = ckpt_every > 0 ? conv_ckpt_out : nullptr;
        }
        cudaStream_t s = (cudaStream_t)stream;
        cudaError_t e = gdn::launch_chunk_split(d, workspace, ws_bytes, s);
        if (e == cudaSuccess && in_place) {
            gdn::ConvArgs c;
            memset(&c, 0, sizeof(c));
            c.x = x; c.w = conv_w; c.cu = cu_seqlens; c.n_seq = n_seq; c.T = T_tot;
            c.C = (int)conv_dim_of(dims);
            c.state_in = conv_state_in; c.state_out = conv_state_out;
            c.ckpt_every = ckpt_every; c.ckpt = ckpt_every > 0 ? conv_ckpt_out : nullptr;
            c.ckpt_rows = ckpt_rows; c.silu = 1;
            e = gdn::launch_conv1d_state(c, dtype, s);
        }
        if (e == cudaSuccess)
            e = gdn::launch_rmsnorm_gated(out, z, norm_w, norm_eps, T_tot, dims.H_v, dims.d_v, out, dtype, s);
        return cuda_status(e);
    }
    const size_t ybytes = T_tot > 0 ? ((size_t)T_tot * (size_t)conv_dim_of(dims) * elem_size(dtype) + 255) &
                                          ~(size_t)255
                                    : 0;
    void* y = T_tot > 0 ? workspace : nullptr;
    void* cws = need > ybytes ? static_cast<uint8_t*>(workspace) + ybytes : nullptr;
    st = gdn_conv1d_fwd(x, conv_w, cu_seqlens, n_seq, T_tot, conv_state_in, conv_state_out, ckpt_every,
                        conv_ckpt_out, ckpt_rows, 1, y, dims, dtype, stream);
    if (st != GDN_OK) return st;
    return gdn_chunk_prefill_norm(y, a, b, A_log, dt_bias, nullptr, nullptr, cu_seqlens, n_seq, T_tot,
                                  initial_state, final_state, ckpt_every, state_ckpt_out, ckpt_rows, scale, flags,
                                  z, norm_w, norm_eps, out, cws, need - ybytes, dims, dtype, stream);
}

gdn_status_t gdn_chunk_prefill_noalloc(const void* qkv, const void* a, const void* b,
                                       const float* A_log, const float* dt_bias, const float* g,
                                       const float* beta, const int32_t* cu_seqlens, int32_t n_seq,
                                       int64_t T_tot, const float* initial_state, float* final_state,
                                       int32_t ckpt_every, float* state_ckpt_out, int64_t ckpt_rows,
                                       float scale, uint32_t flags, void* o, gdn_dims_t dims,
                                       gdn_dtype_t dtype, void* stream) {
    gdn_status_t st = check_dims(dims, dtype);
    if (st != GDN_OK) return st;
    if (dtype != GDN_BF16 || dims.d_k != 128) return GDN_ERR_UNSUPPORTED;
    if ((st = check_seqs(cu_seqlens, n_seq, T_tot)) != GDN_OK) return st;
    if ((st = check_ckpt(ckpt_every, state_ckpt_out, ckpt_rows)) != GDN_OK) return st;
    if (T_tot > 0 && (st = check_gates(a, b, A_log, dt_bias, g, beta, dtype)) != GDN_OK) return st;
    if (flags & ~GDN_QK_L2NORM) return GDN_ERR_INVALID_ARG;
    if (!isfinite(scale)) return GDN_ERR_INVALID_ARG;
    if (final_state == nullptr) return GDN_ERR_INVALID_ARG;
    if (T_tot > 0 && (qkv == nullptr || o == nullptr)) return GDN_ERR_INVALID_ARG;
    if (!aligned16(qkv) || !aligned16(o) || !aligned16(initial_state) || !aligned16(final_state) ||
        !aligned16(state_ckpt_out))
        return GDN_ERR_ALIGN;
    if (!gdn::chunk_split_static_fits(n_seq, dims.H_v)) return GDN_ERR_WORKSPACE;
    if (T_tot == 0) {
        // nothing to compute: the final state of every (empty) sequence is its initial state
        const size_t bytes = (size_t)n_seq * dims.H_v * dims.d_k * dims.d_v * sizeof(float);
        cudaError_t e = initial_state != nullptr
                            ? (initial_state == final_state
                                   ? cudaSuccess
                                   : cudaMemcpyAsync(final_state, initial_state, bytes,
                                                     cudaMemcpyDeviceToDevice, (cudaStream_t)stream))
                            : cudaMemsetAsync(final_state, 0, bytes, (cudaStream_t)stream);
        return cuda_status(e);
    }
    gdn::DeltaArgs d;
    memset(&d, 0, sizeof(d));
    d.qkv = qkv; d.a = a; d.b = b; d.A_log = A_log; d.dt_bias = dt_bias;
    const bool pre = g && beta;
    d.g = pre ? g : nullptr; d.beta = pre ? beta : nullptr;
    d.cu = cu_seqlens; d.n_seq = n_seq; d.T = T_tot;
    d.H_k = dims.H_k; d.H_v = dims.H_v; d.D = dims.d_k;
    d.S0 = initial_state; d.S_final = final_state;
    d.ckpt_every = ckpt_every; d.ckpt = ckpt_every > 0 ? state_ckpt_out : nullptr;
    d.ckpt_rows = ckpt_rows;
    d.scale = scale == 0.f ? 1.0f / sqrtf((float)dims.d_k) : scale;
    d.l2norm = (flags & GDN_QK_L2NORM) != 0;
    d.o = o;
    return cuda_status(gdn::launch_chunk_split_static(d, (cudaStream_t)stream));
}

gdn_status_t gdn_recurrent_decode(const void* qkv, const void* a, const void* b,
                                  const float* A_log, const float* dt_bias, const float* g,
                                  const float* beta, float* state, int32_t B, float scale,
                                  uint32_t flags, void* o, gdn_dims_t dims, gdn_dtype_t dtype,
                                  void* stream) {
    gdn_status_t st = check_dims(dims, dtype);
    if (st != GDN_OK) return st;
    if (B < 0 || (int64_t)B * dims.H_v > INT32_MAX) return GDN_ERR_INVALID_ARG;
    if (B > 0 && (st = check_gates(a, b, A_log, dt_bias, g, beta, dtype)) != GDN_OK) return st;
    if (flags & ~GDN_QK_L2NORM) return GDN_ERR_INVALID_ARG;
    if (!isfinite(scale)) return GDN_ERR_INVALID_ARG;
    if (B > 0 && (qkv == nullptr || state == nullptr || o == nullptr)) return GDN_ERR_INVALID_ARG;
    if (!aligned16(qkv) || !aligned16(state) || !aligned16(o)) return GDN_ERR_ALIGN;
    gdn::DeltaArgs d;
    memset(&d, 0, sizeof(d));
    d.qkv = qkv; d.a = a; d.b = b; d.A_log = A_log; d.dt_bias = dt_bias;
    const bool pre = g && beta;
    d.g = pre ? g : nullptr; d.beta = pre ? beta : nullptr;
    d.n_seq = B; d.T = B;
    d.H_k = dims.H_k; d.H_v = dims.H_v; d.D = dims.d_k;
    d.S0 = state; d.S_final = state;
    d.scale = scale == 0.f ? 1.0f / sqrtf((float)dims.d_k) : scale;
    d.l2norm = (flags & GDN_QK_L2NORM) != 0;
    d.o = o;
    return cuda_status(gdn::launch_recurrent_decode(d, dtype, (cudaStream_t)stream));
}

gdn_status_t gdn_rmsnorm_gated(const void* o, const void* z, const void* w, float eps, int64_t T,
                               void* out, gdn_dims_t dims, gdn_dtype_t dtype, void* stream) {
    gdn_status_t st = check_dims(dims, dtype);
    if (st != GDN_OK) return st;
    if (T < 0 || !(eps > 0.f) || !isfinite(eps)) return GDN_ERR_INVALID_ARG;
    if (w == nullptr || (T > 0 && (o == nullptr || z == nullptr || out == nullptr)))
        return GDN_ERR_INVALID_ARG;
    if (!aligned16(o) || !aligned16(z) || !aligned16(w) || !aligned16(out)) return GDN_ERR_ALIGN;
    return cuda_status(gdn::launch_rmsnorm_gated(o, z, w, eps, T, dims.H_v, dims.d_v, out, dtype,
                                                 (cudaStream_t)stream));
}

// ---------------------------------------------------------------- paged cache, drafted tokens
namespace {
gdn_status_t check_cache(int32_t H_kv, int32_t D, int32_t page_size, int32_t n_pages, int32_t max_pages,
                         gdn_dtype_t dt) {
    if (dt != GDN_F32 && dt != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (H_kv <= 0 || D <= 0 || page_size <= 0 || n_pages <= 0 || max_pages <= 0) return GDN_ERR_INVALID_ARG;
    if (D % 8 != 0 || D > 256 || H_kv > 65536) return GDN_ERR_UNSUPPORTED;
    // positions fit 32 bits with room for a tile, rows of a page fit 31
    if ((int64_t)max_pages * page_size > (1 << 30) || (int64_t)H_kv * page_size > (1 << 30))
        return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

gdn_status_t fill_attn(gdn::AttnArgs& a, int32_t B, int32_t K, int32_t H_q, int32_t H_kv, int32_t D,
                       int32_t page_size, int32_t n_pages, int32_t max_pages, gdn_dtype_t dt) {
    memset(&a, 0, sizeof(a));
    const gdn_status_t st = check_cache(H_kv, D, page_size, n_pages, max_pages, dt);
    if (st != GDN_OK) return st;
    if (B < 0 || B > (1 << 24) || K < 0 || K > gdn::kAttnMaxK || H_q <= 0 || H_q % H_kv != 0)
        return GDN_ERR_INVALID_ARG;
    if (H_q > 65536) return GDN_ERR_UNSUPPORTED;
    a.B = B; a.K = K; a.H_q = H_q; a.H_kv = H_kv; a.D = D;
    a.page_size = page_size; a.n_pages = n_pages; a.max_pages = max_pages;
    a.stop_at = -1;
    return GDN_OK;
}

gdn_status_t attn_decode(const void* q, const void* k_cache, const void* v_cache, const int32_t* page_table,
                         const int32_t* seq_lens, float scale, const void* gate, void* out, float* lse, int32_t B,
                         int32_t K, int32_t H_q, int32_t H_kv, int32_t D, int32_t page_size, int32_t n_pages,
                         int32_t max_pages, void* workspace, size_t ws_bytes, gdn_dtype_t dtype, int32_t stop_at,
                         void* stream) {
    gdn::AttnArgs a;
    const gdn_status_t st = fill_attn(a, B, K, H_q, H_kv, D, page_size, n_pages, max_pages, dtype);
    if (st != GDN_OK) return st;
    if (!isfinite(scale) || scale < 0.f) return GDN_ERR_INVALID_ARG;
    if (B == 0 || K == 0) return GDN_OK;
    if (q == nullptr || k_cache == nullptr || v_cache == nullptr || page_table == nullptr || seq_lens == nullptr ||
        out == nullptr)
        return GDN_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned_n(page_table, 4) ||
        !aligned_n(seq_lens, 4) || !aligned16(gate) || !aligned16(out) || !aligned_n(lse, 4) || !aligned16(workspace))
        return GDN_ERR_ALIGN;
    a.q = q; a.k_cache = k_cache; a.v_cache = v_cache; a.table = page_table; a.lens = seq_lens;
    a.gate = gate; a.out = out; a.lse = lse;
    a.ws = static_cast<float*>(workspace);
    a.stop_at = stop_at;
    a.scale_log2 = (scale == 0.f ? 1.0f / sqrtf((float)D) : scale) * 1.4426950408889634f;
    const size_t need = gdn::attn_plan(a, dtype);
    if (workspace == nullptr || ws_bytes < need) return GDN_ERR_WORKSPACE;
    return cuda_status(gdn::launch_attn_decode(a, dtype, (cudaStream_t)stream));
}
}  // namespace

gdn_status_t gdn_kv_append(const void* k, const void* v, void* k_cache, void* v_cache, const int32_t* page_table,
                           const int32_t* seq_lens, const int32_t* cu_seqlens, int32_t B, int64_t T_tot,
                           int32_t H_kv, int32_t D, int32_t page_size, int32_t n_pages, int32_t max_pages,
                           gdn_dtype_t dtype, void* stream) {
    const gdn_status_t st = check_cache(H_kv, D, page_size, n_pages, max_pages, dtype);
    if (st != GDN_OK) return st;
    if (B < 0 || B > (1 << 24) || T_tot < 0 || T_tot > (int64_t)INT32_MAX) return GDN_ERR_INVALID_ARG;
    if (T_tot == 0) return GDN_OK;
    if (B == 0 || (cu_seqlens == nullptr && T_tot % B != 0)) return GDN_ERR_INVALID_ARG;
    if (k == nullptr || v == nullptr || k_cache == nullptr || v_cache == nullptr || page_table == nullptr ||
        seq_lens == nullptr)
        return GDN_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned_n(page_table, 4) ||
        !aligned_n(seq_lens, 4) || !aligned_n(cu_seqlens, 4))
        return GDN_ERR_ALIGN;
    gdn::KvAppendArgs a;
    memset(&a, 0, sizeof(a));
    a.k = k; a.v = v; a.k_cache = k_cache; a.v_cache = v_cache;
    a.table = page_table; a.lens = seq_lens; a.cu = cu_seqlens;
    a.T = T_tot; a.B = B; a.H_kv = H_kv; a.row_bytes = (int)(D * elem_size(dtype));
    a.page_size = page_size; a.n_pages = n_pages; a.max_pages = max_pages;
    return cuda_status(gdn::launch_kv_append(a, (cudaStream_t)stream));
}

namespace {
// Strides of a [T, H, D] tensor of rows of D contiguous elements.
gdn_status_t check_rows(int64_t tok, int64_t head, int64_t T, int32_t H, gdn_dtype_t dt) {
    const int64_t per16 = 16 / (int64_t)elem_size(dt);
    if ((T > 1 && tok < 0) || (H > 1 && head < 0)) return GDN_ERR_INVALID_ARG;
    if ((T > 1 && tok > INT64_MAX / 16 / T) || (H > 1 && head > INT64_MAX / 16 / H)) return GDN_ERR_INVALID_ARG;
    if ((T > 1 && tok % per16 != 0) || (H > 1 && head % per16 != 0)) return GDN_ERR_ALIGN;
    return GDN_OK;
}

gdn_status_t check_rotation(int32_t n_axes, const int32_t* axes, const float* inv_freq, const float* w0, const float* w1,
                            float eps, float mscale, uint32_t flags, int64_t T, int32_t H, int32_t D, int32_t R,
                            gdn_dtype_t dt) {
    if (dt != GDN_F32 && dt != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (T < 0 || T > (int64_t)INT32_MAX || H <= 0 || D <= 0 || R < 2 || R > D || R % 2 != 0 || n_axes < 1 ||
        (flags & ~GDN_ROPE_INTERLEAVED) != 0 || !isfinite(mscale))
        return GDN_ERR_INVALID_ARG;
    if ((w0 != nullptr || w1 != nullptr) && (!(eps > 0.f) || !isfinite(eps))) return GDN_ERR_INVALID_ARG;
    if (D % 8 != 0 || D > 256 || H > 65536 || n_axes > 16) return GDN_ERR_UNSUPPORTED;
    if (T > 0 && inv_freq == nullptr) return GDN_ERR_INVALID_ARG;
    if (!aligned_n(axes, 4) || !aligned_n(inv_freq, 4) || !aligned_n(w0, 4) || !aligned_n(w1, 4)) return GDN_ERR_ALIGN;
    return GDN_OK;
}

void fill_rotation(gdn::RopeArgs& a, const int32_t* positions, int32_t n_axes, const int32_t* axes, const float* inv_freq,
                   const float* q_w, const float* k_w, float eps, float mscale, uint32_t flags, int64_t T, int32_t D,
                   int32_t R) {
    memset(&a, 0, sizeof(a));
    a.positions = positions; a.axes = axes; a.inv_freq = inv_freq; a.n_axes = n_axes;
    a.q_w = q_w; a.k_w = k_w; a.eps = eps; a.mscale = mscale;
    a.neighbours = (flags & GDN_ROPE_INTERLEAVED) != 0;
    a.T = T; a.D = D; a.R = R;
}
}  // namespace

gdn_status_t gdn_rope(const void* x, int64_t x_token_stride, int64_t x_head_stride, const int32_t* positions,
                      int32_t n_axes, const int32_t* axes, const float* inv_freq, const float* norm_w, float norm_eps,
                      float mscale, uint32_t flags, void* out, int64_t out_token_stride, int64_t out_head_stride,
                      int64_t T, int32_t H, int32_t D, int32_t R, gdn_dtype_t dtype, void* stream) {
    gdn_status_t st = check_rotation(n_axes, axes, inv_freq, norm_w, nullptr, norm_eps, mscale, flags, T, H, D, R, dtype);
    if (st != GDN_OK) return st;
    if (T == 0) return GDN_OK;
    if (x == nullptr || out == nullptr || positions == nullptr) return GDN_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(out) || !aligned_n(positions, 4)) return GDN_ERR_ALIGN;
    if ((st = check_rows(x_token_stride, x_head_stride, T, H, dtype)) != GDN_OK ||
        (st = check_rows(out_token_stride, out_head_stride, T, H, dtype)) != GDN_OK)
        return st;
    const int64_t ot = T > 1 ? out_token_stride : 0, oh = H > 1 ? out_head_stride : 0;
    const int64_t xt = T > 1 ? x_token_stride : 0, xh = H > 1 ? x_head_stride : 0;
    // rows of the output do not overlap, whichever of the two dims is the outer one
    const bool heads_inside = (H == 1 || oh >= D) && (T == 1 || ot >= oh * (H - 1) + D);
    const bool tokens_inside = (T == 1 || ot >= D) && (H == 1 || oh >= ot * (T - 1) + D);
    if (!heads_inside && !tokens_inside) return GDN_ERR_INVALID_ARG;
    if (x == out && (xt != ot || xh != oh)) return GDN_ERR_INVALID_ARG;
    gdn::RopeArgs a;
    fill_rotation(a, positions, n_axes, axes, inv_freq, norm_w, nullptr, norm_eps, mscale, flags, T, D, R);
    a.q = x; a.q_tok = xt; a.q_head = xh; a.q_out = out; a.o_tok = ot; a.o_head = oh;
    a.B = 1; a.H_q = H;
    return cuda_status(gdn::launch_rope(a, dtype, (cudaStream_t)stream));
}

gdn_status_t gdn_rope_kv_append(const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k,
                                int64_t k_token_stride, int64_t k_head_stride, const void* v, int64_t v_token_stride,
                                int64_t v_head_stride, void* q_out, void* k_cache, void* v_cache,
                                const int32_t* page_table, const int32_t* seq_lens, const int32_t* cu_seqlens,
                                const int32_t* positions, int32_t n_axes, const int32_t* axes, const float* inv_freq,
                                const float* q_norm_w, const float* k_norm_w, float norm_eps, float mscale,
                                uint32_t flags, int32_t B, int64_t T_tot, int32_t H_q, int32_t H_kv, int32_t D, int32_t R,
                                int32_t page_size, int32_t n_pages, int32_t max_pages, gdn_dtype_t dtype, void* stream) {
    gdn_status_t st = check_cache(H_kv, D, page_size, n_pages, max_pages, dtype);
    if (st != GDN_OK) return st;
    st = check_rotation(n_axes, axes, inv_freq, q_norm_w, k_norm_w, norm_eps, mscale, flags, T_tot, H_q, D, R, dtype);
    if (st != GDN_OK) return st;
    if (B < 0 || B > (1 << 24) || (positions == nullptr && n_axes != 1)) return GDN_ERR_INVALID_ARG;
    if (T_tot == 0) return GDN_OK;
    if (B == 0 || (cu_seqlens == nullptr && T_tot % B != 0)) return GDN_ERR_INVALID_ARG;
    if (q == nullptr || k == nullptr || v == nullptr || q_out == nullptr || k_cache == nullptr || v_cache == nullptr ||
        page_table == nullptr || seq_lens == nullptr)
        return GDN_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(k_cache) ||
        !aligned16(v_cache) || !aligned_n(page_table, 4) || !aligned_n(seq_lens, 4) || !aligned_n(cu_seqlens, 4) ||
        !aligned_n(positions, 4))
        return GDN_ERR_ALIGN;
    if ((st = check_rows(q_token_stride, q_head_stride, T_tot, H_q, dtype)) != GDN_OK ||
        (st = check_rows(k_token_stride, k_head_stride, T_tot, H_kv, dtype)) != GDN_OK ||
        (st = check_rows(v_token_stride, v_head_stride, T_tot, H_kv, dtype)) != GDN_OK)
        return st;
    gdn::RopeArgs a;
    fill_rotation(a, positions, n_axes, axes, inv_freq, q_norm_w, k_norm_w, norm_eps, mscale, flags, T_tot, D, R);
    const bool many = T_tot > 1;
    a.q = q; a.q_tok = many ? q_token_stride : 0; a.q_head = H_q > 1 ? q_head_stride : 0;
    a.k = k; a.k_tok = many ? k_token_stride : 0; a.k_head = H_kv > 1 ? k_head_stride : 0;
    a.v = v; a.v_tok = many ? v_token_stride : 0; a.v_head = H_kv > 1 ? v_head_stride : 0;
    a.q_out = q_out; a.o_tok = (int64_t)H_q * D; a.o_head = D;
    if (q == q_out && ((many && a.q_tok != a.o_tok) || (H_q > 1 && a.q_head != a.o_head))) return GDN_ERR_INVALID_ARG;
    a.k_cache = k_cache; a.v_cache = v_cache; a.table = page_table; a.lens = seq_lens; a.cu = cu_seqlens;
    a.B = B; a.H_q = H_q; a.H_kv = H_kv; a.page_size = page_size; a.n_pages = n_pages; a.max_pages = max_pages;
    return cuda_status(gdn::launch_rope(a, dtype, (cudaStream_t)stream));
}

size_t gdn_attn_decode_workspace_size(int32_t B, int32_t K, int32_t H_q, int32_t H_kv, int32_t D,
                                      int32_t page_size, gdn_dtype_t dtype) {
    gdn::AttnArgs a;
    if (fill_attn(a, B, K, H_q, H_kv, D, page_size, 1, 1, dtype) != GDN_OK || B == 0 || K == 0) return 0;
    return gdn::attn_plan(a, dtype);
}

gdn_status_t gdn_attn_decode(const void* q, const void* k_cache, const void* v_cache, const int32_t* page_table,
                             const int32_t* seq_lens, float scale, const void* gate, void* out, float* lse,
                             int32_t B, int32_t K, int32_t H_q, int32_t H_kv, int32_t D, int32_t page_size,
                             int32_t n_pages, int32_t max_pages, void* workspace, size_t ws_bytes,
                             gdn_dtype_t dtype, void* stream) {
    return attn_decode(q, k_cache, v_cache, page_table, seq_lens, scale, gate, out, lse, B, K, H_q, H_kv, D, page_size,
                       n_pages, max_pages, workspace, ws_bytes, dtype, -1, stream);
}

gdn_status_t gdn_selftest_attn_decode(const void* q, const void* k_cache, const void* v_cache,
                                      const int32_t* page_table, const int32_t* seq_lens, void* out, int32_t B,
                                      int32_t K, int32_t H_q, int32_t H_kv, int32_t D, int32_t page_size,
                                      int32_t n_pages, int32_t max_pages, void* workspace, size_t ws_bytes,
                                      int32_t stop_at, void* stream) {
    if (stop_at < 0) return GDN_ERR_INVALID_ARG;
    if (page_size % 4 != 0) return GDN_ERR_UNSUPPORTED;  // the CUDA-core kernel waits for nothing
    return attn_decode(q, k_cache, v_cache, page_table, seq_lens, 0.f, nullptr, out, nullptr, B, K, H_q, H_kv, D,
                       page_size, n_pages, max_pages, workspace, ws_bytes, GDN_BF16, stop_at, stream);
}

namespace {
gdn_status_t fill_shared(gdn::ShareArgs& s, int32_t B, int32_t K, int32_t H_q, int32_t H_kv, int32_t D, int32_t page_size,
                         int32_t n_pages, int32_t max_pages, int32_t G, gdn_dtype_t dt) {
    memset(&s, 0, sizeof(s));
    const gdn_status_t st = fill_attn(s.a, B, K, H_q, H_kv, D, page_size, n_pages, max_pages, dt);
    if (st != GDN_OK) return st;
    if (G < 1 || G > (1 << 24)) return GDN_ERR_INVALID_ARG;
    if ((int64_t)B * K * H_q > (1 << 30)) return GDN_ERR_UNSUPPORTED;  // rows fit 31 bits
    s.G = G;
    return GDN_OK;
}

gdn_status_t attn_decode_shared(const void* q, const void* k_cache, const void* v_cache, const int32_t* page_table,
                                const int32_t* seq_lens, const int32_t* prefix_lens, const int32_t* cu_groups, float scale,
                                const void* gate, void* out, float* lse, int32_t B, int32_t K, int32_t H_q, int32_t H_kv,
                                int32_t D, int32_t page_size, int32_t n_pages, int32_t max_pages, int32_t G, void* workspace,
                                size_t ws_bytes, gdn_dtype_t dtype, int32_t stop_at, void* stream) {
    gdn::ShareArgs s;
    const gdn_status_t st = fill_shared(s, B, K, H_q, H_kv, D, page_size, n_pages, max_pages, G, dtype);
    if (st != GDN_OK) return st;
    if (!isfinite(scale) || scale < 0.f || (cu_groups == nullptr && G != 1)) return GDN_ERR_INVALID_ARG;
    if (B == 0 || K == 0) return GDN_OK;
    if (q == nullptr || k_cache == nullptr || v_cache == nullptr || page_table == nullptr || seq_lens == nullptr ||
        prefix_lens == nullptr || out == nullptr)
        return GDN_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned_n(page_table, 4) ||
        !aligned_n(seq_lens, 4) || !aligned_n(prefix_lens, 4) || !aligned_n(cu_groups, 4) || !aligned16(gate) ||
        !aligned16(out) || !aligned_n(lse, 4) || !aligned16(workspace))
        return GDN_ERR_ALIGN;
    gdn::AttnArgs& a = s.a;
    a.q = q; a.k_cache = k_cache; a.v_cache = v_cache; a.table = page_table; a.lens = seq_lens;
    a.gate = gate; a.out = out; a.lse = lse;
    a.stop_at = stop_at;
    a.scale_log2 = (scale == 0.f ? 1.0f / sqrtf((float)D) : scale) * 1.4426950408889634f;
    s.prefix = prefix_lens; s.cu = cu_groups;
    const size_t need = gdn::attn_share_plan(s, dtype, workspace);
    if (workspace == nullptr || ws_bytes < need) return GDN_ERR_WORKSPACE;
    return cuda_status(gdn::launch_attn_shared(s, dtype, (cudaStream_t)stream));
}
}  // namespace

size_t gdn_attn_decode_shared_workspace_size(int32_t B, int32_t K, int32_t H_q, int32_t H_kv, int32_t D, int32_t page_size,
                                             int32_t G, gdn_dtype_t dtype) {
    gdn::ShareArgs s;
    if (fill_shared(s, B, K, H_q, H_kv, D, page_size, 1, 1, G, dtype) != GDN_OK || B == 0 || K == 0) return 0;
    return gdn::attn_share_plan(s, dtype, nullptr);
}

gdn_status_t gdn_attn_decode_shared(const void* q, const void* k_cache, const void* v_cache, const int32_t* page_table,
                                    const int32_t* seq_lens, const int32_t* prefix_lens, const int32_t* cu_groups,
                                    float scale, const void* gate, void* out, float* lse, int32_t B, int32_t K, int32_t H_q,
                                    int32_t H_kv, int32_t D, int32_t page_size, int32_t n_pages, int32_t max_pages, int32_t G,
                                    void* workspace, size_t ws_bytes, gdn_dtype_t dtype, void* stream) {
    return attn_decode_shared(q, k_cache, v_cache, page_table, seq_lens, prefix_lens, cu_groups, scale, gate, out, lse, B, K,
                              H_q, H_kv, D, page_size, n_pages, max_pages, G, workspace, ws_bytes, dtype, -1, stream);
}

gdn_status_t gdn_selftest_attn_decode_shared(const void* q, const void* k_cache, const void* v_cache,
                                             const int32_t* page_table, const int32_t* seq_lens, const int32_t* prefix_lens,
                                             void* out, int32_t B, int32_t K, int32_t H_q, int32_t H_kv, int32_t D,
                                             int32_t page_size, int32_t n_pages, int32_t max_pages, void* workspace,
                                             size_t ws_bytes, int32_t stop_at, void* stream) {
    if (stop_at < 0) return GDN_ERR_INVALID_ARG;
    if (page_size % 4 != 0) return GDN_ERR_UNSUPPORTED;  // the CUDA-core kernels wait for nothing
    return attn_decode_shared(q, k_cache, v_cache, page_table, seq_lens, prefix_lens, nullptr, 0.f, nullptr, out, nullptr, B,
                              K, H_q, H_kv, D, page_size, n_pages, max_pages, 1, workspace, ws_bytes, GDN_BF16, stop_at,
                              stream);
}

gdn_status_t gdn_draft_accept(const void* p, const void* q, const int32_t* draft, const float* u,
                              const int32_t* n_draft, const int32_t* slots, int32_t B, int32_t K, int32_t V,
                              int32_t* n_accept, int32_t* tokens, int32_t* next_slot, gdn_dtype_t dtype,
                              void* stream) {
    if (dtype != GDN_F32 && dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (B < 0 || B > (1 << 24) || K < 0 || K > gdn::kAcceptMaxK || V <= 0 || V > (1 << 24)) return GDN_ERR_INVALID_ARG;
    if (B == 0) return GDN_OK;
    if (p == nullptr || (K > 0 && draft == nullptr) || u == nullptr || n_accept == nullptr || tokens == nullptr ||
        (slots == nullptr) != (next_slot == nullptr))
        return GDN_ERR_INVALID_ARG;
    if (!aligned16(p) || !aligned16(q) || !aligned_n(draft, 4) || !aligned_n(u, 4) || !aligned_n(n_draft, 4) ||
        !aligned_n(slots, 4) || !aligned_n(n_accept, 4) || !aligned_n(tokens, 4) || !aligned_n(next_slot, 4))
        return GDN_ERR_ALIGN;
    gdn::DraftAcceptArgs a;
    memset(&a, 0, sizeof(a));
    a.p = p; a.q = q; a.draft = draft; a.u = u; a.n_draft = n_draft; a.slots = slots;
    a.B = B; a.K = K; a.V = V; a.n_accept = n_accept; a.tokens = tokens; a.next_slot = next_slot;
    return cuda_status(gdn::launch_draft_accept(a, dtype, (cudaStream_t)stream));
}

}  // extern "C"
