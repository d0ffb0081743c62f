// Host-side launchers of the GDN kernels (one translation unit per kernel
// family).  Arguments are already validated by the C ABI layer in gdn_api.cu.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn.h"

#include <cudaTypedefs.h>

namespace gdn {

struct ConvArgs {
    const void* x;
    const void* w;
    const int32_t* cu;
    int n_seq;
    int64_t T;
    int C;  // conv_dim
    const void* state_in;
    void* state_out;
    int ckpt_every;
    void* ckpt;
    int64_t ckpt_rows;
    int silu;
    void* y;
    int fused_state;  // set by launch_conv1d_fwd: the tile kernel writes the state and checkpoints
};
cudaError_t launch_conv1d_fwd(const ConvArgs& a, gdn_dtype_t dt, cudaStream_t s);
// Only the conv state after each sequence and the conv checkpoints (no y): the
// state pass of launch_conv1d_fwd, for callers that compute y elsewhere.
cudaError_t launch_conv1d_state(const ConvArgs& a, gdn_dtype_t dt, cudaStream_t s);
cudaError_t launch_conv1d_update(const void* x, const void* w, void* state, int B, int C,
                                 int silu, void* y, gdn_dtype_t dt, cudaStream_t s);

struct DeltaArgs {
    const void* qkv;  // [T, conv_dim]
    const void* a;
    const void* b;
    const float* A_log;
    const float* dt_bias;
    const float* g;
    const float* beta;
    const int32_t* cu;
    int n_seq;
    int64_t T;
    int H_k, H_v, D;
    const float* S0;
    float* S_final;
    int ckpt_every;
    float* ckpt;
    int64_t ckpt_rows;
    float scale;
    int l2norm;
    void* o;  // [T, H_v, D]
    int neumann;  // chunk inverse by the Neumann-style product (tensor-core path)
    int chunk;    // tokens per chunk: 16, 32 or 64 (0: 64)
    // Conv1d + SiLU inside the chunk kernels (tensor-core path): with conv_w
    // set, qkv is the raw conv input x and the kernels compute y themselves
    // from x, these taps ([conv_dim][4]) and the sequences' conv states before
    // their first tokens ([n_seq][conv_dim][3], null: zeros).
    const void* conv_w;
    const void* conv_state0;
    // ... and, when set, the kernels also write the conv state after each
    // sequence ([n_seq][conv_dim][3]; never the conv_state0 array) and the
    // conv checkpoints ([ckpt_rows][conv_dim][3], every ckpt_every tokens)
    void* conv_state_out;
    void* conv_ckpt;
};
// Chunked prefill on CUDA cores (f32 arithmetic; any supported D and dtype).
cudaError_t launch_chunk_ffma(const DeltaArgs& a, gdn_dtype_t dt, cudaStream_t s);
// Recurrent decode: T = B tokens, sequence i = token i, state in place (S0 == S_final).
cudaError_t launch_recurrent_decode(const DeltaArgs& a, gdn_dtype_t dt, cudaStream_t s);

// Fused decode step: conv update, gates, recurrence and RMSNormGated for one
// token per sequence; conv state and state in place at slots[b] (or b).
struct DecodeStepArgs {
    const void* x;         // [B, conv_dim]
    const void* conv_w;    // [conv_dim, 4]
    void* conv_state;      // [slots, conv_dim, 3]
    const void *z, *a, *b; // [B, H_v*D], [B, H_v], [B, H_v]
    const float *A_log, *dt_bias;
    float* state;          // [slots, H_v, D, D]
    const void* norm_w;    // [D]
    const int32_t* slots;  // [B] or null
    int B, H_k, H_v, D;
    float scale, eps;
    int l2norm;
    void* out;             // [B, H_v*D]
};
cudaError_t launch_decode_step(const DecodeStepArgs& a, gdn_dtype_t dt, cudaStream_t s);

// K draft tokens per sequence from the states in slot slots[b][0]; the conv
// state and the recurrent state after draft token t go to slot slots[b][t + 1].
struct DecodeVerifyArgs {
    const void* x;         // [B, K, conv_dim]
    const void* conv_w;    // [conv_dim, 4]
    void* conv_state;      // [slots, conv_dim, 3]
    const void *z, *a, *b; // [B, K, H_v*D], [B, K, H_v], [B, K, H_v]
    const float *A_log, *dt_bias;
    float* state;          // [slots, H_v, D, D]
    const void* norm_w;    // [D]
    const int32_t* slots;  // [B, K + 1]
    int B, K, H_k, H_v, D;
    float scale, eps;
    int l2norm;
    void* out;             // [B, K, H_v*D]
};
constexpr int kVerifyMaxK = 16;
cudaError_t launch_decode_verify(const DecodeVerifyArgs& a, gdn_dtype_t dt, cudaStream_t s);

// cuTensorMapEncodeTiled from the driver (nullptr if unavailable).
PFN_cuTensorMapEncodeTiled_v12000 tensormap_encoder();
// Unique id of the calling thread's current CUDA context, 0 if there is none
// (or the driver cannot tell).  Caches of device objects key on it, so that a
// context destroyed and created again (a device reset) never reuses objects of
// the old one.
unsigned long long current_context_id();

// Chunked prefill on tcgen05 tensor cores (bf16 operands, f32 state, D = 128)
// in two kernels: the state-independent work of every chunk in parallel (into
// `workspace`), then the sequential state recurrence.
size_t chunk_split_workspace_bytes(int n_seq, int64_t T, int H_v);
// ... when the conv is computed inside the kernels (DeltaArgs::conv_w): the
// same plus the conv'd q tiles of each segment's chunks and key heads.
size_t chunk_split_conv_workspace_bytes(int n_seq, int64_t T, int H_k, int H_v);
cudaError_t launch_chunk_split(const DeltaArgs& a, void* workspace, size_t ws_bytes,
                               cudaStream_t s);
// The same with the chunk offsets and intra kernels on s_pre and the chain on
// s_chain after ev_pre (recorded on s_pre, waited on s_chain); with more than
// one workspace segment everything runs on s_chain after ev_pre.
cudaError_t launch_chunk_split_two(const DeltaArgs& a, void* workspace, size_t ws_bytes, cudaStream_t s_pre,
                                   cudaStream_t s_chain, cudaEvent_t ev_pre);
// Kernel launches launch_chunk_split issues: chunk offsets, then intra + chain per segment
// (chunk: tokens per chunk, 16, 32 or 64).
int chunk_split_launches(int n_seq, int64_t T, int H_v, bool has_cu, int chunk);

// The same chunked prefill with its scratch in a fixed device array of the
// library (gdn_chunk_prefill_noalloc): no allocation; final_state required.
bool chunk_split_static_fits(int n_seq, int H_v);
cudaError_t launch_chunk_split_static(const DeltaArgs& a, cudaStream_t s);

// Reads (synchronising `s`) and clears the library's device error word.
cudaError_t copy_device_error(cudaStream_t s, int* word);
cudaError_t clear_device_error(cudaStream_t s);
// One CTA whose bounded wait runs out after limit_ns and sets the error word.
cudaError_t launch_bounded_wait_selftest(uint64_t limit_ns, cudaStream_t s);
// The same for the conv kernels' own error word.
cudaError_t copy_conv_error(cudaStream_t s, int* word);
cudaError_t clear_conv_error(cudaStream_t s);

cudaError_t launch_rmsnorm_gated(const void* o, const void* z, const void* w, float eps, int64_t T,
                                 int H, int D, void* out, gdn_dtype_t dt, cudaStream_t s);

// Attention of the K newest tokens of B sequences over the paged cache
// (gdn_attn_decode): arguments, and how the call is cut up (attn_common.cuh).
struct AttnArgs {
    const void* q;         // [B, K, H_q, D]
    const void *k_cache, *v_cache;  // [n_pages, H_kv, page_size, D]
    const int32_t* table;  // [B, max_pages]
    const int32_t* lens;   // [B]
    const void* gate;      // [B, K, H_q, D] or null
    void* out;             // [B, K, H_q, D]
    float* lse;            // [B, K, H_q] or null
    float* ws;             // what to join per CTA, then slots of partial results
    int64_t slot_floats;   // floats per slot
    int stat_floats;       // of which maxima and sums come first
    int B, K, H_q, H_kv, D;
    int page_size, max_pages, n_pages;
    float scale_log2;      // score scale times log2 e
    int group, rows;       // H_q / H_kv, K * group
    int rb_rows, n_rb;     // rows per row block, row blocks
    int setup;             // units that starting an item counts as, beside its tiles
    int stop_at;           // self-test: the MMAs stop at a CTA's tile of this number (-1: never)
    // behind shared prefixes (gdn_attn_decode_shared); null otherwise
    const int32_t* skip;   // [B] tokens of the shared prefix, a multiple of kShareStep
    float* part_o;         // [B, K, H_q, D] the items' first parts: unnormalised outputs,
    float4* part_stat;     // [B, K, H_q] maximum, sum, first CTA | CTAs << 16, row in its block
};
constexpr int kAttnMaxK = 16;
constexpr int kAttnMaxCtas = 152;  // CTAs of a call, at most: one per SM
// Fills the derived fields from the sizes; returns the workspace bytes.
size_t attn_plan(AttnArgs& a, gdn_dtype_t dt);
int attn_ctas();
cudaError_t launch_attn_decode(const AttnArgs& a, gdn_dtype_t dt, cudaStream_t s);
constexpr int kAttnFfmaRows = 8;  // rows per block of launch_attn_ffma, at most
cudaError_t launch_attn_ffma(const AttnArgs& a, int n_cta, gdn_dtype_t dt, cudaStream_t s);
// The tensor-core kernel: which calls it takes, and its launch with the join.
bool attn_tc_takes(const AttnArgs& a, gdn_dtype_t dt);
cudaError_t launch_attn_tc(const AttnArgs& a, int n_cta, cudaStream_t s);
cudaError_t copy_attn_error(cudaStream_t s, int* word);
cudaError_t clear_attn_error(cudaStream_t s);
cudaError_t launch_attn_join(const AttnArgs& a, int n_cta, gdn_dtype_t dt, cudaStream_t s);

// Attention behind shared prefixes (gdn_attn_decode_shared; attn_shared.cuh).
constexpr int kPrefixFfmaRows = 64;
constexpr int kShareStep = 128;  // a prefix is shared down to a multiple of this many tokens
// Tokens that one or several sequences attend to through one page table.
struct alignas(16) ShareRecord {
    int64_t unit0;      // first unit of its items
    int seq0, seqs;     // the sequences
    int tile0, tiles;   // the tokens, in tiles
    int leader;         // the sequence whose pages are read
    int blocks;         // row blocks
};
struct ShareArgs {
    AttnArgs a;                        // (its work division holds for what the sequences have of their own on CUDA cores)
    const int32_t *prefix, *cu;        // [G] tokens; [G + 1] sequences or null: one group
    int G;
    int records;                       // G prefixes, then (unless launch_attn_ffma takes them) B sequences' own tokens
    int few;                           // a lane of a warp can hold each: every CTA makes the records for itself
    int rows_per_block, tile, setup;   // rows and tokens per tile, units of an item's start
    int* gather;                       // [3 G] scratch of the plan where there are many groups
    ShareRecord* rec;                  // [records + 1], the last one's unit0 all units
    float* pre_o;                      // [B, K, H_q, D], [B, K, H_q]: the prefix items' first parts, as a.part_o and a.part_stat
    float4* pre_stat;
    float* slots;                      // per CTA: a part that starts inside an item
    int64_t slot_floats;
};
// Fills the derived fields from the sizes (and with a workspace the pointers into it); returns the workspace bytes.
size_t attn_share_plan(ShareArgs& s, gdn_dtype_t dt, void* ws);
cudaError_t launch_attn_shared(const ShareArgs& s, gdn_dtype_t dt, cudaStream_t st);
cudaError_t launch_shared_tc(const ShareArgs& s, int n_cta, cudaStream_t st);
cudaError_t launch_prefix_ffma(const ShareArgs& s, int n_cta, gdn_dtype_t dt, cudaStream_t st);
cudaError_t copy_shared_error(cudaStream_t s, int* word);
cudaError_t clear_shared_error(cudaStream_t s);

// New keys and values into their pages (gdn_kv_append).
struct KvAppendArgs {
    const void *k, *v;     // [T, H_kv, D]
    void *k_cache, *v_cache;
    const int32_t *table, *lens;
    const int32_t* cu;     // [B + 1] or null: T / B tokens each
    int64_t T;
    int B, H_kv, row_bytes, page_size, max_pages, n_pages;
};
cudaError_t launch_kv_append(const KvAppendArgs& a, cudaStream_t s);

// Head norm and rotary positions of q, and with a cache of k on the way into it beside v (gdn_rope,
// gdn_rope_kv_append).  Strides in elements.
struct RopeArgs {
    const void *q, *k, *v;
    int64_t q_tok, q_head, k_tok, k_head, v_tok, v_head;
    void* q_out;
    int64_t o_tok, o_head;
    void *k_cache, *v_cache;  // null: q alone
    const int32_t *table, *lens;
    const int32_t* cu;         // [B + 1] or null: T / B tokens each
    const int32_t* positions;  // [n_axes, T] or null: the cache's
    const int32_t* axes;       // [R / 2] or null: axis 0
    const float* inv_freq;     // [R / 2]
    const float *q_w, *k_w;    // [D] or null
    float eps, mscale;
    int64_t T;
    int B, H_q, H_kv, D, R, n_axes, neighbours, page_size, max_pages, n_pages;
};
cudaError_t launch_rope(const RopeArgs& a, gdn_dtype_t dt, cudaStream_t s);

// Acceptance of drafted tokens (gdn_draft_accept).
struct DraftAcceptArgs {
    const void *p, *q;     // [B, K + 1, V], [B, K, V] or null
    const int32_t* draft;  // [B, K]
    const float* u;        // [B, K + 1]
    const int32_t *n_draft, *slots;  // [B] or null, [B, K + 2] or null
    int B, K, V;
    int32_t *n_accept, *tokens, *next_slot;  // [B], [B, K + 1], [B] or null
};
constexpr int kAcceptMaxK = 15;
cudaError_t launch_draft_accept(const DraftAcceptArgs& a, gdn_dtype_t dt, cudaStream_t s);

// The layer core for one sequence streamed from page-locked host memory
// (gdn_layer_prefill_host).
struct HostLayerArgs {
    const void *h_qkv, *h_z, *h_a, *h_b;  // host, page-locked
    const void* conv_w;
    const float *A_log, *dt_bias;
    const void* norm_w;
    int64_t T;
    int H_k, H_v, D;
    const float* initial_state;
    float* final_state;
    const void* conv_state_in;
    void* conv_state_out;
    float scale, eps;
    int l2norm;
    void* h_out;  // host, page-locked
};
size_t layer_prefill_host_workspace_bytes(int64_t T, int H_k, int H_v, int D, int es, bool tensor_core);
int64_t layer_prefill_host_piece(int64_t T, int H_k, int H_v, int D, int es, bool tensor_core);
int64_t layer_prefill_host_pieces(int64_t T, int H_k, int H_v, int D, int es, bool tensor_core);
cudaError_t launch_layer_prefill_host(const HostLayerArgs& h, gdn_dtype_t dt, void* workspace, cudaStream_t s);

}  // namespace gdn
