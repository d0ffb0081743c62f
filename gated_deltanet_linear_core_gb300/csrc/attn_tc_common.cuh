// What the tensor-core attention kernels (attn_tc.cu, attn_shared_tc.cu) share: cache
// tiles of 128 tokens loaded by TMA in page pieces, bounded waits of their roles,
// MMAs with 128-byte-swizzled operands.
#pragma once

#include <cuda.h>

#include "attn_common.cuh"
#include "tc_ptx.cuh"

namespace gdn {
namespace attn {

using namespace tc;

constexpr int TILE = 128;
constexpr int SLAB = TILE * 128;      // bytes of 128 tokens x 64 dims
constexpr int SLOT = 2 * SLAB;        // ... x 128 dims
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr int kSmemMax = 232448;

// Bounded wait; returns at once when another role has given up.
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    if (mbar_test(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
        if (mbar_test(bar, parity)) return true;
        if ((it & 31) == 0) {
            if (*abort_flag) return false;
            if (globaltimer_ns() - t0 > kWaitNs) {
                *abort_flag = 1;
                return false;
            }
        }
    }
}

// The same for a slot's position counter to reach `pos`.
__device__ __forceinline__ bool loaded_or_abort(volatile int* filled, int pos, volatile int* abort_flag) {
    if (*filled >= pos) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
        if (*filled >= pos) return true;
        if ((it & 31) == 0) {
            if (*abort_flag) return false;
            if (globaltimer_ns() - t0 > kWaitNs) {
                *abort_flag = 1;
                return false;
            }
        }
    }
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ bool finite_bf16x8(uint4 u) {
    bool ok = true;
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) ok = ok && (w[i] & 0x7f80u) != 0x7f80u && (w[i] & 0x7f800000u) != 0x7f800000u;
    return ok;
}
__device__ __forceinline__ uint32_t zero_non_finite(uint32_t w) {
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
    return w;
}

// Operand descriptors by their low words (address and lbo in units of 16 bytes); the high word is the same for
// all (sbo 1024, version, 128-byte swizzle: sdesc_sw128).
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return (saddr >> 4) | ((lbo >> 4) << 16); }
__device__ __forceinline__ void mma_lo(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
    constexpr uint32_t hi = (1024u >> 4) | (1u << 14) | (2u << 29);
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
        "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(hi)
        : "memory");
}

inline bool encode_cache(CUtensorMap* map, const void* base, const AttnArgs& a, int piece) {
    const PFN_cuTensorMapEncodeTiled_v12000 enc = tensormap_encoder();
    if (enc == nullptr) return false;
    cuuint64_t dim[3] = {(cuuint64_t)a.D, (cuuint64_t)a.H_kv * a.page_size, (cuuint64_t)a.n_pages};
    cuuint64_t str[2] = {(cuuint64_t)a.D * 2, (cuuint64_t)a.D * 2 * a.H_kv * a.page_size};
    cuuint32_t box[3] = {64, (cuuint32_t)piece, 1};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dim, str, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of a page that one TMA box takes: the largest power of two that divides the page size, a tile at most.
inline int page_piece(int page_size) {
    const int p = page_size & -page_size;
    return p < TILE ? p : TILE;
}

}  // namespace attn
}  // namespace gdn
