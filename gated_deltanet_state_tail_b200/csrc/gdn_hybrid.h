// gdn_hybrid.h -- what the full-attention layers' operators add to gdn_internal.h and
// gdn_sm100.h.  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "gdn_internal.h"
#include "gdn_sm100.h"

namespace gdn {

// The driver's tensor map encoder, looked up once; null if the driver lacks it.
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                  CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                  CUtensorMapFloatOOBfill);
EncodeTiledFn tensor_map_encoder();

// tag_merge inlined, for kernels that report at one or two places: a call by the ABI
// would spill around it.
__device__ __forceinline__ void tag_merge_inline(unsigned long long* word, unsigned int epoch, unsigned int val,
                                                 bool first_only) {
    unsigned long long old = *reinterpret_cast<volatile unsigned long long*>(word);
    for (int i = 0; i < 64; ++i) {
        const unsigned int low = (unsigned int)(old >> 32) == epoch ? (unsigned int)old : 0u;
        const unsigned int nlow = first_only ? (low ? low : val) : (low | val);
        const unsigned long long want = ((unsigned long long)epoch << 32) | nlow;
        if (want == old) return;
        const unsigned long long seen = atomicCAS(word, old, want);
        if (seen == old) return;
        old = seen;
    }
}

// Norm, rotation and cache append of new tokens' projections (no plan, no workspace).
struct NormRopeArgs {
    int dtype;                   // gdn_dtype of q, k, v, the outputs and the cache
    int num_heads, num_kv_heads;
    int dim, rotary_dim;
    int interleaved;             // pairs (2i, 2i + 1) instead of (i, i + rotary_dim / 2)
    long long rows;
    long long rs_q, rs_k, rs_v;  // elements between consecutive rows
    float eps;
    const void* q;
    const void* k;
    const void* v;               // with a cache only
    const long long* positions;  // [rows]
    const double* inv_freq;      // [rotary_dim / 2]
    const float* q_weight;       // [dim] or null: q is not normalised
    const float* k_weight;
    void* q_out;                 // [rows, num_heads, dim] packed
    void* k_out;                 // [rows, num_kv_heads, dim] packed, or null
    // the paged cache, or slots = null
    const long long* slots;      // [rows]: page * page_size + row in the page; outside the pool = not written
    void* k_pages;
    void* v_pages;
    int num_pages, page_size;
    long long page_stride, cache_row_stride, cache_head_stride;   // elements
};

cudaError_t launch_norm_rope(const NormRopeArgs& a, cudaStream_t stream);

namespace sm100 {

// 4-D tiled load (no multicast), as tma_load_3d.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1,
                                            int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

// 32 lanes x 16 consecutive 32-bit columns, to this thread's lane.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

}  // namespace sm100
}  // namespace gdn
