// spv_tma.cuh -- tensor maps over a page pool: a page's rows of one head are
// copied into an operand tile by the copy engine, permuted on the way as the
// tensor cores read them.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "spv_internal.h"
#include "spv_stream.cuh"

namespace spv {

// The driver's call that describes a tensor; null where it has none.
using EncodeMap = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                               const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                               CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline EncodeMap encode_map()
{
    static const EncodeMap encode = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeMap>(f);
    }();
    return encode;
}

// The map of a 16-bit pool: element, slot, head, page; a box is 64 elements
// (the width of an operand's panel) of min(page_size, `slots`) slots, or, with
// `rows` (e4m3 pools too), the whole rows of so many, as they lie.  False where
// the pool cannot be described so (pages under 8 slots, a driver without the
// call): the kernels then copy row by row.
inline bool pool_map(CUtensorMap *map, const KvLaunch &L, bool v, int slots = 128, bool rows = false)
{
    const spv_kv_cache &c = L.cache;
    const bool eight = c.dtype == SPV_E4M3;
    if ((eight && !rows) || c.page_size < 8 || c.head_dim % 64 != 0) return false;
    const EncodeMap encode = encode_map();
    if (!encode) return false;
    const cuuint64_t sizes[4] = {static_cast<cuuint64_t>(c.head_dim), static_cast<cuuint64_t>(c.page_size),
                                 static_cast<cuuint64_t>(c.kv_heads), static_cast<cuuint64_t>(c.num_pages)};
    const int64_t strides[3] = {v ? c.v_slot_stride : c.k_slot_stride, v ? c.v_head_stride : c.k_head_stride,
                                v ? c.v_page_stride : c.k_page_stride};
    cuuint64_t bytes[3];
    for (int i = 0; i < 3; ++i) {
        // a dimension of one entry is never stepped over, but its stride has to be one
        if (strides[i] <= 0 && sizes[i + 1] > 1) return false;
        bytes[i] = static_cast<cuuint64_t>(strides[i] > 0 ? strides[i] : c.head_dim) * (eight ? 1 : 2);
        if (bytes[i] >= (1ull << 40)) return false;
    }
    const cuuint32_t box[4] = {static_cast<cuuint32_t>(rows ? c.head_dim : 64), static_cast<cuuint32_t>(c.page_size < slots ? c.page_size : slots), 1, 1};
    const cuuint32_t steps[4] = {1, 1, 1, 1};
    return encode(map, eight ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : c.dtype == SPV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                  v ? c.v : c.k, sizes, bytes, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, rows ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The map of q [B, T, q_heads, D]: element, head, token, sequence; a box is 64
// elements of the `group` query heads of a key head and of the tokens that make
// `rows` rows with them.  False where a key head's rows do not come out even.
inline bool query_map(CUtensorMap *map, const void *q, const KvLaunch &L, int group, int rows)
{
    const EncodeMap encode = encode_map();
    const int D = L.cache.head_dim;
    if (!encode || rows % group != 0 || D % 64 != 0) return false;
    const cuuint64_t sizes[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(L.q_heads), static_cast<cuuint64_t>(L.T),
                                 static_cast<cuuint64_t>(L.B)};
    const cuuint64_t bytes[3] = {sizes[0] * 2, sizes[0] * sizes[1] * 2, sizes[0] * sizes[1] * sizes[2] * 2};
    if (bytes[2] >= (1ull << 40)) return false;
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(group), static_cast<cuuint32_t>(rows / group), 1};
    const cuuint32_t steps[4] = {1, 1, 1, 1};
    return encode(map, L.dtype == SPV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void *>(q),
                  sizes, bytes, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Copies the box at (d, slot, head, page) -- d a multiple of 64 -- to shared
// memory; its bytes count on `bar`.  What lies outside the pool becomes zero.
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap *map, int d, int slot, int head, int page, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(d), "r"(slot), "r"(head), "r"(page), "r"(smem_u32(bar))
        : "memory");
}

}  // namespace spv
