// paged_tma.cuh -- tensor maps of the paged cache and of q for the tensor-core kernels (not part of the ABI).
#pragma once

#include "paged.cuh"
#include "tc_common.cuh"

namespace usp {

// One cache as (hd, hkv * page_size, num_pages), bf16, in boxes of 64 columns x `rows` rows of one page,
// 128-byte swizzle. A page outside the cache is out of bounds in the last dimension: the box reads zeros.
inline bool make_cache_tmap(CUtensorMap *m, const void *base, int64_t pages, int64_t page_stride, int32_t hkv,
                            int32_t ps, int32_t hd, uint32_t rows) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)hd, (cuuint64_t)hkv * ps, (cuuint64_t)pages};
    const cuuint64_t strides[2] = {(cuuint64_t)hd * 2, (cuuint64_t)page_stride * 2};
    const cuuint32_t box[3] = {64, rows, 1}, estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 3-D tiled load global -> shared, completion counted on an mbarrier
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void *tmap, int32_t c0, int32_t c1, int32_t c2,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}

// 3-D tiled store shared -> global (the calling thread's bulk group), and waits for it: until the shared memory is
// read, until all is written
__device__ __forceinline__ void tma_store_3d(const void *tmap, int32_t c0, int32_t c1, int32_t c2, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];\n\t"
                 "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(tmap)),
                 "r"(c0), "r"(c1), "r"(c2), "r"(src)
                 : "memory");
}
__device__ __forceinline__ void tma_stores_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void tma_stores_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// the same box into L2 only
__device__ __forceinline__ void tma_prefetch_3d(const void *tmap, int32_t c0, int32_t c1, int32_t c2) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                     reinterpret_cast<uint64_t>(tmap)),
                 "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}

}  // namespace usp
