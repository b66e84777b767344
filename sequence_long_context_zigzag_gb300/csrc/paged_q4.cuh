// paged_q4.cuh -- what the translation units of the attention over a 4-bit paged cache share (not part of the ABI).
#pragma once

#include "paged_sched.cuh"
#include "q4.cuh"
#include "tc_common.cuh"

namespace usp {

// usp_paged_attn_q4's arguments, checked and with the defaults filled in (q's and out's strides in elements, the pages' in
// bytes)
struct PagedQ4Args {
    const void *q;
    const uint8_t *k, *v, *ks, *vs;
    const int32_t *table, *cu, *kv;
    void *out;
    float *lse;
    int64_t tokens, q_stride, out_stride, table_stride, num_pages, k_page, v_page, ks_page, vs_page;
    int32_t nreq, max_pages, max_new, hq, hkv, G, hd, log_ps, causal, dtype;
    float scale_log2;  // softmax scale * log2(e)
};

// Keys a request can have (as paged_max_keys)
inline int64_t q4_max_keys(const PagedQ4Args &a) {
    const int64_t held = (int64_t)a.max_pages << a.log_ps, most = (int64_t(1) << 31) - 1024;
    return held < most ? held : most;
}

// A cache's codes as bytes (hd / 2, hkv * page_size, num_pages), in boxes of whole rows, `rows` of one page; rows of 64
// bytes in the 64-byte swizzle (16-byte piece c of row r at c ^ ((r >> 1) & 3)), rows of 32 as they are. A page outside the
// cache is out of bounds in the last dimension: the box reads zeros, codes that stand for 0.
inline bool make_codes_tmap(CUtensorMap *m, const void *base, int64_t pages, int64_t page_stride, int32_t hkv, int32_t ps,
                            int32_t hd, uint32_t rows) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)q4_code_bytes(hd), (cuuint64_t)hkv * ps, (cuuint64_t)pages};
    const cuuint64_t strides[2] = {(cuuint64_t)q4_code_bytes(hd), (cuuint64_t)page_stride};
    const cuuint32_t box[3] = {(cuuint32_t)q4_code_bytes(hd), rows, 1}, estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, hd == 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_NONE,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// `bytes` (a multiple of 16) from global to shared memory, both 16-byte aligned, completion counted on an mbarrier
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
                 : "memory");
}

// Units of up to `rows` (8 or 16) query rows, G query heads each (a divisor of the group's); requests with at most n_hi new
// tokens. `second`: the call's other kernel is in the stream before it.
int launch_paged_q4_few(const PagedQ4Args &a, int G, int rows, int n_hi, bool second, const PartSpace &w, cudaStream_t s);
int q4_few_ctas(int sms, int rows, int dtype);

}  // namespace usp
