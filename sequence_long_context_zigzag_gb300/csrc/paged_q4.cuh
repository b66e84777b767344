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

// A cache's codes as lines of 128 bytes, 2 keys of hd 128 or 4 of hd 64 each: (128, lines of a page, num_pages), in boxes
// of `rows` keys of one page, 128-byte swizzle: 16-byte piece c of line l lies at c ^ (l % 8). (As rows of a key, 64 bytes,
// the copies of a page of 16 tokens ran at a bit over half the rate.) A page outside the cache is out of bounds in the last
// dimension: the box reads zeros, codes that stand for 0.
inline bool make_codes_tmap(CUtensorMap *m, const void *base, int64_t pages, int64_t page_stride, int32_t hkv, int32_t ps,
                            int32_t hd, uint32_t rows) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const uint32_t keys = 128 / q4_code_bytes(hd);  // of a line
    const cuuint64_t dims[3] = {128, (cuuint64_t)hkv * ps / keys, (cuuint64_t)pages};
    const cuuint64_t strides[2] = {128, (cuuint64_t)page_stride};
    const cuuint32_t box[3] = {128, rows / keys, 1}, estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// where byte b of a key's codes lies in a tile (1024-byte aligned) that the boxes filled
template <int HD> __device__ __forceinline__ uint32_t codes_at(uint32_t key, uint32_t b) {
    const uint32_t x = key * q4_code_bytes(HD) + b;
    return x ^ ((x >> 3) & 0x70u);
}

// 16 bytes from global to shared memory, asynchronously (the 256 bytes around them come to L2 for the CTAs of the other KV
// heads: a page's scales are hd / 32 bytes a token and head); and an arrival on an mbarrier when this thread's copies so far
// have landed
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// ---- codes to operands: (136 + c) s - 136 s in bf16, exact (see paged_q4_few.cu) ----
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
// two scale bytes as bf16 numbers: (b << 4) + the exponent field's 107 (see q4_scale)
__device__ __forceinline__ uint32_t q4_scales2(uint32_t lo, uint32_t hi) { return lo * 0x10u + (hi * 0x100000u + 0x35803580u); }
__device__ __forceinline__ uint32_t q4_scales2(uint32_t b) { return b * 0x100010u + 0x35803580u; }
__device__ __forceinline__ uint32_t q4_minus136(uint32_t s2) {
    return fma_bf16x2(s2, 0xc308c308u, 0x80008000u);  // -136 s - 0
}
// The codes j of a word (the low nibbles of the halves of word >> 4 j) as values. One of the conversion's two constants is
// held in a register: an instruction has room for one of its own, and with both known the compiler takes two
// instructions (143 instead of 72 logic operations per 16 keys).
struct Q4Nibbles {
    uint32_t magic;
    __device__ __forceinline__ Q4Nibbles() { asm volatile("mov.b32 %0, 0x43084308;" : "=r"(magic)); }
    __device__ __forceinline__ uint32_t values(uint32_t word, int j, uint32_t s2, uint32_t off) const {
        uint32_t x;
        asm("lop3.b32 %0, %1, 0x000f000f, %2, 0x6a;" : "=r"(x) : "r"(word >> (4 * j)), "r"(magic));  // (a & b) ^ c
        return fma_bf16x2(x, s2, off);
    }
};

// Units of up to `rows` (a multiple of 8, at most 32; fp32: 16) query rows, G query heads each (a divisor of the group's); requests with at most n_hi new
// tokens. `second`: the call's other kernel is in the stream before it.
int launch_paged_q4_few(const PagedQ4Args &a, int G, int rows, int n_hi, bool second, const PartSpace &w, cudaStream_t s);
int q4_few_ctas(int sms, int rows, int dtype);

// bf16, units of up to kChunkRows query rows, one CTA per SM; requests with more than n_lo new tokens (paged_chunk.cu). join:
// a scratch of q4_join_bytes.
int launch_paged_q4_chunk(const PagedQ4Args &a, int n_lo, const PartSpace &w, float *join, cudaStream_t s);
size_t q4_join_bytes(int ctas, int hd);

}  // namespace usp
