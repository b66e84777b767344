// paged.cuh -- what the paged K/V cache's translation units share (not part of the ABI).
#pragma once

#include "usp_internal.cuh"

namespace usp {

inline bool valid_page_size(int32_t ps) { return ps >= 16 && ps <= 256 && (ps & (ps - 1)) == 0; }

// requests of a call: loops step over them by up to 1024 in 32 bits
constexpr int32_t kMaxRequests = 1 << 30;

int check_cache_dims(const usp_cache_dims &d);

// usp_paged_attn's arguments, checked and with the defaults filled in (strides in elements)
struct PagedArgs {
    const void *q, *k, *v;
    const int32_t *table, *cu, *kv;
    void *out;
    float *lse;
    int64_t tokens, q_stride, out_stride, table_stride, num_pages, k_page, v_page;
    int32_t nreq, max_pages, max_new, hq, hkv, G, hd, log_ps, causal;
    float scale_log2;  // softmax scale * log2(e)
};

// Keys a request can have: what the table holds, and 32-bit key tile arithmetic with room for a tile.
inline int64_t paged_max_keys(const PagedArgs &a) {
    const int64_t held = (int64_t)a.max_pages << a.log_ps, most = (int64_t(1) << 31) - 1024;
    return held < most ? held : most;
}

// Every kernel of these calls may start while the grid before it in the stream still runs (programmatic
// dependent launch), so that its launch and set-up lie under that grid's end: four short decodes in a row
// take 11.5 us each instead of 14.3, one after a matrix product 11.7 instead of 12.3.
//   The first kernel of a call waits for the grid before (wait_grid_before, in every CTA) before it touches
//   global memory, and lets the next one start (let_next_start) only after that.
//   A second kernel of a call, independent of the first, so starts when the grid before the call has
//   completed; it runs beside the first as SMs come free, and ends after it (one CTA waits for that, the
//   others make room), so that what waits for the second one only follows both.
//   The combine waits for the kernel before it before it reads.
//   Inputs are read with plain loads. The read-only path is for data that nothing writes during the kernel's life,
// and here that begins while the grid that makes them may still be writing.
template <typename K, typename P>
inline int launch_overlapped(K kernel, dim3 grid, int threads, int smem, cudaStream_t s, const P &p) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? USP_OK : USP_ERR_CUDA;
}
__device__ __forceinline__ void wait_grid_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// the beginning and the end of a kernel that may be the first or the second of its call
__device__ __forceinline__ void begin_in_order(bool second) {
    if (!second) wait_grid_before();
    let_next_start();
}
__device__ __forceinline__ void end_in_order(bool second) {
    if (second && blockIdx.x == 0) wait_grid_before();
}

// The new tokens [t0, t0 + n) and keys of request i, clamped to what the tensors and the table hold.
struct Request {
    int64_t t0;
    int32_t n, kv;
};
__device__ __forceinline__ Request paged_request(const int32_t *cu, const int32_t *kv, int32_t i, int64_t tokens,
                                                 int64_t max_keys) {
    const int64_t a = min(max((int64_t)cu[i], (int64_t)0), tokens);
    const int64_t b = min(max((int64_t)cu[i + 1], a), tokens);
    return Request{a, (int32_t)(b - a), (int32_t)min(max((int64_t)kv[i], (int64_t)0), max_keys)};
}

}  // namespace usp
