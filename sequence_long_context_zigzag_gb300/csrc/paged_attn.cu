// paged_attn.cu -- usp_paged_attn: argument checks and dispatch.
#include <math.h>

#include "paged.cuh"

namespace usp {
namespace {

int check_paged_desc(const usp_paged_desc &d) {
    int rc = check_cache_dims(d.cache);
    if (rc) return rc;
    if (d.tokens < 0 || d.q_stride < 0 || d.out_stride < 0 || d.nreq < 0 || d.max_pages < 0 || d.hq <= 0 ||
        d.max_new < 0)
        return USP_ERR_INVALID_ARG;
    if (!(d.scale == d.scale) || isinf(d.scale)) return USP_ERR_INVALID_ARG;
    if (d.hq % d.cache.hkv != 0 || d.table_stride < d.max_pages) return USP_ERR_SHAPE;
    if (d.hq / d.cache.hkv > 128) return USP_ERR_UNSUPPORTED;
    const int64_t row = (int64_t)d.hq * d.cache.hd;
    for (int64_t st : {d.q_stride, d.out_stride}) {
        if (st != 0 && st < row) return USP_ERR_SHAPE;
        if (st * elem_size(d.cache.dtype) % 16 != 0) return USP_ERR_ALIGN;
        if (st >= (int64_t(1) << 38)) return USP_ERR_UNSUPPORTED;
    }
    if (d.tokens >= (int64_t(1) << 31) / d.hq) return USP_ERR_UNSUPPORTED;
    return USP_OK;
}

PagedArgs paged_args(const usp_paged_desc &d) {
    PagedArgs a{};
    a.hq = d.hq; a.hkv = d.cache.hkv; a.G = d.hq / d.cache.hkv; a.hd = d.cache.hd;
    a.tokens = d.tokens;
    a.q_stride = d.q_stride ? d.q_stride : (int64_t)d.hq * a.hd;
    a.out_stride = d.out_stride ? d.out_stride : (int64_t)d.hq * a.hd;
    a.table_stride = d.table_stride;
    a.num_pages = d.cache.num_pages;
    const int64_t dense = (int64_t)a.hkv * d.cache.page_size * a.hd;
    a.k_page = d.cache.k_page_stride ? d.cache.k_page_stride : dense;
    a.v_page = d.cache.v_page_stride ? d.cache.v_page_stride : dense;
    a.nreq = d.nreq; a.max_pages = d.max_pages;
    a.max_new = (int32_t)(d.max_new < d.tokens ? d.max_new : d.tokens);
    a.log_ps = 0;
    while ((1 << a.log_ps) < d.cache.page_size) ++a.log_ps;
    a.causal = d.causal ? 1 : 0;
    a.scale_log2 = (d.scale > 0.f ? d.scale : 1.0f / sqrtf((float)a.hd)) * 1.4426950408889634f;
    return a;
}

}  // namespace
}  // namespace usp

using namespace usp;

extern "C" {

size_t usp_paged_attn_workspace_size(usp_paged_desc d) {
    if (check_paged_desc(d)) return 0;
    return 256;
}

int usp_paged_attn(const void *q, const void *k_cache, const void *v_cache, const int32_t *block_table,
                   const int32_t *cu_new, const int32_t *kv_lens, void *out, float *lse, usp_paged_desc d,
                   void *workspace, size_t workspace_bytes, usp_stream_t stream) {
    int rc = check_paged_desc(d);
    if (rc) return rc;
    if (d.tokens == 0 || d.nreq == 0) return USP_OK;
    if (!q || !cu_new || !kv_lens || !out || !lse || !workspace) return USP_ERR_INVALID_ARG;
    // a cache without pages and a table without columns may be null: no request has a key then
    if ((d.cache.num_pages > 0 && (!k_cache || !v_cache)) || (d.max_pages > 0 && !block_table))
        return USP_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) || !aligned(lse, 4) ||
        !aligned(block_table, 4) || !aligned(cu_new, 4) || !aligned(kv_lens, 4) || !aligned(workspace, 256))
        return USP_ERR_ALIGN;
    if (workspace_bytes < usp_paged_attn_workspace_size(d)) return USP_ERR_INVALID_ARG;
    PagedArgs a = paged_args(d);
    a.q = q; a.k = k_cache; a.v = v_cache;
    a.table = block_table; a.cu = cu_new; a.kv = kv_lens;
    a.out = out; a.lse = lse;
    return launch_paged_simt(a, d.cache.dtype, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
