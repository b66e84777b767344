// paged_attn.cu -- usp_paged_attn: argument checks and dispatch.
#include <limits.h>
#include <math.h>

#include <algorithm>

#include "paged_sched.cuh"

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
        if (st >= (int64_t(1) << 38)) return USP_ERR_UNSUPPORTED;
        if (st * elem_size(d.cache.dtype) % 16 != 0) return USP_ERR_ALIGN;
    }
    if (d.tokens >= (int64_t(1) << 31) / d.hq || d.nreq > kMaxRequests) return USP_ERR_UNSUPPORTED;
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

// Which kernels run: one for units of few query rows (a request's new tokens x G), one for units of many,
// or both, each with the CTAs (0: not launched) and unit rows of its partials.
struct Route {
    int few_ctas, few_rows, many_ctas, many_rows;
    int split;   // the most new tokens of a request that the kernel for few rows takes
    bool alone;  // the kernel for many rows takes all requests (the other's workspace counts all the same)
};

// bf16: up to 32 rows of a KV head a call is bound by reading the cache, and the kernel for few rows reads it
// at the HBM rate; above, its re-reading of K/V per unit costs more than the other one's idle rows. fp32: the
// kernel for few rows computes 17 (hd 64) to 25 TFLOP/s at any number of rows, the other one 52 at 128 rows and
// a row's share of that below (40000 keys, 4 requests: 48 rows of 128 1204 against 1600 us, 64 1577 against 1601;
// 40 rows of 64 741 against 811, 48 883 against 812).
Route route(const usp_paged_desc &d, int sms) {
    Route r{};
    const bool bf16 = d.cache.dtype == USP_BF16;
    const int G = d.hq / d.cache.hkv, most = bf16 ? 32 : d.cache.hd == 128 ? 64 : 40;
    const int64_t rows = G * (int64_t)std::max(1, d.max_new);
    r.split = INT_MAX;
    if (rows > most || G > (bf16 ? 32 : f32_rows(false))) {
        r.many_ctas = bf16 ? sms : f32_ctas(sms, true);
        r.many_rows = bf16 ? kChunkRows : f32_rows(true);
        // beside chunks, the few-row requests are mostly single tokens: the 16-row kernel (two CTAs per SM)
        // takes those, the other one all chunks (33 requests, 26 of one token: a fifth less time)
        r.split = G > (bf16 ? 32 : f32_rows(false)) ? 0 : (bf16 && G <= 16 ? 16 : most) / G;
    }
    if (r.split > 0) {
        r.few_rows = bf16 ? (std::min<int64_t>(rows, (int64_t)r.split * G) <= 16 ? 16 : 32) : f32_rows(false);
        r.few_ctas = bf16 ? decode_ctas(sms, r.few_rows) : f32_ctas(sms, false);
    }
    if (r.many_ctas && r.few_ctas) {
        // A second kernel costs its launch (3 to 5 us), also with nothing to do. The requests for it are at most `few`, as
        // many as may be short when the rows add up to `tokens`. None, or with hd 128, where a key costs an SM the
        // same in both bf16 kernels, three units per SM: the kernel for many rows takes them too (one prompt of
        // 500 tokens 24.6 -> 21.5 us; 2 chunks and 30 single tokens over 500 to 4096 keys 63.8 -> 59.5, 46 single tokens
        // 84.5 -> 79.5; 6 prompts 316 -> 313; with 6 units per SM slower, 70 -> 80). With hd 64 reading is twice as fast in
        // the kernel for few rows (2 chunks and 14 single tokens over 4000 to 32000 keys 101 -> 120 us), in fp32 several
        // times.
        const int64_t M = std::min<int64_t>(d.max_new, d.tokens), all = d.nreq * M;
        const int64_t few = M > r.split ? (all - std::min(d.tokens, all)) / (M - r.split) : d.nreq;
        r.alone = few * d.cache.hkv <= (bf16 && d.cache.hd == 128 ? 3 * sms : 0);
    }
    return r;
}

size_t workspace_bytes_of(const Route &r, int hd) {
    return (r.few_ctas ? part_bytes(r.few_ctas, r.few_rows, hd) : 0) +
           (r.many_ctas ? part_bytes(r.many_ctas, r.many_rows, hd) : 0);
}

// What the caller provides: what every call with this max_new or a smaller one uses. The one layout that is smaller
// than that of fewer tokens is the bf16 kernel's for up to 32 rows on its own (half the headers of the 16-row one).
size_t workspace_bytes_for(const usp_paged_desc &d, int sms) {
    const Route r = route(d, sms);
    size_t most = workspace_bytes_of(r, d.cache.hd);
    if (r.few_rows == 32 && d.hq / d.cache.hkv <= 16)
        most = std::max(most, part_bytes(decode_ctas(sms, 16), 16, d.cache.hd));
    return most;
}

PartSpace part_space(char *&at, int ctas, int rows, int hd) {
    PartSpace w{};
    w.ctas = ctas;
    w.rows = rows;
    w.head = reinterpret_cast<PartHeader *>(at);
    w.data = reinterpret_cast<float *>(at + (size_t)ctas * sizeof(PartHeader));
    at += part_bytes(ctas, rows, hd);
    return w;
}

}  // namespace
}  // namespace usp

using namespace usp;

extern "C" {

size_t usp_paged_attn_workspace_size(usp_paged_desc d) {
    const DeviceInfo *di = nullptr;
    if (check_paged_desc(d) || !(di = device_info())) return 0;
    return workspace_bytes_for(d, di->sm_count);
}

int usp_paged_attn(const void *q, const void *k_cache, const void *v_cache, const int32_t *block_table,
                   const int32_t *cu_new, const int32_t *kv_lens, void *out, float *lse, usp_paged_desc d,
                   void *workspace, size_t workspace_bytes, usp_stream_t stream) {
    int rc = check_paged_desc(d);
    if (rc) return rc;
    if (d.tokens == 0 || d.nreq == 0) return USP_OK;
    if (!q || !k_cache || !v_cache || !cu_new || !kv_lens || !out || !lse || !workspace) return USP_ERR_INVALID_ARG;
    if (d.max_pages > 0 && !block_table) return USP_ERR_INVALID_ARG;  // without columns no request has a key
    if (d.cache.num_pages == 0) return USP_ERR_SHAPE;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) || !aligned(lse, 4) ||
        !aligned(block_table, 4) || !aligned(cu_new, 4) || !aligned(kv_lens, 4) || !aligned(workspace, 256))
        return USP_ERR_ALIGN;
    const DeviceInfo *di = device_info();
    if (!di) return USP_ERR_CUDA;
    const Route r = route(d, di->sm_count);
    if (workspace_bytes < workspace_bytes_of(r, d.cache.hd)) return USP_ERR_INVALID_ARG;
    PagedArgs a = paged_args(d);
    a.q = q; a.k = k_cache; a.v = v_cache;
    a.table = block_table; a.cu = cu_new; a.kv = kv_lens;
    a.out = out; a.lse = lse;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool bf16 = d.cache.dtype == USP_BF16;
    char *at = static_cast<char *>(workspace);
    CombineArgs c{};
    c.out = out; c.lse = lse; c.out_stride = a.out_stride;
    c.G = a.G; c.hq = a.hq; c.by_G = FastDiv((uint32_t)a.G);
    if (r.many_ctas) {
        c.w[0] = part_space(at, r.many_ctas, r.many_rows, a.hd);
        const int lo = r.alone ? 0 : r.split;
        rc = bf16 ? launch_paged_chunk(a, lo, c.w[0], s) : launch_paged_f32(a, true, lo, INT_MAX, false, c.w[0], s);
        if (rc) return rc;
    }
    if (r.few_ctas && !r.alone) {
        c.w[1] = part_space(at, r.few_ctas, r.few_rows, a.hd);
        rc = bf16 ? launch_paged_decode(a, r.few_rows, r.split, r.many_ctas > 0, c.w[1], s)
                  : launch_paged_f32(a, false, 0, r.split, r.many_ctas > 0, c.w[1], s);
        if (rc) return rc;
    }
    return launch_paged_combine(c, a.hd, d.cache.dtype, s);
}

}  // extern "C"
