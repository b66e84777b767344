// paged_q4.cu -- usp_paged_attn_q4: attention over a 4-bit paged cache: argument checks and dispatch.
#include <limits.h>
#include <math.h>

#include <algorithm>

#include "paged_q4.cuh"

namespace usp {
namespace {

int check_paged_q4_desc(const usp_paged_q4_desc &d) {
    int rc = check_q4_dims(d.cache);
    if (rc) return rc;
    const int es = elem_size(d.dtype);
    if (es == 0) return USP_ERR_DTYPE;
    if (d.tokens < 0 || d.q_stride < 0 || d.out_stride < 0 || d.nreq < 0 || d.max_pages < 0 || d.hq <= 0 || d.max_new < 0)
        return USP_ERR_INVALID_ARG;
    if (!(d.scale == d.scale) || isinf(d.scale)) return USP_ERR_INVALID_ARG;
    if (d.hq % d.cache.hkv != 0 || d.table_stride < d.max_pages) return USP_ERR_SHAPE;
    if (d.hq / d.cache.hkv > 128) return USP_ERR_UNSUPPORTED;
    const int64_t row = (int64_t)d.hq * d.cache.hd;
    for (int64_t st : {d.q_stride, d.out_stride}) {
        if (st != 0 && st < row) return USP_ERR_SHAPE;
        if (st >= (int64_t(1) << 38)) return USP_ERR_UNSUPPORTED;
        if (st * es % 16 != 0) return USP_ERR_ALIGN;
    }
    if (d.tokens >= (int64_t(1) << 31) / d.hq || d.nreq > kMaxRequests) return USP_ERR_UNSUPPORTED;
    return USP_OK;
}

PagedQ4Args paged_q4_args(const usp_paged_q4_desc &d) {
    PagedQ4Args a{};
    a.hq = d.hq; a.hkv = d.cache.hkv; a.G = d.hq / d.cache.hkv; a.hd = d.cache.hd;
    a.tokens = d.tokens;
    a.q_stride = d.q_stride ? d.q_stride : (int64_t)d.hq * a.hd;
    a.out_stride = d.out_stride ? d.out_stride : (int64_t)d.hq * a.hd;
    a.table_stride = d.table_stride;
    a.num_pages = d.cache.num_pages;
    const int64_t rows = (int64_t)a.hkv * d.cache.page_size;
    a.k_page = d.cache.k_page_stride ? d.cache.k_page_stride : rows * q4_code_bytes(a.hd);
    a.v_page = d.cache.v_page_stride ? d.cache.v_page_stride : rows * q4_code_bytes(a.hd);
    a.ks_page = d.cache.k_scale_stride ? d.cache.k_scale_stride : rows * q4_scale_bytes(a.hd);
    a.vs_page = d.cache.v_scale_stride ? d.cache.v_scale_stride : rows * q4_scale_bytes(a.hd);
    a.nreq = d.nreq; a.max_pages = d.max_pages;
    a.max_new = (int32_t)std::min<int64_t>(d.max_new, d.tokens);
    while ((1 << a.log_ps) < d.cache.page_size) ++a.log_ps;
    a.causal = d.causal ? 1 : 0;
    a.dtype = d.dtype;
    a.scale_log2 = (d.scale > 0.f ? d.scale : 1.0f / sqrtf((float)a.hd)) * 1.4426950408889634f;
    return a;
}

// The heads of a unit: the KV head's G, or where these are more than the kernel for few rows takes, the largest divisor of
// G that it does.
int few_heads(int G, int most) {
    int h = std::min(G, most);
    while (G % h != 0) --h;
    return h;
}

// Which kernels run: one for units of few query rows (a request's new tokens x G), one for units of many (bf16), or both,
// each with the CTAs (0: not launched) and unit rows of its partials.
struct Route {
    int few_ctas, few_rows, few_G, many_ctas;
    int split;   // the most new tokens of a request that the kernel for few rows takes
    bool alone;  // the kernel for many rows takes all requests (the other's workspace counts all the same)
};
Route route(const usp_paged_q4_desc &d, int sms) {
    Route r{};
    // bf16: the kernel for few rows against the one for many, 32 requests of 8000 keys, 20 to 24 and 32 rows 107 and 133 us against
    // 150; 100 requests of 1000 61 and 76 against 98; 36 rows would take two units
    const int G = d.hq / d.cache.hkv, most = d.dtype == USP_BF16 ? 32 : 16;
    const int64_t rows = G * (int64_t)std::max(1, d.max_new);
    r.few_G = few_heads(G, most);
    r.split = INT_MAX;
    if (d.dtype == USP_BF16 && (rows > most || G > most)) {
        r.many_ctas = sms;
        // beside chunks, the few-row requests are mostly single tokens: the kernel of 8 rows takes those where it can, else that of
        // as few tiles of rows as a token's heads need
        r.split = G > most ? 0 : G > 16 ? 1 : (G > 8 ? 16 : 8) / G;
    }
    if (r.split > 0) {
        // (a multiple of 8; a request of more rows than the host knows of has several units)
        r.few_rows = (int)std::min<int64_t>(most, (r.few_G * std::min<int64_t>(std::max(1, d.max_new), r.split) + 7) / 8 * 8);
        r.few_ctas = q4_few_ctas(sms, r.few_rows, d.dtype);
    }
    if (r.many_ctas && r.few_ctas) {
        // A second kernel costs its launch, but a key of a short request costs the kernel for many rows half as much again
        // and more (26 single tokens beside 7 chunks, hd 64: 27.4 us, all in one kernel 30.7; 14 of 4000 to 32000 keys
        // 164, 226). Only where the tokens' number tells that no request is short does that kernel run alone.
        const int64_t M = std::min<int64_t>(d.max_new, d.tokens);
        r.alone = M > r.split && (d.nreq * M - std::min(d.tokens, d.nreq * M)) / (M - r.split) == 0;
    }
    return r;
}

size_t workspace_bytes_of(const Route &r, int hd) {
    return (r.few_ctas ? part_bytes(r.few_ctas, r.few_rows, hd) : 0) + (r.many_ctas ? part_bytes(r.many_ctas, kChunkRows, hd) + q4_join_bytes(r.many_ctas, hd) : 0);
}

// What the caller provides: what every call with this max_new or a smaller one uses. The layouts of few rows alone are
// larger than those of more rows (in headers) or beside chunks.
size_t workspace_bytes_for(const usp_paged_q4_desc &d, int sms) {
    const Route r = route(d, sms);
    size_t most = workspace_bytes_of(r, d.cache.hd);
    if (r.few_ctas)
        for (int rows = 8; rows <= (d.dtype == USP_BF16 ? 32 : 16); rows += 8)
            most = std::max(most, part_bytes(q4_few_ctas(sms, rows, d.dtype), rows, d.cache.hd));
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

size_t usp_paged_attn_q4_workspace_size(usp_paged_q4_desc d) {
    const DeviceInfo *di = nullptr;
    if (check_paged_q4_desc(d) || !(di = device_info())) return 0;
    return workspace_bytes_for(d, di->sm_count);
}

int usp_paged_attn_q4(const void *q, const void *k_cache, const void *v_cache, const uint8_t *k_scales,
                      const uint8_t *v_scales, const int32_t *block_table, const int32_t *cu_new, const int32_t *kv_lens,
                      void *out, float *lse, usp_paged_q4_desc d, void *workspace, size_t workspace_bytes,
                      usp_stream_t stream) {
    int rc = check_paged_q4_desc(d);
    if (rc) return rc;
    if (d.tokens == 0 || d.nreq == 0) return USP_OK;
    if (!q || !k_cache || !v_cache || !k_scales || !v_scales || !cu_new || !kv_lens || !out || !lse || !workspace)
        return USP_ERR_INVALID_ARG;
    if (d.max_pages > 0 && !block_table) return USP_ERR_INVALID_ARG;  // without columns no request has a key
    if (d.cache.num_pages == 0) return USP_ERR_SHAPE;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_scales, 16) ||
        !aligned(v_scales, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(block_table, 4) ||
        !aligned(cu_new, 4) || !aligned(kv_lens, 4) || !aligned(workspace, 256))
        return USP_ERR_ALIGN;
    const DeviceInfo *di = device_info();
    if (!di) return USP_ERR_CUDA;
    const Route r = route(d, di->sm_count);
    if (workspace_bytes < workspace_bytes_of(r, d.cache.hd)) return USP_ERR_INVALID_ARG;
    PagedQ4Args a = paged_q4_args(d);
    a.q = q;
    a.k = static_cast<const uint8_t *>(k_cache); a.v = static_cast<const uint8_t *>(v_cache);
    a.ks = k_scales; a.vs = v_scales;
    a.table = block_table; a.cu = cu_new; a.kv = kv_lens;
    a.out = out; a.lse = lse;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    char *at = static_cast<char *>(workspace);
    CombineArgs c{};
    c.out = out; c.lse = lse; c.out_stride = a.out_stride;
    // (a unit's heads: the KV head's, or fewer in the kernel for few rows, which then runs alone)
    const int G = r.many_ctas ? a.G : r.few_G;
    c.G = G; c.hq = a.hq; c.by_G = FastDiv((uint32_t)G);
    if (r.many_ctas) {
        c.w[0] = part_space(at, r.many_ctas, kChunkRows, a.hd);
        float *join = reinterpret_cast<float *>(at);
        at += q4_join_bytes(r.many_ctas, a.hd);
        rc = launch_paged_q4_chunk(a, r.alone ? 0 : r.split, c.w[0], join, s);
        if (rc) return rc;
    }
    if (r.few_ctas && !r.alone) {
        c.w[1] = part_space(at, r.few_ctas, r.few_rows, a.hd);
        rc = launch_paged_q4_few(a, r.few_G, r.few_rows, r.split, r.many_ctas > 0, c.w[1], s);
        if (rc) return rc;
    }
    return launch_paged_combine(c, a.hd, a.dtype, s);
}

}  // extern "C"
