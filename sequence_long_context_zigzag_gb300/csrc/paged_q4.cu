// paged_q4.cu -- usp_paged_attn_q4: attention over a 4-bit paged cache. Argument checks, and a first kernel.
#include <limits.h>
#include <math.h>

#include <algorithm>

#include "paged.cuh"
#include "q4.cuh"
#include "tc_ptx.cuh"
#include "usp_device.cuh"

namespace usp {
namespace {

constexpr float kLn2 = 0.69314718055994531f;

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

// A warp per query row: 32 keys at a time, a key per lane for the scores, hd / 32 columns per lane for the products.
template <typename T, int HD> __global__ void __launch_bounds__(128) paged_q4_rows_kernel(const PagedQ4Args p) {
    constexpr int kPer = HD / 32;
    __shared__ float q_s[4][HD];
    wait_grid_before();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 4 + warp;
    if (row >= p.tokens * p.hq) return;
    const int64_t t = row / p.hq;
    const int h = (int)(row % p.hq), head = h / p.G;
    int lo = 0, hi = p.nreq;  // the last request with cu <= t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    const Request r = paged_request(p.cu, p.kv, lo, p.tokens, min((int64_t)p.max_pages << p.log_ps, (int64_t)INT_MAX - 1024));
    if (t < r.t0 || t >= r.t0 + r.n) return;
    const int64_t pos = (int64_t)r.kv - r.n + (t - r.t0);
    const int keys = p.causal ? (int)max((int64_t)0, min((int64_t)r.kv, pos + 1)) : r.kv;
    const T *q = static_cast<const T *>(p.q) + t * p.q_stride + (int64_t)h * HD;
    for (int e = lane; e < HD; e += 32) q_s[warp][e] = (float)q[e];
    __syncwarp();
    float m = -INFINITY, l = 0.f, o[kPer] = {};
    const int32_t *pages = p.table + lo * p.table_stride;
    for (int base = 0; base < keys; base += 32) {
        const int key = base + lane;
        int32_t page = -1;
        int64_t in = 0;
        float s = -INFINITY;
        if (key < keys) {
            page = pages[key >> p.log_ps];
            if (page >= p.num_pages) page = -1;
            in = ((int64_t)head << p.log_ps) + (key & ((1 << p.log_ps) - 1));
            s = 0.f;
            if (page >= 0) {
                const uint32_t *w = reinterpret_cast<const uint32_t *>(p.k + page * p.k_page + in * q4_code_bytes(HD));
                const uint8_t *sc = p.ks + page * p.ks_page + in * q4_scale_bytes(HD);
                for (int x = 0; x < HD / 8; ++x) {
                    const float f = q4_scale(sc[x / 4]);
                    for (int e = 0; e < 8; ++e) {
                        const int n = e / 2 + 4 * (e % 2), c = (int)(w[x] << (28 - 4 * n)) >> 28;
                        s = fmaf(q_s[warp][x * 8 + e], (float)c * f, s);
                    }
                }
            }
            s *= p.scale_log2;
        }
        float mx = s;
        for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        const float mn = fmaxf(m, mx), mb = mn == -INFINITY ? 0.f : mn, a = exp2f(m - mb);
        const float w = exp2f(s - mb);
        l = l * a + w;
        m = mn;
        for (int e = 0; e < kPer; ++e) o[e] *= a;
        for (int j = 0; j < min(32, keys - base); ++j) {
            const float pj = __shfl_sync(0xffffffffu, w, j);
            const int32_t pg = __shfl_sync(0xffffffffu, page, j);
            const int64_t ij = __shfl_sync(0xffffffffu, in, j);
            if (pg < 0) continue;
            const uint8_t *b = p.v + pg * p.v_page + ij * q4_code_bytes(HD);
            const uint8_t *sc = p.vs + pg * p.vs_page + ij * q4_scale_bytes(HD);
            for (int e = 0; e < kPer; ++e) {
                const int d = lane + 32 * e, n = (d & 7) / 2 + 4 * (d & 1);
                const uint32_t w32 = *reinterpret_cast<const uint32_t *>(b + d / 8 * 4);
                const int c = (int)(w32 << (28 - 4 * n)) >> 28;
                o[e] = fmaf(pj, (float)c * q4_scale(sc[e]), o[e]);
            }
        }
    }
    for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    T *out = static_cast<T *>(p.out) + t * p.out_stride + (int64_t)h * HD;
    for (int e = 0; e < kPer; ++e) out[lane + 32 * e] = (T)(l == 0.f ? 0.f : o[e] / l);
    if (lane == 0) p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

}  // namespace
}  // namespace usp

using namespace usp;

extern "C" {

size_t usp_paged_attn_q4_workspace_size(usp_paged_q4_desc d) { return check_paged_q4_desc(d) ? 0 : 256; }

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
    if (workspace_bytes < 256) return USP_ERR_INVALID_ARG;
    PagedQ4Args a = paged_q4_args(d);
    a.q = q;
    a.k = static_cast<const uint8_t *>(k_cache); a.v = static_cast<const uint8_t *>(v_cache);
    a.ks = k_scales; a.vs = v_scales;
    a.table = block_table; a.cu = cu_new; a.kv = kv_lens;
    a.out = out; a.lse = lse;
    const dim3 grid((unsigned)((a.tokens * a.hq + 3) / 4));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    auto go = [&](auto kernel) { return launch_overlapped(kernel, grid, 128, 0, s, a); };
    if (a.dtype == USP_BF16)
        return a.hd == 128 ? go(paged_q4_rows_kernel<__nv_bfloat16, 128>) : go(paged_q4_rows_kernel<__nv_bfloat16, 64>);
    return a.hd == 128 ? go(paged_q4_rows_kernel<float, 128>) : go(paged_q4_rows_kernel<float, 64>);
}

}  // extern "C"
