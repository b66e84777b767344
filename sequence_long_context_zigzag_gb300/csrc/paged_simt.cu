// paged_simt.cu -- attention over the paged cache on the CUDA cores: one warp per query row, key by key.
#include "paged.cuh"
#include "usp_device.cuh"

namespace usp {
namespace {

template <typename T, int EPL> __device__ __forceinline__ void load_row(const T *p, float (&x)[EPL]) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) x[i] = (float)p[i];
}

template <typename T, int HD>
__global__ void __launch_bounds__(256) paged_simt_kernel(const PagedArgs p) {
    constexpr int EPL = HD / 32;
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int64_t tok = row / p.hq;
    const int head = (int)(row % p.hq), kh = head / p.G;
    if (tok >= p.tokens) return;
    // the request: the last one that begins at or before the token (empty ones come before)
    int lo = 0, hi = p.nreq;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(p.cu + mid) <= tok) lo = mid;
        else hi = mid;
    }
    const Request r = paged_request(p.cu, p.kv, lo, p.tokens, (int64_t)p.max_pages << p.log_ps);
    if (tok < r.t0 || tok >= r.t0 + r.n) return;
    const int64_t limit = p.causal ? max((int64_t)0, min((int64_t)r.kv, r.kv - r.n + (tok - r.t0) + 1)) : r.kv;
    float q[EPL], acc[EPL];
    load_row<T, EPL>(static_cast<const T *>(p.q) + tok * p.q_stride + head * HD + lane * EPL, q);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        q[i] *= p.scale_log2;
        acc[i] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    const int ps = 1 << p.log_ps;
    for (int64_t j = 0; j < limit; ++j) {
        const int32_t page = __ldg(p.table + lo * p.table_stride + (j >> p.log_ps));
        float k[EPL] = {}, v[EPL] = {};
        if (page >= 0 && page < p.num_pages) {
            const int64_t in = ((int64_t)kh * ps + (j & (ps - 1))) * HD + lane * EPL;
            load_row<T, EPL>(static_cast<const T *>(p.k) + page * p.k_page + in, k);
            load_row<T, EPL>(static_cast<const T *>(p.v) + page * p.v_page + in, v);
        }
        float sc = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) sc = fmaf(q[i], k[i], sc);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sc += __shfl_xor_sync(0xffffffffu, sc, o);
        const float mn = fmaxf(m, sc), a = exp2f(m - mn), e = exp2f(sc - mn);
        m = mn;
        l = l * a + e;
#pragma unroll
        for (int i = 0; i < EPL; ++i) acc[i] = fmaf(acc[i], a, e * v[i]);
    }
    T *o = static_cast<T *>(p.out) + tok * p.out_stride + head * HD + lane * EPL;
#pragma unroll
    for (int i = 0; i < EPL; ++i) o[i] = (T)(l > 0.f ? acc[i] / l : 0.f);
    if (lane == 0) p.lse[row] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace

int launch_paged_simt(const PagedArgs &a, int dtype, cudaStream_t s) {
    const unsigned grid = (unsigned)((a.tokens * a.hq + 7) / 8);
    if (dtype == USP_BF16) {
        if (a.hd == 128) paged_simt_kernel<__nv_bfloat16, 128><<<grid, 256, 0, s>>>(a);
        else paged_simt_kernel<__nv_bfloat16, 64><<<grid, 256, 0, s>>>(a);
    } else {
        if (a.hd == 128) paged_simt_kernel<float, 128><<<grid, 256, 0, s>>>(a);
        else paged_simt_kernel<float, 64><<<grid, 256, 0, s>>>(a);
    }
    return cudaGetLastError() == cudaSuccess ? USP_OK : USP_ERR_CUDA;
}

}  // namespace usp
