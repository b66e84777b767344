// rope.cu -- rotary position embedding: of whole sequences (usp_rope; its inverse is the gradient), and on the way
// into the paged cache (usp_rope_append, usp_rope_append_q4), with the 4-bit cache's plain append (usp_cache_append_q4).
//
// Mathematics: a head's first `rot` elements are rot / 2 pairs (i, i + rot / 2), or (2 i, 2 i + 1) where interleaved; a
// pair (u, v) of a token at position p becomes (u c - v s, v c + u s) with c, s = table[p][i], table[p][rot / 2 + i]. Every
// product and sum is rounded to fp32 on its own (no fused multiply-add): what a 4-bit cache stores then depends on the
// formula alone, and not on how a compiler contracts it.
//
// What bounds it: HBM for long sequences (each element is read and written once for 3 operations), latency for a decode
// step. A row (one head of one token) has hd / 16 threads, 16 elements each: 8 of either half of its pairs. Rows of q, K and V
// of a token lie one after the other in a CTA's range, so the accesses in flight are close together.
#include <algorithm>

#include "paged.cuh"
#include "q4.cuh"
#include "usp_device.cuh"

namespace usp {
namespace {

constexpr int kThreads = 256;
constexpr int kMostPasses = 4;
constexpr int kSearch = 1024;  // entries of cu that a CTA searches in shared memory

enum RopeMode { ROPE_PLAIN = 0, ROPE_CACHE = 1, ROPE_Q4 = 2 };

struct RopeArgs {
    const char *q, *k, *v;
    char *q_out, *k_out, *v_out;      // k_out, v_out: the caches, except for ROPE_PLAIN
    uint8_t *k_scales, *v_scales;
    const float *table;
    const int32_t *slots, *positions, *cu, *kv;
    int64_t q_stride, k_stride, v_stride, qo_stride, ko_stride;  // bytes between tokens
    int64_t k_page, v_page, ks_page, vs_page;                    // bytes between pages
    int64_t max_pos;
    uint32_t rows, tokens, per_cta, nslots;
    int32_t nreq;                                                // entries of kv, or packed samples
    int32_t hq, hkv, per_token;                                  // per_token: heads of q, K and V together
    int32_t rot, log_ps;
    bool interleaved, inverse, quads;                            // quads: see group_max
    FastDiv by_heads, by_L;
    uint32_t L;
};

template <typename T> __device__ __forceinline__ void load8(const char *p, float (&x)[8]) {
    if constexpr (sizeof(T) == 2) {
        const uint4 w = *reinterpret_cast<const uint4 *>(p);
        const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = bf16x2_to_float2(a[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 f = reinterpret_cast<const float4 *>(p)[i];
            x[4 * i] = f.x; x[4 * i + 1] = f.y; x[4 * i + 2] = f.z; x[4 * i + 3] = f.w;
        }
    }
}
template <typename T> __device__ __forceinline__ void store8(char *p, const float (&x)[8]) {
    if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(float2_to_bf16x2(x[0], x[1]), float2_to_bf16x2(x[2], x[3]),
                                                   float2_to_bf16x2(x[4], x[5]), float2_to_bf16x2(x[6], x[7]));
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            reinterpret_cast<float4 *>(p)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    }
}

__device__ __forceinline__ void turn(float &u, float &v, float c, float s) {
    const float a = __fsub_rn(__fmul_rn(u, c), __fmul_rn(v, s));
    v = __fadd_rn(__fmul_rn(v, c), __fmul_rn(u, s));
    u = a;
}

__device__ __forceinline__ float max8(const float (&x)[8]) {
    float m = 0.f;  // a NaN is left out
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x[e]));
    return m;
}

// The largest magnitudes of the groups that a lane's two runs of 8 (with maxima a, b) belong to; all lanes of the warp
// call it. A row's lane c holds runs c and R + c for c < R, 2 c and 2 c + 1 behind that (R: the lanes of its row that hold the
// halves of pairs). Where R is a multiple of 4 a group is a run of four lanes or both runs of two; else each member
// is fetched from its lane.
template <int kLanes> __device__ __forceinline__ void group_max(float a, float b, int c, int R, bool quads, float &ga, float &gb) {
    if (quads) {
        const bool split = c < R;
        float x = split ? a : fmaxf(a, b), y = b;
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 1));
        const float x2 = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2)), y2 = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 2));
        ga = split ? x2 : x;
        gb = split ? y2 : x;
        return;
    }
    const int ja = c < R ? c : 2 * c, jb = c < R ? R + c : 2 * c + 1;
    ga = gb = 0.f;
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int j = ((h ? jb : ja) & ~3) + m;
            const int lane = j < R ? j : j < 2 * R ? j - R : j / 2;
            const float x = __shfl_sync(0xffffffffu, a, lane, kLanes), y = __shfl_sync(0xffffffffu, b, lane, kLanes);
            const float z = j < R ? x : j < 2 * R || (j & 1) ? y : x;
            if (h) gb = fmaxf(gb, z);
            else ga = fmaxf(ga, z);
        }
}

// the last entry i < n with cu[i] <= t, cu non-decreasing with cu[0] <= t; part: every step-th entry, in shared memory
__device__ __forceinline__ int find_sample(const int32_t *cu, int n, const int32_t *part, int step, int64_t t) {
    int lo = 0, hi = (n + step - 1) / step;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (part[mid] <= t) lo = mid;
        else hi = mid;
    }
    lo *= step;
    hi = min(lo + step, n);
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

template <typename T, int HD, int kMode> __global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs p) {
    constexpr int kLanes = HD / 16, kRows = kThreads / kLanes;  // lanes of a row; rows of a pass
    constexpr int kMostTokens = kMostPasses * kRows + 1;
    __shared__ int32_t part[kSearch];
    __shared__ int32_t pos_s[kMostTokens], slot_s[kMostTokens];
    wait_grid_before();
    const uint32_t r0 = blockIdx.x * p.per_cta, r1 = min(r0 + p.per_cta, p.rows);
    const uint32_t t0 = p.by_heads.div(r0), ntok = p.by_heads.div(r1 - 1) + 1 - t0;
    // ---- positions (-1: none) and slots of the CTA's tokens ----
    const bool search = p.rot > 0 && !p.positions && p.cu && p.nreq > 0;
    const int step = (p.nreq + kSearch - 1) / kSearch;
    if (search) {
        for (int i = threadIdx.x; i * step < p.nreq; i += kThreads) part[i] = p.cu[i * step];
        __syncthreads();
    }
    for (uint32_t i = threadIdx.x; i < ntok; i += kThreads) {
        const uint32_t t = t0 + i;
        int64_t pos = -1;
        if (p.rot > 0) {
            if (p.positions) {
                pos = p.positions[t];
            } else if constexpr (kMode == ROPE_PLAIN) {
                uint32_t b, l;
                p.by_L.divmod(t, b, l);
                pos = l;
                if (search && part[0] <= (int)l) pos = (int64_t)l - p.cu[find_sample(p.cu, p.nreq, part, step, l)];
            } else if (search && part[0] <= (int)t) {
                const int r = find_sample(p.cu, p.nreq, part, step, t);
                const int64_t end = p.cu[r + 1];  // a token behind the last request has no position
                if (t < end) pos = (int64_t)p.kv[r] - end + t;
            }
            if (pos >= p.max_pos) pos = -1;
        }
        pos_s[i] = (int32_t)max(pos, (int64_t)-1);
        if (kMode != ROPE_PLAIN) {
            const uint32_t slot = (uint32_t)p.slots[t];
            slot_s[i] = slot < p.nslots && (p.rot == 0 || pos >= 0) ? (int32_t)slot : -1;
        }
    }
    __syncthreads();
    // ---- rows ----
    const int c = threadIdx.x % kLanes;
    for (uint32_t first = r0; first < r1; first += kRows) {
        const uint32_t r = first + threadIdx.x / kLanes;
        uint32_t t, h;
        p.by_heads.divmod(min(r, r1 - 1), t, h);
        const int32_t pos = pos_s[t - t0], slot = kMode != ROPE_PLAIN ? slot_s[t - t0] : 0;
        const bool is_q = (int)h < p.hq, is_k = !is_q && (int)h < p.hq + p.hkv, is_v = !is_q && !is_k;
        const int head = is_q ? (int)h : is_k ? (int)h - p.hq : (int)h - p.hq - p.hkv;
        const bool turned = !is_v && p.rot > 0;
        const int R = turned && !p.interleaved ? p.rot / 16 : 0;
        const bool ok = r < r1 && (kMode == ROPE_PLAIN || (is_q ? pos >= 0 : slot >= 0));
        const int d0 = c < R ? 8 * c : 16 * c, d1 = c < R ? p.rot / 2 + 8 * c : 16 * c + 8;
        float x[8] = {}, y[8] = {};
        if (ok) {
            const char *src = (is_q ? p.q + t * p.q_stride : is_k ? p.k + t * p.k_stride : p.v + t * p.v_stride) +
                              (int64_t)head * HD * sizeof(T);
            load8<T>(src + d0 * sizeof(T), x);
            load8<T>(src + d1 * sizeof(T), y);
            if (turned && 16 * c < p.rot && pos >= 0) {
                float cs[8], sn[8];
                const char *row = reinterpret_cast<const char *>(p.table + (int64_t)pos * p.rot + 8 * c);
                load8<float>(row, cs);
                load8<float>(row + p.rot * 2, sn);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (p.inverse) sn[e] = -sn[e];
                if (p.interleaved) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        turn(x[2 * e], x[2 * e + 1], cs[e], sn[e]);
                        turn(y[2 * e], y[2 * e + 1], cs[4 + e], sn[4 + e]);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) turn(x[e], y[e], cs[e], sn[e]);
                }
            }
        }
        const int64_t page = slot >> p.log_ps;
        const int64_t in_page = ((int64_t)head << p.log_ps) + (slot & ((1 << p.log_ps) - 1));  // row of the page
        if (kMode == ROPE_Q4) {
            float ga, gb;
            group_max<kLanes>(max8(x), max8(y), c, R, p.quads, ga, gb);
            if (ok && !is_q) {
                const uint32_t ba = q4_scale_for(ga), bb = q4_scale_for(gb);
                char *row = (is_k ? p.k_out + page * p.k_page : p.v_out + page * p.v_page) + in_page * q4_code_bytes(HD);
                *reinterpret_cast<uint32_t *>(row + d0 / 2) = q4_pack(x, ba);
                *reinterpret_cast<uint32_t *>(row + d1 / 2) = q4_pack(y, bb);
                uint8_t *sc = (is_k ? p.k_scales + page * p.ks_page : p.v_scales + page * p.vs_page) + in_page * q4_scale_bytes(HD);
                if (d0 % kQ4Group == 0) sc[d0 / kQ4Group] = (uint8_t)ba;
                if (d1 % kQ4Group == 0) sc[d1 / kQ4Group] = (uint8_t)bb;
            }
        }
        if (ok && (kMode != ROPE_Q4 || is_q)) {
            char *dst;
            if (is_q) dst = p.q_out + t * p.qo_stride + (int64_t)head * HD * sizeof(T);
            else if (kMode == ROPE_PLAIN) dst = p.k_out + t * p.ko_stride + (int64_t)head * HD * sizeof(T);
            else dst = (is_k ? p.k_out + page * p.k_page : p.v_out + page * p.v_page) + in_page * (HD * (int64_t)sizeof(T));
            store8<T>(dst + d0 * sizeof(T), x);
            store8<T>(dst + d1 * sizeof(T), y);
        }
    }
}

template <int kMode> int launch_rope(RopeArgs a, int hd, int dtype, cudaStream_t s) {
    const DeviceInfo *di = device_info();
    if (!di) return USP_ERR_CUDA;
    a.by_heads = FastDiv((uint32_t)a.per_token);
    a.rows = a.tokens * (uint32_t)a.per_token;
    a.quads = a.interleaved || a.rot % 64 == 0;
    // passes per CTA: as many as leave every SM eight CTAs
    const uint32_t pass = (uint32_t)(kThreads / (hd / 16));
    const uint32_t passes = std::max(1u, std::min((uint32_t)kMostPasses, a.rows / (pass * 8u * (uint32_t)di->sm_count)));
    a.per_cta = pass * passes;
    const dim3 grid((a.rows + a.per_cta - 1) / a.per_cta);
    auto go = [&](auto kernel) { return launch_overlapped(kernel, grid, kThreads, 0, s, a); };
    if (dtype == USP_BF16)
        return hd == 128 ? go(rope_kernel<__nv_bfloat16, 128, kMode>) : go(rope_kernel<__nv_bfloat16, 64, kMode>);
    return hd == 128 ? go(rope_kernel<float, 128, kMode>) : go(rope_kernel<float, 64, kMode>);
}

int log2_of(int64_t x) {
    int l = 0;
    while ((int64_t(1) << l) < x) ++l;
    return l;
}

int check_stride(int64_t st, int64_t row, int es) {
    if (st < 0) return USP_ERR_INVALID_ARG;
    if (st != 0 && st < row) return USP_ERR_SHAPE;
    if (st >= (int64_t(1) << 38)) return USP_ERR_UNSUPPORTED;
    return st * es % 16 != 0 ? USP_ERR_ALIGN : USP_OK;
}

int check_rotation(int32_t rot, int32_t hd, int64_t max_pos) {
    if (rot < 0 || max_pos < 0) return USP_ERR_INVALID_ARG;
    if (rot > hd || rot % 16 != 0) return USP_ERR_SHAPE;
    return max_pos >= (int64_t(1) << 31) ? USP_ERR_UNSUPPORTED : USP_OK;
}

// what the appends share, up to where K and V go
int check_append(const usp_rope_append_desc &d, int32_t hkv, int32_t hd) {
    const int es = elem_size(d.dtype);
    if (es == 0) return USP_ERR_DTYPE;
    if (d.tokens < 0 || d.hq < 0 || d.nreq < 0) return USP_ERR_INVALID_ARG;
    int rc = check_rotation(d.rot, hd, d.max_pos);
    if (rc) return rc;
    if (d.rot == 0 && d.hq != 0) return USP_ERR_SHAPE;
    for (int64_t st : {d.q_stride, d.q_out_stride})
        if ((rc = check_stride(st, (int64_t)d.hq * hd, es))) return rc;
    for (int64_t st : {d.k_stride, d.v_stride})
        if ((rc = check_stride(st, (int64_t)hkv * hd, es))) return rc;
    if (d.nreq > kMaxRequests || d.hq > (1 << 20)) return USP_ERR_UNSUPPORTED;
    return d.tokens >= (int64_t(1) << 31) / (d.hq + 2 * (int64_t)hkv) ? USP_ERR_UNSUPPORTED : USP_OK;
}

int append_pointers(const void *q, const void *q_out, const void *k, const void *v, const int32_t *slots,
                    const int32_t *positions, const int32_t *cu, const int32_t *kv, const float *table,
                    const usp_rope_append_desc &d) {
    if (!k || !v || !slots || (d.hq > 0 && (!q || !q_out))) return USP_ERR_INVALID_ARG;
    if (d.rot > 0 && d.max_pos > 0 && !table) return USP_ERR_INVALID_ARG;
    if (d.rot > 0 && !positions && d.nreq > 0 && (!cu || !kv)) return USP_ERR_INVALID_ARG;
    for (const void *x : {q, q_out, k, v, static_cast<const void *>(table)})
        if (!aligned(x, 16)) return USP_ERR_ALIGN;
    for (const int32_t *x : {slots, positions, cu, kv})
        if (!aligned(x, 4)) return USP_ERR_ALIGN;
    return USP_OK;
}

RopeArgs append_args(const void *q, void *q_out, const void *k, const void *v, const int32_t *slots,
                     const int32_t *positions, const int32_t *cu, const int32_t *kv, const float *table,
                     const usp_rope_append_desc &d, int32_t hkv, int32_t hd, int32_t page_size, int64_t num_pages) {
    RopeArgs a{};
    const int es = elem_size(d.dtype);
    a.q = static_cast<const char *>(q); a.q_out = static_cast<char *>(q_out);
    a.k = static_cast<const char *>(k); a.v = static_cast<const char *>(v);
    a.slots = slots; a.positions = positions; a.cu = cu; a.kv = kv; a.table = table;
    a.q_stride = (d.q_stride ? d.q_stride : (int64_t)d.hq * hd) * es;
    a.qo_stride = (d.q_out_stride ? d.q_out_stride : (int64_t)d.hq * hd) * es;
    a.k_stride = (d.k_stride ? d.k_stride : (int64_t)hkv * hd) * es;
    a.v_stride = (d.v_stride ? d.v_stride : (int64_t)hkv * hd) * es;
    a.max_pos = d.max_pos;
    a.tokens = (uint32_t)d.tokens;
    a.nslots = (uint32_t)(num_pages * page_size);
    a.nreq = d.nreq;
    a.hq = d.hq; a.hkv = hkv; a.per_token = d.hq + 2 * hkv;
    a.rot = d.rot; a.log_ps = log2_of(page_size);
    a.interleaved = d.interleaved != 0;
    return a;
}

}  // namespace

int check_q4_dims(const usp_q4_dims &d) {
    // (the same limits as a bf16 cache's, whose elements these bytes stand for)
    usp_cache_dims c{};
    c.num_pages = d.num_pages; c.page_size = d.page_size; c.hkv = d.hkv; c.hd = d.hd; c.dtype = USP_BF16;
    const int rc = check_cache_dims(c);
    if (rc) return rc;
    const int64_t rows = (int64_t)d.hkv * d.page_size;
    const int64_t strides[4] = {d.k_page_stride, d.v_page_stride, d.k_scale_stride, d.v_scale_stride};
    for (int i = 0; i < 4; ++i) {
        if (strides[i] < 0) return USP_ERR_INVALID_ARG;
        if (strides[i] != 0 && strides[i] < rows * (i < 2 ? q4_code_bytes(d.hd) : q4_scale_bytes(d.hd))) return USP_ERR_SHAPE;
        if (strides[i] >= (int64_t(1) << 39)) return USP_ERR_UNSUPPORTED;
        if (strides[i] % 16 != 0) return USP_ERR_ALIGN;
    }
    return USP_OK;
}

}  // namespace usp

using namespace usp;

extern "C" {

int usp_rope(const void *q, void *q_out, const void *k, void *k_out, const float *table, const int32_t *positions,
             const int32_t *cu_seqlens, usp_rope_desc d, usp_stream_t stream) {
    const int es = elem_size(d.dtype);
    if (es == 0) return USP_ERR_DTYPE;
    if (d.bs < 0 || d.L < 0 || d.hq <= 0 || d.hkv < 0 || d.nseq < 0) return USP_ERR_INVALID_ARG;
    if (d.hd != 64 && d.hd != 128) return USP_ERR_UNSUPPORTED;
    int rc = check_rotation(d.rot, d.hd, d.max_pos);
    if (rc) return rc;
    if (d.rot == 0) return USP_ERR_SHAPE;
    for (int64_t st : {d.q_stride, d.q_out_stride})
        if ((rc = check_stride(st, (int64_t)d.hq * d.hd, es))) return rc;
    for (int64_t st : {d.k_stride, d.k_out_stride})
        if ((rc = check_stride(st, (int64_t)d.hkv * d.hd, es))) return rc;
    if (!positions && d.L > d.max_pos) return USP_ERR_SHAPE;
    if (d.nseq > kMaxRequests || d.hq > (1 << 20) || d.hkv > (1 << 20) || d.L >= (int64_t(1) << 31)) return USP_ERR_UNSUPPORTED;
    if (d.bs == 0 || d.L == 0) return USP_OK;
    if (d.bs >= (int64_t(1) << 31) / (d.hq + d.hkv) / d.L + 1 || d.bs * d.L >= (int64_t(1) << 31) / (d.hq + d.hkv))
        return USP_ERR_UNSUPPORTED;
    if (!q || !q_out || (d.hkv > 0 && (!k || !k_out)) || (d.max_pos > 0 && !table) || (d.nseq > 0 && !positions && !cu_seqlens))
        return USP_ERR_INVALID_ARG;
    for (const void *x : {q, static_cast<const void *>(q_out), k, static_cast<const void *>(k_out), static_cast<const void *>(table)})
        if (!aligned(x, 16)) return USP_ERR_ALIGN;
    if (!aligned(positions, 4) || !aligned(cu_seqlens, 4)) return USP_ERR_ALIGN;
    RopeArgs a{};
    a.q = static_cast<const char *>(q); a.q_out = static_cast<char *>(q_out);
    a.k = static_cast<const char *>(k); a.k_out = static_cast<char *>(k_out);
    a.table = table; a.positions = positions;
    a.cu = d.nseq > 0 ? cu_seqlens : nullptr;
    a.q_stride = (d.q_stride ? d.q_stride : (int64_t)d.hq * d.hd) * es;
    a.qo_stride = (d.q_out_stride ? d.q_out_stride : (int64_t)d.hq * d.hd) * es;
    a.k_stride = (d.k_stride ? d.k_stride : (int64_t)d.hkv * d.hd) * es;
    a.ko_stride = (d.k_out_stride ? d.k_out_stride : (int64_t)d.hkv * d.hd) * es;
    a.max_pos = d.max_pos;
    a.tokens = (uint32_t)(d.bs * d.L);
    a.nreq = d.nseq;
    a.hq = d.hq; a.hkv = d.hkv; a.per_token = d.hq + d.hkv;
    a.rot = d.rot;
    a.interleaved = d.interleaved != 0; a.inverse = d.inverse != 0;
    a.by_L = FastDiv((uint32_t)d.L); a.L = (uint32_t)d.L;
    return launch_rope<ROPE_PLAIN>(a, d.hd, d.dtype, reinterpret_cast<cudaStream_t>(stream));
}

int usp_rope_append(const void *q, void *q_out, const void *k, const void *v, void *k_cache, void *v_cache,
                    const int32_t *slot_map, const int32_t *positions, const int32_t *cu_new, const int32_t *kv_lens,
                    const float *table, usp_rope_append_desc d, usp_cache_dims c, usp_stream_t stream) {
    int rc = check_cache_dims(c);
    if (rc) return rc;
    if ((rc = check_append(d, c.hkv, c.hd))) return rc;
    if (c.dtype != d.dtype) return USP_ERR_DTYPE;
    if (d.rot == 0) return USP_ERR_SHAPE;  // (usp_cache_append)
    if (d.tokens == 0) return USP_OK;
    if ((rc = append_pointers(q, q_out, k, v, slot_map, positions, cu_new, kv_lens, table, d))) return rc;
    if (c.num_pages > 0 && (!k_cache || !v_cache)) return USP_ERR_INVALID_ARG;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16)) return USP_ERR_ALIGN;
    RopeArgs a = append_args(q, q_out, k, v, slot_map, positions, cu_new, kv_lens, table, d, c.hkv, c.hd, c.page_size, c.num_pages);
    const int es = elem_size(c.dtype);
    const int64_t dense = (int64_t)c.hkv * c.page_size * c.hd;
    a.k_out = static_cast<char *>(k_cache); a.v_out = static_cast<char *>(v_cache);
    a.k_page = (c.k_page_stride ? c.k_page_stride : dense) * es;
    a.v_page = (c.v_page_stride ? c.v_page_stride : dense) * es;
    return launch_rope<ROPE_CACHE>(a, c.hd, d.dtype, reinterpret_cast<cudaStream_t>(stream));
}

int usp_rope_append_q4(const void *q, void *q_out, const void *k, const void *v, void *k_cache, void *v_cache,
                       uint8_t *k_scales, uint8_t *v_scales, const int32_t *slot_map, const int32_t *positions,
                       const int32_t *cu_new, const int32_t *kv_lens, const float *table, usp_rope_append_desc d,
                       usp_q4_dims c, usp_stream_t stream) {
    int rc = check_q4_dims(c);
    if (rc) return rc;
    if ((rc = check_append(d, c.hkv, c.hd))) return rc;
    if (d.tokens == 0) return USP_OK;
    if ((rc = append_pointers(q, q_out, k, v, slot_map, positions, cu_new, kv_lens, table, d))) return rc;
    if (c.num_pages > 0 && (!k_cache || !v_cache || !k_scales || !v_scales)) return USP_ERR_INVALID_ARG;
    for (const void *x : {static_cast<const void *>(k_cache), static_cast<const void *>(v_cache),
                          static_cast<const void *>(k_scales), static_cast<const void *>(v_scales)})
        if (!aligned(x, 16)) return USP_ERR_ALIGN;
    RopeArgs a = append_args(q, q_out, k, v, slot_map, positions, cu_new, kv_lens, table, d, c.hkv, c.hd, c.page_size, c.num_pages);
    const int64_t rows = (int64_t)c.hkv * c.page_size;
    a.k_out = static_cast<char *>(k_cache); a.v_out = static_cast<char *>(v_cache);
    a.k_scales = k_scales; a.v_scales = v_scales;
    a.k_page = c.k_page_stride ? c.k_page_stride : rows * q4_code_bytes(c.hd);
    a.v_page = c.v_page_stride ? c.v_page_stride : rows * q4_code_bytes(c.hd);
    a.ks_page = c.k_scale_stride ? c.k_scale_stride : rows * q4_scale_bytes(c.hd);
    a.vs_page = c.v_scale_stride ? c.v_scale_stride : rows * q4_scale_bytes(c.hd);
    return launch_rope<ROPE_Q4>(a, c.hd, d.dtype, reinterpret_cast<cudaStream_t>(stream));
}

int usp_cache_append_q4(const void *k, const void *v, void *k_cache, void *v_cache, uint8_t *k_scales, uint8_t *v_scales,
                        const int32_t *slot_map, int64_t tokens, int64_t k_stride, int64_t v_stride, int32_t dtype,
                        usp_q4_dims c, usp_stream_t stream) {
    usp_rope_append_desc d{};
    d.tokens = tokens; d.k_stride = k_stride; d.v_stride = v_stride; d.dtype = dtype;
    return usp_rope_append_q4(nullptr, nullptr, k, v, k_cache, v_cache, k_scales, v_scales, slot_map, nullptr, nullptr,
                              nullptr, nullptr, d, c, stream);
}

}  // extern "C"
