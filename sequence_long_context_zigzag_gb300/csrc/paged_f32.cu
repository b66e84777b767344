// paged_f32.cu -- fp32 attention over the paged cache on the CUDA cores, fp32 throughout (weights by the
// special-function unit's 2^x, whose error of 2^-22 is that of the scores' own sums).
//
// Mathematics and division of the work as in the bf16 kernels (online softmax with lazy rescale, spans of
// equal cost, cut units merged by the combine). Two kernels:
//
// few rows (paged_f32_few_kernel, units of up to 8 query rows): bound by HBM. A warp takes 4 keys of
//   each tile of 32, a lane hd / 32 elements of every row: K and V are read straight from global memory,
//   whole rows per load, no shared memory and no synchronisation inside a unit. The 8 x 4 scores are
//   reduced over the lanes by a butterfly that halves the values each lane holds, which ends with one
//   score per lane (row lane / 4, key lane % 4): 31 shuffles for 32 sums. 32 requests of 8000 keys, 8 heads of 128:
//   356 us, 5.9 TB/s (0.88 of the copy rate); 4 query heads on each of 8 KV heads of 64: 249 us, 4.2 TB/s (0.63), bound
//   by the shuffles and multiply-adds.
// many rows (paged_f32_many_kernel, units of up to 128 query rows): bound by the fp32 pipes
//   (128 lanes per SM). 256 threads compute 128 x 64 scores, 8 x 4 each, and 128 x hd outputs, 8 x hd / 16
//   each, from shared memory, with packed fp32 pairs (half the issue slots): a score's pair sums its even and
//   its odd elements, so that Q's and K's rows serve as they are, 12 16-byte words for 64 pair products; an
//   output's pair is two rows, from P written transposed. K and V come by asynchronous copies: V during a tile's scores, the next K during its outputs,
//   so the copies hold no registers (with register prefetch the loop had none left to run its loads ahead). 2048 tokens
//   over 8192 keys, 8 heads: 756 us at hd 64, 1493 at 128, 51 to 52 TFLOP/s, two thirds of what packed multiply-adds
//   alone reach (79): the operands' shared-memory reads share the issue slots. The products' loops are unrolled all
//   the way for their addresses (2 and 4 steps at a time 805 and 1660 us).
#include <math.h>

#include <algorithm>
#include <mutex>

#include "paged_sched.cuh"
#include "tc_ptx.cuh"

namespace usp {
namespace {

constexpr float kRescale = 8.0f;  // log2 units
constexpr float kLn2 = 0.69314718055994531f;

struct F32Params {
    SchedIn s;
    PartSpace w;
    const float *q, *k, *v;
    float *out, *lse;
    const int32_t *table;
    int64_t q_stride, out_stride, table_stride, k_page, v_page;
    int32_t num_pages, log_ps, hq;
    float scale_log2;
    bool second;  // the call's other kernel is in the stream before this one
};

__device__ __forceinline__ float finite_or_0(float m) { return m == -INFINITY ? 0.f : m; }

// ------------------------------------------------------------------------------------------------
// few rows
// ------------------------------------------------------------------------------------------------
constexpr int kFewRows = 8;
constexpr int kFewWarps = 8;
constexpr int kFewThreads = kFewWarps * 32;
constexpr int kFewKT = kFewWarps * 4;
constexpr int kFewOver = 64, kFewMinSpan = 64;  // (8 requests of up to 2000 keys: 14.5 us, spans of 160 keys up 18.4)
static_assert(kFewMinSpan > kFewKT, "a span holds more than a tile");

template <int E> struct Vec;
template <> struct Vec<4> { typedef float4 T; };
template <> struct Vec<2> { typedef float2 T; };
template <int E> __device__ __forceinline__ void load_vec(const float *p, float (&x)[E]) {
    const typename Vec<E>::T t = *reinterpret_cast<const typename Vec<E>::T *>(p);
    const float *f = reinterpret_cast<const float *>(&t);
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = f[e];
}

template <int HD>
__global__ void __launch_bounds__(kFewThreads, 2) paged_f32_few_kernel(const __grid_constant__ F32Params p) {
    constexpr int E = HD / 32;  // elements of a row per lane
    __shared__ SchedShared sh;
    __shared__ __align__(16) float qs[kFewRows][HD];
    __shared__ float xch[kFewWarps][kFewRows][HD];
    __shared__ float2 ml[kFewWarps][kFewRows];
    begin_in_order(p.second);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int srow = lane >> 2, skey = lane & 3;  // the score this lane ends up with
    // thread 0 walks the span; its state stays in shared memory, out of the products' registers
    __shared__ Sched sc;
    __shared__ Segment seg;
    __shared__ PartHeader opened;
    if (tid == 0) opened = PartHeader{};
    if (sched_scan<kFewThreads, kFewKT>(p.s, sh)) {
        __syncthreads();
        if (tid == 0) sched_begin<kFewKT>(p.s, sh, sc);
        for (;;) {
            if (tid == 0) {
                if (!sched_next<kFewKT>(p.s, sc, seg)) seg.ntok = 0;
                else if (seg.t0 == 0 && seg.t1 < seg.tiles) opened = part_header(p.s, sh, sc, seg);
            }
            __syncthreads();
            const Segment g = seg;
            if (g.ntok == 0) break;
            const int rows = g.ntok * p.s.G;
            __syncthreads();  // the previous unit's reads of qs, xch and ml are done
            for (int x = tid; x < kFewRows * HD; x += kFewThreads) {
                const int r = x / HD, c = x % HD;
                uint32_t tok, h;
                p.s.by_G.divmod((uint32_t)min(r, rows - 1), tok, h);
                qs[r][c] = p.q[(g.tok0 + tok) * p.q_stride + (int64_t)(g.head * p.s.G + (int)h) * HD + c] * p.scale_log2;
            }
            __syncthreads();
            const int stok = (int)p.s.by_G.div((uint32_t)min(srow, rows - 1));
            const int lim = p.s.causal ? max(0, min(g.kv, g.p0 + stok + 1)) : g.kv;
            float o[kFewRows][E], m = -INFINITY, l = 0.f;
#pragma unroll
            for (int r = 0; r < kFewRows; ++r)
#pragma unroll
                for (int e = 0; e < E; ++e) o[r][e] = 0.f;
            const int32_t *row = p.table + (int64_t)g.req * p.table_stride;
            const int ps = 1 << p.log_ps;
            // the 4 keys of a warp's batch share a page; -1 where there is none
            auto page_of = [&](int t) {
                const int64_t key = (int64_t)t * kFewKT + warp * 4;
                if (key >= g.kv) return -1;
                const int32_t x = row[key >> p.log_ps];
                return x < p.num_pages ? x : -1;
            };
            int32_t page = g.t0 < g.t1 ? page_of(g.t0) : -1;
            for (int t = g.t0; t < g.t1; ++t) {
                const int key0 = t * kFewKT + warp * 4;
                float k[4][E], v[4][E];
                const int64_t in = ((int64_t)g.head * ps + (key0 & (ps - 1))) * HD + lane * E;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bool ok = page >= 0 && key0 + j < g.kv;
                    if (ok) load_vec<E>(p.k + page * p.k_page + in + j * HD, k[j]);
                    else for (int e = 0; e < E; ++e) k[j][e] = 0.f;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bool ok = page >= 0 && key0 + j < g.kv;
                    if (ok) load_vec<E>(p.v + page * p.v_page + in + j * HD, v[j]);
                    else for (int e = 0; e < E; ++e) v[j][e] = 0.f;
                }
                page = t + 1 < g.t1 ? page_of(t + 1) : -1;  // the next tile's
                float s[32];
#pragma unroll
                for (int r = 0; r < kFewRows; ++r) {
                    float q[E];
#pragma unroll
                    for (int e = 0; e < E; ++e) q[e] = qs[r][lane * E + e];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float d = q[0] * k[j][0];
#pragma unroll
                        for (int e = 1; e < E; ++e) d = fmaf(q[e], k[j][e], d);
                        s[r * 4 + j] = d;
                    }
                }
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) {
                    const bool up = lane & d;
#pragma unroll
                    for (int i = 0; i < d; ++i) {
                        const float keep = up ? s[i + d] : s[i], send = up ? s[i] : s[i + d];
                        s[i] = keep + __shfl_xor_sync(0xffffffffu, send, d);
                    }
                }
                const float score = key0 + skey < lim ? s[0] : -INFINITY;
                if (__any_sync(0xffffffffu, score > m + kRescale)) {
                    float mx = fmaxf(score, __shfl_xor_sync(0xffffffffu, score, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    const float mn = fmaxf(m, mx), a = mn == -INFINITY ? 1.f : tc::ex2(m - mn);
                    m = mn;
                    l *= a;
#pragma unroll
                    for (int r = 0; r < kFewRows; ++r) {
                        const float ar = __shfl_sync(0xffffffffu, a, r * 4);
#pragma unroll
                        for (int e = 0; e < E; ++e) o[r][e] *= ar;
                    }
                }
                const float w = tc::ex2(score - finite_or_0(m));
                l += w;
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int r = 0; r < kFewRows; ++r) {
                        const float wr = __shfl_sync(0xffffffffu, w, r * 4 + j);
#pragma unroll
                        for (int e = 0; e < E; ++e) o[r][e] = fmaf(wr, v[j][e], o[r][e]);
                    }
            }
            // merge the warps' states and write the rows
            l += __shfl_xor_sync(0xffffffffu, l, 1);
            l += __shfl_xor_sync(0xffffffffu, l, 2);
            if (skey == 0) ml[warp][srow] = make_float2(m, l);
#pragma unroll
            for (int r = 0; r < kFewRows; ++r)
#pragma unroll
                for (int e = 0; e < E; ++e) xch[warp][r][lane * E + e] = o[r][e];
            __syncthreads();
            const bool whole = g.t0 == 0 && g.t1 == g.tiles;
            float *slot = part_slot(p.w, HD, blockIdx.x, g.t0 == 0 ? 1 : 0);
            for (int x = tid; x < rows * HD; x += kFewThreads) {
                const int r = x / HD, c = x % HD;
                float M = -INFINITY, L = 0.f, acc = 0.f;
#pragma unroll
                for (int w = 0; w < kFewWarps; ++w) M = fmaxf(M, ml[w][r].x);
                const float Mb = finite_or_0(M);
#pragma unroll
                for (int w = 0; w < kFewWarps; ++w) {
                    const float a = exp2f(ml[w][r].x - Mb);
                    L = fmaf(a, ml[w][r].y, L);
                    acc = fmaf(a, xch[w][r][c], acc);
                }
                uint32_t tok, h;
                p.s.by_G.divmod((uint32_t)r, tok, h);
                const int head = g.head * p.s.G + (int)h;
                if (whole) {
                    p.out[(g.tok0 + tok) * p.out_stride + (int64_t)head * HD + c] = L == 0.f ? 0.f : acc / L;
                    if (c == 0) p.lse[(g.tok0 + tok) * p.hq + head] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
                } else {
                    slot[(size_t)r * HD + c] = acc;
                    if (c == 0) {
                        slot[(size_t)p.w.rows * HD + r] = M;
                        slot[(size_t)p.w.rows * (HD + 1) + r] = L;
                    }
                }
            }
        }
    }
    __syncthreads();  // sh.any_long, also where this CTA has no work
    if (tid == 0) {
        opened.any_long = sh.any_long;
        p.w.head[blockIdx.x] = opened;
    }
    end_in_order(p.second);
}

// ------------------------------------------------------------------------------------------------
// many rows
// ------------------------------------------------------------------------------------------------
constexpr int kManyRows = 128;
constexpr int kManyThreads = 256;
constexpr int kManyKT = 64;
constexpr int kManyOver = 64, kManyMinSpan = 66;  // (6 prompts of up to 814 tokens: 28 us, spans of 256 keys up 41)
static_assert(kManyMinSpan > kManyKT, "a span holds more than a tile");

template <int HD> struct Many {
    static constexpr int kRow = HD + 4;          // floats per row of Q and K: 16 keys' pieces then lie on all banks
    static constexpr int kPRow = kManyRows + 4;  // of the transposed P
    static constexpr int kQ = 0;                       // [kManyRows][kRow]
    static constexpr int kK = kQ + kManyRows * kRow;   // [kManyKT][kRow]
    static constexpr int kV = kK + kManyKT * kRow;     // [kManyKT][HD]
    static constexpr int kP = kV + kManyKT * HD;       // [kManyKT][kPRow]
    static constexpr int kFloats = kP + kManyKT * kPRow;
};

// 16 bytes global -> shared; zeros when !ok (src is not read then)
__device__ __forceinline__ void copy16(uint32_t dst, const float *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copies_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ void load_pairs(const float *p, uint64_t (&x)[4]) {  // 8 floats as 4 pairs
    const ulonglong2 a = *reinterpret_cast<const ulonglong2 *>(p), b = *reinterpret_cast<const ulonglong2 *>(p + 4);
    x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
}

template <int HD>
__global__ void __launch_bounds__(kManyThreads, 1) paged_f32_many_kernel(const __grid_constant__ F32Params p) {
    using C = Many<HD>;
    constexpr int kCols = HD / 64;             // groups of 4 output columns per thread
    constexpr int kLd = kManyKT * HD / 4 / kManyThreads;  // 16-byte copies of K (and V) per thread
    extern __shared__ __align__(16) float sm[];
    __shared__ SchedShared sh;
    begin_in_order(false);
    float *qs = sm + C::kQ, *ks = sm + C::kK, *vs = sm + C::kV, *pt = sm + C::kP;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    // thread 0 walks the span; its state stays in shared memory, out of the products' registers
    __shared__ Sched sc;
    __shared__ Segment seg;
    __shared__ PartHeader opened;
    if (tid == 0) opened = PartHeader{};
    if (sched_scan<kManyThreads, kManyKT>(p.s, sh)) {
        __syncthreads();
        if (tid == 0) sched_begin<kManyKT>(p.s, sh, sc);
        for (;;) {
            if (tid == 0) {
                if (!sched_next<kManyKT>(p.s, sc, seg)) seg.ntok = 0;
                else if (seg.t0 == 0 && seg.t1 < seg.tiles) opened = part_header(p.s, sh, sc, seg);
            }
            __syncthreads();
            const Segment g = seg;
            if (g.ntok == 0) break;
            const int rows = g.ntok * p.s.G;
            __syncthreads();  // the previous unit's products are done
            constexpr int kQ = HD == 128 ? 8 : 4;  // pieces per thread and round: plain loads stay behind stores
            for (int x0 = tid; x0 < kManyRows * (HD / 4); x0 += kQ * kManyThreads) {
                float4 f[kQ];
#pragma unroll
                for (int i = 0; i < kQ; ++i) {
                    const int x = x0 + i * kManyThreads, r = x / (HD / 4), c = x % (HD / 4) * 4;
                    f[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (r < rows) {
                        uint32_t tok, h;
                        p.s.by_G.divmod((uint32_t)r, tok, h);
                        f[i] = *reinterpret_cast<const float4 *>(p.q + (g.tok0 + tok) * p.q_stride +
                                                                 (int64_t)(g.head * p.s.G + (int)h) * HD + c);
                    }
                }
#pragma unroll
                for (int i = 0; i < kQ; ++i) {
                    const int x = x0 + i * kManyThreads, r = x / (HD / 4), c = x % (HD / 4) * 4;
                    *reinterpret_cast<float4 *>(qs + r * C::kRow + c) = make_float4(
                        f[i].x * p.scale_log2, f[i].y * p.scale_log2, f[i].z * p.scale_log2, f[i].w * p.scale_log2);
                }
            }
            const int32_t *row = p.table + (int64_t)g.req * p.table_stride;
            const int ps = 1 << p.log_ps;
            // whole rows over consecutive threads; zeros behind the request's keys and for pages outside the cache
            auto fetch = [&](int t, const float *base, int64_t stride, const float *to, int to_row) {
#pragma unroll
                for (int i = 0; i < kLd; ++i) {
                    const int x = tid + i * kManyThreads, r = x / (HD / 4), c = x % (HD / 4) * 4;
                    const int key = t * kManyKT + r;
                    int32_t page = -1;
                    if (key < g.kv) page = row[key >> p.log_ps];
                    const bool ok = page >= 0 && page < p.num_pages;
                    const float *from = ok ? base + page * stride + ((int64_t)g.head * ps + (key & (ps - 1))) * HD + c : base;
                    copy16(tc::smem_u32(to + r * to_row + c), from, ok);
                }
                copies_commit();
            };
            // keys each of this thread's rows sees
            int lim[8];
            float m[8], l[8];
            uint64_t o[4][4 * kCols];  // [row pair][column]
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int tok = (int)p.s.by_G.div((uint32_t)min(ty * 8 + i, rows - 1));
                lim[i] = p.s.causal ? max(0, min(g.kv, g.p0 + tok + 1)) : g.kv;
                m[i] = -INFINITY;
                l[i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < 4 * kCols; ++c) o[i][c] = 0;
            const int lim_all = p.s.causal ? max(0, min(g.kv, g.p0 + 1)) : g.kv;
            if (g.t0 < g.t1) fetch(g.t0, p.k, p.k_page, ks, C::kRow);
            for (int t = g.t0; t < g.t1; ++t) {
                copies_wait_all();  // K of this tile
                __syncthreads();    // everyone's; and the previous tile's outputs are done with V
                fetch(t, p.v, p.v_page, vs, HD);
                uint64_t s[8][4];  // [row][key]: the sums over even and over odd elements
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[i][j] = 0;
#pragma unroll 16
                for (int d = 0; d < HD; d += 4) {
                    ulonglong2 k2[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        k2[j] = *reinterpret_cast<const ulonglong2 *>(ks + (tx + 16 * j) * C::kRow + d);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const ulonglong2 q2 = *reinterpret_cast<const ulonglong2 *>(qs + (ty * 8 + i) * C::kRow + d);
#pragma unroll
                        for (int j = 0; j < 4; ++j) s[i][j] = tc::fma2(q2.x, k2[j].x, s[i][j]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) s[i][j] = tc::fma2(q2.y, k2[j].y, s[i][j]);
                    }
                }
                const int key0 = t * kManyKT + tx;  // this thread's keys: key0 + 16 j
                const bool edge = (t + 1) * kManyKT > lim_all;
                float w[8][4];
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float even, odd;
                        tc::unpack2(s[i][j], even, odd);
                        w[i][j] = even + odd;
                    }
                float mx[8];
                bool need = false;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (edge) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (key0 + 16 * j >= lim[i]) w[i][j] = -INFINITY;
                    }
                    // the row's maximum over its 16 lanes is needed only when some lane's own exceeds the bound
                    mx[i] = fmaxf(fmaxf(w[i][0], w[i][1]), fmaxf(w[i][2], w[i][3]));
                    need |= mx[i] > m[i] + kRescale;
                }
                if (__any_sync(0xffffffffu, need)) {
                    float a[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
#pragma unroll
                        for (int d = 8; d > 0; d >>= 1) mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], d));
                        const float mn = fmaxf(m[i], mx[i]);
                        a[i] = mn == -INFINITY ? 1.f : tc::ex2(m[i] - mn);
                        m[i] = mn;
                        l[i] *= a[i];
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint64_t a2 = tc::pack2(a[2 * i], a[2 * i + 1]);
#pragma unroll
                        for (int c = 0; c < 4 * kCols; ++c) o[i][c] = tc::fma2(o[i][c], a2, 0ull);
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float mb = finite_or_0(m[i]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[i][j] = tc::ex2(w[i][j] - mb);
                    l[i] += (w[i][0] + w[i][1]) + (w[i][2] + w[i][3]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float4 *d = reinterpret_cast<float4 *>(pt + (tx + 16 * j) * C::kPRow + ty * 8);
                    d[0] = make_float4(w[0][j], w[1][j], w[2][j], w[3][j]);
                    d[1] = make_float4(w[4][j], w[5][j], w[6][j], w[7][j]);
                }
                copies_wait_all();  // V
                __syncthreads();    // everyone's; and all are done with K
                if (t + 1 < g.t1) fetch(t + 1, p.k, p.k_page, ks, C::kRow);
#pragma unroll
                for (int d = 0; d < kManyKT; ++d) {
                    uint64_t p2[4];
                    load_pairs(pt + d * C::kPRow + ty * 8, p2);
#pragma unroll
                    for (int c = 0; c < kCols; ++c) {
                        const float4 v4 = *reinterpret_cast<const float4 *>(vs + d * HD + c * 64 + tx * 4);
                        const uint64_t vv[4] = {tc::pack2(v4.x, v4.x), tc::pack2(v4.y, v4.y), tc::pack2(v4.z, v4.z),
                                                tc::pack2(v4.w, v4.w)};
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int j = 0; j < 4; ++j) o[i][c * 4 + j] = tc::fma2(p2[i], vv[j], o[i][c * 4 + j]);
                    }
                }
            }
            const bool whole = g.t0 == 0 && g.t1 == g.tiles;
            float *slot = part_slot(p.w, HD, blockIdx.x, g.t0 == 0 ? 1 : 0);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = ty * 8 + i;
#pragma unroll
                for (int d = 8; d > 0; d >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
                if (r >= rows) continue;
                uint32_t tok, h;
                p.s.by_G.divmod((uint32_t)r, tok, h);
                const int head = g.head * p.s.G + (int)h;
                const float inv = whole && l[i] != 0.f ? 1.f / l[i] : 1.f;
                float *dst = whole ? p.out + (g.tok0 + tok) * p.out_stride + (int64_t)head * HD : slot + (size_t)r * HD;
#pragma unroll
                for (int c = 0; c < kCols; ++c) {
                    float f[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float a, b;
                        tc::unpack2(o[i / 2][c * 4 + j], a, b);
                        f[j] = (i & 1 ? b : a) * inv;
                    }
                    *reinterpret_cast<float4 *>(dst + c * 64 + tx * 4) = make_float4(f[0], f[1], f[2], f[3]);
                }
                if (tx == 0) {
                    if (whole) {
                        p.lse[(g.tok0 + tok) * p.hq + head] = l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * kLn2;
                    } else {
                        slot[(size_t)p.w.rows * HD + r] = m[i];
                        slot[(size_t)p.w.rows * (HD + 1) + r] = l[i];
                    }
                }
            }
        }
    }
    __syncthreads();  // sh.any_long, also where this CTA has no work
    if (tid == 0) {
        opened.any_long = sh.any_long;
        p.w.head[blockIdx.x] = opened;
    }
}

template <int HD>
int launch_many(const F32Params &p, int grid, cudaStream_t s) {
    constexpr int kSmem = Many<HD>::kFloats * 4;
    static_assert(kSmem <= 226 * 1024, "shared memory per CTA");
    static std::mutex mu;
    static bool attr_set[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return USP_ERR_CUDA;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (dev < 0 || dev >= 64) return USP_ERR_UNSUPPORTED;
        if (!attr_set[dev]) {
            if (cudaFuncSetAttribute(paged_f32_many_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) !=
                cudaSuccess)
                return USP_ERR_CUDA;
            attr_set[dev] = true;
        }
    }
    return launch_overlapped(paged_f32_many_kernel<HD>, dim3((unsigned)grid), kManyThreads, kSmem, s, p);
}

}  // namespace

// one CTA per SM for many rows also at hd 64, where two fit: with half the registers the products' operands
// spill (2048 tokens over 8192: 1196 us against 824)
int f32_ctas(int sms, bool many) { return many ? sms : 2 * sms; }
int f32_rows(bool many) { return many ? kManyRows : kFewRows; }

int launch_paged_f32(const PagedArgs &a, bool many, int n_lo, int n_hi, bool second, const PartSpace &w,
                     cudaStream_t s) {
    F32Params p{};
    p.s.cu = a.cu; p.s.kv = a.kv;
    p.s.tokens = a.tokens; p.s.max_keys = paged_max_keys(a);
    p.s.nreq = a.nreq; p.s.hkv = a.hkv; p.s.G = a.G;
    p.s.tb = f32_rows(many) / a.G; p.s.causal = a.causal;
    p.s.n_lo = n_lo; p.s.n_hi = n_hi;
    p.s.over = many ? kManyOver : kFewOver;
    p.s.long_parts = many ? kManyParts : kFewParts;
    p.s.min_span = many ? kManyMinSpan : kFewMinSpan;
    p.s.inv_ctas = 1.0f / (float)w.ctas;
    p.s.by_tb = FastDiv((uint32_t)p.s.tb); p.s.by_G = FastDiv((uint32_t)a.G);
    p.w = w;
    p.q = static_cast<const float *>(a.q); p.k = static_cast<const float *>(a.k); p.v = static_cast<const float *>(a.v);
    p.out = static_cast<float *>(a.out); p.lse = a.lse;
    p.table = a.table;
    p.q_stride = a.q_stride; p.out_stride = a.out_stride; p.table_stride = a.table_stride;
    p.k_page = a.k_page; p.v_page = a.v_page;
    p.num_pages = (int32_t)a.num_pages; p.log_ps = a.log_ps; p.hq = a.hq;
    p.scale_log2 = a.scale_log2;
    p.second = second;
    if (many) return a.hd == 128 ? launch_many<128>(p, w.ctas, s) : launch_many<64>(p, w.ctas, s);
    return launch_overlapped(a.hd == 128 ? paged_f32_few_kernel<128> : paged_f32_few_kernel<64>, dim3((unsigned)w.ctas),
                             kFewThreads, 0, s, p);
}

}  // namespace usp
