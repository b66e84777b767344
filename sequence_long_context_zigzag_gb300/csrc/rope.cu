// rope.cu -- rotary position embedding: of whole sequences (usp_rope; its inverse is the gradient), and on the way
// into the paged cache (usp_rope_append, usp_rope_append_q4), with the 4-bit cache's plain append (usp_cache_append_q4).
//
// Mathematics: a head's first `rot` elements are rot / 2 pairs (i, i + rot / 2), or (2 i, 2 i + 1) where interleaved; a
// pair (u, v) of a token at position p becomes (u c - v s, v c + u s) with c, s = table[p][i], table[p][rot / 2 + i]. Every
// product and sum is rounded to fp32 on its own (no fused multiply-add): what a 4-bit cache stores then depends on the
// formula alone, and not on how a compiler contracts it.
//
// What bounds it: HBM for long sequences (each element is read and written once for 3 operations), latency for a decode
// step. A row (one head of one token) has hd / 16 threads, 16 elements each: 8 of either half of its pairs. A thread stays
// with its token, whose cosines and sines it holds, and walks the heads of q, K and V, the next row's loads in flight; the
// threads of a token side by side read a few KB in a row. Measured: 32768 tokens of 40 heads of 128 rotated 107 us, 0.95 of the
// copy rate; 48 heads of 46000 tokens rotated and appended 169 us, 1.01. What goes to a 4-bit cache has its own rows
// (quant_rows). A call of 64 tokens takes 3.7 us, quantising 5.1: launch and latency.
#include <string.h>

#include <algorithm>
#include <type_traits>

#include "paged.cuh"
#include "q4.cuh"
#include "usp_device.cuh"

namespace usp {
namespace {

constexpr int kThreads = 256;
constexpr int kSearch = 1024;  // entries of cu that a CTA searches in shared memory

enum RopeMode { ROPE_PLAIN, ROPE_CACHE, ROPE_Q4 };  // whole sequences; into the pages; q of an append to a 4-bit cache

struct RopeArgs {
    const char *q, *k, *v;
    char *q_out, *k_out, *v_out;      // k_out, v_out: the caches, except for ROPE_PLAIN
    uint8_t *k_scales, *v_scales;
    const float *table;
    const int32_t *slots, *positions, *cu, *kv;
    int64_t q_stride, k_stride, v_stride, qo_stride, ko_stride;  // bytes between tokens
    int64_t k_page, v_page, ks_page, vs_page;                    // bytes between pages
    int64_t max_pos;
    uint32_t tokens, nslots;
    int32_t nreq;                                                // entries of kv, or packed samples
    int32_t hq, hkv, heads;                                      // heads: of q, K and V together
    int32_t log_side, log_side_kv;                               // rows of a token side by side: 1 << log_side; in quant_rows
    uint32_t kv_blocks;                                          // CTAs of quant_rows
    int32_t rot, log_ps;
    bool interleaved, inverse, quads;                            // quads: see group_max
    FastDiv by_L;
};

__device__ __forceinline__ void load8(const char *p, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float4 f = reinterpret_cast<const float4 *>(p)[i];
        x[4 * i] = f.x; x[4 * i + 1] = f.y; x[4 * i + 2] = f.z; x[4 * i + 3] = f.w;
    }
}

__device__ __forceinline__ void turn(float &u, float &v, float c, float s) {
    const float a = __fsub_rn(__fmul_rn(u, c), __fmul_rn(v, s));
    v = __fadd_rn(__fmul_rn(v, c), __fmul_rn(u, s));
    u = a;
}

// the largest magnitude; NaN if there is one
__device__ __forceinline__ float max8(const float (&x)[8]) {
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(x[e])));
    return m;
}

// The largest magnitudes of the groups that a lane's two runs of 8 (with maxima a, b) belong to; all lanes of the warp
// call it. A row's lane c holds runs c and R + c for c < R, 2 c and 2 c + 1 behind that (R: the lanes of its row that hold the
// halves of pairs). Where R is a multiple of 4 a group is a run of four lanes or both runs of two; else each member
// is fetched from its lane.
template <int kLanes> __device__ __forceinline__ void group_max(float a, float b, int c, int R, bool none, bool quads,
                                                                        float &ga, float &gb) {
    if (none) {  // no row of the call has halves
        ga = fmaxf(a, b);
        ga = gb = fmaxf(ga, __shfl_xor_sync(0xffffffffu, ga, 1));
        return;
    }
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

// 8 elements as they lie in memory
template <typename T> struct Raw8 {
    uint4 w[sizeof(T) / 2];
    __device__ __forceinline__ void load(const char *p) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[i] = reinterpret_cast<const uint4 *>(p)[i];
    }
    __device__ __forceinline__ void store(char *p) const {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4 *>(p)[i] = w[i];
    }
    __device__ __forceinline__ void values(float (&x)[8]) const {
        if constexpr (sizeof(T) == 2) {
            const uint32_t a[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = bf16x2_to_float2(a[i]);
                x[2 * i] = f.x;
                x[2 * i + 1] = f.y;
            }
        } else {
            memcpy(x, w, sizeof(x));
        }
    }
    __device__ __forceinline__ void set(const float (&x)[8]) {
        if constexpr (sizeof(T) == 2)
            w[0] = make_uint4(float2_to_bf16x2(x[0], x[1]), float2_to_bf16x2(x[2], x[3]), float2_to_bf16x2(x[4], x[5]),
                              float2_to_bf16x2(x[6], x[7]));
        else
            memcpy(w, x, sizeof(x));
    }
};

// rows of a thread whose loads are in flight at once, at three CTAs per SM
template <typename T> constexpr int rope_batch(int mode) {
    const int n = mode == ROPE_CACHE ? 3 : 4;
    return sizeof(T) == 2 ? n : (n + 1) / 2;
}

struct Places {
    int32_t part[kSearch], pos[kThreads / 4], slot[kThreads / 4];  // (4: the fewest lanes of a row)
};
// The positions (-1: none) and slots of a CTA's ntok tokens from t0 on; all of its threads call it.
template <int kMode> __device__ __forceinline__ void find_places(const RopeArgs &p, uint32_t t0, uint32_t ntok, Places &sh) {
    const bool search = p.rot > 0 && !p.positions && p.cu && p.nreq > 0;
    const int step = (p.nreq + kSearch - 1) / kSearch;
    if (search) {
        for (int i = threadIdx.x; (int64_t)i * step < p.nreq; i += kThreads) sh.part[i] = p.cu[i * step];
        __syncthreads();
    }
    if (threadIdx.x < ntok) {
        const uint32_t u = t0 + threadIdx.x;
        const uint32_t slot = kMode != ROPE_PLAIN ? (uint32_t)p.slots[u] : 0;
        int64_t pos = -1;
        if (p.rot > 0) {
            if (p.positions) {
                pos = p.positions[u];
            } else if constexpr (kMode == ROPE_PLAIN) {
                uint32_t s, l;
                p.by_L.divmod(u, s, l);
                pos = l;
                if (search && sh.part[0] <= (int)l) pos = (int64_t)l - p.cu[find_sample(p.cu, p.nreq, sh.part, step, l)];
            } else if (search && sh.part[0] <= (int)u) {
                const int r = find_sample(p.cu, p.nreq, sh.part, step, u);
                const int64_t end = p.cu[r + 1];  // a token behind the last request has no position
                if (u < end) pos = (int64_t)p.kv[r] - end + u;
            }
            if (pos >= p.max_pos) pos = -1;
        }
        sh.pos[threadIdx.x] = (int32_t)max(pos, (int64_t)-1);
        if (kMode != ROPE_PLAIN) sh.slot[threadIdx.x] = slot < p.nslots && (p.rot == 0 || pos >= 0) ? (int32_t)slot : -1;
    }
    __syncthreads();
}

// Rows rotated and copied: the CTA's share of the tokens, q (and K and V, except for ROPE_Q4) of each; all threads call it.
template <typename T, int HD, int kMode> __device__ __forceinline__ void rope_rows(const RopeArgs &p, uint32_t block, Places &sh) {
    constexpr int kLanes = HD / 16, kRows = kThreads / kLanes;  // lanes of a row; rows side by side in a CTA
    constexpr int kRowBytes = HD * (int)sizeof(T);
    constexpr int kBatch = rope_batch<T>(kMode);
    // ---- this thread's token, and its part of the token's rows ----
    const int side = 1 << p.log_side;
    const uint32_t t0 = block * (kRows >> p.log_side), ntok = min((uint32_t)(kRows >> p.log_side), p.tokens - t0);
    const int c = threadIdx.x % kLanes, row = threadIdx.x / kLanes, h0 = row & (side - 1);
    const uint32_t tl = (uint32_t)row >> p.log_side, t = t0 + tl;
    const bool live = tl < ntok;
    // runs of 8: one of either half of the pairs, or neighbours (V, what is not rotated, interleaved pairs)
    const int R = p.interleaved ? 0 : p.rot / 16;
    struct Row {
        int head, d0, d1;
        bool q, k, ok;
    };
    auto row_of = [&](int h) {
        Row r;
        r.q = kMode == ROPE_Q4 || h < p.hq;
        r.k = !r.q && h < p.hq + p.hkv;
        r.head = r.q ? h : r.k ? h - p.hq : h - p.hq - p.hkv;
        r.ok = live && h < p.heads;
        const bool halves = (r.q || r.k) && c < R;
        r.d0 = halves ? 8 * c : 16 * c;
        r.d1 = halves ? p.rot / 2 + 8 * c : 16 * c + 8;
        return r;
    };
    Raw8<T> a[kBatch], b[kBatch];
    // (also of tokens that turn out to have no place: their rows are there)
    auto fetch = [&](int first) {
        const char *q = p.q + t * p.q_stride, *k = p.k + t * p.k_stride, *v = p.v + t * p.v_stride;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const Row r = row_of(first + i * side + h0);
            if (!r.ok) continue;
            const char *src = (r.q ? q : r.k ? k : v) + r.head * kRowBytes;
            a[i].load(src + r.d0 * sizeof(T));
            b[i].load(src + r.d1 * sizeof(T));
        }
    };
    fetch(0);
    find_places<kMode>(p, t0, ntok, sh);  // under the first loads
    const int32_t pos = live ? sh.pos[tl] : -1, slot = live && kMode != ROPE_PLAIN ? sh.slot[tl] : -1;
    const bool angles = 16 * c < p.rot && pos >= 0;
    float cs[8], sn[8];
    if (angles) {
        const char *at = reinterpret_cast<const char *>(p.table + (int64_t)pos * p.rot + 8 * c);
        load8(at, cs);
        load8(at + p.rot * 2, sn);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (p.inverse) sn[e] = -sn[e];
    }
    // ---- rows: head h's is h rows (of the page: h << log_ps rows) from the token's first ----
    char *q_out = p.q_out + t * p.qo_stride, *k_out, *v_out = nullptr;
    int k_step = kRowBytes;
    if constexpr (kMode == ROPE_PLAIN) {
        k_out = p.k_out + t * p.ko_stride;
    } else {
        const int64_t page = slot >> p.log_ps;
        const int in_page = slot & ((1 << p.log_ps) - 1);
        k_out = p.k_out + page * p.k_page + in_page * kRowBytes;
        v_out = p.v_out + page * p.v_page + in_page * kRowBytes;
        k_step = kRowBytes << p.log_ps;
    }
    for (int first = 0;;) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (i > 0 && first + i * side >= p.heads) break;
            const Row r = row_of(first + i * side + h0);
            const bool turned = (r.q || r.k) && angles, ok = r.ok && (kMode == ROPE_PLAIN || (r.q ? pos >= 0 : slot >= 0));
            float x[8], y[8];
            if (turned) {
                a[i].values(x);
                b[i].values(y);
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
            if (ok) {
                if (turned) {
                    a[i].set(x);
                    b[i].set(y);
                }
                char *to = r.q ? q_out + r.head * kRowBytes : (r.k ? k_out : v_out) + (int64_t)r.head * k_step;
                a[i].store(to + r.d0 * sizeof(T));
                b[i].store(to + r.d1 * sizeof(T));
            }
        }
        first += side * kBatch;
        if (first >= p.heads) break;
        fetch(first);
    }
}

// K and V rows quantised. A thread has 16 elements of the K and of the V row of a head at a time, the next head's loads under
// the arithmetic. Without a rotation it is about 100 operations a row and thread, which leave the kernel 0.94 of the copy
// rate (73000 tokens of 8 heads of 128 59 us; with 32 heads of q, rotated, 265 us, 0.90). One walk over q's, K's and V's
// rows alike, as rope_rows does it, took three times the operations (120 and 351 us).
enum Turn { TURN_NONE, TURN_NEIGHBOURS, TURN_HALVES };  // how K is rotated on the way

template <typename T> struct QuantRow {
    Raw8<T> a, b;
    __device__ __forceinline__ void load(const char *p, int d0, int d1) {
        a.load(p + d0 * sizeof(T));
        b.load(p + d1 * sizeof(T));
    }
};

template <typename T, int HD, int kTurn> __device__ __forceinline__ void quant_rows(const RopeArgs &p, uint32_t block, Places &sh) {
    constexpr int kLanes = HD / 16, kRows = kThreads / kLanes, kRowBytes = HD * (int)sizeof(T);
    constexpr int kCode = q4_code_bytes(HD), kScale = q4_scale_bytes(HD);
    const int side = 1 << p.log_side_kv;
    const uint32_t t0 = block * (kRows >> p.log_side_kv), ntok = min((uint32_t)(kRows >> p.log_side_kv), p.tokens - t0);
    const int c = threadIdx.x % kLanes, row = threadIdx.x / kLanes, h0 = row & (side - 1);
    const uint32_t tl = (uint32_t)row >> p.log_side_kv, t = t0 + tl;
    const bool live = tl < ntok;
    const int R = kTurn == TURN_HALVES ? p.rot / 16 : 0;
    const bool halves = c < R;
    const int d0 = halves ? 8 * c : 16 * c, d1 = halves ? p.rot / 2 + 8 * c : 16 * c + 8;
    const char *k = p.k + t * p.k_stride + h0 * kRowBytes, *v = p.v + t * p.v_stride + h0 * kRowBytes;
    QuantRow<T> kr, vr;
    if (live && h0 < p.hkv) {
        kr.load(k, d0, d1);
        vr.load(v, 16 * c, 16 * c + 8);
    }
    int32_t pos = -1, slot = -1;
    if constexpr (kTurn == TURN_NONE) {
        if (live && (uint32_t)p.slots[t] < p.nslots) slot = p.slots[t];
    } else {
        find_places<ROPE_Q4>(p, t0, ntok, sh);
        if (live) pos = sh.pos[tl], slot = sh.slot[tl];
    }
    float cs[8], sn[8];
    const bool angles = kTurn != TURN_NONE && 16 * c < p.rot && pos >= 0;
    if (angles) {
        const char *at = reinterpret_cast<const char *>(p.table + (int64_t)pos * p.rot + 8 * c);
        load8(at, cs);
        load8(at + p.rot * 2, sn);
    }
    const int64_t page = slot >> p.log_ps;
    const int at = (h0 << p.log_ps) + (slot & ((1 << p.log_ps) - 1));  // the row in its page
    char *ko = p.k_out + page * p.k_page + (int64_t)at * kCode, *vo = p.v_out + page * p.v_page + (int64_t)at * kCode;
    uint8_t *ks = p.k_scales + page * p.ks_page + (int64_t)at * kScale, *vs = p.v_scales + page * p.vs_page + (int64_t)at * kScale;
    // x, y: the lane's runs at e0 and e1 of a row
    auto store = [&](auto turned, float (&x)[8], float (&y)[8], char *to, uint8_t *sc, bool ok, int e0, int e1) {
        constexpr bool kHalves = decltype(turned)::value && kTurn == TURN_HALVES;
        constexpr bool kExact = sizeof(T) == 2 && !(decltype(turned)::value && kTurn != TURN_NONE);
        float ma = max8(x), mb = max8(y), ga, gb;
        if (__any_sync(0xffffffffu, ma != ma || mb != mb)) {  // NaN is stored as 0
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[e] = x[e] == x[e] ? x[e] : 0.f;
                y[e] = y[e] == y[e] ? y[e] : 0.f;
            }
            ma = max8(x);
            mb = max8(y);
        }
        group_max<kLanes>(ma, mb, c, R, !kHalves, p.quads, ga, gb);
        if (!ok) return;
        const Q4Scale sa(ga), sb = kHalves ? Q4Scale(gb) : sa;
        const uint32_t wa = q4_pack<kExact>(x, sa), wb = q4_pack<kExact>(y, sb);
        if (kHalves) {
            *reinterpret_cast<uint32_t *>(to + e0 / 2) = wa;
            *reinterpret_cast<uint32_t *>(to + e1 / 2) = wb;
            if (e0 % kQ4Group == 0) sc[e0 / kQ4Group] = (uint8_t)sa.b;
            if (e1 % kQ4Group == 0) sc[e1 / kQ4Group] = (uint8_t)sb.b;
        } else {
            *reinterpret_cast<uint2 *>(to + 8 * c) = make_uint2(wa, wb);
            if (c % 2 == 0) sc[c / 2] = (uint8_t)sa.b;
        }
    };
    for (int first = 0;;) {
        const bool ok = slot >= 0 && first + h0 < p.hkv;
        float x[8], y[8];
        kr.a.values(x);
        kr.b.values(y);
        if (angles) {
            if (kTurn == TURN_NEIGHBOURS) {
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
        first += side;
        const bool more = live && first + h0 < p.hkv;
        k += side * kRowBytes;
        v += side * kRowBytes;
        if (more) kr.load(k, d0, d1);  // the next head's K under this one's
        store(std::true_type{}, x, y, ko, ks, ok, d0, d1);
        vr.a.values(x);
        vr.b.values(y);
        if (more) vr.load(v, 16 * c, 16 * c + 8);
        store(std::false_type{}, x, y, vo, vs, ok, 16 * c, 16 * c + 8);
        if (first >= p.hkv) break;
        ko += (int64_t)(side * kCode) << p.log_ps;
        vo += (int64_t)(side * kCode) << p.log_ps;
        ks += (int64_t)(side * kScale) << p.log_ps;
        vs += (int64_t)(side * kScale) << p.log_ps;
    }
}

template <typename T, int HD, int kMode> __global__ void __launch_bounds__(kThreads, 3) rope_kernel(const RopeArgs p) {
    __shared__ Places sh;
    wait_grid_before();
    rope_rows<T, HD, kMode>(p, blockIdx.x, sh);
}

// CTAs per SM: as many as the registers of the bf16 kinds allow without a spill (a fourth costs the rotating ones 20 to 30%). The
// rotating fp32 kinds spill 84 to 152 bytes (30000 tokens of 8 + 8 heads of 128 117 us, 0.68 of the copy rate).
template <typename T> constexpr int quant_ctas(int turn) { return turn == TURN_NONE && sizeof(T) == 2 ? 4 : 3; }

// K and V, and q's rows (the last blocks)
template <typename T, int HD, int kTurn> __global__ void __launch_bounds__(kThreads, quant_ctas<T>(kTurn)) quant_kernel(const RopeArgs p) {
    __shared__ Places sh;
    wait_grid_before();
    if (blockIdx.x < p.kv_blocks) quant_rows<T, HD, kTurn>(p, blockIdx.x, sh);
    else if constexpr (kTurn != TURN_NONE) rope_rows<T, HD, ROPE_Q4>(p, blockIdx.x - p.kv_blocks, sh);
}

// Rows of a token side by side: all, as far as a CTA has place, where there are few; in large calls 1 << large.
int side_by_side(int64_t tokens, int heads, int rows, int large, int sms) {
    const int most = tokens * heads < (int64_t)rows * 8 * sms ? 30 : large;
    int log_side = 0;
    while (log_side < most && (1 << log_side) < heads && (2 << log_side) <= rows) ++log_side;
    return log_side;
}
uint32_t blocks_of(uint32_t tokens, int rows, int log_side) {
    const uint32_t per_cta = (uint32_t)rows >> log_side;
    return (tokens + per_cta - 1) / per_cta;
}

template <int kMode> int launch_rope(RopeArgs a, int hd, int dtype, cudaStream_t s) {
    const DeviceInfo *di = device_info();
    if (!di) return USP_ERR_CUDA;
    // In large calls eight, or four where the rows go to pages (40 heads of 128 of 32768 tokens: 2, 4, 8, 16, 32 of them 126,
    // 114, 107, 119, 174 us; 48 heads of 46000 into a cache 172, 169, 176, 211, 307).
    const int rows = kThreads / (hd / 16);
    a.log_side = side_by_side(a.tokens, a.heads, rows, kMode == ROPE_PLAIN ? 3 : 2, di->sm_count);
    const dim3 grid(blocks_of(a.tokens, rows, a.log_side));
    auto go = [&](auto kernel) { return launch_overlapped(kernel, grid, kThreads, 0, s, a); };
    if (dtype == USP_BF16)
        return hd == 128 ? go(rope_kernel<__nv_bfloat16, 128, kMode>) : go(rope_kernel<__nv_bfloat16, 64, kMode>);
    return hd == 128 ? go(rope_kernel<float, 128, kMode>) : go(rope_kernel<float, 64, kMode>);
}

template <typename T, int HD> int launch_quant(RopeArgs a, cudaStream_t s) {
    const DeviceInfo *di = device_info();
    if (!di) return USP_ERR_CUDA;
    const int rows = kThreads / (HD / 16);
    a.quads = a.rot % 64 == 0;
    a.heads = a.hq;  // (of rope_rows)
    a.log_side = side_by_side(a.tokens, a.hq, rows, 3, di->sm_count);
    // (73000 tokens, 8 heads: 1, 2, 4, 8 of them side by side 66.1, 65.2, 65.7, 69.0 us; rotated, with 32 of q, 278, 283, 294, 317)
    a.log_side_kv = side_by_side(a.tokens, a.hkv, rows, a.rot == 0 ? 1 : 0, di->sm_count);
    a.kv_blocks = blocks_of(a.tokens, rows, a.log_side_kv);
    const dim3 grid(a.kv_blocks + (a.hq > 0 ? blocks_of(a.tokens, rows, a.log_side) : 0));
    auto go = [&](auto kernel) { return launch_overlapped(kernel, grid, kThreads, 0, s, a); };
    return a.rot == 0 ? go(quant_kernel<T, HD, TURN_NONE>)
           : a.interleaved ? go(quant_kernel<T, HD, TURN_NEIGHBOURS>) : go(quant_kernel<T, HD, TURN_HALVES>);
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
    a.hq = d.hq; a.hkv = hkv; a.heads = d.hq + 2 * hkv;
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
    a.hq = d.hq; a.hkv = d.hkv; a.heads = d.hq + d.hkv;
    a.rot = d.rot;
    a.interleaved = d.interleaved != 0; a.inverse = d.inverse != 0;
    a.by_L = FastDiv((uint32_t)d.L);
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
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (d.dtype == USP_BF16) return c.hd == 128 ? launch_quant<__nv_bfloat16, 128>(a, st) : launch_quant<__nv_bfloat16, 64>(a, st);
    return c.hd == 128 ? launch_quant<float, 128>(a, st) : launch_quant<float, 64>(a, st);
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
