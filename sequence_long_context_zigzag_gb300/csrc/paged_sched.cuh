// paged_sched.cuh -- how the work of one usp_paged_attn call is divided among the CTAs of a kernel.
//
// A unit is one request, one KV head and one block of `tb` new tokens (tb * G query rows); its cost is
// the keys its last token sees plus a constant `over` for its start and end. Units are ordered request
// by request, KV head by KV head, block by block, and the total cost W is cut into spans of one length, a
// span per CTA, at key-tile boundaries inside units. So every CTA gets the same number of keys however ragged
// the lengths are, and a long sequence with few rows is spread over all SMs. The lengths are device
// data: every CTA sums the costs itself (one scan over the requests, about a microsecond for the first
// few hundred), which costs less than a planning launch and keeps the call free of host copies.
// A unit cut by a span's end is finished by paged_combine_kernel: the CTA that opens it writes its
// partial to its slot 1 with a header, the CTAs that continue it to their slot 0; spans are longer than
// a tile, so each of these has a tile, and a CTA has at most one of each. (A span that ends within a unit's
// constant cost leaves the whole unit to the next one.)
#pragma once

#include <string.h>

#include "paged.cuh"

namespace usp {

struct SchedIn {
    const int32_t *cu, *kv;
    int64_t tokens, max_keys;
    int32_t nreq, hkv, G;
    int32_t tb;          // new tokens per unit
    int32_t causal;
    int32_t n_lo, n_hi;  // the requests of this kernel: n_lo < new tokens <= n_hi
    int32_t over;        // constant cost of a unit, in keys
    int32_t min_span;    // keys per CTA below which fewer CTAs work (more than a key tile)
    int32_t long_parts;  // parts of a unit above which the combine shares it out (kManyParts, kFewParts)
    float inv_ctas;      // 1 / CTAs of the launch
    FastDiv by_tb, by_G;
};

// A request's units: block b of each head holds new tokens [b tb, min((b + 1) tb, n)).
struct ReqUnits {
    int64_t t0, p0;  // first row of q; position of the first new token
    int32_t n, kv, nb;
    int64_t head_cost;
};

__device__ __forceinline__ int64_t unit_keys(const SchedIn &s, const ReqUnits &r, int32_t b) {
    if (!s.causal) return r.kv;
    return max((int64_t)0, r.p0 + min((int64_t)(b + 1) * s.tb, (int64_t)r.n));
}

// cost of blocks [0, b), b < nb (all of them full): sum of over + max(0, p0 + (b' + 1) tb)
__device__ __forceinline__ int64_t unit_prefix(const SchedIn &s, const ReqUnits &r, int32_t b) {
    if (!s.causal) return (int64_t)b * (s.over + (int64_t)r.kv);
    const int64_t b0 = r.p0 >= 0 ? 0 : min((int64_t)b, -r.p0 / s.tb);  // blocks that see nothing
    const int64_t nb = b, tri = nb * (nb + 1) / 2 - b0 * (b0 + 1) / 2;
    return nb * s.over + (nb - b0) * r.p0 + tri * s.tb;
}

__device__ __forceinline__ ReqUnits req_units(const SchedIn &s, int32_t i) {
    const Request q = paged_request(s.cu, s.kv, i, s.tokens, s.max_keys);
    ReqUnits r;
    r.t0 = q.t0;
    r.n = q.n > s.n_lo && q.n <= s.n_hi ? q.n : 0;
    r.kv = q.kv;
    r.p0 = (int64_t)q.kv - q.n;
    r.nb = (int32_t)s.by_tb.div((uint32_t)(r.n + s.tb - 1));
    r.head_cost = r.n > 0 ? unit_prefix(s, r, r.nb - 1) + s.over + unit_keys(s, r, r.nb - 1) : 0;
    return r;
}

// A place in the order of units: key tile t of a unit. req == nreq: the end.
struct UnitPos {
    int32_t req, head, b, t;
};

struct SchedShared {
    int64_t warp_sum[32];
    UnitPos at, end;  // of this CTA's span
    ReqUnits r;       // the request of `at`
    int64_t before;   // cost before that request
    int64_t span;
    int32_t any_long;  // some unit may have more than long_parts parts
};

// One stretch of a unit's key tiles [t0, t1), of `tiles` in all, that this CTA computes.
struct Segment {
    int64_t tok0;        // first row of q
    int32_t ntok, head;  // tokens of the block; KV head
    int32_t req, b;
    int32_t p0, kv;      // position of the block's first token; keys of the request
    int32_t t0, t1, tiles;
};

struct Sched {
    int64_t span;      // cost per CTA: CTA c covers [c span, (c + 1) span)
    UnitPos at, end;   // this CTA's span
    ReqUnits r;        // the request of `at`
    int64_t before;    // cost before that request
    Segment tail;      // a segment put off to the end (see sched_begin)
    bool put_off;
};

// floor(x / d), 0 <= x, 0 < d, for quotients below 2^20: a rounded estimate and its correction (a 64-bit
// division costs a few hundred cycles, and the start of a short call is a chain of these)
__device__ __forceinline__ int32_t div_small(int64_t x, int64_t d) {
    int32_t k = (int32_t)__fdividef((float)x, (float)d);
    while ((int64_t)k * d > x) --k;
    while ((int64_t)(k + 1) * d <= x) ++k;
    return k;
}

template <int KT>
__device__ __forceinline__ UnitPos unit_pos(const SchedIn &s, const ReqUnits &r, int32_t req, int64_t off) {
    UnitPos p;
    p.req = req;
    p.head = div_small(off, r.head_cost);  // fewer than 2^16 heads
    off -= p.head * r.head_cost;
    int32_t lo = 0, hi = r.nb;  // the last block that begins at or before off
    while (hi - lo > 1) {
        const int32_t mid = (lo + hi) >> 1;
        if (unit_prefix(s, r, mid) <= off) lo = mid;
        else hi = mid;
    }
    p.b = lo;
    off -= unit_prefix(s, r, lo);
    p.t = off <= s.over ? 0 : (int32_t)((off - s.over) / KT);
    return p;
}

// the next segment in the order of the units
template <int KT>
__device__ __forceinline__ bool sched_step(const SchedIn &s, Sched &o, Segment &g) {
    for (;;) {
        const bool last = o.at.req == o.end.req && o.at.head == o.end.head && o.at.b == o.end.b;
        if (o.at.req >= s.nreq || (last && o.end.t <= o.at.t)) return false;
        g.tiles = (int32_t)((unit_keys(s, o.r, o.at.b) + KT - 1) / KT);
        g.t0 = o.at.t;
        g.t1 = last ? o.end.t : g.tiles;
        g.head = o.at.head;
        g.req = o.at.req;
        g.b = o.at.b;
        const int32_t first = o.at.b * s.tb;
        g.tok0 = o.r.t0 + first;
        g.ntok = min(s.tb, o.r.n - first);
        g.p0 = (int32_t)(o.r.p0 + first);
        g.kv = o.r.kv;
        // step to the next unit (the end of the span when this one is cut)
        if (last) {
            o.at = o.end;
        } else {
            o.at.t = 0;
            if (++o.at.b == o.r.nb) {
                o.at.b = 0;
                if (++o.at.head == s.hkv) {
                    o.at.head = 0;
                    o.before += o.r.head_cost * s.hkv;
                    do {
                        if (++o.at.req >= s.nreq) break;
                        o.r = req_units(s, o.at.req);
                    } while (o.r.n == 0);
                }
            }
        }
        return true;
    }
}

// Called by all NT threads of the CTA: finds the requests in which the CTA's span begins and ends. False
// when this CTA has no work. `sh` is complete after the caller's next barrier.
template <int NT, int KT>
__device__ bool sched_scan(const SchedIn &s, SchedShared &sh) {
    static_assert(NT % 32 == 0 && NT <= 1024, "whole warps");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // inclusive scan of x over the CTA; total: the sum
    auto scan = [&](int64_t x, int64_t &total) {
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        __syncthreads();
        if (lane == 31) sh.warp_sum[warp] = x;
        __syncthreads();
        total = 0;
        for (int w = 0; w < NT / 32; ++w) {
            const int64_t y = sh.warp_sum[w];
            if (w < warp) x += y;
            total += y;
        }
        return x;
    };
    // (also where it begins, for sums past 64 bits: 2^13 requests that all claim the same 2^30 tokens)
    if (tid == 0) {
        sh.at = sh.end = UnitPos{s.nreq, 0, 0, 0};
        sh.any_long = 0;
    }
    int64_t mine = 0, W;
    int32_t longest = 0;  // keys
    ReqUnits r{};
    for (int32_t i = tid; i < s.nreq; i += NT) {
        r = req_units(s, i);
        mine += r.head_cost * s.hkv;
        if (r.n > 0) longest = max(longest, r.kv);
    }
    int64_t incl = scan(mine, W);
    // one length for all spans; the factor covers the estimate's roundings, so that they cover W
    const int64_t span = max((int64_t)s.min_span, (int64_t)((float)W * s.inv_ctas * 1.000001f) + 1);
    const int64_t x0 = blockIdx.x * span, x1 = x0 + span;
    if (tid == 0) sh.span = span;
    // a unit of cost u has at most u / span + 2 parts
    if (longest + s.over > (s.long_parts - 2) * span) sh.any_long = 1;
    if (x0 >= W) return false;
    int64_t carry = 0;
    for (int32_t base = 0; base < s.nreq; base += NT) {
        int64_t total = W;
        if (s.nreq > NT) {
            mine = 0;
            if (base + tid < s.nreq) {
                r = req_units(s, base + tid);
                mine = r.head_cost * s.hkv;
            }
            incl = scan(mine, total);
        }
        const int64_t a = carry + incl - mine;
        // the threads of the requests in which the span begins and ends find the places
        if (mine > 0 && a <= x0 && x0 < a + mine) {
            sh.at = unit_pos<KT>(s, r, base + tid, x0 - a);
            sh.before = a;
            sh.r = r;
        }
        if (mine > 0 && a <= x1 && x1 < a + mine) sh.end = unit_pos<KT>(s, r, base + tid, x1 - a);
        carry += total;
        if (carry > x1) break;
    }
    return true;
}

// The CTA's span as a walk, from what sched_scan found: for the one thread (or warp) that hands out the
// segments.
template <int KT>
__device__ __forceinline__ void sched_begin(const SchedIn &s, const SchedShared &sh, Sched &o) {
    o.span = sh.span;
    o.before = sh.before;
    o.r = sh.r;
    o.at = sh.at;
    o.end = sh.end;
    // A span that begins inside a unit takes that unit's rest last, if there is more: so all CTAs sweep
    // the keys from the front at the same time, and those that share a KV head read it from L2 (chunk
    // of 900 tokens over 64000 keys, 152 spans: every span at its own place re-reads 4 GB from HBM).
    o.put_off = false;
    if (o.at.t > 0 && !(o.end.req == o.at.req && o.end.head == o.at.head && o.end.b == o.at.b)) {
        Segment g;
        sched_step<KT>(s, o, g);
        o.tail = g;
        o.put_off = true;
    }
}

// the next segment of the span; false at its end
template <int KT>
__device__ __forceinline__ bool sched_next(const SchedIn &s, Sched &o, Segment &g) {
    if (sched_step<KT>(s, o, g)) return true;
    if (!o.put_off) return false;
    o.put_off = false;
    g = o.tail;
    return true;
}


// ---- handing segments to a CTA's roles ---------------------------------------------------------------
// One warp walks the span and passes each segment on through a small ring in shared memory, so that the
// other roles hold none of the walk's state (whose registers would spill in the softmax) and never wait
// for its arithmetic at a unit's end.
constexpr int kSegSlots = 4;
struct SegMsg {
    int64_t tok0;
    int32_t ntok, head;  // ntok == 0: the end
    int32_t req, p0, kv, t0;
    int32_t t1, tiles;
    int32_t act[2], full[2];  // per tile of rows (paged_chunk.cu): key tiles needed; key tiles without a mask
    int32_t pad[2];
};
static_assert(sizeof(SegMsg) == 64, "four 16-byte words");

// Reads the message at shared address `at`. `never` is false, but known only when all words have arrived: an arrive
// does not wait for loads in flight, so the one that releases the slot takes its address from it.
__device__ __forceinline__ SegMsg read_segment(uint32_t at, bool &never) {
    uint4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w)
                     : "r"(at + 16u * i)
                     : "memory");
    SegMsg m;
    memcpy(&m, w, sizeof(m));
    never = (m.ntok | m.t0 | m.t1 | m.full[0]) < 0;  // one of each word
    return m;
}

// What the CTA that opens a unit and does not finish it leaves for the combine.
struct __align__(16) PartHeader {
    int32_t rows;  // valid rows (ntok * G); 0: this CTA opens no cut unit
    int32_t head;
    int32_t last;  // the CTA that finishes the unit
    int32_t any_long;  // a unit of the call may have more than long_parts parts
    int64_t tok0, pad;
};
static_assert(sizeof(PartHeader) == 32, "two 16-byte words");

__device__ __forceinline__ PartHeader no_part(const SchedShared &sh) {
    PartHeader h{};
    h.any_long = sh.any_long;
    return h;
}

// The header of the segment just returned, with t0 == 0 and t1 < tiles: the last one in the order of
// the units, so `o` still holds its request.
__device__ __forceinline__ PartHeader part_header(const SchedIn &s, const SchedShared &sh, const Sched &o,
                                                   const Segment &g) {
    PartHeader h = no_part(sh);
    h.tok0 = g.tok0;
    h.rows = g.ntok * s.G;
    h.head = g.head;
    const int64_t end = o.before + (int64_t)g.head * o.r.head_cost +
                        (g.b + 1 < o.r.nb ? unit_prefix(s, o.r, g.b + 1) : o.r.head_cost);
    h.last = div_small(end - 1, o.span);  // fewer than 2^16 CTAs
    return h;
}

// parts of a unit up to which the combine leaves its rows to one CTA each 16: units of many rows, of few
constexpr int kManyParts = 16, kFewParts = 40;

// ---- partials: per CTA two slots of `rows` rows: o (rows x hd, relative to the maximum m), m, l ------
struct PartSpace {
    PartHeader *head;  // [ctas]
    float *data;       // [ctas][2][rows * (hd + 2)]
    int32_t ctas, rows;
};
__host__ __device__ inline size_t part_bytes(int ctas, int rows, int hd) {
    const size_t b = (size_t)ctas * (sizeof(PartHeader) + 2 * (size_t)rows * (hd + 2) * 4);
    return (b + 255) / 256 * 256;
}
__device__ __forceinline__ float *part_slot(const PartSpace &w, int hd, int cta, int slot) {
    return w.data + ((size_t)cta * 2 + slot) * (size_t)w.rows * (hd + 2);
}

struct CombineArgs {
    PartSpace w[2];  // one per kernel of the call (ctas == 0: not launched)
    void *out;
    float *lse;
    int64_t out_stride;
    int32_t hq, G;
    FastDiv by_G;
};
int launch_paged_combine(const CombineArgs &a, int hd, int dtype, cudaStream_t s);

// bf16, units of up to `rows` (16 or 32) query rows; requests with at most n_hi new tokens. `second`: the
// call's other kernel is in the stream before it
int launch_paged_decode(const PagedArgs &a, int rows, int n_hi, bool second, const PartSpace &w, cudaStream_t s);
int decode_ctas(int sms, int rows);

// bf16, units of up to kChunkRows query rows, one CTA per SM; requests with more than n_lo new tokens
constexpr int kChunkRows = 256;
int launch_paged_chunk(const PagedArgs &a, int n_lo, const PartSpace &w, cudaStream_t s);

// fp32: units of few (8) or many (128) query rows; requests with n_lo < new tokens <= n_hi
int launch_paged_f32(const PagedArgs &a, bool many, int n_lo, int n_hi, bool second, const PartSpace &w,
                     cudaStream_t s);
int f32_ctas(int sms, bool many);
int f32_rows(bool many);

}  // namespace usp
