// paged_decode.cu -- bf16 attention of few query rows per KV head over the paged cache (sm_103a): single
// tokens and short chunks, up to 32 query rows (tokens x G heads) per unit.
//
// Mathematics: online softmax over key tiles, o = sum_j 2^(s_j - m) v_j / l with s = scale log2(e) <q, k>,
// m the running maximum (rescaled only when it grows by more than 2^8: exact, the same stale maximum
// normalises), l the sum of the unrounded weights in fp32. The weights are rounded to bf16 for the product
// with V, whose products take both operands in one type: up to 2^-8 of each weight, at random signs, which over
// the keys adds less to o than o's own rounding to bf16 (whole outputs are 0.0018 to 0.0023 off in the norm against 64
// bits, the formula with fp32 weights 0.0016 to 0.0017).
//
// What bounds it: every K/V row is read once for 2 x rows multiply-adds per element, so HBM is the limit
// (an SM's share of the copy rate is about 23 bytes per clock). Layout of the work:
//  - spans of equal key counts per CTA (paged_sched.cuh); two CTAs per SM for 16 rows, one for 32;
//  - one producer warp walks the span, hands its segments to the others, and streams K and V tiles of 64 or
//    128 keys through a ring of shared-memory stages with TMA: one box of a page per lane, 128-byte swizzle,
//    the next tile's page numbers read ahead;
//  - four consumer warps per 16 rows, each with a quarter of the tile's keys and a softmax state of its own:
//    no synchronisation among them inside a unit. A tile is a chain of about 1000 cycles per warp (products,
//    maximum, exponentials, products), so a warp takes 32 keys of it, as two interleaved chains, where 16
//    would not keep HBM busy: rows of 64 elements, or one CTA per SM. S = Q K^T and O += P V run as m16n8k16 products
//    (mma.sync: at 16 rows a product uses an eighth of a tcgen05 tile, and the rate needed is far below
//    the legacy pipe's); P goes from S's registers straight into the next product;
//  - the four states merge through shared memory at a unit's end.
// Measured, a whole call with the combine (8 KV heads of 128, 4 query heads each, L2 cold): 64 requests of 2000 to
// 16384 keys (1.59 GB) 234 to 238 us and 2 of 200000 to 262143 (1.93 GB) 281 to 286 us, 1.00 to 1.03 of the measured copy
// rate; 64 of 8000 keys at hd 64 158 to 161 us, 0.98; 4 of 300 to 1024 keys 11 us, where 7 are the start (instructions, lengths, table,
// keys, one after the other) and 2 to 3 the combine.
// Rows behind the request's last key may hold NaN: scores are replaced, and V's registers of such keys
// are cleared, since 0 x NaN would spread.
#include <cuda_bf16.h>

#include <algorithm>
#include <mutex>

#include "paged_sched.cuh"
#include "paged_tma.cuh"
#include "tc_ptx.cuh"
#include "usp_device.cuh"

namespace usp {
namespace {

// A unit's constant cost, in keys: its start and end take a CTA about 2.5 us, in which the other CTAs read
// that many keys each. 256 tokens over up to 2000 keys: 64 in its place 101 us, 128 78, 192 and 256 67 (61 to 67 over the runs); 26
// single tokens and 7 chunks 38, 34.5, 32, 31.
constexpr int kOver = 256;
constexpr int kMinSpan = 194;     // keys per CTA below which fewer CTAs work
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr float kRescale = 8.0f;  // log2 units
constexpr float kLn2 = 0.69314718055994531f;

// RT: row tiles of 16 rows, each with four consumer warps
template <int HD, int RT> struct Cfg {
    static constexpr int kW = HD == 128 && RT == 1 ? 1 : 2;  // 16-key steps per warp and tile
    static constexpr int kKT = 64 * kW;                      // keys per tile
    static constexpr int kConsumers = 4 * RT;
    static constexpr int kThreads = (kConsumers + 1) * 32;
    static constexpr int kBoxes = HD / 64;
    static constexpr int kTile = kKT * HD * 2;  // bytes of K (or V) of one tile
    static constexpr int kStages = RT == 1 ? 3 : HD == 128 ? 3 : 5;  // 96 KB per CTA at two per SM, 160-192 KB at one
    static_assert(kMinSpan > kKT, "a span holds more than a tile");
    static constexpr int kXRow = 36;            // exchange row: 32 columns + padding
    static constexpr int kXGroup = 4 * 16 * kXRow * 4;
    static constexpr int kX = kStages * 2 * kTile;
    static constexpr int kML = kX + RT * kXGroup;  // m and l per warp and row
    static constexpr int kSeg = kML + kConsumers * 16 * 8;
    static constexpr int kBar = kSeg + kSegSlots * (int)sizeof(SegMsg);
    static constexpr int FULL = 0, EMPTY = kStages, SEG_FULL = 2 * kStages, SEG_EMPTY = SEG_FULL + kSegSlots;
    static constexpr int kSmem = kBar + (SEG_EMPTY + kSegSlots) * 8 + 1024;  // + slack for the alignment
};

struct DecodeParams {
    CUtensorMap tk, tv;
    SchedIn s;
    PartSpace w;
    const __nv_bfloat16 *q;
    __nv_bfloat16 *out;
    float *lse;
    const int32_t *table;
    int *status;
    int64_t q_stride, out_stride, table_stride;
    int32_t num_pages, log_ps, hq;
    float scale_log2;
    bool second;  // the call's other kernel is in the stream before this one
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// c += a (16x16, row) * b (16x8, column), bf16 in, fp32 out
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the four warps of a row tile
__device__ __forceinline__ void group_sync(int group) { asm volatile("bar.sync %0, 128;" ::"r"(group + 1) : "memory"); }
__device__ __forceinline__ bool group_all(int group, bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %2, 0;\n\t"
        "bar.red.and.pred p, %1, 128, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"(group + 1), "r"((uint32_t)x)
        : "memory");
    return r != 0;
}

// The producer warp: walks the span; lane b loads box b of each tile (page piece x column half, K then V).
template <int HD, int RT>
__device__ void producer(const DecodeParams &p, const SchedShared &sh, uint8_t *smem, uint32_t sbase) {
    using C = Cfg<HD, RT>;
    const int lane = threadIdx.x & 31;
    auto BAR = [&](int i) { return sbase + C::kBar + 8u * i; };
    auto wait = [&](int bar, uint32_t parity) {
        const bool r = tc::mbar_wait(BAR(bar), parity, p.status, USP_ERR_TIMEOUT, kWaitLimitNs);
        return (bool)__all_sync(0xffffffffu, r);
    };
    SegMsg *ring = reinterpret_cast<SegMsg *>(smem + C::kSeg);
    const int ps = 1 << p.log_ps, piece = min(ps, C::kKT), pieces = C::kKT / piece;
    const int nbox = pieces * C::kBoxes * 2;  // at most 32
    const int kv = lane >= nbox / 2, within = lane - kv * (nbox / 2);
    const int half = within / pieces, pc = within % pieces;
    const uint32_t dst0 = sbase + kv * C::kTile + half * (C::kKT * 128) + pc * piece * 128;
    const void *map = kv ? &p.tv : &p.tk;
    Sched sc;
    sched_begin<C::kKT>(p.s, sh, sc);
    PartHeader opened = no_part(sh);
    uint32_t fill = 0, nseg = 0;
    bool ok = true, more = true;
    while (more) {
        Segment g;
        more = sched_next<C::kKT>(p.s, sc, g);
        if (!(ok = wait(C::SEG_EMPTY + nseg % kSegSlots, ((nseg / kSegSlots) & 1u) ^ 1u))) break;
        if (lane == 0) {
            SegMsg m{};
            if (more) {
                m.tok0 = g.tok0; m.ntok = g.ntok; m.head = g.head; m.req = g.req; m.p0 = g.p0; m.kv = g.kv;
                m.t0 = g.t0; m.t1 = g.t1; m.tiles = g.tiles;
            }
            ring[nseg % kSegSlots] = m;
            tc::mbar_arrive(BAR(C::SEG_FULL + nseg % kSegSlots));
        }
        ++nseg;
        if (!more) break;
        const int32_t *row = p.table + (int64_t)g.req * p.table_stride;
        // page of this lane's piece of tile t; num_pages (a box of zeros) behind the request's keys
        auto page_of = [&](int t) {
            const int64_t key = (int64_t)t * C::kKT + pc * piece;
            if (lane >= nbox || key >= g.kv) return p.num_pages;
            const int32_t x = row[key >> p.log_ps];
            return x >= 0 && x < p.num_pages ? x : p.num_pages;
        };
        int32_t page = page_of(g.t0);
        for (int t = g.t0; t < g.t1; ++t) {
            const int32_t next = t + 1 < g.t1 ? page_of(t + 1) : 0;
            const uint32_t st = fill % C::kStages;
            if (!(ok = wait(C::EMPTY + st, ((fill / C::kStages) & 1u) ^ 1u))) break;
            if (lane == 0) tc::mbar_arrive_expect_tx(BAR(C::FULL + st), 2 * C::kTile);
            __syncwarp();
            if (lane < nbox)
                tma_load_3d(dst0 + st * 2 * C::kTile, map, half * 64,
                            g.head * ps + (int)(((int64_t)t * C::kKT + pc * piece) & (ps - 1)), page, BAR(C::FULL + st));
            ++fill;
            page = next;
        }
        if (!ok) break;
        if (g.t0 == 0 && g.t1 < g.tiles) opened = part_header(p.s, sh, sc, g);
    }
    if (!ok) {  // drain (bounded): no copy may land after the CTA has gone
        opened = no_part(sh);
        for (uint32_t f = fill > C::kStages ? fill - C::kStages : 0; f < fill; ++f)
            wait(C::FULL + f % C::kStages, (f / C::kStages) & 1u);
    }
    if (lane == 0) p.w.head[blockIdx.x] = opened;
}

template <int HD, int RT>
__device__ void consumer(const DecodeParams &p, uint8_t *smem, uint32_t sbase) {
    using C = Cfg<HD, RT>;
    constexpr int kNT = HD / 8;   // 8-column tiles of O
    constexpr int kKS = HD / 16;  // 16-element steps of the head dim
    const int lane = threadIdx.x & 31, group = threadIdx.x >> 7, tid = threadIdx.x & 127, warp = tid >> 5;
    auto BAR = [&](int i) { return sbase + C::kBar + 8u * i; };
    auto wait = [&](int bar, uint32_t parity) {
        const bool r = tc::mbar_wait(BAR(bar), parity, p.status, USP_ERR_TIMEOUT, kWaitLimitNs);
        return (bool)__all_sync(0xffffffffu, r);
    };
    float *xch = reinterpret_cast<float *>(smem + C::kX + group * C::kXGroup);
    float2 *ml = reinterpret_cast<float2 *>(smem + C::kML) + group * 64;  // [warp][16]
    const int qr = lane >> 2, qc = (lane & 3) * 2;  // fragment row and column of this lane
    // ldmatrix addresses inside a tile: 16-byte piece c of key row r lies at (c / 8) * kKT * 128 + r * 128 +
    // ((c % 8) ^ (r % 8)) * 16
    const int mi = lane >> 3, mr = lane & 7;
    const int krow = warp * 16 * C::kW + (mi >> 1) * 8 + mr, kc0 = mi & 1;
    const int vrow = warp * 16 * C::kW + (mi & 1) * 8 + mr, vc0 = mi >> 1;
    auto piece_at = [](int row, int c) { return (uint32_t)((c >> 3) * (C::kKT * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4)); };
    uint32_t fill = 0;
    for (uint32_t nseg = 0;; ++nseg) {
        // Every warp of the group reaches exactly one group_all per segment, also after a failed wait and
        // at the end, and leaves only by its result: so no warp waits for one that has gone.
        bool ok = wait(C::SEG_FULL + nseg % kSegSlots, (nseg / kSegSlots) & 1u);
        SegMsg g;
        g.ntok = 0;
        if (ok) {
            bool never;
            g = read_segment(sbase + C::kSeg + nseg % kSegSlots * (uint32_t)sizeof(SegMsg), never);
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(BAR(C::SEG_EMPTY + nseg % kSegSlots) + (never ? 8u : 0u));
        }
        const int rows = g.ntok * p.s.G - group * 16;  // rows of this group's tile
        uint32_t qf[kKS][4];
        float o[kNT][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        if (g.ntok > 0) {
            auto q_row = [&](int r) -> const uint32_t * {
                if (r >= rows) return nullptr;
                uint32_t tok, h;
                p.s.by_G.divmod((uint32_t)(group * 16 + r), tok, h);
                return reinterpret_cast<const uint32_t *>(p.q + (g.tok0 + tok) * p.q_stride +
                                                          (int64_t)(g.head * p.s.G + (int)h) * HD + qc);
            };
            const uint32_t *q0 = q_row(qr), *q1 = q_row(qr + 8);
#pragma unroll
            for (int k = 0; k < kKS; ++k) {
                qf[k][0] = q0 ? q0[k * 8] : 0u;
                qf[k][1] = q1 ? q1[k * 8] : 0u;
                qf[k][2] = q0 ? q0[k * 8 + 4] : 0u;
                qf[k][3] = q1 ? q1[k * 8 + 4] : 0u;
            }
        }
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
        // keys each of this lane's rows sees (rows beyond the valid ones like the last)
        int lim[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int tok = (int)p.s.by_G.div((uint32_t)(group * 16 + max(0, min(qr + h * 8, rows - 1))));
            lim[h] = p.s.causal ? max(0, min(g.kv, g.p0 + tok + 1)) : g.kv;
        }
        const int lim_all = p.s.causal ? max(0, min(g.kv, g.p0 + 1)) : g.kv;  // keys that every row sees
        for (int t = g.t0; ok && g.ntok > 0 && t < g.t1; ++t, ++fill) {
            const uint32_t st = fill % C::kStages;
            if (!(ok = wait(C::FULL + st, (fill / C::kStages) & 1u))) break;
            const uint32_t sk = sbase + st * 2 * C::kTile, sv = sk + C::kTile;
            const int key0 = t * C::kKT + warp * 16 * C::kW;  // this warp's first key
            if (RT == 1 || rows > 0) {
                float s[2 * C::kW][4];
#pragma unroll
                for (int n = 0; n < 2 * C::kW; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
                for (int k = 0; k < kKS; ++k)
#pragma unroll
                    for (int w = 0; w < C::kW; ++w) {
                        uint32_t b[4];
                        ldsm4(sk + piece_at(krow + w * 16, k * 2 + kc0), b);
                        mma16816(s[2 * w], qf[k], b[0], b[1]);
                        mma16816(s[2 * w + 1], qf[k], b[2], b[3]);
                    }
                if (key0 + 16 * C::kW > lim_all) {
#pragma unroll
                    for (int n = 0; n < 2 * C::kW; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (key0 + n * 8 + qc + (e & 1) >= lim[e >> 1]) s[n][e] = -INFINITY;
                }
                // a row's maximum over its four lanes is needed only when some lane's own exceeds the bound
                float mx[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    mx[h] = fmaxf(s[0][2 * h], s[0][2 * h + 1]);
#pragma unroll
                    for (int n = 1; n < 2 * C::kW; ++n) mx[h] = tc::max3(mx[h], s[n][2 * h], s[n][2 * h + 1]);
                    mx[h] *= p.scale_log2;
                }
                const bool need = mx[0] > m[0] + kRescale || mx[1] > m[1] + kRescale;
                if (__any_sync(0xffffffffu, need)) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
                        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
                        const float mn = fmaxf(m[h], mx[h]);
                        const float a = mn == -INFINITY ? 1.f : tc::ex2(m[h] - mn);
                        m[h] = mn;
                        l[h] *= a;
#pragma unroll
                        for (int n = 0; n < kNT; ++n) {
                            o[n][2 * h] *= a;
                            o[n][2 * h + 1] *= a;
                        }
                    }
                }
                uint32_t pf[C::kW][4], keep[C::kW][2];
#pragma unroll
                for (int w = 0; w < C::kW; ++w) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float mb = m[h] == -INFINITY ? 0.f : m[h];
                        float x[4];
#pragma unroll
                        for (int n = 0; n < 2; ++n)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                x[2 * n + e] = tc::ex2(fmaf(s[2 * w + n][2 * h + e], p.scale_log2, -mb));
                        l[h] += (x[0] + x[1]) + (x[2] + x[3]);
                        pf[w][h] = float2_to_bf16x2(x[0], x[1]);
                        pf[w][2 + h] = float2_to_bf16x2(x[2], x[3]);
                    }
                    // keys behind the request's last one: cleared in V's fragments (this lane's keys qc, qc+1, +8)
                    keep[w][0] = keep[w][1] = 0xffffffffu;
                    if (key0 + w * 16 + 16 > g.kv) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int k = key0 + w * 16 + h * 8 + qc;
                            keep[w][h] = (k < g.kv ? 0xffffu : 0u) | (k + 1 < g.kv ? 0xffff0000u : 0u);
                        }
                    }
                }
#pragma unroll
                for (int c = 0; c < kNT; c += 2)
#pragma unroll
                    for (int w = 0; w < C::kW; ++w) {
                        uint32_t b[4];
                        ldsm4t(sv + piece_at(vrow + w * 16, c + vc0), b);
                        mma16816(o[c], pf[w], b[0] & keep[w][0], b[1] & keep[w][1]);
                        mma16816(o[c + 1], pf[w], b[2] & keep[w][0], b[3] & keep[w][1]);
                    }
            }
            // The stage is released only when its rows have arrived in registers: an arrive does not wait for
            // ldmatrix reads in flight, and beside another kernel's load on the shared memory pipe these came after
            // the next tile had landed (one call in 10^4: the last columns of a unit a few keys wrong). The arrive's
            // address depends on a result of every product of V, compared with a NaN that no product gives.
            bool never = false;
#pragma unroll
            for (int c = 0; c < kNT; ++c) never |= __float_as_uint(o[c][0]) == 0x7fa5a5a5u;
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(BAR(C::EMPTY + st) + (never ? 8u : 0u));
        }
        // ---- merge the four warps' states and write the rows ---------------------------------------
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
            if ((lane & 3) == 0) ml[warp * 16 + qr + h * 8] = make_float2(m[h], l[h]);
        }
        if (!group_all(group, ok) || g.ntok == 0) return;
        if (rows <= 0) {
            group_sync(group);  // before the next segment's writes of ml
            continue;
        }
        const bool whole = g.t0 == 0 && g.t1 == g.tiles;
        float *slot = part_slot(p.w, HD, blockIdx.x, g.t0 == 0 ? 1 : 0) + (size_t)group * 16 * HD;
        // this thread's output row, its 4 columns of each 32, and the merged statistics
        const int orow = tid >> 3, ocol = (tid & 7) * 4;
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) M = fmaxf(M, ml[w * 16 + orow].x);
        const float Mb = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int w = 0; w < 4; ++w) L += ml[w * 16 + orow].y * tc::ex2(ml[w * 16 + orow].x - Mb);
        float a[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float mm = -INFINITY;
#pragma unroll
            for (int w = 0; w < 4; ++w) mm = fmaxf(mm, ml[w * 16 + qr + h * 8].x);
            a[h] = mm == -INFINITY ? 0.f : tc::ex2(m[h] - mm);
        }
        const float inv = whole && L != 0.f ? 1.f / L : 1.f;
        uint32_t tok, hr;
        p.s.by_G.divmod((uint32_t)(group * 16 + orow), tok, hr);
        const int head = g.head * p.s.G + (int)hr;
#pragma unroll
        for (int c = 0; c < HD / 32; ++c) {
            if (c > 0) group_sync(group);  // the exchange buffer is free
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const float *f = o[c * 4 + n];
                float *d = xch + (warp * 16 + qr) * C::kXRow + n * 8 + qc;
                *reinterpret_cast<float2 *>(d) = make_float2(f[0] * a[0], f[1] * a[0]);
                *reinterpret_cast<float2 *>(d + 8 * C::kXRow) = make_float2(f[2] * a[1], f[3] * a[1]);
            }
            group_sync(group);
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float4 x = *reinterpret_cast<const float4 *>(xch + (w * 16 + orow) * C::kXRow + ocol);
                v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
            }
            if (orow < rows) {
                if (whole) {
                    *reinterpret_cast<uint2 *>(p.out + (g.tok0 + tok) * p.out_stride + (int64_t)head * HD + c * 32 + ocol) =
                        make_uint2(float2_to_bf16x2(v.x * inv, v.y * inv), float2_to_bf16x2(v.z * inv, v.w * inv));
                } else {
                    *reinterpret_cast<float4 *>(slot + (size_t)orow * HD + c * 32 + ocol) = v;
                }
            }
        }
        if (orow < rows && (tid & 7) == 0) {
            if (whole) {
                p.lse[(g.tok0 + tok) * p.hq + head] = L == 0.f ? -INFINITY : (M + __log2f(L)) * kLn2;
            } else {
                float *st = part_slot(p.w, HD, blockIdx.x, g.t0 == 0 ? 1 : 0) + (size_t)p.w.rows * HD + group * 16 + orow;
                st[0] = M;
                st[p.w.rows] = L;
            }
        }
        group_sync(group);  // xch and ml are free for the next segment
    }
}

template <int HD, int RT>
__global__ void __launch_bounds__(Cfg<HD, RT>::kThreads, RT == 1 ? 2 : 1)
    paged_decode_kernel(const __grid_constant__ DecodeParams p) {
    using C = Cfg<HD, RT>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = tc::smem_u32(smem_raw);
    const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
    uint8_t *smem = smem_raw + pad;
    const uint32_t sbase = raw + pad;
    __shared__ SchedShared sh;
    __shared__ uint32_t skip;
    if (threadIdx.x == 0) {
        tc::prefetch_tmap(&p.tk);
        tc::prefetch_tmap(&p.tv);
        const uint32_t bar = sbase + C::kBar;
        for (int i = 0; i < C::kStages; ++i) {
            tc::mbar_init(bar + 8 * (C::FULL + i), 1);
            tc::mbar_init(bar + 8 * (C::EMPTY + i), C::kConsumers);
        }
        for (int i = 0; i < kSegSlots; ++i) {
            tc::mbar_init(bar + 8 * (C::SEG_FULL + i), 1);
            tc::mbar_init(bar + 8 * (C::SEG_EMPTY + i), C::kConsumers);
        }
        tc::fence_barrier_init();
    }
    begin_in_order(p.second);
    // a bounded wait of an earlier kernel ran out: do no work until usp_check clears it
    if (threadIdx.x == 0) skip = *reinterpret_cast<volatile int *>(p.status) != 0;
    const bool work = sched_scan<C::kThreads, C::kKT>(p.s, sh);
    __syncthreads();
    if (!work || skip) {
        if (threadIdx.x == 0) p.w.head[blockIdx.x] = no_part(sh);
    } else if ((threadIdx.x >> 5) == C::kConsumers) {
        producer<HD, RT>(p, sh, smem, sbase);
    } else {
        consumer<HD, RT>(p, smem, sbase);
    }
    end_in_order(p.second);
}

// ------------------------------------------------------------------------------------------------
// combine: out and lse of the units that spans cut
// ------------------------------------------------------------------------------------------------
// o = sum_i 2^(m_i - M) o_i / l over a row's parts, online, in an order that depends on their number alone, so the
// result does not depend on timing. A group of threads, 4 columns each, holds a row. What bounds it is
// latency: the header, then the parts, so a group fetches 8 (row, part) pairs at once: 8 parts of a row in
// the few-row kernels' units, 2 parts of 4 rows in the others' (prompts of 16334 tokens: 16 us with a row at a
// time).
// A CTA takes 16 rows of the unit that one header names. Units of many parts (a long sequence with few KV heads:
// up to 304) would leave that to a few CTAs, round after round: where the headers say that there are any, all
// CTAs then read all headers and share these units' rows evenly, and the groups of a CTA share a row's parts
// and join through shared memory. One token over 100000 keys, 16 heads on one KV head: 125 us a call with the first
// way alone, 25 to 28 with both; 32 tokens of 8 heads 69, 36.
// A part whose rows saw nothing has m = -inf, and its o (perhaps unwritten) is not used; a NaN score leaves l
// NaN, which is kept. Small CTAs: some fit beside the decode kernel's and are in place when it ends.
constexpr int kCombineThreads = 128;
constexpr int kCombineRows = 16;  // rows of a header's unit per CTA
constexpr int kHeadersPer = 4;    // headers per thread
constexpr int kMaxHeaders = kCombineThreads * kHeadersPer;
constexpr int kRowCost = 4;       // a row's constant cost, in parts
constexpr int kSharing = 608;     // CTAs that share the long units: all that run at once

// the running combination of a row's parts, 4 columns
struct RowSum {
    float M, L;
    float4 acc;
    __device__ __forceinline__ void clear() {
        M = -INFINITY;
        L = 0.f;
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __device__ __forceinline__ void rescale(float to, float base) {  // base: to, or 0 for -inf
        const float g = tc::ex2(M - base);
        M = to;
        L *= g;
        acc.x *= g; acc.y *= g; acc.z *= g; acc.w *= g;
    }
    __device__ __forceinline__ void add(float m, float l, const float4 &o, float base) {
        const float g = tc::ex2(m - base);
        if (g > 0.f || l != l) {
            L = fmaf(g, l, L);
            acc.x = fmaf(g, o.x, acc.x);
            acc.y = fmaf(g, o.y, acc.y);
            acc.z = fmaf(g, o.z, acc.z);
            acc.w = fmaf(g, o.w, acc.w);
        }
    }
};

// The partials of one unit, as a group's thread sees them (its columns start at col).
struct Parts {
    const float *open, *cont;  // part 0; parts 1, 2, ... a CTA's slots apart
    size_t step;
    int32_t cap, hd, col;      // rows of a slot; head dim
    __device__ __forceinline__ Parts(const PartSpace &w, int hd_, int c, int col_)
        : open(part_slot(w, hd_, c, 1)), cont(part_slot(w, hd_, c + 1, 0)), step(2 * (size_t)w.rows * (hd_ + 2)),
          cap(w.rows), hd(hd_), col(col_) {}
    // parts [base, base + NP) of the rows first, first + row_step, ..., below `end`, into sum[NR]
    template <int NR, int NP>
    __device__ __forceinline__ void fold(int first, int row_step, int end, int base, int parts, RowSum (&sum)[NR]) const {
        float m[NR][NP], l[NR][NP];
        float4 o[NR][NP];
#pragma unroll
        for (int j = 0; j < NR; ++j)
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int r = first + j * row_step;
                m[j][i] = -INFINITY;
                l[j][i] = 0.f;
                o[j][i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (base + i < parts && r < end) {
                    const float *s = base + i == 0 ? open : cont + (base + i - 1) * step;
                    m[j][i] = s[(size_t)cap * hd + r];
                    l[j][i] = s[(size_t)cap * (hd + 1) + r];
                    o[j][i] = *reinterpret_cast<const float4 *>(s + (size_t)r * hd + col);
                }
            }
#pragma unroll
        for (int j = 0; j < NR; ++j) {
            float mx = sum[j].M;
#pragma unroll
            for (int i = 0; i < NP; ++i) mx = fmaxf(mx, m[j][i]);
            const float mb = mx == -INFINITY ? 0.f : mx;
            sum[j].rescale(mx, mb);
#pragma unroll
            for (int i = 0; i < NP; ++i) sum[j].add(m[j][i], l[j][i], o[j][i], mb);
        }
    }
};

template <typename T, int HD>
__device__ __forceinline__ void write_row(const CombineArgs &a, const PartHeader &h, int r, int col, const RowSum &x) {
    constexpr bool kExact = sizeof(T) == 4;  // log2f for the fp32 path
    const float inv = x.L == 0.f ? 0.f : 1.f / x.L;
    uint32_t tok, hr;
    a.by_G.divmod((uint32_t)r, tok, hr);
    const int head = h.head * a.G + (int)hr;
    T *to = static_cast<T *>(a.out) + (h.tok0 + tok) * a.out_stride + (int64_t)head * HD + col;
    if constexpr (kExact)
        *reinterpret_cast<float4 *>(to) = make_float4(x.acc.x * inv, x.acc.y * inv, x.acc.z * inv, x.acc.w * inv);
    else
        *reinterpret_cast<uint2 *>(to) =
            make_uint2(float2_to_bf16x2(x.acc.x * inv, x.acc.y * inv), float2_to_bf16x2(x.acc.z * inv, x.acc.w * inv));
    if (col == 0)
        a.lse[(h.tok0 + tok) * a.hq + head] =
            x.L == 0.f ? -INFINITY : (x.M + (kExact ? log2f(x.L) : __log2f(x.L))) * kLn2;
}

// the rows [r0, end) of the unit that header c names, NR rows and NP parts at a time
template <typename T, int HD, int NR, int NP>
__device__ __forceinline__ void combine_rows(const CombineArgs &a, const Parts &p, const PartHeader &h, int parts, int r0,
                                             int end) {
    constexpr int kGroups = kCombineThreads / (HD / 4);
    for (int first = r0 + (int)threadIdx.x / (HD / 4); first < end; first += NR * kGroups) {
        RowSum x[NR];
#pragma unroll
        for (int j = 0; j < NR; ++j) x[j].clear();
        for (int base = 0; base < parts; base += NP) p.fold<NR, NP>(first, kGroups, end, base, parts, x);
#pragma unroll
        for (int j = 0; j < NR; ++j)
            if (first + j * kGroups < end) write_row<T, HD>(a, h, first + j * kGroups, p.col, x[j]);
    }
}

// CTA x of `ctas`: its share of the rows of all units of more than `limit` parts
template <typename T, int HD>
__device__ void combine_long(const CombineArgs &a, const PartSpace &w, int limit, int x, int ctas) {
    constexpr int kLanes = HD / 4, kGroups = kCombineThreads / kLanes;
    __shared__ int32_t before[kMaxHeaders + 1];  // cost of the rows before each header's
    __shared__ int32_t warp_sum[kCombineThreads / 32];
    __shared__ float4 xo[kGroups][kLanes];
    __shared__ float2 xml[kGroups];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int32_t cost[kHeadersPer], mine = 0;
#pragma unroll
    for (int e = 0; e < kHeadersPer; ++e) {
        const int c = tid * kHeadersPer + e;
        cost[e] = 0;
        if (c < w.ctas) {
            const int4 h = *reinterpret_cast<const int4 *>(w.head + c);  // rows, head, last
            if (h.x > 0 && h.z - c + 1 > limit) cost[e] = h.x * (h.z - c + 1 + kRowCost);
        }
        mine += cost[e];
    }
    int32_t incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += y;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int32_t all = 0, at = incl - mine;
#pragma unroll
    for (int i = 0; i < kCombineThreads / 32; ++i) {
        if (i < warp) at += warp_sum[i];
        all += warp_sum[i];
    }
#pragma unroll
    for (int e = 0; e < kHeadersPer; ++e) {
        before[tid * kHeadersPer + e] = at;
        at += cost[e];
    }
    if (tid == 0) before[kMaxHeaders] = all;
    __syncthreads();
    const int32_t share = (all + ctas - 1) / ctas, x0 = x * share, x1 = min(x0 + share, all);
    if (x0 >= all) return;
    int c = 0;  // the last header that begins at or before x0
#pragma unroll
    for (int d = kMaxHeaders / 2; d > 0; d >>= 1)
        if (before[c + d] <= x0) c += d;
    const int group = tid / kLanes, in_group = tid % kLanes;
    for (; c < w.ctas && before[c] < x1; ++c) {
        if (before[c + 1] == before[c]) continue;
        const PartHeader h = w.head[c];
        const int parts = h.last - c + 1;
        // the rows whose cost begins in this CTA's share
        const int32_t per = parts + kRowCost;
        const int r0 = max(0, (x0 - before[c] + per - 1) / per), r1 = min(h.rows, (x1 - before[c] + per - 1) / per);
        const Parts p(w, HD, c, in_group * 4);
        for (int r = r0; r < r1; ++r) {
            RowSum x[1];
            x[0].clear();
            for (int base = group * 8; base < parts; base += kGroups * 8) p.fold<1, 8>(r, 0, r1, base, parts, x);
            xo[group][in_group] = x[0].acc;
            if (in_group == 0) xml[group] = make_float2(x[0].M, x[0].L);
            __syncthreads();
            if (group == 0) {
                float mx = x[0].M;
#pragma unroll
                for (int g = 1; g < kGroups; ++g) mx = fmaxf(mx, xml[g].x);
                const float mb = mx == -INFINITY ? 0.f : mx;
                x[0].rescale(mx, mb);
#pragma unroll
                for (int g = 1; g < kGroups; ++g) x[0].add(xml[g].x, xml[g].y, xo[g][in_group], mb);
                write_row<T, HD>(a, h, r, p.col, x[0]);
            }
            __syncthreads();
        }
    }
}

template <typename T, int HD>
__global__ void __launch_bounds__(kCombineThreads) paged_combine_kernel(const CombineArgs a) {
    wait_grid_before();
    const int per0 = (a.w[0].rows + kCombineRows - 1) / kCombineRows;
    const int per1 = (a.w[1].rows + kCombineRows - 1) / kCombineRows;
    const int n0 = a.w[0].ctas * per0, n1 = a.w[1].ctas * per1;
    const bool many = (int)blockIdx.x < n0;
    const PartSpace &w = many ? a.w[0] : a.w[1];
    const int x = many ? (int)blockIdx.x : (int)blockIdx.x - n0, per = many ? per0 : per1;
    const int limit = many ? kManyParts : kFewParts, c = x / per, r0 = x % per * kCombineRows;
    const PartHeader h = w.head[c];
    const int parts = h.last - c + 1, end = min(r0 + kCombineRows, h.rows);
    if (r0 < end && parts <= limit) {
        const Parts p(w, HD, c, (int)threadIdx.x % (HD / 4) * 4);
        if (many) combine_rows<T, HD, 4, 2>(a, p, h, parts, r0, end);
        else combine_rows<T, HD, 1, 8>(a, p, h, parts, r0, end);
    }
    const int sharing = min(many ? n0 : n1, kSharing);
    if (h.any_long && x < sharing) combine_long<T, HD>(a, w, limit, x, sharing);
}

template <int HD, int RT>
int launch_typed(const DecodeParams &p, int grid, cudaStream_t s) {
    using C = Cfg<HD, RT>;
    constexpr int kSmem = C::kSmem;
    static_assert(kSmem + 2048 <= (RT == 1 ? 114 : 227) * 1024, "shared memory per CTA");
    static std::mutex mu;
    static bool attr_set[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return USP_ERR_CUDA;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (dev < 0 || dev >= 64) return USP_ERR_UNSUPPORTED;
        if (!attr_set[dev]) {
            if (cudaFuncSetAttribute(paged_decode_kernel<HD, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) !=
                cudaSuccess)
                return USP_ERR_CUDA;
            attr_set[dev] = true;
        }
    }
    return launch_overlapped(paged_decode_kernel<HD, RT>, dim3((unsigned)grid), C::kThreads, kSmem, s, p);
}

}  // namespace

int decode_ctas(int sms, int rows) { return rows == 16 ? 2 * sms : sms; }

int launch_paged_decode(const PagedArgs &a, int rows, int n_hi, bool second, const PartSpace &w, cudaStream_t s) {
    const DeviceInfo *di = device_info();
    if (!di) return USP_ERR_CUDA;
    DecodeParams p{};
    const int ps = 1 << a.log_ps;
    const uint32_t box = (uint32_t)std::min(ps, a.hd == 128 && rows == 16 ? Cfg<128, 1>::kKT : Cfg<64, 1>::kKT);
    static_assert(Cfg<64, 1>::kKT == Cfg<64, 2>::kKT && Cfg<64, 1>::kKT == Cfg<128, 2>::kKT, "one box height for these");
    if (!make_cache_tmap(&p.tk, a.k, a.num_pages, a.k_page, a.hkv, ps, a.hd, box) ||
        !make_cache_tmap(&p.tv, a.v, a.num_pages, a.v_page, a.hkv, ps, a.hd, box))
        return USP_ERR_CUDA;
    p.s.cu = a.cu; p.s.kv = a.kv;
    p.s.tokens = a.tokens; p.s.max_keys = paged_max_keys(a);
    p.s.nreq = a.nreq; p.s.hkv = a.hkv; p.s.G = a.G;
    p.s.tb = rows / a.G; p.s.causal = a.causal;
    p.s.n_lo = 0; p.s.n_hi = n_hi;
    p.s.over = kOver; p.s.min_span = kMinSpan; p.s.long_parts = kFewParts;
    p.s.inv_ctas = 1.0f / (float)w.ctas;
    p.s.by_tb = FastDiv((uint32_t)p.s.tb); p.s.by_G = FastDiv((uint32_t)a.G);
    p.w = w;
    p.q = static_cast<const __nv_bfloat16 *>(a.q);
    p.out = static_cast<__nv_bfloat16 *>(a.out);
    p.lse = a.lse;
    p.table = a.table;
    p.status = di->status;
    p.q_stride = a.q_stride; p.out_stride = a.out_stride; p.table_stride = a.table_stride;
    p.num_pages = (int32_t)a.num_pages; p.log_ps = a.log_ps; p.hq = a.hq;
    p.scale_log2 = a.scale_log2;
    p.second = second;
    if (rows == 16)
        return a.hd == 128 ? launch_typed<128, 1>(p, w.ctas, s) : launch_typed<64, 1>(p, w.ctas, s);
    return a.hd == 128 ? launch_typed<128, 2>(p, w.ctas, s) : launch_typed<64, 2>(p, w.ctas, s);
}

int launch_paged_combine(const CombineArgs &a, int hd, int dtype, cudaStream_t s) {
    if (std::max(a.w[0].ctas, a.w[1].ctas) > kMaxHeaders) return USP_ERR_UNSUPPORTED;
    const int per = kCombineRows;
    const dim3 grid((unsigned)(a.w[0].ctas * ((a.w[0].rows + per - 1) / per) + a.w[1].ctas * ((a.w[1].rows + per - 1) / per)));
    auto go = [&](auto kernel) { return launch_overlapped(kernel, grid, kCombineThreads, 0, s, a); };
    if (dtype == USP_BF16)
        return hd == 128 ? go(paged_combine_kernel<__nv_bfloat16, 128>) : go(paged_combine_kernel<__nv_bfloat16, 64>);
    return hd == 128 ? go(paged_combine_kernel<float, 128>) : go(paged_combine_kernel<float, 64>);
}

}  // namespace usp
