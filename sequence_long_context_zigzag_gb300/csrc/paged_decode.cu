// paged_decode.cu -- bf16 attention of few query rows per KV head over the paged cache (sm_103a): single
// tokens and short chunks, up to 32 query rows (tokens x G heads) per unit.
//
// Mathematics: online softmax over key tiles, o = sum_j 2^(s_j - m) v_j / l with s = scale log2(e) <q, k>,
// m the running maximum (rescaled only when it grows by more than 2^8: exact, the same stale maximum
// normalises), l the sum of the unrounded weights in fp32.
//
// What bounds it: every K/V row is read once for 2 x rows multiply-adds per element, so HBM is the limit
// (an SM's share of the copy rate is about 23 bytes per clock). Layout of the work:
//  - spans of equal key counts per CTA (paged_sched.cuh), two CTAs per SM;
//  - one producer warp streams K and V tiles of 64 keys through a ring of shared-memory stages with TMA:
//    one box of a page per lane, 128-byte swizzle, the next tile's page numbers read ahead;
//  - four consumer warps, each with 16 of the tile's 64 keys and a softmax state of its own: no
//    synchronisation among them inside a unit. S = Q K^T and O += P V run as m16n8k16 products
//    (mma.sync: at 16 rows a product uses an eighth of a tcgen05 tile, and the rate needed is far below
//    the legacy pipe's); P goes from S's registers straight into the next product;
//  - the four states merge through shared memory at a unit's end.
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

constexpr int kKT = 64;           // keys per tile
constexpr int kConsumers = 4;     // warps; 16 keys each
constexpr int kThreads = (kConsumers + 1) * 32;
constexpr int kOver = 64;         // a unit's constant cost, in keys
constexpr int kMinSpan = 192;     // keys per CTA below which fewer CTAs work
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr float kRescale = 8.0f;  // log2 units
constexpr float kLn2 = 0.69314718055994531f;

template <int HD, int MT> struct Cfg {
    static constexpr int kRows = 16 * MT;
    static constexpr int kBoxes = HD / 64;
    static constexpr int kTile = kKT * HD * 2;          // bytes of K (or V) of one tile
    static constexpr int kStages = HD == 128 ? 3 : 6;   // 96 KB in flight per CTA
    static constexpr int kXRow = 36;                    // exchange row: 32 columns + padding
    static constexpr int kXBytes = kConsumers * 16 * kXRow * 4;
    static constexpr int kQBytes = MT > 1 ? kRows * HD * 2 : 0;
    static constexpr int kX = kStages * 2 * kTile;
    static constexpr int kQ = kX + kXBytes;
    static constexpr int kML = kQ + kQBytes;            // m and l per warp and row
    static constexpr int kBar = kML + kConsumers * 16 * 8;
    static constexpr int kSmem = kBar + 2 * kStages * 8 + 16;
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
    int32_t max_pages, num_pages, log_ps, hq;
    float scale_log2;
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
__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kConsumers * 32) : "memory"); }

// The producer warp: lane b of it loads box b of each tile (page piece x column half, K then V).
template <int HD, int MT>
__device__ void producer(const DecodeParams &p, Sched &sc, uint32_t sbase) {
    using C = Cfg<HD, MT>;
    const int lane = threadIdx.x & 31;
    const uint32_t full = sbase + C::kBar, empty = full + 8 * C::kStages;
    const int ps = 1 << p.log_ps, piece = min(ps, kKT), pieces = kKT / piece;
    const int nbox = pieces * C::kBoxes * 2;  // at most 16
    const int kv = lane >= nbox / 2, within = lane - kv * (nbox / 2);
    const int half = within / pieces, pc = within % pieces;
    const uint32_t dst0 = sbase + kv * C::kTile + half * (kKT * 128) + pc * piece * 128;
    const void *map = kv ? &p.tv : &p.tk;
    uint32_t fill = 0;
    bool ok = true;
    Segment g;
    while (ok && sched_next<kKT>(p.s, sc, g)) {
        const int32_t *row = p.table + (int64_t)g.req * p.table_stride;
        // page of this lane's piece of tile t; num_pages (a box of zeros) behind the request's keys
        auto page_of = [&](int t) {
            const int64_t key = (int64_t)t * kKT + pc * piece;
            if (lane >= nbox || key >= g.kv) return p.num_pages;
            const int32_t x = __ldg(row + (key >> p.log_ps));
            return x >= 0 && x < p.num_pages ? x : p.num_pages;
        };
        int32_t page = page_of(g.t0);
        for (int t = g.t0; t < g.t1; ++t) {
            const int32_t next = t + 1 < g.t1 ? page_of(t + 1) : 0;
            const uint32_t st = fill % C::kStages;
            ok = tc::mbar_wait(empty + 8 * st, ((fill / C::kStages) & 1u) ^ 1u, p.status, USP_ERR_TIMEOUT, kWaitLimitNs);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (lane == 0) tc::mbar_arrive_expect_tx(full + 8 * st, 2 * C::kTile);
            __syncwarp();
            if (lane < nbox)
                tma_load_3d(dst0 + st * 2 * C::kTile, map, half * 64,
                            g.head * ps + (int)(((int64_t)t * kKT + pc * piece) & (ps - 1)), page, full + 8 * st);
            ++fill;
            page = next;
        }
    }
    if (!ok)  // drain (bounded): no copy may land after the CTA has gone
        for (uint32_t f = fill > C::kStages ? fill - C::kStages : 0; f < fill; ++f)
            tc::mbar_wait(full + 8 * (f % C::kStages), (f / C::kStages) & 1u, p.status, USP_ERR_TIMEOUT, kWaitLimitNs);
}

template <int HD, int MT>
__device__ void consumer(const DecodeParams &p, Sched &sc, uint8_t *smem, uint32_t sbase, PartHeader &opened) {
    using C = Cfg<HD, MT>;
    constexpr int kNT = HD / 8;   // 8-column tiles of O
    constexpr int kKS = HD / 16;  // 16-element steps of the head dim
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tid = threadIdx.x;
    const uint32_t full = sbase + C::kBar, empty = full + 8 * C::kStages;
    float *xch = reinterpret_cast<float *>(smem + C::kX);
    float2 *ml = reinterpret_cast<float2 *>(smem + C::kML);  // [warp][16]
    const int qr = lane >> 2, qc = (lane & 3) * 2;  // fragment row and column of this lane
    // ldmatrix addresses inside a tile: 16-byte piece c of key row r lies at (c / 8) * 64 rows + r * 128 +
    // ((c % 8) ^ (r % 8)) * 16
    const int mi = lane >> 3, mr = lane & 7;
    const int krow = warp * 16 + (mi >> 1) * 8 + mr, kc0 = mi & 1;
    const int vrow = warp * 16 + (mi & 1) * 8 + mr, vc0 = mi >> 1;
    auto piece_at = [](int row, int c) { return (uint32_t)((c >> 3) * (kKT * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4)); };
    uint32_t fill = 0;
    bool ok = true;
    Segment g;
    while (sched_next<kKT>(p.s, sc, g)) {
        const int rows = g.ntok * p.s.G;
        // ---- Q: fragments in registers (one 16-row tile), or in shared memory ---------------------
        uint32_t qf[MT > 1 ? 1 : kKS][4];
        auto q_word = [&](int r, int c) -> uint32_t {
            if (r >= rows) return 0u;
            uint32_t tok, h;
            p.s.by_G.divmod((uint32_t)r, tok, h);
            const int head = g.head * p.s.G + (int)h;
            return __ldg(reinterpret_cast<const uint32_t *>(p.q + (g.tok0 + tok) * p.q_stride + (int64_t)head * HD + c));
        };
        if constexpr (MT == 1) {
#pragma unroll
            for (int k = 0; k < kKS; ++k) {
                qf[k][0] = q_word(qr, k * 16 + qc);
                qf[k][1] = q_word(qr + 8, k * 16 + qc);
                qf[k][2] = q_word(qr, k * 16 + qc + 8);
                qf[k][3] = q_word(qr + 8, k * 16 + qc + 8);
            }
        } else {
            // rows of HD bf16, 16-byte pieces swizzled by row
            consumer_sync();  // the previous unit's reads are done
            for (int x = tid; x < C::kRows * HD / 2; x += kConsumers * 32) {
                const int r = x / (HD / 2), c = (x % (HD / 2)) * 2;
                *reinterpret_cast<uint32_t *>(smem + C::kQ + r * HD * 2 + (((c >> 3) ^ (r & 7)) << 4) + (c & 7) * 2) = q_word(r, c);
            }
            consumer_sync();
        }
        float o[MT][kNT][4], m[MT][2], l[MT][2];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            m[t][0] = m[t][1] = -INFINITY;
            l[t][0] = l[t][1] = 0.f;
#pragma unroll
            for (int n = 0; n < kNT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[t][n][e] = 0.f;
        }
        // keys each of this lane's rows sees (rows beyond the valid ones like the last)
        int lim[MT][2];
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int tok = (int)p.s.by_G.div((uint32_t)min(t * 16 + qr + h * 8, rows - 1));
                lim[t][h] = p.s.causal ? max(0, min(g.kv, g.p0 + tok + 1)) : g.kv;
            }
        const int lim_all = p.s.causal ? max(0, min(g.kv, g.p0 + 1)) : g.kv;  // keys that every row sees
        for (int t = g.t0; t < g.t1; ++t, ++fill) {
            const uint32_t st = fill % C::kStages;
            if (ok) ok = tc::mbar_wait(full + 8 * st, (fill / C::kStages) & 1u, p.status, USP_ERR_TIMEOUT, kWaitLimitNs);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) continue;  // the walk goes on without work, so that every warp reaches the same barriers
            const uint32_t sk = sbase + st * 2 * C::kTile, sv = sk + C::kTile;
            const int key0 = t * kKT + warp * 16;  // this warp's first key
            float s[MT][2][4];
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[i][n][e] = 0.f;
#pragma unroll
            for (int k = 0; k < kKS; ++k) {
                uint32_t b[4];
                ldsm4(sk + piece_at(krow, k * 2 + kc0), b);
                if constexpr (MT == 1) {
                    mma16816(s[0][0], qf[k], b[0], b[1]);
                    mma16816(s[0][1], qf[k], b[2], b[3]);
                } else {
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        uint32_t a[4];
                        const int r = i * 16 + (mi & 1) * 8 + mr, c = k * 2 + (mi >> 1);
                        ldsm4(sbase + C::kQ + r * HD * 2 + ((c ^ (r & 7)) << 4), a);
                        mma16816(s[i][0], a, b[0], b[1]);
                        mma16816(s[i][1], a, b[2], b[3]);
                    }
                }
            }
            const bool edge = key0 + 16 > lim_all;
            uint32_t pf[MT][4];
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                if (edge) {
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (key0 + n * 8 + qc + (e & 1) >= lim[i][e >> 1]) s[i][n][e] = -INFINITY;
                }
                float mx[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float x = fmaxf(fmaxf(s[i][0][2 * h], s[i][0][2 * h + 1]), fmaxf(s[i][1][2 * h], s[i][1][2 * h + 1]));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                    mx[h] = x * p.scale_log2;
                }
                const bool need = mx[0] > m[i][0] + kRescale || mx[1] > m[i][1] + kRescale;
                if (__any_sync(0xffffffffu, need)) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float mn = fmaxf(m[i][h], mx[h]);
                        const float a = mn == -INFINITY ? 1.f : tc::ex2(m[i][h] - mn);
                        m[i][h] = mn;
                        l[i][h] *= a;
#pragma unroll
                        for (int n = 0; n < kNT; ++n) {
                            o[i][n][2 * h] *= a;
                            o[i][n][2 * h + 1] *= a;
                        }
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float mb = m[i][h] == -INFINITY ? 0.f : m[i][h];
                    float w[4];
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) w[2 * n + e] = tc::ex2(fmaf(s[i][n][2 * h + e], p.scale_log2, -mb));
                    l[i][h] += (w[0] + w[1]) + (w[2] + w[3]);
                    pf[i][h] = float2_to_bf16x2(w[0], w[1]);
                    pf[i][2 + h] = float2_to_bf16x2(w[2], w[3]);
                }
            }
            // keys behind the request's last one: cleared in V's fragments (this lane's keys qc, qc+1, +8)
            uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
            if (key0 + 16 > g.kv) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int k = key0 + h * 8 + qc;
                    keep[h] = (k < g.kv ? 0xffffu : 0u) | (k + 1 < g.kv ? 0xffff0000u : 0u);
                }
            }
#pragma unroll
            for (int c = 0; c < kNT; c += 2) {
                uint32_t b[4];
                ldsm4t(sv + piece_at(vrow, c + vc0), b);
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    mma16816(o[i][c], pf[i], b[0] & keep[0], b[1] & keep[1]);
                    mma16816(o[i][c + 1], pf[i], b[2] & keep[0], b[3] & keep[1]);
                }
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(empty + 8 * st);
        }
        // ---- merge the four warps' states and write the rows ---------------------------------------
        const bool whole = g.t0 == 0 && g.t1 == g.tiles;
        float *slot = part_slot(p.w, HD, blockIdx.x, g.t0 == 0 ? 1 : 0);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                l[i][h] += __shfl_xor_sync(0xffffffffu, l[i][h], 1);
                l[i][h] += __shfl_xor_sync(0xffffffffu, l[i][h], 2);
                if ((lane & 3) == 0) ml[warp * 16 + qr + h * 8] = make_float2(m[i][h], l[i][h]);
            }
            consumer_sync();
            // this thread's output row, its 4 columns of each 32, and the merged statistics
            const int orow = tid >> 3, ocol = (tid & 7) * 4, r = i * 16 + orow;
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int w = 0; w < kConsumers; ++w) M = fmaxf(M, ml[w * 16 + orow].x);
            const float Mb = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int w = 0; w < kConsumers; ++w) L += ml[w * 16 + orow].y * tc::ex2(ml[w * 16 + orow].x - Mb);
            float a[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float mm = -INFINITY;
#pragma unroll
                for (int w = 0; w < kConsumers; ++w) mm = fmaxf(mm, ml[w * 16 + qr + h * 8].x);
                a[h] = mm == -INFINITY ? 0.f : tc::ex2(m[i][h] - mm);
            }
            const float inv = whole ? (L > 0.f ? 1.f / L : 0.f) : 1.f;
            uint32_t tok, hr;
            p.s.by_G.divmod((uint32_t)r, tok, hr);
            const int head = g.head * p.s.G + (int)hr;
#pragma unroll
            for (int c = 0; c < HD / 32; ++c) {
                consumer_sync();  // the exchange buffer is free
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const float *f = o[i][c * 4 + n];
                    float *d = xch + (warp * 16 + qr) * C::kXRow + n * 8 + qc;
                    *reinterpret_cast<float2 *>(d) = make_float2(f[0] * a[0], f[1] * a[0]);
                    *reinterpret_cast<float2 *>(d + 8 * C::kXRow) = make_float2(f[2] * a[1], f[3] * a[1]);
                }
                consumer_sync();
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kConsumers; ++w) {
                    const float4 x = *reinterpret_cast<const float4 *>(xch + (w * 16 + orow) * C::kXRow + ocol);
                    v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
                }
                if (r < rows && ok) {
                    if (whole) {
                        *reinterpret_cast<uint2 *>(p.out + (g.tok0 + tok) * p.out_stride + (int64_t)head * HD + c * 32 + ocol) =
                            make_uint2(float2_to_bf16x2(v.x * inv, v.y * inv), float2_to_bf16x2(v.z * inv, v.w * inv));
                    } else {
                        *reinterpret_cast<float4 *>(slot + (size_t)r * HD + c * 32 + ocol) = v;
                    }
                }
            }
            if (r < rows && ok && (tid & 7) == 0) {
                if (whole) {
                    p.lse[(g.tok0 + tok) * p.hq + head] = L > 0.f ? (M + __log2f(L)) * kLn2 : -INFINITY;
                } else {
                    slot[(size_t)p.w.rows * HD + r] = M;
                    slot[(size_t)p.w.rows * (HD + 1) + r] = L;
                }
            }
            consumer_sync();  // ml is free for the next tile of rows
        }
        if (!whole && g.t0 == 0 && ok) opened = part_header(p.s, sc, g);
    }
}

template <int HD, int MT>
__global__ void __launch_bounds__(kThreads, MT == 1 ? 2 : 1) paged_decode_kernel(const __grid_constant__ DecodeParams p) {
    using C = Cfg<HD, MT>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = tc::smem_u32(smem_raw);
    const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
    uint8_t *smem = smem_raw + pad;
    const uint32_t sbase = raw + pad;
    __shared__ SchedShared sh;
    __shared__ uint32_t skip;
    const uint32_t full = sbase + C::kBar, empty = full + 8 * C::kStages;
    // the combine may take its place on the SMs already; it waits for this kernel's end before it reads
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) {
        tc::prefetch_tmap(&p.tk);
        tc::prefetch_tmap(&p.tv);
        // a bounded wait of an earlier kernel ran out: do no work until usp_check clears it
        skip = *reinterpret_cast<volatile int *>(p.status) != 0;
        for (int i = 0; i < C::kStages; ++i) {
            tc::mbar_init(full + 8 * i, 1);
            tc::mbar_init(empty + 8 * i, kConsumers);
        }
        tc::fence_barrier_init();
    }
    Sched sc;
    const bool work = sched_init<kThreads, kKT>(p.s, sh, sc);
    __syncthreads();
    PartHeader opened{};
    if (work && !skip) {
        if ((threadIdx.x >> 5) == kConsumers) producer<HD, MT>(p, sc, sbase);
        else consumer<HD, MT>(p, sc, smem, sbase, opened);
    }
    if (threadIdx.x == 0) p.w.head[blockIdx.x] = opened;
}

// ------------------------------------------------------------------------------------------------
// combine: out and lse of the units that spans cut
// ------------------------------------------------------------------------------------------------
// A CTA per span and up to 8 rows at a time: a warp per row, the columns over its lanes. The parts' maxima
// and sums are read a part per lane; o = sum_i 2^(m_i - M) o_i / l in the parts' order, so the result does
// not depend on timing. A part whose rows saw nothing has m = -inf, and its o (perhaps unwritten) no part.
template <typename T, int HD>
__global__ void __launch_bounds__(256) paged_combine_kernel(const CombineArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int E = HD / 32;
    int c = blockIdx.x;
    const int which = c >= a.w[0].ctas;
    if (which) c -= a.w[0].ctas;
    const PartSpace w = which ? a.w[1] : a.w[0];
    const PartHeader h = w.head[c];
    const int lane = threadIdx.x & 31;
    const int parts = h.last - c + 1;
    auto slot = [&](int i) { return part_slot(w, HD, c + i, i == 0 ? 1 : 0); };
    for (int r = blockIdx.y * 8 + (threadIdx.x >> 5); r < h.rows; r += gridDim.y * 8) {
        float M = -INFINITY;
        for (int i = lane; i < parts; i += 32) M = fmaxf(M, slot(i)[(size_t)w.rows * HD + r]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        const float Mb = M == -INFINITY ? 0.f : M;
        float L = 0.f, acc[E] = {};
        for (int base = 0; base < parts; base += 32) {
            float wgt = 0.f, l = 0.f;
            if (base + lane < parts) {
                const float *s = slot(base + lane);
                const float d = s[(size_t)w.rows * HD + r] - Mb;
                wgt = sizeof(T) == 4 ? exp2f(d) : tc::ex2(d);  // the fp32 path has no fast functions
                l = wgt * s[(size_t)w.rows * (HD + 1) + r];
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            L += l;
            const int n = min(32, parts - base);
#pragma unroll 8
            for (int i = 0; i < n; ++i) {
                const float wi = __shfl_sync(0xffffffffu, wgt, i);
                const float *s = slot(base + i) + (size_t)r * HD + lane * E;
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] = wi > 0.f ? fmaf(wi, s[e], acc[e]) : acc[e];
            }
        }
        const float inv = L > 0.f ? 1.f / L : 0.f;
        const int64_t tok = h.tok0 + r / a.G;
        const int head = h.head * a.G + r % a.G;
        T *o = static_cast<T *>(a.out) + tok * a.out_stride + (int64_t)head * HD + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = (T)(acc[e] * inv);
        if (lane == 0) a.lse[tok * a.hq + head] = L > 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
    }
}

template <int HD, int MT>
int launch_typed(const DecodeParams &p, int grid, cudaStream_t s) {
    using C = Cfg<HD, MT>;
    constexpr int kSmem = C::kSmem + 1024;
    static std::mutex mu;
    static bool attr_set[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return USP_ERR_CUDA;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (dev < 0 || dev >= 64) return USP_ERR_UNSUPPORTED;
        if (!attr_set[dev]) {
            if (cudaFuncSetAttribute(paged_decode_kernel<HD, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) !=
                cudaSuccess)
                return USP_ERR_CUDA;
            attr_set[dev] = true;
        }
    }
    paged_decode_kernel<HD, MT><<<grid, kThreads, kSmem, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? USP_OK : USP_ERR_CUDA;
}

}  // namespace

int decode_ctas(int sms, int rows) { return rows == 16 ? 2 * sms : sms; }

int launch_paged_decode(const PagedArgs &a, int rows, int n_hi, const PartSpace &w, cudaStream_t s) {
    const DeviceInfo *di = device_info();
    if (!di) return USP_ERR_CUDA;
    DecodeParams p{};
    const int ps = 1 << a.log_ps;
    const uint32_t box = (uint32_t)std::min(ps, kKT);
    if (!make_cache_tmap(&p.tk, a.k, a.num_pages, a.k_page, a.hkv, ps, a.hd, box) ||
        !make_cache_tmap(&p.tv, a.v, a.num_pages, a.v_page, a.hkv, ps, a.hd, box))
        return USP_ERR_CUDA;
    p.s.cu = a.cu; p.s.kv = a.kv;
    p.s.tokens = a.tokens; p.s.max_keys = (int64_t)a.max_pages << a.log_ps;
    p.s.nreq = a.nreq; p.s.hkv = a.hkv; p.s.G = a.G;
    p.s.tb = rows / a.G; p.s.causal = a.causal;
    p.s.n_lo = 0; p.s.n_hi = n_hi;
    p.s.over = kOver; p.s.min_span = kMinSpan;
    p.s.inv_ctas = 1.0f / (float)w.ctas;
    p.s.by_tb = FastDiv((uint32_t)p.s.tb); p.s.by_G = FastDiv((uint32_t)a.G);
    p.w = w;
    p.q = static_cast<const __nv_bfloat16 *>(a.q);
    p.out = static_cast<__nv_bfloat16 *>(a.out);
    p.lse = a.lse;
    p.table = a.table;
    p.status = di->status;
    p.q_stride = a.q_stride; p.out_stride = a.out_stride; p.table_stride = a.table_stride;
    p.max_pages = a.max_pages; p.num_pages = (int32_t)a.num_pages; p.log_ps = a.log_ps; p.hq = a.hq;
    p.scale_log2 = a.scale_log2;
    if (rows == 16)
        return a.hd == 128 ? launch_typed<128, 1>(p, w.ctas, s) : launch_typed<64, 1>(p, w.ctas, s);
    return a.hd == 128 ? launch_typed<128, 2>(p, w.ctas, s) : launch_typed<64, 2>(p, w.ctas, s);
}

int launch_paged_combine(const CombineArgs &a, int hd, int dtype, cudaStream_t s) {
    // launched while the kernel before it still runs; griddepcontrol.wait is its first instruction
    cudaLaunchConfig_t cfg{};
    const int rows = std::max(a.w[0].ctas ? a.w[0].rows : 0, a.w[1].ctas ? a.w[1].rows : 0);
    cfg.gridDim = dim3((unsigned)(a.w[0].ctas + a.w[1].ctas), (unsigned)std::min(8, (rows + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    cudaError_t e;
    if (dtype == USP_BF16)
        e = hd == 128 ? cudaLaunchKernelEx(&cfg, paged_combine_kernel<__nv_bfloat16, 128>, a)
                      : cudaLaunchKernelEx(&cfg, paged_combine_kernel<__nv_bfloat16, 64>, a);
    else
        e = hd == 128 ? cudaLaunchKernelEx(&cfg, paged_combine_kernel<float, 128>, a)
                      : cudaLaunchKernelEx(&cfg, paged_combine_kernel<float, 64>, a);
    return e == cudaSuccess ? USP_OK : USP_ERR_CUDA;
}

}  // namespace usp
