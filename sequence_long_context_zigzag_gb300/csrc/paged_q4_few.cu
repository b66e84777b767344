// paged_q4_few.cu -- attention of few query rows per KV head over the 4-bit paged cache (sm_103a): single tokens and short
// chunks, up to 32 query rows (tokens x G heads; fp32: 16) per unit; fp32 queries at any length.
//
// Mathematics: as paged_decode.cu (online softmax over key tiles, lazy rescale, weights rounded to bf16 for the product
// with V; fp32 queries and weights enter as three bf16 terms each, x = x0 + x1 + x2 to 24 bits). The products run
// transposed, S^T = K Q^T and O^T = V^T P^T as m16n8k16 (mma.sync), so that the cache is the operand of 16 rows and 8
// query rows fill the other: a value of the cache is converted once for all rows, and with up to 8 rows no product is idle.
//   A code pair becomes an operand in registers: (word >> 4 j) has two codes in the low nibbles of its halves; with
// 0x4308 exclusive-ored in they are the bf16 numbers 136 + c, and one bf16x2 multiply-add gives (136 + c) s - 136 s =
// c s. It is exact: 136 s = 17 (8 .. 15) 2^e has 8 bits, c s 7.
//
// What bounds it: reading the cache (0.53 bytes a value, an SM's share of the copy rate 42 values a clock) and, close to
// it, the conversion: about 1.5 instructions a value beside some 0.6 of products, loads and softmax, where an SM issues
// 128 lanes a clock. Layout of the work:
//  - spans of equal key counts per CTA (paged_sched.cuh); a producer warp walks the span and streams K, V (TMA boxes) and
//    their scales (16-byte asynchronous copies) of 128 keys a tile (256 of hd 64) through a ring of stages; four consumer
//    warps, each with a quarter of the tile and a softmax state of its own, which merge through shared memory at a unit's
//    end;
//  - S^T comes out of the product with a key per lane group and rows along lanes; two 8x8 transposes (movmatrix) make
//    the weights the operand of the second product;
//  - lane (g, t) converts for K the 32 values of group t of keys g and g + 8, and for V the 16 columns from 16 g on of four
//    keys: loads of 16 and 8 bytes, a scale byte each. Which key is row k of a product is free: key_of makes both loads
//    meet all banks.
// Measured (8 KV heads of 128, 4 query heads each, pages of 64): 64 requests of 11000 keys 155 us, 0.73 of the copy rate; with
// pages of 16 tokens 176, hd 64 90 (0.63), two requests of 230000 keys 107 (0.69); 16 rows 209. Loading alone
// runs at 0.95 to 1.05 of the copy rate. Per 16 keys a warp issues 306 instructions; 16 operands of four shifts, four logic
// operations, four bf16x2 multiply-adds and a product take 22 to 24 cycles each of a scheduler, as the logic pipe takes one
// instruction in two cycles and the multiply-adds do not quite hide under them: 486 cycles, where HBM would take 372. More
// warps do not change that (7 consumers in each of 2 CTAs 164 us, 15 in one 177), nor do shifts as products on the other
// pipe. Up to four requests of 1000 keys take 10 us a call, start-up of two kernels and the chain over a tile.
#include <cuda_bf16.h>

#include <algorithm>
#include <mutex>

#include "paged_q4.cuh"
#include "paged_tma.cuh"
#include "tc_ptx.cuh"
#include "usp_device.cuh"

namespace usp {
namespace {

// a unit's constant cost, in keys (64 requests of 2000 to 32768 keys with 128, 256, 512, 1024: 155, 154, 156, 161 us; 26 single
// tokens beside chunks 27.4, 25.5, 25.1, 25.1)
constexpr int kOver = 256;
constexpr int kWarps = 4;      // consumers
constexpr int kThreads = (kWarps + 1) * 32;
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr float kRescale = 8.0f;  // log2 units
constexpr float kLn2 = 0.69314718055994531f;

// NT: tiles of 8 query rows; F32: q, out and the weights in three bf16 terms
template <int HD, int NT, bool F32> struct Cfg {
    static constexpr int kTerms = F32 ? 3 : 1;
    static constexpr bool kWide = NT > 1 && !F32;         // see consumer_wide
    static constexpr int kCtas = F32 || NT >= 3 ? 2 : 3;  // per SM, as registers allow (24, 32 rows in three: 117, 146 us for 107, 133)
    static constexpr int kW = HD == 64 && NT == 1 && !F32 ? 4 : 2;  // 16-key steps per warp and tile
    static constexpr int kKT = 16 * kW * kWarps;          // keys per tile
    // Tiles of a segment that O's accumulator takes, a piece, before it is added to a sum in the workspace: 512 products, kWide
    // 1024. They cut their sum to fp32, by half a unit in the last place each on average, always towards zero; the sum of the pieces is
    // rounded. (In one piece, a unit of 2^20 keys in one CTA was off by 0.35% with 8 rows and by 0.6% with 16, where bf16's half
    // step is 0.4%. Pieces of 512 instead of 1024 cost 64 requests of 200000 keys with 16 rows 1.2%.) fp32 adds every tile.
    static constexpr int kPiece = F32 ? 1 << 30 : kWide ? 1024 / (kKT / 16) : 512 / kW;
    // keys per CTA below which fewer CTAs work (one request of 8000 keys with kKT + 1, 64, 128, 320: 17.6, 13.7, 12.3, 12.4 us; four
    // of 2000 11.4, 11.2, 11.7, 11.7)
    static constexpr int kMinSpan = kKT + 128;
    static_assert(kMinSpan > kKT, "a span holds more than a tile");
    static constexpr int kRow = q4_code_bytes(HD), kSRow = q4_scale_bytes(HD);
    static constexpr int kCodes = kKT * kRow, kScales = kKT * kSRow;
    static constexpr int kStages = (NT >= 3 ? 4 : 3) * (kKT * HD == 128 * 128 ? 1 : 2);
    static constexpr int kXRow = HD + 4;                  // exchange row in floats
    static constexpr int kSc = kStages * 2 * kCodes;      // scales, behind all stages' codes (K, V each)
    static constexpr int kX = kSc + kStages * 2 * kScales;  // [warp][row][kXRow]
    static constexpr int kML = kX + (kWide ? 0 : kWarps * NT * 8 * kXRow * 4);
    static constexpr int kQ = kML + kWarps * NT * 8 * 8;  // q's terms as operands: [term][step][row tile][lane]
    static constexpr int kP = kQ + (F32 || kWide ? kTerms * (HD / 16) * NT * 256 : 0);  // kWide: P: [two steps][row tile][lane]
    static constexpr int kVS = kP + (kWide ? kKT / 16 * NT * 256 : 0);  // kWide: V's scales as operands: [warp][step, t]
    static constexpr int kSeg = kVS + (kWide ? kWarps * 256 : 0);
    static constexpr int kBar = kSeg + kSegSlots * (int)sizeof(SegMsg);
    static constexpr int FULL = 0, EMPTY = kStages, SEG_FULL = 2 * kStages, SEG_EMPTY = SEG_FULL + kSegSlots;
    static constexpr int kSmem = kBar + (SEG_EMPTY + kSegSlots) * 8 + 1024;  // + slack for the alignment
    static_assert(kCodes % 1024 == 0, "the swizzle's pattern of 1024 bytes");
};

struct FewParams {
    CUtensorMap tk, tv;
    SchedIn s;
    PartSpace w;
    const void *q;
    const uint8_t *ks, *vs;
    void *out;
    float *lse;
    const int32_t *table;
    int *status;
    int64_t q_stride, out_stride, table_stride, ks_page, vs_page;
    int32_t num_pages, log_ps, hq;
    FastDiv by_sub;  // row groups (heads of the walk) per KV head
    float scale_log2;
    bool second;  // the call's other kernel is in the stream before this one
};

// c += a (16x16, row) * b (16x8, column), bf16 in, fp32 out
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t x;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x) : "r"(a) : "memory");
    return x;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 x;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(x.x), "=r"(x.y) : "r"(a) : "memory");
    return x;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 x;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(a) : "memory");
    return x;
}
__device__ __forceinline__ void sts64(uint32_t a, uint32_t x, uint32_t y) {
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 x) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w) : "memory");
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
    uint32_t x;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(x) : "r"(a) : "memory");
    return x;
}
__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory"); }
__device__ __forceinline__ bool consumers_all(bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
        "bar.red.and.pred p, 1, %2, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x), "n"(kWarps * 32)
        : "memory");
    return r != 0;
}
// x as kTerms bf16 numbers, the first pair of two values (low half: x)
template <int kTerms> __device__ __forceinline__ void split2(float x, float y, uint32_t (&t)[kTerms]) {
#pragma unroll
    for (int i = 0; i < kTerms; ++i) {
        t[i] = float2_to_bf16x2(x, y);
        if (i + 1 < kTerms) {
            const float2 f = bf16x2_to_float2(t[i]);
            x -= f.x;
            y -= f.y;
        }
    }
}

// a whole warp's wait that did not end at once (out of line: the loop has no registers for it)
static __device__ __noinline__ bool wait_longer(uint32_t bar, uint32_t parity, int *status) {
    return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, status, USP_ERR_TIMEOUT, kWaitLimitNs));
}

// The state of a row that the pieces before left in this CTA's slot (m, l and O's N columns from col on) with that of the last
// one (M, L, v).
template <int N>
__device__ __forceinline__ void add_piece(float m, float l, const float *o, float &M, float &L, float (&v)[N]) {
    const float to = fmaxf(M, m), base = to == -INFINITY ? 0.f : to, now = tc::ex2(M - base), was = tc::ex2(m - base);
    M = to;
    L = fmaf(l, was, L * now);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = fmaf(o[i], was, v[i] * now);
}

// The key of a step's 16 that is row k of the products (k < 8; row k + 8: 8 further). hd 128: the keys of K's 16-byte loads
// that meet, rows (k, k + 1), and of V's 8-byte loads, rows (k, k + 2, k + 4, k + 6) with k even, then lie in different banks
// of the swizzled lines; hd 64: rows (k, .., k + 3) of K's 8-byte loads and the same rows of V's 4-byte loads.
template <int HD> __device__ __forceinline__ int key_of(int k) {
    return HD == 128 ? (k & 4) + (((k >> 1) & 1) ^ (3 * (k & 1))) : k ^ ((k >> 2) & 1);
}

// The producer warp: walks the span. Lane b < 2 x pieces loads box b of each tile's codes (K, then V; a page piece each) by
// TMA, and every lane 16-byte pieces of the scales with asynchronous copies: as bulk copies of a page piece each (64 bytes
// where a page has 16 tokens) they took as long to issue as the boxes.
template <int HD, int NT, bool F32>
__device__ void producer(const FewParams &p, const SchedShared &sh, uint8_t *smem, uint32_t sbase) {
    using C = Cfg<HD, NT, F32>;
    const int lane = threadIdx.x & 31;
    auto BAR = [&](int i) { return sbase + C::kBar + 8u * i; };
    auto wait = [&](int bar, uint32_t parity) {
        return __all_sync(0xffffffffu, tc::mbar_try_wait(BAR(bar), parity)) || wait_longer(BAR(bar), parity, p.status);
    };
    SegMsg *ring = reinterpret_cast<SegMsg *>(smem + C::kSeg);
    const int ps = 1 << p.log_ps, piece = min(ps, C::kKT), pieces = C::kKT / piece;  // at most 16 pieces
    const bool v = lane >= pieces, loads = lane < 2 * pieces;
    const int pc = v ? lane - pieces : lane;
    const uint32_t dst0 = sbase + (v ? C::kCodes : 0) + pc * piece * C::kRow;
    // this lane's 16 bytes of K's and V's scales: kCopyKeys keys from its key on
    constexpr int kCopyKeys = 16 / C::kSRow;
    const int skey = lane * kCopyKeys;
    const bool copies = lane < C::kScales / 16;
    Sched sc;
    sched_begin<C::kKT>(p.s, sh, sc);
    PartHeader opened = no_part(sh);
    uint32_t fill = 0, nseg = 0;
    bool ok = true, more = true;
    while (more) {
        Segment g{};
        more = sched_next<C::kKT>(p.s, sc, g);
        const int32_t *row = p.table + (int64_t)g.req * p.table_stride;
        const int kv_head = (int)p.by_sub.div((uint32_t)g.head);
        // The next tile's page numbers are read a tile ahead and looked at only when that tile's stage is free. -1: behind the
        // request's keys.
        auto page_of = [&](int t, int in, bool on) {
            const int key = t * C::kKT + in;
            return on && key < g.kv ? row[key >> p.log_ps] : -1;
        };
        const int mask = ps - 1, row0 = kv_head * ps;
        int32_t raw = -1, sraw = -1;
        if (more) raw = page_of(g.t0, pc * piece, loads), sraw = page_of(g.t0, skey, copies);
        int t = g.t0;
        do {  // a piece
            const int t1 = min(g.t1, t + C::kPiece);
            if (!(ok = wait(C::SEG_EMPTY + nseg % kSegSlots, ((nseg / kSegSlots) & 1u) ^ 1u))) break;
            if (lane == 0) {
                SegMsg m{};
                if (more) {
                    m.tok0 = g.tok0; m.ntok = g.ntok; m.head = g.head; m.req = g.req; m.p0 = g.p0; m.kv = g.kv;
                    m.t0 = t; m.t1 = t1; m.tiles = g.tiles; m.first = g.t0;
                }
                ring[nseg % kSegSlots] = m;
                tc::mbar_arrive(BAR(C::SEG_FULL + nseg % kSegSlots));
            }
            ++nseg;
            if (!more) break;
            for (; t < t1; ++t) {
                const uint32_t st = fill % C::kStages;
                if (!(ok = wait(C::EMPTY + st, ((fill / C::kStages) & 1u) ^ 1u))) break;
                if (lane == 0) tc::mbar_arrive_expect_tx(BAR(C::FULL + st), 2 * C::kCodes);
                __syncwarp();
                // a page outside the cache: a box of zeros, and page 0's scales
                const int32_t page = (uint32_t)raw < (uint32_t)p.num_pages ? raw : p.num_pages;
                const int64_t spage = (uint32_t)sraw < (uint32_t)p.num_pages ? sraw : 0;
                if (loads)
                    tma_load_3d(dst0 + st * 2 * C::kCodes, v ? &p.tv : &p.tk, 0,
                                (row0 + ((t * C::kKT + pc * piece) & mask)) / (128 / C::kRow), page, BAR(C::FULL + st));
                if (copies) {
                    const int at = (row0 + ((t * C::kKT + skey) & mask)) * C::kSRow;
                    const uint32_t dst = sbase + C::kSc + st * 2 * C::kScales + lane * 16;
                    copy16(dst, p.ks + spage * p.ks_page + at);
                    copy16(dst + C::kScales, p.vs + spage * p.vs_page + at);
                }
                copies_arrive(BAR(C::FULL + st));
                raw = page_of(t + 1, pc * piece, loads);
                sraw = page_of(t + 1, skey, copies);
                ++fill;
            }
        } while (ok && t < g.t1);
        if (!ok || !more) break;
        if (g.t0 == 0 && g.t1 < g.tiles) opened = part_header(p.s, sh, sc, g);
    }
    if (!ok) {  // drain (bounded): no copy may land after the CTA has gone
        opened = no_part(sh);
        for (uint32_t f = fill > C::kStages ? fill - C::kStages : 0; f < fill; ++f)
            wait(C::FULL + f % C::kStages, (f / C::kStages) & 1u);
    }
    if (lane == 0) p.w.head[blockIdx.x] = opened;
}

template <int HD, int NT, bool F32> __device__ void consumer(const FewParams &p, uint8_t *smem, uint32_t sbase) {
    using C = Cfg<HD, NT, F32>;
    using T = typename std::conditional<F32, float, __nv_bfloat16>::type;
    constexpr int kMT = HD / 16;  // 16-column tiles of O^T; 16-element steps of the head dim
    constexpr int kT = C::kTerms;
    constexpr int kW = C::kW, kWords = HD / 32;  // K's words of a lane and key; a lane converts 8 kWords values of a key
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    auto BAR = [&](int i) { return sbase + C::kBar + 8u * i; };
    auto wait = [&](int bar, uint32_t parity) {
        return __all_sync(0xffffffffu, tc::mbar_try_wait(BAR(bar), parity)) || wait_longer(BAR(bar), parity, p.status);
    };
    float *xch = reinterpret_cast<float *>(smem + C::kX);
    float2 *ml = reinterpret_cast<float2 *>(smem + C::kML);  // [warp][8 NT rows]
    uint2 *q_s = reinterpret_cast<uint2 *>(smem + C::kQ);
    const Q4Nibbles nib;
    // addresses inside a stage: K's row k = g (and + 8), this lane's values; V's rows 2 t, 2 t + 1 (and + 8), its columns; a
    // step's rows are 16 further
    const int kkey = warp * 16 * kW + key_of<HD>(g);
    const uint32_t k_at = codes_at<HD>(kkey, t * (C::kRow / 4));
    const uint32_t ks_at = kkey * C::kSRow + (HD == 128 ? t : t >> 1);
    // the address of the same codes n keys further (a multiple of 8; no carry reaches the swizzled bits)
    auto further = [](uint32_t at, int n) { return (at ^ ((n * C::kRow >> 3) & 0x70)) + n * C::kRow; };
    uint32_t v_at[2], vs_at[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int key = warp * 16 * kW + key_of<HD>(2 * t + e);
        v_at[e] = C::kCodes + codes_at<HD>(key, g * (C::kRow / 8));
        vs_at[e] = C::kScales + key * C::kSRow + (HD == 128 ? g >> 1 : g >> 2);
    }
    uint32_t st = 0, st_phase = 0;  // the stage of the next tile, and its fill's parity
    for (uint32_t nseg = 0;; ++nseg) {
        // Every warp reaches exactly one consumers_all per segment, also after a failed wait and at the end, and
        // leaves only by its result: so no warp waits for one that has gone.
        bool ok = wait(C::SEG_FULL + nseg % kSegSlots, (nseg / kSegSlots) & 1u);
        SegMsg s;
        s.ntok = 0;
        if (ok) {
            bool never;
            s = read_segment(sbase + C::kSeg + nseg % kSegSlots * (uint32_t)sizeof(SegMsg), never);
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(BAR(C::SEG_EMPTY + nseg % kSegSlots) + (never ? 8u : 0u));
        }
        const int rows = s.ntok * p.s.G;
        // q as the products' second operand: row g of each tile, values 4 step .. + 3 of this lane's
        uint2 qf[F32 ? 1 : kMT][NT];
        if (s.ntok > 0) {
            auto q_row = [&](int r) -> const T * {
                if (r >= rows) return nullptr;
                uint32_t tok, h;
                p.s.by_G.divmod((uint32_t)r, tok, h);
                return static_cast<const T *>(p.q) + (s.tok0 + tok) * p.q_stride + (int64_t)(s.head * p.s.G + (int)h) * HD +
                       t * (8 * kWords);
            };
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const T *q = q_row(n * 8 + g);
                if constexpr (F32) {
                    for (int k = warp; k < kMT; k += kWarps) {
                        const float4 x = q ? *reinterpret_cast<const float4 *>(q + k * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
                        uint32_t a[kT], b[kT];
                        split2(x.x, x.y, a);
                        split2(x.z, x.w, b);
#pragma unroll
                        for (int i = 0; i < kT; ++i) q_s[((i * kMT + k) * NT + n) * 32 + lane] = make_uint2(a[i], b[i]);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < kMT; ++k)
                        qf[k][n] = q ? *reinterpret_cast<const uint2 *>(q + k * 4) : make_uint2(0u, 0u);
                }
            }
        }
        if constexpr (F32) consumers_sync();  // (the end of the segment before has a barrier behind its reads)
        float o[NT][kMT][4], m[NT][2], l[NT][2], nmb[NT][2];  // nmb: -m, or 0 before the first key
        int lim[NT][2];  // keys that this lane's rows 2 t, 2 t + 1 see (rows beyond the valid ones like the last)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < kMT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][i][e] = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[n][e] = -INFINITY;
                l[n][e] = nmb[n][e] = 0.f;
                const int tok = (int)p.s.by_G.div((uint32_t)max(0, min(n * 8 + 2 * t + e, rows - 1)));
                lim[n][e] = p.s.causal ? max(0, min(s.kv, s.p0 + tok + 1)) : s.kv;
            }
        }
        const int lim_all = p.s.causal ? max(0, min(s.kv, s.p0 + 1)) : s.kv;  // keys that every row sees
        const int t1 = s.ntok > 0 ? s.t1 : s.t0;
        for (int kt = s.t0; ok && kt < t1; ++kt) {
            if (!(ok = wait(C::FULL + st, st_phase))) break;
            const uint32_t base = sbase + st * 2 * C::kCodes, sbs = sbase + C::kSc + st * 2 * C::kScales;
            const int key0 = kt * C::kKT + warp * 16 * kW;
            // ---- S^T = K Q^T ----
            float sc[kW][NT][4];
            float low[kW][NT][4];  // F32: of q's second and third terms
#pragma unroll
            for (int i0 = 0; i0 < kW; i0 += 2) {  // two steps at a time: products of two chains in turn, q's terms loaded once
                uint32_t w[2][2][kWords], s2[2][2], off[2][2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t at = base + further(k_at, (i0 + i) * 16 + e * 8);
                        if constexpr (HD == 128) {
                            const uint4 x = lds128(at);
                            w[i][e][0] = x.x; w[i][e][1] = x.y; w[i][e][2] = x.z; w[i][e][3] = x.w;
                        } else {
                            const uint2 x = lds64(at);
                            w[i][e][0] = x.x; w[i][e][1] = x.y;
                        }
                        s2[i][e] = q4_scales2(lds8(sbs + ks_at + ((i0 + i) * 16 + e * 8) * C::kSRow));
                        off[i][e] = q4_minus136(s2[i][e]);
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sc[i0 + i][n][e] = low[i0 + i][n][e] = 0.f;
                }
#pragma unroll
                for (int k = 0; k < kMT; ++k) {
                    uint32_t a[2][4];
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            a[i][e] = nib.values(w[i][e][k / 2], k % 2 * 2, s2[i][e], off[i][e]);
                            a[i][2 + e] = nib.values(w[i][e][k / 2], k % 2 * 2 + 1, s2[i][e], off[i][e]);
                        }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        if constexpr (F32) {
#pragma unroll
                            for (int x = kT - 1; x >= 0; --x) {
                                const uint2 b = lds64(sbase + C::kQ + (((x * kMT + k) * NT + n) * 32 + lane) * 8);
#pragma unroll
                                for (int i = 0; i < 2; ++i) mma16816(x ? low[i0 + i][n] : sc[i0 + i][n], a[i], b.x, b.y);
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 2; ++i) mma16816(sc[i0 + i][n], a[i], qf[k][n].x, qf[k][n].y);
                        }
                    }
                }
            }
            // ---- softmax ----
            uint32_t pf[kW][NT][kT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                // sc: key g rows 2t, 2t+1; key g + 8
                if constexpr (F32)
#pragma unroll
                    for (int i = 0; i < kW; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sc[i][n][e] += low[i][n][e];
                if (key0 + 16 * kW > lim_all) {
                    const int key = key0 + key_of<HD>(g);
#pragma unroll
                    for (int i = 0; i < kW; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (key + i * 16 + (e >> 1) * 8 >= lim[n][e & 1]) sc[i][n][e] = -INFINITY;
                }
                // a row's maximum over its eight lanes is needed only when some lane's own exceeds the bound
                float mx[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    mx[e] = fmaxf(sc[0][n][e], sc[0][n][2 + e]);
#pragma unroll
                    for (int i = 1; i < kW; ++i) mx[e] = tc::max3(mx[e], sc[i][n][e], sc[i][n][2 + e]);
                    mx[e] *= p.scale_log2;
                }
                const bool need = mx[0] > m[n][0] + kRescale || mx[1] > m[n][1] + kRescale;
                if (__any_sync(0xffffffffu, need)) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], d));
                        const float mn = fmaxf(m[n][e], mx[e]);
                        const float a = mn == -INFINITY ? 1.f : tc::ex2(m[n][e] - mn);
                        m[n][e] = mn;
                        nmb[n][e] = mn == -INFINITY ? 0.f : -mn;
                        l[n][e] *= a;
#pragma unroll
                        for (int i = 0; i < kMT; ++i) {
                            o[n][i][e] *= a;
                            o[n][i][2 + e] *= a;
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < kW; ++i) {
                    float x[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float y = fmaf(sc[i][n][e], p.scale_log2, nmb[n][e & 1]);
                        x[e] = F32 ? exp2f(y) : tc::ex2(y);
                    }
                    l[n][0] += x[0] + x[2];
                    l[n][1] += x[1] + x[3];
                    uint32_t lo[kT], hi[kT];
                    split2(x[0], x[1], lo);
                    split2(x[2], x[3], hi);
#pragma unroll
                    for (int c = 0; c < kT; ++c) {
                        pf[i][n][c][0] = transpose8x8(lo[c]);
                        pf[i][n][c][1] = transpose8x8(hi[c]);
                    }
                }
            }
            // ---- O^T += V^T P^T ----
            struct VRows {
                uint32_t w[2][2][kMT / 4], s2[2], off[2];  // [half of the step's keys][pair's element][word]
            };
            auto load_v = [&](int i, VRows &v) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t b[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if constexpr (HD == 128) {
                            const uint2 x = lds64(base + further(v_at[e], i * 16 + h * 8));
                            v.w[h][e][0] = x.x; v.w[h][e][1] = x.y;
                        } else {
                            v.w[h][e][0] = lds32(base + further(v_at[e], i * 16 + h * 8));
                        }
                        b[e] = lds8(sbs + vs_at[e] + (i * 16 + h * 8) * C::kSRow);
                    }
                    v.s2[h] = q4_scales2(b[0], b[1]);
                    v.off[h] = q4_minus136(v.s2[h]);
                }
            };
            // columns 2 j, 2 j + 1 of word x: the even and the odd columns of 8 are four codes of either key of a pair
            auto operand = [&](const VRows &v, int x, int j, uint32_t (&a)[4]) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    a[2 * h] = nib.values(__byte_perm(v.w[h][0][x], v.w[h][1][x], 0x5410), j, v.s2[h], v.off[h]);
                    a[2 * h + 1] = nib.values(__byte_perm(v.w[h][0][x], v.w[h][1][x], 0x7632), j, v.s2[h], v.off[h]);
                }
            };
            if constexpr (F32) {
                // a tile's sum on its own: the products' accumulation truncates, which over a thousand tiles would show
                VRows v[kW];
#pragma unroll
                for (int i = 0; i < kW; ++i) load_v(i, v[i]);
#pragma unroll
                for (int x = 0; x < kMT; ++x) {
                    float sum[NT][4] = {};
#pragma unroll
                    for (int i = 0; i < kW; ++i) {
                        uint32_t a[4];
                        operand(v[i], x / 4, x % 4, a);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int c = kT - 1; c >= 0; --c) mma16816(sum[n], a, pf[i][n][c][0], pf[i][n][c][1]);
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[n][x][e] += sum[n][e];
                }
            } else {
#pragma unroll
                for (int i = 0; i < kW; ++i) {
                    VRows v;
                    load_v(i, v);
#pragma unroll
                    for (int x = 0; x < kMT; ++x) {
                        uint32_t a[4];
                        operand(v, x / 4, x % 4, a);
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma16816(o[n][x], a, pf[i][n][0][0], pf[i][n][0][1]);
                    }
                }
            }
            // The stage is released only when its rows have arrived in registers (see paged_decode.cu): the arrive's
            // address depends on a result of every product of V. Their bits' conjunction is this NaN only if each is a NaN
            // and not all the one that products give.
            uint32_t all = 0xffffffffu;
#pragma unroll
            for (int i = 0; i < kMT; ++i) all &= __float_as_uint(o[0][i][0]);
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(BAR(C::EMPTY + st) + (all == 0x7fa5a5a5u ? 8u : 0u));
            if (++st == C::kStages) {
                st = 0;
                st_phase ^= 1u;
            }
        }
        // ---- merge the warps' states and write the rows ----
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], d);
                if (g == 0) ml[(warp * NT + n) * 8 + 2 * t + e] = make_float2(m[n][e], l[n][e]);
            }
        if (!consumers_all(ok) || s.ntok == 0) return;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float mm = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, ml[(w * NT + n) * 8 + 2 * t + e].x);
                const float a = mm == -INFINITY ? 0.f : tc::ex2(m[n][e] - mm);
                float *d = xch + ((warp * NT + n) * 8 + 2 * t + e) * C::kXRow + g * (HD / 8);
#pragma unroll
                for (int i = 0; i < kMT; i += 2)  // columns 2 i .. 2 i + 3 of the lane's
                    *reinterpret_cast<float4 *>(d + 2 * i) = make_float4(o[n][i][e] * a, o[n][i][2 + e] * a, o[n][i + 1][e] * a,
                                                                         o[n][i + 1][2 + e] * a);
            }
        consumers_sync();
        const bool whole = s.first == 0 && s.t1 == s.tiles;
        float *slot = part_slot(p.w, HD, blockIdx.x, s.first == 0 ? 1 : 0);
        constexpr int kLanes = HD / 4, kAtOnce = kWarps * 32 / kLanes;  // threads of a row, 4 columns each
        const int col = tid % kLanes * 4;
        for (int r = tid / kLanes; r < rows; r += kAtOnce) {
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[w * NT * 8 + r].x);
            const float Mb = M == -INFINITY ? 0.f : M;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float2 x = ml[w * NT * 8 + r];
                L = fmaf(x.y, tc::ex2(x.x - Mb), L);
                const float4 f = *reinterpret_cast<const float4 *>(xch + (w * NT * 8 + r) * C::kXRow + col);
                v.x += f.x; v.y += f.y; v.z += f.z; v.w += f.w;
            }
            if (!F32 && s.t0 != s.first) {
                const float was_m = slot[(size_t)p.w.rows * HD + r], was_l = slot[(size_t)p.w.rows * (HD + 1) + r];
                __syncwarp(kLanes == 32 ? 0xffffffffu : 0xffffu << (lane & 16));  // (the row's threads, one of which writes these anew)
                float x[4] = {v.x, v.y, v.z, v.w};
                add_piece(was_m, was_l, slot + (size_t)r * HD + col, M, L, x);
                v = make_float4(x[0], x[1], x[2], x[3]);
            }
            uint32_t tok, h;
            p.s.by_G.divmod((uint32_t)r, tok, h);
            const int head = s.head * p.s.G + (int)h;
            if (whole) {
                const float inv = L == 0.f ? 1.f : 1.f / L;
                T *to = static_cast<T *>(p.out) + (s.tok0 + tok) * p.out_stride + (int64_t)head * HD + col;
                if constexpr (F32)
                    *reinterpret_cast<float4 *>(to) = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
                else
                    *reinterpret_cast<uint2 *>(to) =
                        make_uint2(float2_to_bf16x2(v.x * inv, v.y * inv), float2_to_bf16x2(v.z * inv, v.w * inv));
                if (col == 0)
                    p.lse[(s.tok0 + tok) * p.hq + head] =
                        L == 0.f ? -INFINITY : (M + (F32 ? log2f(L) : __log2f(L))) * kLn2;
            } else {
                *reinterpret_cast<float4 *>(slot + (size_t)r * HD + col) = v;
                if (col == 0) {
                    slot[(size_t)p.w.rows * HD + r] = M;
                    slot[(size_t)p.w.rows * (HD + 1) + r] = L;
                }
            }
        }
        consumers_sync();  // xch, ml and q_s are free for the next segment
    }
}

// Units of 9 to 32 rows (bf16). A warp takes a quarter of the tile's keys for S^T, as above, but a quarter of the head's
// columns, over all of the tile's keys, for O^T: so it holds O of 32 rows in the registers of one row tile, no value of the cache
// is converted twice, and there is one softmax state: the weights go through shared memory. Two barriers a tile: where a
// maximum has to move (one for all warps), and before the weights are read. Measured: 32 requests of 8000 keys, 16, 24, 32 rows 87, 107,
// 133 us, hd 64 61, 78, 91 (with the division above 16 rows take 97 and spill); for 8 rows the barriers cost more than the
// smaller O gives (64 requests of 11000 keys 173 us, the division above 155).
template <int HD, int NT> __device__ void consumer_wide(const FewParams &p, uint8_t *smem, uint32_t sbase) {
    using C = Cfg<HD, NT, false>;
    constexpr int kMT = HD / 16, kX = HD / 64;  // 16-element steps of the head dim; this warp's 16-column tiles of O^T
    constexpr int kW = C::kW, kWords = HD / 32;
    static_assert(kW == 2, "four score pairs a row tile");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    auto BAR = [&](int i) { return sbase + C::kBar + 8u * i; };
    auto wait = [&](int bar, uint32_t parity) {
        return __all_sync(0xffffffffu, tc::mbar_try_wait(BAR(bar), parity)) || wait_longer(BAR(bar), parity, p.status);
    };
    float *wm = reinterpret_cast<float *>(smem + C::kML), *wl = wm + kWarps * NT * 8;  // [warp][row]: maxima, sums
    const Q4Nibbles nib;
    const int kkey = warp * 16 * kW + key_of<HD>(g);
    const uint32_t k_at = codes_at<HD>(kkey, t * (C::kRow / 4));
    const uint32_t ks_at = kkey * C::kSRow + (HD == 128 ? t : t >> 1);
    auto further = [](uint32_t at, int n) { return (at ^ ((n * C::kRow >> 3) & 0x70)) + n * C::kRow; };
    // V's rows 2 t, 2 t + 1 (and + 8) of a step: the word with this lane's columns. Of the 8 columns of a word it has the even
    // or the odd ones (hd 64: two of these)
    uint32_t v_at[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
        v_at[e] = C::kCodes + codes_at<HD>(key_of<HD>(2 * t + e), warp * (C::kRow / 4) + (HD == 128 ? g >> 1 : g >> 2) * 4);
    // V's scales: the warp's columns are of one group, so a pair of keys has one operand; lane 4 i + t makes those of step i's
    // rows 2 t, 2 t + 1 (and + 8)
    const uint32_t my_vs = sbase + C::kVS + warp * 256;
    uint32_t vs_at[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
        vs_at[e] = C::kScales + (g * 16 + key_of<HD>(2 * t + e)) * C::kSRow + (HD == 128 ? warp : warp >> 1);
    const uint32_t half = g & 1 ? 0x7632u : 0x5410u;
    const int v_shift = HD == 128 ? 0 : (g >> 1 & 1) * 8;
    uint32_t st = 0, st_phase = 0;  // the stage of the next tile, and its fill's parity
    for (uint32_t nseg = 0;; ++nseg) {
        bool ok = wait(C::SEG_FULL + nseg % kSegSlots, (nseg / kSegSlots) & 1u);
        SegMsg s;
        s.ntok = 0;
        if (ok) {
            bool never;
            s = read_segment(sbase + C::kSeg + nseg % kSegSlots * (uint32_t)sizeof(SegMsg), never);
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(BAR(C::SEG_EMPTY + nseg % kSegSlots) + (never ? 8u : 0u));
        }
        const int rows = s.ntok * p.s.G;
        if (s.ntok > 0) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int r = n * 8 + g;
                const __nv_bfloat16 *q = nullptr;
                if (r < rows) {
                    uint32_t tok, h;
                    p.s.by_G.divmod((uint32_t)r, tok, h);
                    q = static_cast<const __nv_bfloat16 *>(p.q) + (s.tok0 + tok) * p.q_stride +
                        (int64_t)(s.head * p.s.G + (int)h) * HD + t * (8 * kWords);
                }
                for (int k = warp; k < kMT / 2; k += kWarps)  // two steps of the head dim
                    sts128(sbase + C::kQ + ((k * NT + n) * 32 + lane) * 16,
                           q ? *reinterpret_cast<const uint4 *>(q + k * 8) : make_uint4(0u, 0u, 0u, 0u));
            }
        }
        // The barriers of the tiles need all warps: a failed wait ends the segment for all of them here or at a tile's first
        ok = consumers_all(ok);
        float o[NT][kX][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int x = 0; x < kX; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][x][e] = 0.f;
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.f;
        }
        const int lim_all = p.s.causal ? max(0, min(s.kv, s.p0 + 1)) : s.kv;  // keys that every row sees
        const int t1 = s.ntok > 0 ? s.t1 : s.t0;
        for (int kt = s.t0; ok && kt < t1; ++kt) {
            ok = wait(C::FULL + st, st_phase);
            const uint32_t base = sbase + st * 2 * C::kCodes, sbs = sbase + C::kSc + st * 2 * C::kScales;
            const int key0 = kt * C::kKT + warp * 16 * kW;
            {
                uint32_t b[2][2];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 2; ++e) b[h][e] = lds8(sbs + vs_at[e] + h * 8 * C::kSRow);
                sts64(my_vs + lane * 8, q4_scales2(b[0][0], b[0][1]), q4_scales2(b[1][0], b[1][1]));
            }
            // ---- S^T = K Q^T ----
            float sc[kW][NT][4];
            uint32_t w[kW][2][kWords], s2[kW][2], off[kW][2];
#pragma unroll
            for (int i = 0; i < kW; ++i) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t at = base + further(k_at, i * 16 + e * 8);
                    if constexpr (HD == 128) {
                        const uint4 x = lds128(at);
                        w[i][e][0] = x.x; w[i][e][1] = x.y; w[i][e][2] = x.z; w[i][e][3] = x.w;
                    } else {
                        const uint2 x = lds64(at);
                        w[i][e][0] = x.x; w[i][e][1] = x.y;
                    }
                    s2[i][e] = q4_scales2(lds8(sbs + ks_at + (i * 16 + e * 8) * C::kSRow));
                    off[i][e] = q4_minus136(s2[i][e]);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[i][n][e] = 0.f;
            }
#pragma unroll
            for (int k = 0; k < kMT / 2; ++k) {
                uint32_t a[2][kW][4];
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int i = 0; i < kW; ++i)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            a[j][i][e] = nib.values(w[i][e][k], 2 * j, s2[i][e], off[i][e]);
                            a[j][i][2 + e] = nib.values(w[i][e][k], 2 * j + 1, s2[i][e], off[i][e]);
                        }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint4 b = lds128(sbase + C::kQ + ((k * NT + n) * 32 + lane) * 16);
#pragma unroll
                    for (int i = 0; i < kW; ++i) mma16816(sc[i][n], a[0][i], b.x, b.y);
#pragma unroll
                    for (int i = 0; i < kW; ++i) mma16816(sc[i][n], a[1][i], b.z, b.w);
                }
            }
            // ---- softmax ----
            bool need = !ok;
            float mx[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (key0 + 16 * kW > lim_all) {
                    const int key = key0 + key_of<HD>(g);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int tok = (int)p.s.by_G.div((uint32_t)max(0, min(n * 8 + 2 * t + e, rows - 1)));
                        const int lim = p.s.causal ? max(0, min(s.kv, s.p0 + tok + 1)) : s.kv;
#pragma unroll
                        for (int i = 0; i < kW; ++i)
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                if (key + i * 16 + h * 8 >= lim) sc[i][n][2 * h + e] = -INFINITY;
                    }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    mx[n][e] = fmaxf(tc::max3(sc[0][n][e], sc[0][n][2 + e], sc[1][n][e]), sc[1][n][2 + e]) * p.scale_log2;
                    need |= mx[n][e] > m[n][e] + kRescale;
                }
            }
            if (!consumers_all(!need)) {  // (the same for all warps)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) mx[n][e] = fmaxf(mx[n][e], __shfl_xor_sync(0xffffffffu, mx[n][e], d));
                        if (g == 0) wm[(warp * NT + n) * 8 + 2 * t + e] = mx[n][e];
                    }
                if (!(ok = consumers_all(ok))) break;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mn = m[n][e];
#pragma unroll
                        for (int x = 0; x < kWarps; ++x) mn = fmaxf(mn, wm[(x * NT + n) * 8 + 2 * t + e]);
                        const float a = mn == -INFINITY ? 1.f : tc::ex2(m[n][e] - mn);
                        m[n][e] = mn;
                        l[n][e] *= a;
#pragma unroll
                        for (int x = 0; x < kX; ++x) {
                            o[n][x][e] *= a;
                            o[n][x][2 + e] *= a;
                        }
                    }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float nmb[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) nmb[e] = m[n][e] == -INFINITY ? 0.f : -m[n][e];
                uint32_t pt[kW][2];
#pragma unroll
                for (int i = 0; i < kW; ++i) {
                    float x[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = tc::ex2(fmaf(sc[i][n][e], p.scale_log2, nmb[e & 1]));
                    l[n][0] += x[0] + x[2];
                    l[n][1] += x[1] + x[3];
                    pt[i][0] = transpose8x8(float2_to_bf16x2(x[0], x[1]));
                    pt[i][1] = transpose8x8(float2_to_bf16x2(x[2], x[3]));
                }
                sts128(sbase + C::kP + ((warp * NT + n) * 32 + lane) * 16, make_uint4(pt[0][0], pt[0][1], pt[1][0], pt[1][1]));
            }
            consumers_sync();
            // ---- O^T += V^T P^T ----
#pragma unroll
            for (int j = 0; j < C::kKT / 32; ++j) {
                uint32_t a[2][kX][4];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint2 v2 = lds64(my_vs + (2 * j + i) * 32 + t * 8);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t v[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) v[e] = lds32(base + further(v_at[e], (2 * j + i) * 16 + h * 8));
                        const uint32_t vs2 = h ? v2.y : v2.x, voff = q4_minus136(vs2);
                        const uint32_t word = __byte_perm(v[0], v[1], half) >> v_shift;
#pragma unroll
                        for (int x = 0; x < kX; ++x) {
                            a[i][x][2 * h] = nib.values(word, 2 * x, vs2, voff);
                            a[i][x][2 * h + 1] = nib.values(word, 2 * x + 1, vs2, voff);
                        }
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint4 b = lds128(sbase + C::kP + ((j * NT + n) * 32 + lane) * 16);
#pragma unroll
                    for (int x = 0; x < kX; ++x) mma16816(o[n][x], a[0][x], b.x, b.y);
#pragma unroll
                    for (int x = 0; x < kX; ++x) mma16816(o[n][x], a[1][x], b.z, b.w);
                }
            }
            // (as above)
            uint32_t all = 0xffffffffu;
#pragma unroll
            for (int x = 0; x < kX; ++x) all &= __float_as_uint(o[0][x][0]);
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(BAR(C::EMPTY + st) + (all == 0x7fa5a5a5u ? 8u : 0u));
            if (++st == C::kStages) {
                st = 0;
                st_phase ^= 1u;
            }
        }
        // ---- the rows' sums, and the rows ----
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], d);
                if (g == 0) wl[(warp * NT + n) * 8 + 2 * t + e] = l[n][e];
            }
        if (!consumers_all(ok) || s.ntok == 0) return;
        const bool whole = s.first == 0 && s.t1 == s.tiles;
        float *slot = part_slot(p.w, HD, blockIdx.x, s.first == 0 ? 1 : 0);
        const bool more = s.t0 != s.first;  // pieces before: their m and l, which warp 0 writes anew
        if (more) {
            for (int i = tid; i < 2 * p.w.rows; i += kWarps * 32) wm[i] = slot[(size_t)p.w.rows * HD + i];
            consumers_sync();
        }
        // the lane's columns after the exchange of even and odd ones with its neighbour: 2 kX in a row
        const int col = warp * (HD / 4) + (HD == 128 ? (g >> 1) * 8 + (g & 1) * 4 : (g >> 2) * 8 + (g >> 1 & 1) * 4 + (g & 1) * 2);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = n * 8 + 2 * t + e;
                float L = 0.f;
#pragma unroll
                for (int x = 0; x < kWarps; ++x) L += wl[(x * NT + n) * 8 + 2 * t + e];
                float v[2 * kX], y[2 * kX];
#pragma unroll
                for (int x = 0; x < kX; ++x) v[2 * x] = o[n][x][e], v[2 * x + 1] = o[n][x][2 + e];
#pragma unroll
                for (int j = 0; j < kX; ++j) {  // an even lane gives its upper half for the other's lower one
                    const float got = __shfl_xor_sync(0xffffffffu, g & 1 ? v[j] : v[kX + j], 4);
                    y[2 * j] = g & 1 ? got : v[j];
                    y[2 * j + 1] = g & 1 ? v[kX + j] : got;
                }
                if (r >= rows) continue;
                float M = m[n][e];
                if (more) add_piece(wm[r], wm[p.w.rows + r], slot + (size_t)r * HD + col, M, L, y);
                uint32_t tok, h;
                p.s.by_G.divmod((uint32_t)r, tok, h);
                const int head = s.head * p.s.G + (int)h;
                if (whole) {
                    const float inv = L == 0.f ? 1.f : 1.f / L;
                    __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(p.out) + (s.tok0 + tok) * p.out_stride + (int64_t)head * HD + col;
                    uint32_t z[kX];
#pragma unroll
                    for (int j = 0; j < kX; ++j) z[j] = float2_to_bf16x2(y[2 * j] * inv, y[2 * j + 1] * inv);
                    if constexpr (kX == 2) *reinterpret_cast<uint2 *>(to) = make_uint2(z[0], z[1]);
                    else *reinterpret_cast<uint32_t *>(to) = z[0];
                    if (warp == 0 && g == 0)
                        p.lse[(s.tok0 + tok) * p.hq + head] = L == 0.f ? -INFINITY : (M + __log2f(L)) * kLn2;
                } else {
                    float *to = slot + (size_t)r * HD + col;
                    if constexpr (kX == 2) *reinterpret_cast<float4 *>(to) = make_float4(y[0], y[1], y[2], y[3]);
                    else *reinterpret_cast<float2 *>(to) = make_float2(y[0], y[1]);
                    if (warp == 0 && g == 0) {
                        slot[(size_t)p.w.rows * HD + r] = M;
                        slot[(size_t)p.w.rows * (HD + 1) + r] = L;
                    }
                }
            }
    }
}

template <int HD, int NT, bool F32>
__global__ void __launch_bounds__(kThreads, (Cfg<HD, NT, F32>::kCtas)) paged_q4_few_kernel(const __grid_constant__ FewParams p) {
    using C = Cfg<HD, NT, F32>;
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
            tc::mbar_init(bar + 8 * (C::FULL + i), 33);  // the boxes' bytes, and each lane's copies
            tc::mbar_init(bar + 8 * (C::EMPTY + i), kWarps);
        }
        for (int i = 0; i < kSegSlots; ++i) {
            tc::mbar_init(bar + 8 * (C::SEG_FULL + i), 1);
            tc::mbar_init(bar + 8 * (C::SEG_EMPTY + i), kWarps);
        }
        tc::fence_barrier_init();
    }
    begin_in_order(p.second);
    // a bounded wait of an earlier kernel ran out: do no work until usp_check clears it
    if (threadIdx.x == 0) skip = *reinterpret_cast<volatile int *>(p.status) != 0;
    const bool work = sched_scan<kThreads, C::kKT>(p.s, sh);
    __syncthreads();
    if (!work || skip) {
        if (threadIdx.x == 0) p.w.head[blockIdx.x] = no_part(sh);
    } else if ((threadIdx.x >> 5) == kWarps) {
        producer<HD, NT, F32>(p, sh, smem, sbase);
    } else {
        if constexpr (C::kWide) consumer_wide<HD, NT>(p, smem, sbase);
        else consumer<HD, NT, F32>(p, smem, sbase);
    }
    end_in_order(p.second);
}

template <int HD, int NT, bool F32> int launch_typed(FewParams &p, cudaStream_t s) {
    using C = Cfg<HD, NT, F32>;
    static_assert(C::kSmem + 2048 <= (228 / C::kCtas - 1) * 1024, "shared memory per CTA");
    static std::mutex mu;
    static bool attr_set[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return USP_ERR_CUDA;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (dev < 0 || dev >= 64) return USP_ERR_UNSUPPORTED;
        if (!attr_set[dev]) {
            if (cudaFuncSetAttribute(paged_q4_few_kernel<HD, NT, F32>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) !=
                cudaSuccess)
                return USP_ERR_CUDA;
            attr_set[dev] = true;
        }
    }
    p.s.min_span = C::kMinSpan;
    return launch_overlapped(paged_q4_few_kernel<HD, NT, F32>, dim3((unsigned)p.w.ctas), kThreads, C::kSmem, s, p);
}

}  // namespace

int q4_few_ctas(int sms, int rows, int dtype) {
    return (dtype == USP_BF16 ? rows > 16 ? Cfg<128, 3, false>::kCtas : Cfg<128, 1, false>::kCtas : Cfg<128, 1, true>::kCtas) * sms;
}

int launch_paged_q4_few(const PagedQ4Args &a, int G, int rows, int n_hi, bool second, const PartSpace &w, cudaStream_t s) {
    const DeviceInfo *di = device_info();
    if (!di) return USP_ERR_CUDA;
    FewParams p{};
    const int ps = 1 << a.log_ps;
    const bool f32 = a.dtype == USP_F32;
    const int tile = a.hd == 128 || rows > 8 || f32 ? Cfg<128, 1, false>::kKT : Cfg<64, 1, false>::kKT;
    const uint32_t box = (uint32_t)std::min(ps, tile);
    if (!make_codes_tmap(&p.tk, a.k, a.num_pages, a.k_page, a.hkv, ps, a.hd, box) ||
        !make_codes_tmap(&p.tv, a.v, a.num_pages, a.v_page, a.hkv, ps, a.hd, box))
        return USP_ERR_CUDA;
    p.s.cu = a.cu; p.s.kv = a.kv;
    p.s.tokens = a.tokens; p.s.max_keys = q4_max_keys(a);
    p.s.nreq = a.nreq; p.s.hkv = a.hq / G; p.s.G = G;
    p.s.tb = rows / G; p.s.causal = a.causal;
    p.s.n_lo = 0; p.s.n_hi = n_hi;
    p.s.over = kOver; p.s.long_parts = kFewParts;
    p.s.inv_ctas = 1.0f / (float)w.ctas;
    p.s.by_tb = FastDiv((uint32_t)p.s.tb); p.s.by_G = FastDiv((uint32_t)G);
    p.by_sub = FastDiv((uint32_t)(a.G / G));
    p.w = w;
    p.q = a.q; p.out = a.out; p.lse = a.lse;
    p.ks = a.ks; p.vs = a.vs; p.ks_page = a.ks_page; p.vs_page = a.vs_page;
    p.table = a.table;
    p.status = di->status;
    p.q_stride = a.q_stride; p.out_stride = a.out_stride; p.table_stride = a.table_stride;
    p.num_pages = (int32_t)a.num_pages; p.log_ps = a.log_ps; p.hq = a.hq;
    p.scale_log2 = a.scale_log2;
    p.second = second;
    auto go = [&](auto hd, auto nt, auto f32) {
        return launch_typed<decltype(hd)::value, decltype(nt)::value, decltype(f32)::value>(p, s);
    };
    auto with = [&](auto hd) {
        using One = std::integral_constant<int, 1>;
        using Two = std::integral_constant<int, 2>;
        using Three = std::integral_constant<int, 3>;
        using Four = std::integral_constant<int, 4>;
        if (f32) return rows == 8 ? go(hd, One{}, std::true_type{}) : go(hd, Two{}, std::true_type{});
        return rows == 8 ? go(hd, One{}, std::false_type{}) : rows == 16 ? go(hd, Two{}, std::false_type{})
               : rows == 24 ? go(hd, Three{}, std::false_type{}) : go(hd, Four{}, std::false_type{});
    };
    return a.hd == 128 ? with(std::integral_constant<int, 128>{}) : with(std::integral_constant<int, 64>{});
}

}  // namespace usp
