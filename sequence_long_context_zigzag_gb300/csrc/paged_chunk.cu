// paged_chunk.cu -- bf16 attention of many query rows per KV head over the paged cache, bf16 or 4-bit, on the
// 5th-generation tensor cores (sm_103a): chunks of a prompt, whole prompts.
//
// Mathematics: as paged_decode.cu (online softmax, lazy rescale). A unit is two tiles of up to 128 query
// rows of one request and KV head: a tile packs TQ = 128 / G tokens x the G query heads of the KV head,
// so grouped heads share every K/V tile that is loaded, and a chunk of 128 / G tokens fills a tile.
//
// What bounds it: from about 290 rows per KV head on, the tensor cores and the exponentials (the
// unit's two tiles keep both busy in turn); below that, HBM. Roles of a CTA (one per SM), which run through
// the CTA's span of the work (paged_sched.cuh) without a CTA-wide barrier:
//   warps 0-3, 4-7  softmax of Q tile 0 / 1, one thread per query row: S from tensor memory, mask, running
//                   maximum, P = 2^(S scale log2(e) - m) as bf16 back over S (the A operand of P V), rescale
//                   of O when the maximum grows by more than 2^8; at a segment's end out and lse, or the
//                   fp32 partial of a cut unit;
//   warp 8          TMA: Q per segment (a box of 64 columns x G heads x TQ tokens), K and V tiles of 128 keys
//                   through a ring of stages, one box of a page per lane, page numbers read ahead;
//   warps 9, 10     one MMA issuer per Q tile: S_i = Q_i K^T, O_i += P_i V, taking turns so that one tile's
//                   products run under the other tile's softmax;
//   warp 11         walks the span and hands its segments to the other roles through a ring; with 8-10 it
//                   is the warpgroup that gives registers to the softmax (setmaxnreg). Rows of the last page
//                   behind the request's last key may hold NaN, and 0 x NaN would spread in P V: this warp
//                   clears them in V's stage before the issuers see it.
// Measured, whole calls (8 KV heads of 128, 4 query heads each): 900 tokens over 64000 keys 587 to 600 us, 1580 to
// 1617 TFLOP/s of a measured 1939 for cuBLAS (power-capped: 1748 sustained); 6 prompts of 1500 to 4100 tokens 309 to 314 us,
// 1210 to 1230; a prompt of 16384 tokens 1310 to 1340 us, 1640 to 1680. Below a full tile, 32 requests of 8000 keys (1.06
// GB): 64 rows per KV head 174 to 176 us, 128 rows 179 to 181, 0.91 and 0.89 of the copy rate; 256 rows 213 to 225, 1200
// to 1260 TFLOP/s. A pair of tiles takes about 2750 cycles (its products 2050: each Q tile is one chain of
// products, softmax, products), a unit's end about 6000 more (last products, read-out of O, both Q tiles in step again).
//   TMEM: S0 [0,128) S1 [128,256) O0 [256,256+hd) O1 [256+hd,256+2hd); P_i lies over S_i.
//
// Over a 4-bit cache (Q4) the producer loads codes and scales into a small ring of tiles, and four more warps (12-15), a
// thread per key, convert them into the stages: c s is exact in bf16, so all else is as for a bf16 cache. A tile is
// converted anew for every unit that reads it: 400 instructions a thread for K and V in the 2750 cycles that a pair of
// tiles takes the other roles, where converting the cache once into memory would need that memory, and 13% of the time of
// a chunk of 900 tokens. Rows behind the last key need no clearing: whatever their bytes, they stand for finite numbers.
//   Where a unit's rows fit one Q tile, reading is four times as fast as over a bf16 cache, and one chain of products,
// softmax, products per key tile would bound the kernel: such a segment is split, both Q tiles being the same rows, each
// for every other key tile. At its end the second one's state goes through a scratch in the workspace to the first one's
// threads, which join the two (32 requests of 8000 keys, 20 rows by this kernel: 178 us, split 150).
//   Measured (8 KV heads of 128, 4 query heads each): 1000 tokens over 48000 keys 495 to 525 us (1510 to 1600 TFLOP/s; over a bf16
// cache 437), a prompt of 16384 tokens 1437 to 1450 (1182 to 1266); 32 requests of 8000 keys with 9, 16, 64 tokens each 153,
// 155, 199 us. The converting warps take a tenth of a long chunk. Below a tile of rows both the chain of a tile and
// the conversion, which waits for its own loads and stores, take about as long (20 rows without any conversion 142 us, 121
// with five slots of codes instead of two).
#include <cuda_bf16.h>

#include <algorithm>
#include <mutex>

#include "paged_q4.cuh"
#include "paged_tma.cuh"
#include "tc_ptx.cuh"
#include "usp_device.cuh"

namespace usp {
namespace {

constexpr int kM = 128;  // rows of a Q tile
constexpr int kN = 128;  // keys of a tile
constexpr int kSoftmaxWarps = 8;
template <bool Q4> constexpr int kWarps = kSoftmaxWarps + (Q4 ? 8 : 4);
template <bool Q4> constexpr int kThreads = kWarps<Q4> * 32;
constexpr int kProducerWarp = kSoftmaxWarps;
constexpr int kMmaWarp = kSoftmaxWarps + 1;  // Q tile 0's issuer (tile 1's follows); allocates and frees tensor memory
constexpr int kWalkWarp = kSoftmaxWarps + 3;
constexpr int kConvertWarp = kSoftmaxWarps + 4;  // the first of four (Q4)
template <bool Q4> constexpr int kSegReaders = kSoftmaxWarps + 3 + (Q4 ? 4 : 0);  // the softmax warps, the producer, the issuers, the converters
// the warpgroups' shares (setmaxnreg) add up to exactly the launch's registers
template <bool Q4> constexpr int kLaunchRegs = (65536 / kThreads<Q4>) / 8 * 8;
template <bool Q4> constexpr int kSoftmaxRegs = Q4 ? 192 : 208;
template <bool Q4> constexpr int kConvertRegs = Q4 ? 64 : 0;
template <bool Q4> constexpr int kControlRegs = kLaunchRegs<Q4> * kWarps<Q4> / 4 - 2 * kSoftmaxRegs<Q4> - kConvertRegs<Q4>;
template <bool Q4>
constexpr bool split_ok = kControlRegs<Q4> >= 24 && kControlRegs<Q4> % 8 == 0 &&
                          2 * kSoftmaxRegs<Q4> + kControlRegs<Q4> + kConvertRegs<Q4> == kLaunchRegs<Q4> * kWarps<Q4> / 4;
static_assert(split_ok<false> && split_ok<true>, "register split must use exactly the launch's registers");
constexpr int kOver = 192;     // a unit's constant cost, in keys
constexpr int kMinSpan = 448;  // keys per CTA below which fewer CTAs work
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr float kRescale = 8.0f;  // log2 units
// Tiles of a segment that O takes in tensor memory, a piece, before it is added to a sum in the workspace (the slot that a cut
// unit's part goes to). The products cut their sums to fp32, always towards zero; the sum of the pieces is rounded. (In one piece,
// 2^20 keys of a unit in one CTA were off by 0.45%, over a 4-bit cache by 0.26%, where bf16's half step is 0.4%. 60 requests of
// 300000 keys with 9 tokens each take 2% longer so, 64 tokens 1%.)
constexpr int kPiece = 512;
constexpr float kLn2 = 0.69314718055994531f;

template <int HD, bool Q4> struct Cfg {
    static constexpr int kBoxes = HD / 64;
    static constexpr int kBoxBytes = kM * 128;
    static constexpr int kTileBytes = kM * HD * 2;
    static constexpr int kStages = HD == 128 ? 2 : 4;
    static constexpr int kQ = 0;
    static constexpr int kK = kQ + 2 * kTileBytes;
    static constexpr int kV = kK + kStages * kTileBytes;
    // tiles of codes and scales (K, V, K, V, ..), codes 1024-byte aligned
    static constexpr int kSlots = Q4 ? (HD == 128 ? 2 : 6) : 0;
    static constexpr int kCodes = kN * q4_code_bytes(HD), kScales = kN * q4_scale_bytes(HD);
    static constexpr int kQ4 = kV + kStages * kTileBytes;
    static constexpr int kQ4Scales = kQ4 + kSlots * kCodes;
    // a staging slot per softmax warp for its stores: 32 rows x 128 bytes (1024-byte aligned: a swizzled box), 32 bytes where
    // the slots of codes leave no more (16-byte stores straight from registers cost a unit's end 7 us)
    static constexpr int kStgRow = Q4 && HD == 128 ? 32 : 128;
    static constexpr int kStgSlot = 32 * kStgRow;
    static constexpr int kStg = (kQ4Scales + kSlots * kScales + 1023) / 1024 * 1024;
    static constexpr int kBar = kStg + kSoftmaxWarps * kStgSlot;
    static constexpr int Q_FULL = 0;
    static constexpr int K_FULL = 1;
    static constexpr int K_EMPTY = K_FULL + kStages;
    static constexpr int V_FULL = K_EMPTY + kStages;
    static constexpr int V_EMPTY = V_FULL + kStages;
    static constexpr int S_FULL = V_EMPTY + kStages;  // [2]
    static constexpr int P_FULL = S_FULL + 2;         // [2]
    static constexpr int O_FULL = P_FULL + 2;         // [2]
    static constexpr int DONE = O_FULL + 2;           // [2]
    static constexpr int TURN = DONE + 2;             // [2]
    static constexpr int Q_EMPTY = TURN + 2;
    static constexpr int O_EMPTY = Q_EMPTY + 1;       // [2]
    static constexpr int SEG_FULL = O_EMPTY + 2;      // [kSegSlots]
    static constexpr int SEG_EMPTY = SEG_FULL + kSegSlots;
    static constexpr int TAIL = SEG_EMPTY + kSegSlots;  // [2]: V tiles that the walk warp has to clear the end of
    static constexpr int P_HALF = TAIL + 2;             // [2]: the first half of a tile's P
    static constexpr int Q4_FULL = P_HALF + 2;          // [kSlots]
    static constexpr int Q4_EMPTY = Q4_FULL + kSlots;   // [kSlots]
    static constexpr int JOIN_FULL = Q4_EMPTY + kSlots;  // Q4: a split segment's second state is in the scratch; is read
    static constexpr int JOIN_EMPTY = JOIN_FULL + 1;
    static constexpr int kNumBars = JOIN_EMPTY + 1;
    static constexpr int kSlot = kBar + (kNumBars * 8 + 15) / 16 * 16;  // tensor memory address, skip flag
    static constexpr int kSeg = kSlot + 16;
    static constexpr int kSmem = kSeg + kSegSlots * (int)sizeof(SegMsg) + 1024;  // + slack for the alignment
};

struct ChunkParams {
    CUtensorMap tq, tk, tv;
    SchedIn s;
    PartSpace w;
    __nv_bfloat16 *out;
    float *lse;
    const int32_t *table;
    int *status;
    int64_t out_stride, table_stride;
    int32_t num_pages, log_ps, hq;
    int32_t tq_tokens;  // tokens per Q tile
    float scale_log2;
    CUtensorMap to;  // of the launches with boxes
    const uint8_t *ks, *vs;  // Q4: the scales
    int64_t ks_page, vs_page;
    float *join;  // Q4: per CTA the state of a tile of rows: o in columns of four ([hd / 4][kM][4]), m, l
};

// Waits between the roles last a tile or two, those for a segment's place, message, first scores or end as long as the
// segments before: a tile of 128 keys takes a CTA 1.1 to 1.5 us, so 2^31 keys would outlast any one limit. These waits may take
// ten times the time of the CTA's span.
constexpr uint64_t kKeyLimitNs = 128;
__device__ __forceinline__ bool wait_segment(uint32_t bar, uint32_t parity, int *status, const SchedShared &sh) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    const uint64_t limit = kWaitLimitNs + kKeyLimitNs * (uint64_t)min(sh.span, int64_t(1) << 36);
    return tc::mbar_wait(bar, parity, status, USP_ERR_TIMEOUT, limit);
}

// does key tile t hold rows behind the request's last key? (only a unit's last tile can)
__device__ __forceinline__ bool is_tail(const int32_t t, const int32_t kv) { return (t + 1) * kN > kv; }

// The walk warp hands out the segments and, at the end, the header of a unit left open. It is a segment
// ahead when it clears the end of a segment's last V tile.
template <int HD, bool Q4>
__device__ void walk_role(const ChunkParams &p, const SchedShared &sh, uint8_t *smem, uint32_t bar0) {
    using C = Cfg<HD, Q4>;
    const int lane = threadIdx.x & 31;
    auto wait = [&](int bar, uint32_t parity) {
        const bool r = wait_segment(bar0 + 8u * bar, parity, p.status, sh);
        return (bool)__all_sync(0xffffffffu, r);
    };
    SegMsg *ring = reinterpret_cast<SegMsg *>(smem + C::kSeg);
    Sched sc;
    sched_begin<kN>(p.s, sh, sc);
    PartHeader opened = no_part(sh);
    uint32_t tiles = 0, ntail = 0;  // tiles and tails of the segments handed out
    int tail_row = -1;              // first row to clear in the pending tail tile
    uint32_t tail_stage = 0;
    bool ok = true, more = true;
    for (uint32_t n = 0; ok && more; ++n) {
        Segment g;
        more = sched_next<kN>(p.s, sc, g);
        if (!(ok = wait(C::SEG_EMPTY + n % kSegSlots, ((n / kSegSlots) & 1u) ^ 1u))) break;
        if (lane == 0) {
            SegMsg m{};
            if (more) {
                m.tok0 = g.tok0; m.ntok = g.ntok; m.head = g.head; m.req = g.req; m.p0 = g.p0; m.kv = g.kv;
                m.t0 = g.t0; m.t1 = g.t1; m.tiles = g.tiles;
                for (int i = 0; i < 2; ++i) {
                    const int a = i * p.tq_tokens, b = min(g.ntok, a + p.tq_tokens);  // the Q tile's tokens
                    if (a >= b) continue;
                    const int last = p.s.causal ? max(0, min(g.kv, g.p0 + b)) : g.kv;
                    const int all = p.s.causal ? max(0, min(g.kv, g.p0 + a + 1)) : g.kv;
                    m.act[i] = (last + kN - 1) / kN;
                    m.full[i] = all / kN;
                }
                if (Q4 && g.ntok <= p.tq_tokens) {
                    m.split = 1;
                    m.act[1] = m.act[0];
                    m.full[1] = m.full[0];
                }
            }
            ring[n % kSegSlots] = m;
            tc::mbar_arrive(bar0 + 8u * (C::SEG_FULL + n % kSegSlots));
        }
        __syncwarp();
        if (tail_row >= 0) {
            // the last V tile of the segment before: landed, cleared, handed to the issuers
            if (!(ok = wait(C::TAIL + (ntail & 1u), (ntail >> 1) & 1u))) break;
            uint8_t *v = smem + C::kV + tail_stage * C::kTileBytes;
            for (int x = tail_row * 8 + lane; x < kN * 8; x += 32)
#pragma unroll
                for (int bx = 0; bx < C::kBoxes; ++bx)
                    *reinterpret_cast<uint4 *>(v + bx * C::kBoxBytes + x * 16) = make_uint4(0, 0, 0, 0);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(bar0 + 8u * (C::V_FULL + tail_stage));
            ++ntail;
            tail_row = -1;
        }
        if (more && g.t0 < g.t1) {
            tiles += (uint32_t)(g.t1 - g.t0);
            if (!Q4 && is_tail(g.t1 - 1, g.kv)) {
                tail_row = g.kv - (g.t1 - 1) * kN;
                tail_stage = (tiles - 1) % C::kStages;
            }
        }
        if (more && g.t0 == 0 && g.t1 < g.tiles) opened = part_header(p.s, sh, sc, g);
    }
    if (!ok) opened = no_part(sh);
    if (lane == 0) p.w.head[blockIdx.x] = opened;
}

// The next segment, for a whole warp; ntok == 0 at the end. False after a failed wait.
template <int HD, bool Q4>
__device__ __forceinline__ bool next_segment(const ChunkParams &p, const SchedShared &sh, uint32_t bar0, uint32_t &n,
                                             SegMsg &g) {
    using C = Cfg<HD, Q4>;
    bool ok = wait_segment(bar0 + 8u * (C::SEG_FULL + n % kSegSlots), (n / kSegSlots) & 1u, p.status, sh);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) return false;
    bool never;
    g = read_segment(bar0 + (uint32_t)(C::kSeg - C::kBar) + n % kSegSlots * (uint32_t)sizeof(SegMsg), never);
    __syncwarp();
    if ((threadIdx.x & 31) == 0) tc::mbar_arrive(bar0 + 8u * (C::SEG_EMPTY + n % kSegSlots) + (never ? 8u : 0u));
    ++n;
    return true;
}

// The next piece of a segment, for a warp of the softmax. n: twice the segments taken, and 1 in a segment with more pieces, whose
// message stays where it is; the next piece begins at the last one's end, g.t1. (A register more, and long prompts over a 4-bit
// cache take 3% longer.)
template <int HD, bool Q4>
__device__ __forceinline__ bool next_piece(const ChunkParams &p, const SchedShared &sh, uint32_t bar0, uint32_t &n, SegMsg &g) {
    using C = Cfg<HD, Q4>;
    const uint32_t at = n / 2 % kSegSlots;
    bool ok = wait_segment(bar0 + 8u * (C::SEG_FULL + at), (n / (2 * kSegSlots)) & 1u, p.status, sh);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) return false;
    bool never;
    SegMsg x = read_segment(bar0 + (uint32_t)(C::kSeg - C::kBar) + at * (uint32_t)sizeof(SegMsg), never);
    __syncwarp();
    x.first = x.t0;
    if (n & 1) x.t0 = g.t1;
    if (x.t1 - x.t0 > kPiece) {
        x.t1 = x.t0 + kPiece;
        n |= 1;
    } else {
        if ((threadIdx.x & 31) == 0) tc::mbar_arrive(bar0 + 8u * (C::SEG_EMPTY + at) + (never ? 8u : 0u));
        n = (n | 1) + 1;
    }
    g = x;
    return true;
}

// The producer warp. Lane l < boxes loads box l of each K and V tile: column half l / pieces, page piece
// l % pieces; lane 0 loads Q too.
template <int HD, bool Q4>
__device__ void producer_role(const ChunkParams &p, const SchedShared &sh, uint32_t sbase, uint32_t bar0) {
    using C = Cfg<HD, Q4>;
    const int lane = threadIdx.x & 31;
    auto BAR = [&](int i) { return bar0 + 8u * i; };
    auto wait = [&](int bar, uint32_t parity) {
        const bool r = tc::mbar_wait(BAR(bar), parity, p.status, USP_ERR_TIMEOUT, kWaitLimitNs);
        return (bool)__all_sync(0xffffffffu, r);
    };
    const int ps = 1 << p.log_ps, piece = min(ps, kN), pieces = kN / piece, nbox = pieces * C::kBoxes;
    const int half = lane / pieces, pc = lane % pieces;
    const uint32_t in_tile = half * C::kBoxBytes + pc * piece * 128;
    uint32_t kfills = 0, vfills = 0, nq = 0, nseg = 0, ntail = 0;
    bool ok = true;
    SegMsg g;
    while (ok && (ok = next_segment<HD, Q4>(p, sh, bar0, nseg, g)) && g.ntok > 0) {
        if (g.t0 >= g.t1) continue;
        // Q: the first one at once; later ones when the buffer is free, into L2 meanwhile
        auto q_boxes = [&](auto &&f) {
            for (int i = 0; i < 2; ++i)
                for (int bx = 0; bx < C::kBoxes; ++bx)
                    f(C::kQ + i * C::kTileBytes + bx * C::kBoxBytes, bx * 64, (int32_t)(g.tok0 + i * p.tq_tokens));
        };
        auto load_q = [&]() {
            if (lane != 0) return;
            tc::mbar_arrive_expect_tx(BAR(C::Q_FULL), 2 * C::kBoxes * (uint32_t)(p.tq_tokens * p.s.G) * 128);
            q_boxes([&](int dst, int c, int32_t tok) {
                tma_load_3d(sbase + dst, &p.tq, c, g.head * p.s.G, tok, BAR(C::Q_FULL));
            });
        };
        if (nq == 0) load_q();
        else if (lane == 0) q_boxes([&](int, int c, int32_t tok) { tma_prefetch_3d(&p.tq, c, g.head * p.s.G, tok); });
        ++nq;
        const int32_t *row = p.table + (int64_t)g.req * p.table_stride;
        // page of this lane's piece of tile t; num_pages (a box of zeros) behind the request's keys
        auto page_of = [&](int t) {
            const int64_t key = (int64_t)t * kN + pc * piece;
            if (lane >= nbox || key >= g.kv) return p.num_pages;
            const int32_t x = row[key >> p.log_ps];
            return x >= 0 && x < p.num_pages ? x : p.num_pages;
        };
        int32_t page = page_of(g.t0);
        for (int t = g.t0; t < g.t1; ++t) {
            const int32_t next = t + 1 < g.t1 ? page_of(t + 1) : 0;
            const int32_t c1 = g.head * ps + (int)(((int64_t)t * kN + pc * piece) & (ps - 1));
            const uint32_t st = kfills % C::kStages, ph = ((kfills / C::kStages) & 1u) ^ 1u;
            if (!(ok = wait(C::K_EMPTY + st, ph))) break;
            if (lane == 0) tc::mbar_arrive_expect_tx(BAR(C::K_FULL + st), C::kTileBytes);
            __syncwarp();
            if (lane < nbox)
                tma_load_3d(sbase + C::kK + st * C::kTileBytes + in_tile, &p.tk, half * 64, c1, page, BAR(C::K_FULL + st));
            ++kfills;
            if (t == g.t0 && nq > 1) {
                if (!(ok = wait(C::Q_EMPTY, (nq - 2) & 1u))) break;
                load_q();
            }
            if (!(ok = wait(C::V_EMPTY + st, ph))) break;
            // a tile with rows behind the last key goes to the walk warp first
            const bool tail = is_tail(t, g.kv);
            const uint32_t full = BAR(tail ? C::TAIL + (int)(ntail & 1u) : C::V_FULL + (int)st);
            if (lane == 0) tc::mbar_arrive_expect_tx(full, C::kTileBytes);
            __syncwarp();
            if (lane < nbox) tma_load_3d(sbase + C::kV + st * C::kTileBytes + in_tile, &p.tv, half * 64, c1, page, full);
            ++vfills;
            ntail += tail;
            page = next;
        }
    }
    if (!ok) {
        // drain (bounded), so that no copy lands after the CTA has gone
        if (nq > 0) wait(C::Q_FULL, (nq - 1) & 1u);  // (a load that was not issued ends by the recorded status)
        for (uint32_t f = kfills > C::kStages ? kfills - C::kStages : 0; f < kfills; ++f)
            wait(C::K_FULL + f % C::kStages, (f / C::kStages) & 1u);
        for (uint32_t f = vfills > C::kStages ? vfills - C::kStages : 0; f < vfills; ++f)
            wait(C::V_FULL + f % C::kStages, (f / C::kStages) & 1u);
        if (ntail > 0) wait(C::TAIL + ((ntail - 1) & 1u), ((ntail - 1) >> 1) & 1u);
    }
}

// The issuing warps stay converged and predicate each tensor-core instruction on one elected lane: the
// descriptors are then warp-uniform values in uniform registers. Issued from a branch that one lane takes,
// every product first moves its descriptors there: 75 to 100 cycles per m128n128k16 product (64 at the
// tensor core's rate), and the issue bounds the kernel (measured: a burst of 16 products 1420 cycles).
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r;
}
__device__ __forceinline__ void mma_ss_if(uint32_t elected, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(elected)
        : "memory");
}
__device__ __forceinline__ void mma_ts_if(uint32_t elected, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(elected)
        : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t elected, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(elected)
        : "memory");
}
__device__ __forceinline__ void arrive_if(uint32_t elected, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar),
        "r"(elected)
        : "memory");
}
// a wait of a whole warp, with a warp-uniform result
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, int *status) {
    if (__all_sync(0xffffffffu, tc::mbar_try_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, status, USP_ERR_TIMEOUT, kWaitLimitNs));
}

template <int HD, bool Q4>
__device__ __forceinline__ void issue_s(uint32_t el, uint32_t d_tmem, uint64_t qdesc, uint64_t kdesc) {
    using C = Cfg<HD, Q4>;
    constexpr uint32_t id = tc::idesc_bf16_f32(kM, kN, 0, 0);
#pragma unroll
    for (int k = 0; k < HD / 16; ++k) {
        const uint64_t off = (uint64_t)(((k / 4) * C::kBoxBytes + (k % 4) * 32) >> 4);
        mma_ss_if(el, d_tmem, qdesc + off, kdesc + off, id, k > 0 ? 1u : 0u);
    }
}
// V as (N = hd) x (K = keys), MN-major: 64-column blocks kBoxBytes apart, 8-key groups 1024 bytes apart
template <int HD, int kHalf>  // keys [64 kHalf, 64 kHalf + 64)
__device__ __forceinline__ void issue_pv(uint32_t el, uint32_t d_tmem, uint32_t p_tmem, uint64_t vdesc,
                                         uint32_t accumulate) {
    constexpr uint32_t id = tc::idesc_bf16_f32(kM, HD, 0, 1);
#pragma unroll
    for (int k = kHalf * 4; k < kHalf * 4 + 4; ++k)
        mma_ts_if(el, d_tmem, p_tmem + k * 8, vdesc + (uint64_t)((k * 2048) >> 4), id, (accumulate || k > 0) ? 1u : 0u);
}

// One warp per Q tile. Burst j of issuer i: PV_i(j), then S_i(j+1) unless tile j+1 opens a segment (its
// S leaves the turn order, so that it runs while the other tile finishes the old segment). Every wait
// costs 100 cycles or more even when it need not wait, so the one for P, which comes last in the steady
// state, is the last (with the turn last, 16384 tokens without the mask ran 6% slower). PV_i(j) and
// S_i(j+1) come from one lane, so S_i(j+1) overwrites P_i(j) only after PV_i(j) has read it. Stages are
// released by both issuers; each waits for a stage's fill before releasing it, also when its Q tile skips
// the tile.
template <int HD, bool Q4>
__device__ void mma_role(const ChunkParams &p, const SchedShared &sh, uint32_t sbase, uint32_t bar0, uint32_t tmem, int i) {
    using C = Cfg<HD, Q4>;
    const uint32_t el = elect_one();
    auto BAR = [&](int k) { return bar0 + 8u * k; };
    auto wait = [&](int bar, uint32_t parity) {
        return warp_wait(BAR(bar), parity, p.status);
    };
    const uint64_t qdesc = tc::sw128_desc(sbase + C::kQ + (uint32_t)i * C::kTileBytes, 16, 1024);
    const uint64_t kdesc0 = tc::sw128_desc(sbase + C::kK, 16, 1024);
    const uint64_t vdesc0 = tc::sw128_desc(sbase + C::kV, C::kBoxBytes, 1024);
    auto stage_off = [](uint32_t st) { return (uint64_t)((st * C::kTileBytes) >> 4); };
    const uint32_t tS = tmem + 128u * i, tO = tmem + 256u + (uint32_t)(HD * i);
    const int my_turn = C::TURN + i, other_turn = C::TURN + (1 - i);
    // the current segment's tiles: kt of [., end), in pieces of [., t1); this issuer's Q tile needs those below act_end
    int kt = 0, t1 = 0, end = 0, act_end = 0;
    // a split segment (Q4): this issuer takes every other key tile, and the two go on without turns
    bool split = false, begun = false;
    int t0 = 0;  // the segment's first tile
    auto acts = [&](int t) { return t < act_end && (!split || ((t - t0) & 1) == i); };
    auto s_burst = [&](bool act, uint32_t st) {
        if (act) {
            issue_s<HD, Q4>(el, tS, qdesc, kdesc0 + stage_off(st));
            commit_if(el, BAR(C::S_FULL + i));
        }
        commit_if(el, BAR(C::K_EMPTY + st));
    };
    uint32_t pc = 0, started = 0;  // P waits; a PV of the current segment has been issued
    uint32_t nq = 0, no = 0;       // Q loads consumed; O_i read-outs handed to the softmax
    uint32_t turns = 0, nseg = 0;
    uint32_t j = 0;                // tiles of all segments
    bool ok = true;
    for (;;) {
        // The next piece, or the next segment with a tile. All that the softmax warps need of the one before is issued by now: one
        // taken earlier, with segments without a tile between, would take the issuers up to a ring of segments
        // ahead of the softmax warps, which wait for the O of the last tile while the ring has no place for
        // the segment that the issuers wait for.
        if (kt >= end) {
            int ntok;
            do {
                SegMsg g;
                if (!(ok = next_segment<HD, Q4>(p, sh, bar0, nseg, g))) break;
                // (reductions over equal values: the compiler then knows that they are uniform)
                ntok = __reduce_max_sync(0xffffffffu, g.ntok);
                kt = t0 = __reduce_max_sync(0xffffffffu, g.t0);
                end = __reduce_max_sync(0xffffffffu, g.t1);
                act_end = __reduce_max_sync(0xffffffffu, i ? g.act[1] : g.act[0]);
                if (Q4) split = __reduce_max_sync(0xffffffffu, g.split) != 0;
            } while (ntok > 0 && kt >= end);
            if (!ok || ntok == 0) break;
            if (!(ok = wait(C::Q_FULL, nq & 1u))) break;
            ++nq;
        }
        t1 = min(end, kt + kPiece);
        if (!(ok = wait(C::K_FULL + j % C::kStages, (j / C::kStages) & 1u))) break;
        const bool first = !begun && !split;
        begun |= !split;
        if (first && i == 1 && !(ok = wait(my_turn, (turns++) & 1u))) break;
        s_burst(acts(kt), j % C::kStages);
        if (first) arrive_if(el, BAR(other_turn));
        for (;;) {
            const bool act = acts(kt), last = kt + 1 >= t1;
            const uint32_t st = j % C::kStages, ph = (j / C::kStages) & 1u;
            const uint32_t stn = (j + 1) % C::kStages, phn = ((j + 1) / C::kStages) & 1u;
            if (last && t1 == end) commit_if(el, BAR(C::Q_EMPTY));  // this issuer's S products of the segment are issued
            if (!(ok = wait(C::V_FULL + st, ph))) break;
            if (!last && !(ok = wait(C::K_FULL + stn, phn))) break;
            if (act && !started && no > 0 && !(ok = wait(C::O_EMPTY + i, (no - 1) & 1u))) break;
            if (!split && !(ok = wait(my_turn, (turns++) & 1u))) break;
            if (act) {
                if (!(ok = wait(C::P_HALF + i, pc & 1u))) break;
                tc::fence_after_sync();
                issue_pv<HD, 0>(el, tO, tS, vdesc0 + stage_off(st), started);
                if (!(ok = wait(C::P_FULL + i, pc & 1u))) break;
                ++pc;
                tc::fence_after_sync();
                issue_pv<HD, 1>(el, tO, tS, vdesc0 + stage_off(st), 1);
                started = 1;
            }
            commit_if(el, BAR(C::V_EMPTY + st));
            ++j;
            ++kt;
            if (last) break;
            s_burst(acts(kt), stn);
            if (!split) arrive_if(el, BAR(other_turn));
        }
        if (!ok) break;
        if (started) {
            commit_if(el, BAR(C::O_FULL + i));
            ++no;
        }
        started = 0;
        if (!split) arrive_if(el, BAR(other_turn));
    }
    if (!ok) arrive_if(el, BAR(other_turn));  // let the other issuer reach its own bounded exit
    commit_if(el, BAR(C::DONE + i));           // every MMA of this issuer ends before tensor memory is freed
    wait(C::DONE + i, 0);
}

__device__ __forceinline__ float u2f(uint32_t x) { return __uint_as_float(x); }
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr)
                 : "memory");
    return v;
}

// The producer warp over a 4-bit cache: tiles of codes and scales, K then V, through the ring of slots. Lane l < pieces loads the
// codes of page piece l (a TMA box), every lane 16 bytes of the scales; lane 0 loads Q as above.
template <int HD>
__device__ void producer_q4_role(const ChunkParams &p, const SchedShared &sh, uint32_t sbase, uint32_t bar0) {
    using C = Cfg<HD, true>;
    const int lane = threadIdx.x & 31;
    auto BAR = [&](int i) { return bar0 + 8u * i; };
    auto wait = [&](int bar, uint32_t parity) { return warp_wait(BAR(bar), parity, p.status); };
    const int ps = 1 << p.log_ps, mask = ps - 1, piece = min(ps, kN), pieces = kN / piece;
    constexpr int kCopyKeys = 16 / q4_scale_bytes(HD), kLineKeys = 128 / q4_code_bytes(HD);
    const int skey = lane * kCopyKeys;
    const bool loads = lane < pieces, copies = lane < C::kScales / 16;
    const uint32_t codes0 = sbase + C::kQ4 + lane * piece * q4_code_bytes(HD), scales0 = sbase + C::kQ4Scales + lane * 16;
    uint32_t fills = 0, nq = 0, nseg = 0;
    bool ok = true;
    SegMsg g;
    while (ok && (ok = next_segment<HD, true>(p, sh, bar0, nseg, g)) && g.ntok > 0) {
        if (g.t0 >= g.t1) continue;
        auto q_boxes = [&](auto &&f) {
            for (int i = 0; i < 2; ++i)
                for (int bx = 0; bx < C::kBoxes; ++bx)
                    f(C::kQ + i * C::kTileBytes + bx * C::kBoxBytes, bx * 64, (int32_t)(g.tok0 + (g.split ? 0 : i) * p.tq_tokens));
        };
        auto load_q = [&]() {
            if (lane != 0) return;
            tc::mbar_arrive_expect_tx(BAR(C::Q_FULL), 2 * C::kBoxes * (uint32_t)(p.tq_tokens * p.s.G) * 128);
            q_boxes([&](int dst, int c, int32_t tok) {
                tma_load_3d(sbase + dst, &p.tq, c, g.head * p.s.G, tok, BAR(C::Q_FULL));
            });
        };
        if (nq == 0) load_q();
        else if (lane == 0) q_boxes([&](int, int c, int32_t tok) { tma_prefetch_3d(&p.tq, c, g.head * p.s.G, tok); });
        ++nq;
        // The next tile's page numbers are read a tile ahead and looked at only when that tile's slot is free: this warp alone
        // feeds the SM, and a wait for them in every tile (800 cycles) would show. -1: behind the request's keys.
        const int32_t *row = p.table + (int64_t)g.req * p.table_stride;
        auto page_of = [&](int t, int in, bool on) {
            const int key = t * kN + in;
            return on && key < g.kv ? row[key >> p.log_ps] : -1;
        };
        const int row0 = g.head * ps;
        int32_t raw = page_of(g.t0, lane * piece, loads), sraw = page_of(g.t0, skey, copies);
        for (int t = g.t0; t < g.t1; ++t) {
            uint32_t slot = fills % C::kSlots;
            if (!(ok = wait(C::Q4_EMPTY + slot, ((fills / C::kSlots) & 1u) ^ 1u))) break;
            if (lane == 0) tc::mbar_arrive_expect_tx(BAR(C::Q4_FULL + slot), C::kCodes);
            // a page outside the cache: a box of zeros, and page 0's scales
            const int32_t page = (uint32_t)raw < (uint32_t)p.num_pages ? raw : p.num_pages;
            const int64_t spage = (uint32_t)sraw < (uint32_t)p.num_pages ? sraw : 0;
            const int line = (row0 + ((t * kN + lane * piece) & mask)) / kLineKeys;
            const int in = (row0 + ((t * kN + skey) & mask)) * q4_scale_bytes(HD);
            const uint8_t *ks = p.ks + spage * p.ks_page + in, *vs = p.vs + spage * p.vs_page + in;
            auto load = [&](const CUtensorMap *map, const uint8_t *scales) {
                __syncwarp();
                if (loads) tma_load_3d(codes0 + slot * C::kCodes, map, 0, line, page, BAR(C::Q4_FULL + slot));
                if (copies) copy16(scales0 + slot * C::kScales, scales);
                copies_arrive(BAR(C::Q4_FULL + slot));
                ++fills;
            };
            load(&p.tk, ks);
            raw = page_of(t + 1, lane * piece, loads);
            sraw = page_of(t + 1, skey, copies);
            if (t == g.t0 && nq > 1) {
                if (!(ok = wait(C::Q_EMPTY, (nq - 2) & 1u))) break;
                load_q();
            }
            slot = fills % C::kSlots;
            if (!(ok = wait(C::Q4_EMPTY + slot, ((fills / C::kSlots) & 1u) ^ 1u))) break;
            if (lane == 0) tc::mbar_arrive_expect_tx(BAR(C::Q4_FULL + slot), C::kCodes);
            load(&p.tv, vs);
        }
    }
    if (!ok) {
        // drain (bounded), so that no copy lands after the CTA has gone
        if (nq > 0) wait(C::Q_FULL, (nq - 1) & 1u);  // (a load that was not issued ends by the recorded status)
        for (uint32_t f = fills > C::kSlots ? fills - C::kSlots : 0; f < fills; ++f)
            wait(C::Q4_FULL + f % C::kSlots, (f / C::kSlots) & 1u);
    }
}

// The converting warps: thread r takes key r of each tile of codes to row r of the K or V stage.
template <int HD>
__device__ void convert_role(const ChunkParams &p, const SchedShared &sh, uint32_t sbase, uint32_t bar0) {
    using C = Cfg<HD, true>;
    const int lane = threadIdx.x & 31;
    const uint32_t r = threadIdx.x & 127;
    auto BAR = [&](int i) { return bar0 + 8u * i; };
    auto wait = [&](int bar, uint32_t parity) { return warp_wait(BAR(bar), parity, p.status); };
    const Q4Nibbles nib;
    const uint32_t codes0 = codes_at<HD>(r, 0);
    uint32_t fills = 0, nseg = 0;
    bool ok = true;
    SegMsg g;
    while (ok && (ok = next_segment<HD, true>(p, sh, bar0, nseg, g)) && g.ntok > 0) {
        const int n = 2 * max(g.t1 - g.t0, 0);
        for (int x = 0; x < n; ++x, ++fills) {
            const uint32_t slot = fills % C::kSlots, v = fills & 1u, tile = fills >> 1, st = tile % C::kStages;
            if (!(ok = wait(C::Q4_FULL + slot, (fills / C::kSlots) & 1u))) break;
            const uint32_t codes = sbase + C::kQ4 + slot * C::kCodes + codes0, scales = sbase + C::kQ4Scales + slot * C::kScales;
            uint4 w[HD / 32];
#pragma unroll
            for (int c = 0; c < HD / 32; ++c) w[c] = ld_shared_v4(codes ^ (c * 16));  // (of one line: swizzled alike)
            uint32_t sb;
            if constexpr (HD == 128) asm volatile("ld.shared.b32 %0, [%1];" : "=r"(sb) : "r"(scales + r * 4) : "memory");
            else asm volatile("ld.shared.u16 %0, [%1];" : "=r"(sb) : "r"(scales + r * 2) : "memory");
            // The slot goes back at once, so that all slots are loads in flight; but only when its words are here: an arrive does
            // not wait for loads. The store before it does, for its predicate, which is a word of each load (the word it
            // may write is nobody's).
            uint32_t all = sb;
#pragma unroll
            for (int c = 0; c < HD / 32; ++c) all ^= w[c].x;
            asm volatile("{\n\t.reg .pred p;\n\tsetp.eq.u32 p, %0, 0x9e3779b9;\n\t@p st.shared.b32 [%1], %0;\n\t}" ::"r"(all),
                         "r"(sbase + C::kSlot + 8)
                         : "memory");
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(BAR(C::Q4_EMPTY + slot));
            if (!(ok = wait((v ? C::V_EMPTY : C::K_EMPTY) + st, ((tile / C::kStages) & 1u) ^ 1u))) break;
            const uint32_t to = sbase + (v ? C::kV : C::kK) + st * C::kTileBytes + r * 128;
#pragma unroll
            for (int c = 0; c < HD / 32; ++c) {  // a group of 32 values
                const uint32_t s2 = q4_scales2((sb >> (8 * c)) & 255u), off = q4_minus136(s2);
                const uint32_t words[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int c8 = c * 4 + e;
                    st_shared_v4(to + (c8 >> 3) * C::kBoxBytes + (((uint32_t)(c8 & 7) ^ (r & 7u)) << 4),
                                 nib.values(words[e], 0, s2, off), nib.values(words[e], 1, s2, off),
                                 nib.values(words[e], 2, s2, off), nib.values(words[e], 3, s2, off));
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(BAR((v ? C::V_FULL : C::K_FULL) + st));
        }
    }
}

// One piece of a segment of the softmax of Q tile i; ns (S tiles), no (O read-outs) and nj (joined states) run on across these.
// False after a failed wait (the whole warp leaves; the others' waits end by the recorded status).
template <int HD, bool Q4, bool kBox>  // kBox: whole warps of rows of out are stored as boxes
__device__ __forceinline__ bool softmax_segment(const ChunkParams &p, const SchedShared &sh, const SegMsg &g, uint8_t *smem, uint32_t bar0,
                                                uint32_t tmem, int i, uint32_t &ns, uint32_t &no, uint32_t &nj) {
    using C = Cfg<HD, Q4>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wq = warp & 3;
    const int row = wq * 32 + lane;
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const uint32_t tS = tmem + lane_off + 128u * (uint32_t)i;
    const uint32_t tO = tmem + lane_off + 256u + (uint32_t)(HD * i);
    uint32_t rt, rh;
    p.s.by_G.divmod((uint32_t)row, rt, rh);
    const bool split = Q4 && g.split != 0;
    const int tile = split ? 0 : i;                // of the unit's rows
    const int tok = tile * p.tq_tokens + (int)rt;  // token of the segment's block
    const bool row_ok = row < p.tq_tokens * p.s.G && tok < g.ntok;
    const int lim = p.s.causal ? max(0, min(g.kv, g.p0 + min(tok, g.ntok - 1) + 1)) : g.kv;
    const float sl2 = p.scale_log2;
    const uint64_t sl22 = tc::pack2(sl2, sl2);
    float m = -INFINITY, l = 0.f;
    bool any = false, ok = true;
    const int act_end = min(g.t1, i ? g.act[1] : g.act[0]), full_end = i ? g.full[1] : g.full[0];
    for (int kt = split ? g.t0 + i : g.t0; kt < act_end; kt += split ? 2 : 1) {
        const bool full = kt < full_end;
        // (over a bf16 cache this tile of rows may have skipped segments that the issuers are still in)
        const uint32_t s_full = bar0 + 8u * (C::S_FULL + i);
        ok = Q4 ? tc::mbar_wait(s_full, ns & 1u, p.status, USP_ERR_TIMEOUT, kWaitLimitNs) : wait_segment(s_full, ns & 1u, p.status, sh);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc::fence_after_sync();
        if (!full) {
            // Mask S in place, only the 32-key chunks that some row of the warp sees not all of (a warp's
            // rows are a few tokens with limits close together). A rolled loop of its own keeps 128 selects
            // out of the code that every tile runs through: what runs once per unit mostly waits for its
            // instructions.
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                const int lc = lim - kt * kN - c * 32;
                if (__all_sync(0xffffffffu, lc >= 32)) continue;
                uint32_t x[32];
                tc::tmem_ld32(tS + c * 32, x);
                tc::tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (e >= lc) x[e] = __float_as_uint(-INFINITY);
                tc::tmem_st32(tS + c * 32, x);
                tc::tmem_st_wait();
            }
        }
        uint32_t sr[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tc::tmem_ld32(tS + c * 32, sr[c]);
        tc::tmem_ld_wait();
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            float a = u2f(sr[c][0]), b = u2f(sr[c][1]);
#pragma unroll
            for (int e = 2; e < 30; e += 4) {
                a = tc::max3(a, u2f(sr[c][e]), u2f(sr[c][e + 1]));
                b = tc::max3(b, u2f(sr[c][e + 2]), u2f(sr[c][e + 3]));
            }
            mx = tc::max3(mx, tc::max3(a, u2f(sr[c][30]), u2f(sr[c][31])), b);
        }
        mx *= sl2;
        const bool need = mx > m + kRescale;
        if (__any_sync(0xffffffffu, need)) {
            const float mn = fmaxf(m, mx);
            const float alpha = need ? tc::ex2(m - mn) : 1.f;  // 0 on the first visible tile
            if (need) m = mn;
            if (any) {
#pragma unroll 1
                for (int c = 0; c < HD / 32; ++c) {
                    uint32_t o[32];
                    tc::tmem_ld32(tO + c * 32, o);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(u2f(o[e]) * alpha);
                    tc::tmem_st32(tO + c * 32, o);
                }
            }
            l *= alpha;
        }
        const float mb = m == -INFINITY ? 0.f : m;
        const uint64_t nmb2 = tc::pack2(-mb, -mb);
        uint64_t sum = tc::pack2(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const uint64_t y = tc::fma2(tc::pack2(u2f(sr[c][2 * e]), u2f(sr[c][2 * e + 1])), sl22, nmb2);
                float y0, y1;
                tc::unpack2(y, y0, y1);
                const float p0 = tc::ex2(y0), p1 = tc::ex2(y1);
                sum = tc::add2(sum, tc::pack2(p0, p1));
                pk[e] = float2_to_bf16x2(p0, p1);  // (see paged_decode.cu on this rounding)
            }
            tc::tmem_st16(tS + c * 16, pk);
            if (c == 1) {
                // the products of the first 64 keys run under the exponentials of the others (1% at all lengths)
                tc::tmem_st_wait();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(bar0 + 8u * (C::P_HALF + i));
            }
        }
        float s0, s1;
        tc::unpack2(sum, s0, s1);
        l += s0 + s1;
        tc::tmem_st_wait();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar0 + 8u * (C::P_FULL + i));
        any = true;
        ++ns;
    }
    if (!ok) return false;
    // ---- end of the piece -------------------------------------------------------------------------
    const bool whole = g.first == 0 && g.t1 == g.tiles, more = g.t0 != g.first;  // more: pieces before this one
    const int r = tile * p.tq_tokens * p.s.G + row;  // row of the unit
    float *slot = part_slot(p.w, HD, blockIdx.x, g.first == 0 ? 1 : 0);
    const int head = g.head * p.s.G + (int)rh;
    __nv_bfloat16 *orow = p.out + (g.tok0 + tok) * p.out_stride + (int64_t)head * HD;
    // What the slot holds of the pieces before (o is unwritten where they saw no key: then without weight)
    float now = 1.f, was = 0.f;
    if (more && (!split || i == 0)) {
        const float m0 = slot[(size_t)p.w.rows * HD + r], l0 = slot[(size_t)p.w.rows * (HD + 1) + r], both = fmaxf(m, m0),
                    base = both == -INFINITY ? 0.f : both;
        now = tc::ex2(m - base);
        was = tc::ex2(m0 - base);
        l = fmaf(l0, was, l * now);
        m = both;
    }
    auto before = [&](int at) {
        return was > 0.f ? *reinterpret_cast<const float4 *>(slot + (size_t)r * HD + at) : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    // A split segment: the second tile's state to the scratch, column by column of four, so that a warp's lanes, a row each,
    // write and read whole lines; the first tile's threads scale both to the common maximum.
    float mine_by = 1.f, other_by = 0.f;
    const float *join = nullptr;
    if constexpr (Q4) {
        if (split && g.t0 + 1 < min(g.t1, g.act[1])) {  // (then the first tile of rows has a key tile too)
            float *at = p.join + (size_t)blockIdx.x * (kM * (HD + 2)), *stats = at + kM * HD;
            if (i == 1) {
                ok = tc::mbar_wait(bar0 + 8u * (C::O_FULL + 1), no & 1u, p.status, USP_ERR_TIMEOUT, kWaitLimitNs) &&
                     (nj == 0 || tc::mbar_wait(bar0 + 8u * C::JOIN_EMPTY, (nj - 1) & 1u, p.status, USP_ERR_TIMEOUT, kWaitLimitNs));
                if (!__all_sync(0xffffffffu, ok)) return false;
                ++no;
                tc::fence_after_sync();
#pragma unroll 1
                for (int c = 0; c < HD / 32; ++c) {
                    uint32_t o[32];
                    tc::tmem_ld32(tO + c * 32, o);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        *reinterpret_cast<uint4 *>(at + ((c * 8 + e) * kM + row) * 4) =
                            make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                }
                stats[row] = m;
                stats[kM + row] = l;
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    tc::mbar_arrive(bar0 + 8u * (C::O_EMPTY + 1));
                    tc::mbar_arrive(bar0 + 8u * C::JOIN_FULL);
                }
                ++nj;
                return true;
            }
            ok = tc::mbar_wait(bar0 + 8u * C::JOIN_FULL, nj & 1u, p.status, USP_ERR_TIMEOUT, kWaitLimitNs);
            if (!__all_sync(0xffffffffu, ok)) return false;
            ++nj;
            const float m1 = stats[row], l1 = stats[kM + row], both = fmaxf(m, m1), base = both == -INFINITY ? 0.f : both;
            mine_by = tc::ex2(m - base);
            other_by = tc::ex2(m1 - base);
            l = l * mine_by + l1 * other_by;
            m = both;
            join = at;
        } else if (split && i == 1) {
            return true;
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    auto released = [&]() {  // the scratch is read
        if (Q4 && join) {
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(bar0 + 8u * C::JOIN_EMPTY);
        }
    };
    if (any) {
        ok = tc::mbar_wait(bar0 + 8u * (C::O_FULL + i), no & 1u, p.status, USP_ERR_TIMEOUT, kWaitLimitNs);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return false;
        ++no;
        tc::fence_after_sync();
        // A lane holds a row, and rows lie apart in memory: 128 bytes of each of the 32 rows go through the
        // warp's staging slot, 16-byte pieces swizzled by row % 8 against bank conflicts. A TMA box of out takes the
        // slot, or the lanes write it, four whole lines per instruction (see launch_paged_chunk).
        const uint32_t stg = tc::smem_u32(smem) + C::kStg + warp * C::kStgSlot;
        constexpr int kP = C::kStgRow / 16, kR = 32 / kP;  // pieces of a staged row; rows per instruction
        const int sub = lane / kP, pc = lane % kP;         // the row and the piece that this lane stores
        auto swz = [](uint32_t c, uint32_t r) { return kP == 8 ? c ^ (r & 7u) : c ^ ((r >> 2) & 1u); };
        const uint64_t mine = !row_ok ? 0
                              : whole ? reinterpret_cast<uint64_t>(orow)
                                      : reinterpret_cast<uint64_t>(slot + (size_t)r * HD);
        auto stage_in = [&](int c, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
            st_shared_v4(stg + (uint32_t)lane * C::kStgRow + (swz((uint32_t)c, (uint32_t)lane) << 4), x, y, z, w);
        };
        auto stage_out = [&](uint32_t at) {  // the staged bytes of every row, to byte `at` of the rows
            __syncwarp();
#pragma unroll
            for (int x = 0; x < kP; ++x) {
                const uint32_t rr = (uint32_t)(x * kR + sub);
                const uint4 v = ld_shared_v4(stg + rr * C::kStgRow + (swz((uint32_t)pc, rr) << 4));
                const uint64_t to = __shfl_sync(0xffffffffu, mine, (int)rr);
                if (to) *reinterpret_cast<uint4 *>(to + at + (uint32_t)pc * 16u) = v;
            }
            __syncwarp();
        };
        if (more) {
#pragma unroll 1
            for (int c = 0; c < HD / 32; ++c) {
                uint32_t o[32];
                tc::tmem_ld32(tO + c * 32, o);
                tc::tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float4 x = before(c * 32 + e * 4);
                    const float y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int f = 0; f < 4; ++f) o[e * 4 + f] = __float_as_uint(fmaf(y[f], was, u2f(o[e * 4 + f]) * now));
                }
                tc::tmem_st32(tO + c * 32, o);
            }
            tc::tmem_st_wait();
        }
        const bool box = kBox && whole && __all_sync(0xffffffffu, row_ok);
        if constexpr (kBox) {
            if (lane == 0) tma_stores_read();  // the unit before may have left one
            __syncwarp();
        }
#pragma unroll 1
        for (uint32_t c = 0; c < HD / 64; ++c) {
            uint32_t o[2][32];
            tc::tmem_ld32(tO + c * 64, o[0]);
            tc::tmem_ld32(tO + c * 64 + 32, o[1]);
            tc::tmem_ld_wait();
            if (Q4 && join) {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float4 x = *reinterpret_cast<const float4 *>(join + ((c * 16 + e) * kM + row) * 4);
                    const float y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int f = 0; f < 4; ++f) {
                        uint32_t &w = o[e / 8][e % 8 * 4 + f];
                        w = __float_as_uint(fmaf(y[f], other_by, u2f(w) * mine_by));
                    }
                }
            }
            if (whole) {
                if (c > 0 && box) {
                    if (lane == 0) tma_stores_read();
                    __syncwarp();
                }
#pragma unroll
                for (int c8 = 0; c8 < 8; ++c8) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[e] = float2_to_bf16x2(u2f(o[c8 / 4][c8 % 4 * 8 + 2 * e]) * inv,
                                                u2f(o[c8 / 4][c8 % 4 * 8 + 2 * e + 1]) * inv);
                    stage_in(c8 % kP, w[0], w[1], w[2], w[3]);
                    if (kP < 8 && c8 % kP == kP - 1) stage_out(c * 128 + c8 / kP * C::kStgRow);
                }
                if (kP < 8) continue;
                if (box) {
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) tma_store_3d(&p.to, (int32_t)c * 64, head, (int32_t)(g.tok0 + tok), stg);
                } else {
                    stage_out(c * 128);
                }
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int c8 = 0; c8 < 8; ++c8) {
                        stage_in(c8 % kP, o[h][c8 * 4], o[h][c8 * 4 + 1], o[h][c8 * 4 + 2], o[h][c8 * 4 + 3]);
                        if (c8 % kP == kP - 1) stage_out(c * 256 + h * 128 + c8 / kP * C::kStgRow);
                    }
                }
            }
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar0 + 8u * (C::O_EMPTY + i));
        released();
    } else if (row_ok && whole) {
        for (int e = 0; e < HD; e += 4) {
            const float4 x = before(e);
            const float by = was * inv;
            *reinterpret_cast<uint2 *>(orow + e) =
                make_uint2(float2_to_bf16x2(x.x * by, x.y * by), float2_to_bf16x2(x.z * by, x.w * by));
        }
    }
    if (row_ok) {
        if (whole) {
            p.lse[(g.tok0 + tok) * p.hq + head] = l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2;
        } else {
            // a part without a visible key has m = -inf: the combine gives its (unwritten) o no weight
            slot[(size_t)p.w.rows * HD + r] = m;
            slot[(size_t)p.w.rows * (HD + 1) + r] = l;
        }
    }
    return true;
}

template <int HD, bool Q4, bool kBox>
__global__ void __launch_bounds__(kThreads<Q4>, 1) paged_chunk_kernel(const __grid_constant__ ChunkParams p) {
    using C = Cfg<HD, Q4>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ SchedShared sh;
    const uint32_t raw = tc::smem_u32(smem_raw);
    const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
    uint8_t *smem = smem_raw + pad;
    const uint32_t sbase = raw + pad;
    const uint32_t bar0 = sbase + C::kBar;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kSlot);
    volatile uint32_t *skip_flag = tmem_slot + 1;
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        tc::prefetch_tmap(&p.tq);
        tc::prefetch_tmap(&p.tk);
        tc::prefetch_tmap(&p.tv);
        for (int s = 0; s < C::kStages; ++s) {
            tc::mbar_init(bar0 + 8u * (C::K_FULL + s), Q4 ? 4 : 1);
            tc::mbar_init(bar0 + 8u * (C::K_EMPTY + s), 2);
            tc::mbar_init(bar0 + 8u * (C::V_FULL + s), Q4 ? 4 : 1);
            tc::mbar_init(bar0 + 8u * (C::V_EMPTY + s), 2);
        }
        tc::mbar_init(bar0 + 8u * C::Q_FULL, 1);
        tc::mbar_init(bar0 + 8u * C::Q_EMPTY, 2);
        for (int i = 0; i < kSegSlots; ++i) {
            tc::mbar_init(bar0 + 8u * (C::SEG_FULL + i), 1);
            tc::mbar_init(bar0 + 8u * (C::SEG_EMPTY + i), kSegReaders<Q4>);
        }
        for (int i = 0; i < C::kSlots; ++i) {
            tc::mbar_init(bar0 + 8u * (C::Q4_FULL + i), 33);  // the boxes' bytes, and each lane's copies
            tc::mbar_init(bar0 + 8u * (C::Q4_EMPTY + i), 4);
        }
        tc::mbar_init(bar0 + 8u * C::JOIN_FULL, 4);
        tc::mbar_init(bar0 + 8u * C::JOIN_EMPTY, 4);
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(bar0 + 8u * (C::S_FULL + i), 1);
            tc::mbar_init(bar0 + 8u * (C::P_FULL + i), 4);
            tc::mbar_init(bar0 + 8u * (C::P_HALF + i), 4);
            tc::mbar_init(bar0 + 8u * (C::O_FULL + i), 1);
            tc::mbar_init(bar0 + 8u * (C::O_EMPTY + i), 4);
            tc::mbar_init(bar0 + 8u * (C::DONE + i), 1);
            tc::mbar_init(bar0 + 8u * (C::TURN + i), 1);
            tc::mbar_init(bar0 + 8u * (C::TAIL + i), 1);
        }
        tc::fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        tc::tmem_alloc(tc::smem_u32(tmem_slot), 512);
        tc::tmem_relinquish();
    }
    wait_grid_before();
    // a bounded wait of an earlier kernel ran out: do no work until usp_check clears it
    const int status = *reinterpret_cast<volatile int *>(p.status);
    let_next_start();
    const bool work = sched_scan<kThreads<Q4>, kN>(p.s, sh);  // the same for every thread
    if (threadIdx.x == 0) *skip_flag = status != 0;
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const bool skip = !work || *skip_flag != 0;
    if (Q4 && warp >= kConvertWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Q4 ? kConvertRegs<Q4> : 24));
        if constexpr (Q4)
            if (!skip) convert_role<HD>(p, sh, sbase, bar0);
    } else if (warp >= kSoftmaxWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kControlRegs<Q4>));
        if (!skip) {
            if (warp == kProducerWarp) {
                if constexpr (Q4) producer_q4_role<HD>(p, sh, sbase, bar0);
                else producer_role<HD, Q4>(p, sh, sbase, bar0);
            } else if (warp == kWalkWarp) {
                walk_role<HD, Q4>(p, sh, smem, bar0);
            } else {
                mma_role<HD, Q4>(p, sh, sbase, bar0, tmem, warp - kMmaWarp);
            }
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs<Q4>));
        uint32_t ns = 0, no = 0, nj = 0, nseg = 0;
        SegMsg g{};
        while (!skip && next_piece<HD, Q4>(p, sh, bar0, nseg, g) && g.ntok > 0)
            if (!softmax_segment<HD, Q4, kBox>(p, sh, g, smem, bar0, tmem, warp >> 2, ns, no, nj)) break;
        if (kBox && (threadIdx.x & 31) == 0) tma_stores_done();
    }
    if (skip && threadIdx.x == 0) p.w.head[blockIdx.x] = no_part(sh);
    tc::fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 512);
    }
}

template <int HD, bool Q4, bool kBox>
int launch_typed(const ChunkParams &p, int grid, cudaStream_t s) {
    constexpr int kSmem = Cfg<HD, Q4>::kSmem;
    static_assert(kSmem <= 226 * 1024, "shared memory per CTA");
    static std::mutex mu;
    static bool attr_set[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return USP_ERR_CUDA;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (dev < 0 || dev >= 64) return USP_ERR_UNSUPPORTED;
        if (!attr_set[dev]) {
            // setmaxnreg.inc is granted only from registers the launch holds: never launch a build whose
            // register count would make the split wait forever
            cudaFuncAttributes fa{};
            if (cudaFuncGetAttributes(&fa, paged_chunk_kernel<HD, Q4, kBox>) != cudaSuccess) return USP_ERR_CUDA;
            if ((long)fa.numRegs * kThreads<Q4> < 128L * (2 * kSoftmaxRegs<Q4> + kControlRegs<Q4> + kConvertRegs<Q4>)) return USP_ERR_UNSUPPORTED;
            if (cudaFuncSetAttribute(paged_chunk_kernel<HD, Q4, kBox>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) !=
                cudaSuccess)
                return USP_ERR_CUDA;
            attr_set[dev] = true;
        }
    }
    return launch_overlapped(paged_chunk_kernel<HD, Q4, kBox>, dim3((unsigned)grid), kThreads<Q4>, kSmem, s, p);
}

}  // namespace

int launch_paged_chunk(const PagedArgs &a, int n_lo, const PartSpace &w, cudaStream_t s) {
    const DeviceInfo *di = device_info();
    if (!di) return USP_ERR_CUDA;
    ChunkParams p{};
    const int ps = 1 << a.log_ps;
    const uint32_t box = (uint32_t)std::min(ps, kN);
    p.tq_tokens = kM / a.G;
    // q as (hd, hq, tokens) in boxes of 64 columns x G heads x the tile's tokens
    EncodeTiledFn enc = encode_fn();
    if (!enc) return USP_ERR_CUDA;
    const cuuint64_t dims[3] = {(cuuint64_t)a.hd, (cuuint64_t)a.hq, (cuuint64_t)a.tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)a.hd * 2, (cuuint64_t)a.q_stride * 2};
    const cuuint32_t qbox[3] = {64, (cuuint32_t)a.G, (cuuint32_t)p.tq_tokens}, estr[3] = {1, 1, 1};
    // out likewise, in boxes of a softmax warp's 32 rows where these are whole tokens or parts of one token's heads.
    // With two units per CTA or more a warp goes on while its boxes are written, where its own stores would cost it a
    // thousand cycles per unit (6 prompts of 1500 to 4100 tokens, 13 units per CTA: 320 us, with boxes 313; a
    // prompt of 16384 1353, 1326); with fewer the CTA would only wait for them (a prompt of 500 tokens 1 us more).
    const bool box_out = (32 % a.G == 0 || a.G % 32 == 0) && a.tokens * a.hkv / (2 * p.tq_tokens) >= 2 * (int64_t)w.ctas;
    const cuuint64_t out_strides[2] = {(cuuint64_t)a.hd * 2, (cuuint64_t)a.out_stride * 2};
    const cuuint32_t oheads = box_out ? (cuuint32_t)std::min(a.G, 32) : 1u;
    const cuuint32_t obox[3] = {64, oheads, box_out ? 32 / oheads : 1u};
    if (enc(&p.tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(a.q), dims, strides, qbox, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS ||
        (box_out && enc(&p.to, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.out, dims, out_strides, obox, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS) ||
        !make_cache_tmap(&p.tk, a.k, a.num_pages, a.k_page, a.hkv, ps, a.hd, box) ||
        !make_cache_tmap(&p.tv, a.v, a.num_pages, a.v_page, a.hkv, ps, a.hd, box))
        return USP_ERR_CUDA;
    p.s.cu = a.cu; p.s.kv = a.kv;
    p.s.tokens = a.tokens; p.s.max_keys = paged_max_keys(a);
    p.s.nreq = a.nreq; p.s.hkv = a.hkv; p.s.G = a.G;
    p.s.tb = 2 * p.tq_tokens; p.s.causal = a.causal;
    p.s.n_lo = n_lo; p.s.n_hi = INT32_MAX;
    p.s.over = kOver; p.s.min_span = kMinSpan; p.s.long_parts = kManyParts;
    p.s.inv_ctas = 1.0f / (float)w.ctas;
    p.s.by_tb = FastDiv((uint32_t)p.s.tb); p.s.by_G = FastDiv((uint32_t)a.G);
    p.w = w;
    p.out = static_cast<__nv_bfloat16 *>(a.out);
    p.lse = a.lse;
    p.table = a.table;
    p.status = di->status;
    p.out_stride = a.out_stride; p.table_stride = a.table_stride;
    p.num_pages = (int32_t)a.num_pages; p.log_ps = a.log_ps; p.hq = a.hq;
    p.scale_log2 = a.scale_log2;
    if (box_out) return a.hd == 128 ? launch_typed<128, false, true>(p, w.ctas, s) : launch_typed<64, false, true>(p, w.ctas, s);
    return a.hd == 128 ? launch_typed<128, false, false>(p, w.ctas, s) : launch_typed<64, false, false>(p, w.ctas, s);
}

size_t q4_join_bytes(int ctas, int hd) { return (size_t)ctas * kM * (hd + 2) * 4; }

int launch_paged_q4_chunk(const PagedQ4Args &a, int n_lo, const PartSpace &w, float *join, cudaStream_t s) {
    const DeviceInfo *di = device_info();
    if (!di) return USP_ERR_CUDA;
    ChunkParams p{};
    const int ps = 1 << a.log_ps;
    const uint32_t box = (uint32_t)std::min(ps, kN);
    p.tq_tokens = kM / a.G;
    EncodeTiledFn enc = encode_fn();
    if (!enc) return USP_ERR_CUDA;
    const cuuint64_t dims[3] = {(cuuint64_t)a.hd, (cuuint64_t)a.hq, (cuuint64_t)a.tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)a.hd * 2, (cuuint64_t)a.q_stride * 2};
    const cuuint32_t qbox[3] = {64, (cuuint32_t)a.G, (cuuint32_t)p.tq_tokens}, estr[3] = {1, 1, 1};
    if (enc(&p.tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(a.q), dims, strides, qbox, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS ||
        !make_codes_tmap(&p.tk, a.k, a.num_pages, a.k_page, a.hkv, ps, a.hd, box) ||
        !make_codes_tmap(&p.tv, a.v, a.num_pages, a.v_page, a.hkv, ps, a.hd, box))
        return USP_ERR_CUDA;
    p.ks = a.ks; p.vs = a.vs; p.ks_page = a.ks_page; p.vs_page = a.vs_page;
    p.join = join;
    p.s.cu = a.cu; p.s.kv = a.kv;
    p.s.tokens = a.tokens; p.s.max_keys = q4_max_keys(a);
    p.s.nreq = a.nreq; p.s.hkv = a.hkv; p.s.G = a.G;
    p.s.tb = 2 * p.tq_tokens; p.s.causal = a.causal;
    p.s.n_lo = n_lo; p.s.n_hi = INT32_MAX;
    p.s.over = kOver; p.s.min_span = kMinSpan; p.s.long_parts = kManyParts;
    p.s.inv_ctas = 1.0f / (float)w.ctas;
    p.s.by_tb = FastDiv((uint32_t)p.s.tb); p.s.by_G = FastDiv((uint32_t)a.G);
    p.w = w;
    p.out = static_cast<__nv_bfloat16 *>(a.out);
    p.lse = a.lse;
    p.table = a.table;
    p.status = di->status;
    p.out_stride = a.out_stride; p.table_stride = a.table_stride;
    p.num_pages = (int32_t)a.num_pages; p.log_ps = a.log_ps; p.hq = a.hq;
    p.scale_log2 = a.scale_log2;
    return a.hd == 128 ? launch_typed<128, true, false>(p, w.ctas, s) : launch_typed<64, true, false>(p, w.ctas, s);
}

}  // namespace usp
