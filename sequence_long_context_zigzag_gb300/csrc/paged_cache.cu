// paged_cache.cu -- the paged K/V cache's bookkeeping: pages and slots for the next tokens from the
// requests' lengths (usp_page_plan), and the copy of their K and V rows into the cache
// (usp_cache_append).
#include <algorithm>

#include "paged.cuh"
#include "usp_internal.cuh"

namespace usp {
namespace {

// ------------------------------------------------------------------------------------------------
// usp_page_plan
// ------------------------------------------------------------------------------------------------
// Request i needs fresh_i = ceil((ctx_i + n_i) / ps) - ceil(ctx_i / ps) pages and n_i slots; their
// places are exclusive prefix sums over the requests. Every CTA owns a slice of the slot map and walks
// the requests in tiles of kTile with a running carry of both sums until its slice is done, so one
// launch suffices: repeating the scan costs less than a second launch or a grid-wide wait (64 to 1024
// requests are one tile, about a microsecond, and the lengths come from L2). Calls one after the other take 6.4 us for
// 64 requests and 6.2 to 7.1 for 256 with 272576 slots: the launch, the two dependent loads and the scan, and the host
// side of the call as long. A token finds its request
// by binary search in the tile's cumulative lengths in shared memory. A fresh page always begins with
// a new token of its request (position % ps == 0), so that token's thread writes the table entry; the
// pages of tokens behind max_tokens, which no thread has, are written by CTA 0.
// Sums are 64-bit; what is written saturates.
constexpr int kPlanThreads = 256;
constexpr int kPer = 4;
constexpr int kTile = kPlanThreads * kPer;

struct PlanArgs {
    const int32_t *ctx, *fresh_len, *free_pages, *free_head;
    int32_t *table, *slots, *cu, *kv, *counts;
    int64_t num_pages, table_stride, free_count, max_tokens, slice;
    int32_t nreq, max_pages, log_ps;
};

struct Pair {
    int64_t a, b;
};

// inclusive scan over the CTA's threads; total: the sums of all of them
__device__ __forceinline__ Pair block_scan(Pair x, Pair *warp_sums, Pair &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t a = __shfl_up_sync(0xffffffffu, x.a, o), b = __shfl_up_sync(0xffffffffu, x.b, o);
        if (lane >= o) {
            x.a += a;
            x.b += b;
        }
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    total = Pair{0, 0};
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        const Pair s = warp_sums[w];
        if (w < warp) {
            x.a += s.a;
            x.b += s.b;
        }
        total.a += s.a;
        total.b += s.b;
    }
    return x;
}

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const PlanArgs p) {
    __shared__ Pair warp_sums[kPlanThreads / 32];
    __shared__ int64_t cu_s[kTile + 1];  // cumulative new tokens before each request of the tile
    __shared__ int64_t page_s[kTile];    // place of the request's first fresh page in free_pages
    __shared__ int32_t ctx_s[kTile];
    __shared__ int64_t red[kPlanThreads / 32];
    __shared__ int32_t red_max[kPlanThreads / 32];
    wait_grid_before();
    const int tid = threadIdx.x, ps = 1 << p.log_ps;
    const int64_t t0 = (int64_t)blockIdx.x * p.slice, t1 = min(t0 + p.slice, p.max_tokens);
    const bool writer = blockIdx.x == 0;  // CTA 0 walks all requests and writes the per-request outputs
    const int64_t head = max(*p.free_head, 0);
    Pair carry{0, head};
    int64_t lost = 0;
    int32_t longest = 0;
    for (int base = 0; base < p.nreq && (writer || carry.a < t1); base += kTile) {
        int32_t ctx[kPer], len[kPer];
        Pair mine[kPer], sum{0, 0};
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int i = base + tid * kPer + e;
            ctx[e] = i < p.nreq ? max(p.ctx[i], 0) : 0;
            len[e] = i < p.nreq ? max(p.fresh_len[i], 0) : 0;
            const int64_t end = (int64_t)ctx[e] + len[e];
            mine[e] = sum;  // exclusive within the thread
            sum.a += len[e];
            sum.b += ((end + ps - 1) >> p.log_ps) - (((int64_t)ctx[e] + ps - 1) >> p.log_ps);
        }
        Pair total;
        const Pair incl = block_scan(sum, warp_sums, total);
        const Pair off{carry.a + incl.a - sum.a, carry.b + incl.b - sum.b};
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int l = tid * kPer + e, i = base + l;
            const int64_t cu = off.a + mine[e].a, first = off.b + mine[e].b, end = (int64_t)ctx[e] + len[e];
            cu_s[l] = cu;
            page_s[l] = first;
            ctx_s[l] = ctx[e];
            if (writer && i < p.nreq) {
                p.cu[i] = (int32_t)min(cu, p.max_tokens);
                p.kv[i] = (int32_t)min(end, (int64_t)INT32_MAX);
                // tokens at or behind the first position that has no page, or no place in slot_map
                const int64_t old = ((int64_t)ctx[e] + ps - 1) >> p.log_ps;
                const int64_t cols = min((int64_t)p.max_pages, old + max(p.free_count - first, (int64_t)0));
                const int64_t fit = min(cols << p.log_ps, (int64_t)ctx[e] + max(p.max_tokens - cu, (int64_t)0));
                lost += max(end - max(fit, (int64_t)ctx[e]), (int64_t)0);
                longest = max(longest, (int32_t)min(end, (int64_t)INT32_MAX));
            }
        }
        if (tid == 0) cu_s[kTile] = carry.a + total.a;
        __syncthreads();
        const int64_t a = max(t0, carry.a), b = min(t1, carry.a + total.a);
        for (int64_t t = a + tid; t < b; t += kPlanThreads) {
            int lo = 0;  // the request is the last one with cu_s <= t (empty ones come before)
#pragma unroll
            for (int step = kTile / 2; step > 0; step >>= 1)
                if (cu_s[lo + step] <= t) lo += step;
            const int64_t i = base + lo, pos = (int64_t)ctx_s[lo] + (t - cu_s[lo]);
            const int64_t col = pos >> p.log_ps, old = ((int64_t)ctx_s[lo] + ps - 1) >> p.log_ps;
            int32_t page = -1;
            if (col < p.max_pages) {
                int32_t *entry = p.table + i * p.table_stride + col;
                if (col < old) {
                    page = *entry;
                } else {
                    const int64_t at = page_s[lo] + (col - old);
                    if (at < p.free_count) page = p.free_pages[at];
                    if ((pos & (ps - 1)) == 0) *entry = page;
                }
            }
            const bool ok = page >= 0 && page < p.num_pages;
            p.slots[t] = ok ? (page << p.log_ps) + (int32_t)(pos & (ps - 1)) : -1;
        }
        if (writer && carry.a + total.a > p.max_tokens) {
            // a warp per request, a lane per column, from the first page that a token at max_tokens or behind opens
            for (int l = tid >> 5; l < kTile && base + l < p.nreq; l += kPlanThreads / 32) {
                const int64_t ctx0 = ctx_s[l], end = ctx0 + (cu_s[l + 1] - cu_s[l]);
                const int64_t old = (ctx0 + ps - 1) >> p.log_ps;
                const int64_t from = ctx0 + max(p.max_tokens - cu_s[l], (int64_t)0);  // its first token without a place
                const int64_t cols = min((end + ps - 1) >> p.log_ps, (int64_t)p.max_pages);
                for (int64_t col = ((from + ps - 1) >> p.log_ps) + (tid & 31); col < cols; col += 32) {
                    const int64_t at = page_s[l] + (col - old);
                    p.table[(int64_t)(base + l) * p.table_stride + col] = at < p.free_count ? p.free_pages[at] : -1;
                }
            }
        }
        carry.a += total.a;
        carry.b += total.b;
        __syncthreads();
    }
    for (int64_t t = max(t0, carry.a) + tid; t < t1; t += kPlanThreads) p.slots[t] = -1;
    if (!writer) return;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        lost += __shfl_xor_sync(0xffffffffu, lost, o);
        longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, o));
    }
    if ((tid & 31) == 0) {
        red[tid >> 5] = lost;
        red_max[tid >> 5] = longest;
    }
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < kPlanThreads / 32; ++w) {
            lost += red[w];
            longest = max(longest, red_max[w]);
        }
        p.cu[p.nreq] = (int32_t)min(carry.a, p.max_tokens);
        p.counts[0] = (int32_t)min(carry.a, (int64_t)INT32_MAX);
        p.counts[1] = (int32_t)min(carry.b, (int64_t)INT32_MAX);
        p.counts[2] = (int32_t)min(lost, (int64_t)INT32_MAX);
        p.counts[3] = longest;
    }
}

// ------------------------------------------------------------------------------------------------
// usp_cache_append
// ------------------------------------------------------------------------------------------------
// A pure copy, bound by HBM: 16-byte pieces, kUnroll of K and V each in flight per thread. A token's
// hkv * hd elements are contiguous in the source and go to hkv runs of hd elements in its page. A CTA takes
// consecutive pieces, so that the accesses in flight lie close together: 73055 tokens of 8 heads of 128
// (599 MB) in 87 us, 1.03 of the measured copy rate; with strides of the whole grid between a thread's
// pieces 105 us. More pieces per thread gain nothing and cost a small call CTAs.
constexpr int kAppendThreads = 256;
constexpr int kUnroll = 2;

struct AppendArgs {
    const char *k, *v;
    char *kc, *vc;
    const int32_t *slots;
    int64_t k_stride, v_stride, k_page, v_page;  // bytes
    uint32_t pieces;                             // 16-byte pieces of K in all
    uint32_t nslots;
    int32_t log_ps, log_row;  // page size; 16-byte pieces per head row (hd * es / 16, a power of two)
    FastDiv per_token;        // pieces per token
};

__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(const AppendArgs p) {
    wait_grid_before();
    uint4 k[kUnroll], v[kUnroll];
    int64_t kd[kUnroll], vd[kUnroll];
    bool ok[kUnroll];
#pragma unroll
    for (int e = 0; e < kUnroll; ++e) {
        const uint32_t x = (blockIdx.x * kUnroll + e) * kAppendThreads + threadIdx.x;
        ok[e] = x < p.pieces;
        if (!ok[e]) continue;
        uint32_t t, r;
        p.per_token.divmod(x, t, r);
        const uint32_t slot = (uint32_t)p.slots[t];
        ok[e] = slot < p.nslots;
        if (!ok[e]) continue;
        k[e] = reinterpret_cast<const uint4 *>(p.k + t * p.k_stride)[r];
        v[e] = reinterpret_cast<const uint4 *>(p.v + t * p.v_stride)[r];
        const uint32_t h = r >> p.log_row, c = r & ((1u << p.log_row) - 1);
        const int64_t page = slot >> p.log_ps;
        const int64_t in = (((int64_t)h << p.log_ps) + (slot & ((1u << p.log_ps) - 1))) << p.log_row;
        kd[e] = page * p.k_page + (in + c) * 16;
        vd[e] = page * p.v_page + (in + c) * 16;
    }
#pragma unroll
    for (int e = 0; e < kUnroll; ++e) {
        if (!ok[e]) continue;
        *reinterpret_cast<uint4 *>(p.kc + kd[e]) = k[e];
        *reinterpret_cast<uint4 *>(p.vc + vd[e]) = v[e];
    }
}

int log2_of(int64_t x) {
    int l = 0;
    while ((int64_t(1) << l) < x) ++l;
    return l;
}

}  // namespace

int check_cache_dims(const usp_cache_dims &d) {
    if (d.num_pages < 0 || d.hkv <= 0 || d.k_page_stride < 0 || d.v_page_stride < 0) return USP_ERR_INVALID_ARG;
    const int es = elem_size(d.dtype);
    if (es == 0) return USP_ERR_DTYPE;
    if (d.hd != 64 && d.hd != 128) return USP_ERR_UNSUPPORTED;
    if (!valid_page_size(d.page_size)) return USP_ERR_UNSUPPORTED;
    // the tensor maps count rows in 31 bits; so do slots
    if (d.num_pages >= (int64_t(1) << 31) / d.page_size || d.hkv > 65536) return USP_ERR_UNSUPPORTED;
    const int64_t dense = (int64_t)d.hkv * d.page_size * d.hd;
    for (int64_t st : {d.k_page_stride, d.v_page_stride}) {
        if (st != 0 && st < dense) return USP_ERR_SHAPE;
        if (st >= (int64_t(1) << 38)) return USP_ERR_UNSUPPORTED;  // the tensor maps' strides end at 2^40 bytes
        if (st * es % 16 != 0) return USP_ERR_ALIGN;
    }
    return USP_OK;
}

}  // namespace usp

using namespace usp;

extern "C" {

int usp_page_plan(const int32_t *ctx_lens, const int32_t *new_lens, const int32_t *free_pages,
                  const int32_t *free_head, int32_t *block_table, int32_t *slot_map, int32_t *cu_new,
                  int32_t *kv_lens, int32_t *counts, usp_plan_dims d, usp_stream_t stream) {
    if (d.nreq < 0 || d.max_pages < 0 || d.num_pages < 0 || d.free_count < 0 || d.max_tokens < 0)
        return USP_ERR_INVALID_ARG;
    if (!valid_page_size(d.page_size)) return USP_ERR_UNSUPPORTED;
    if (d.table_stride < d.max_pages) return USP_ERR_SHAPE;
    if (d.num_pages >= (int64_t(1) << 31) / d.page_size || d.max_tokens >= (int64_t(1) << 31) ||
        d.free_count >= (int64_t(1) << 31) || d.nreq > kMaxRequests)
        return USP_ERR_UNSUPPORTED;
    // empty arrays may be null: no request, no free page, no column, no token
    if (!free_head || !cu_new || !counts || (d.nreq > 0 && (!ctx_lens || !new_lens || !kv_lens)) ||
        (d.free_count > 0 && !free_pages) || (d.nreq > 0 && d.max_pages > 0 && !block_table) ||
        (d.max_tokens > 0 && !slot_map))
        return USP_ERR_INVALID_ARG;
    const void *ptrs[] = {ctx_lens, new_lens, free_pages, free_head, block_table, slot_map, cu_new, kv_lens, counts};
    for (const void *x : ptrs)
        if (!aligned(x, 4)) return USP_ERR_ALIGN;
    // CTA 0 writes these while others may still have to read the lengths and the head
    struct Range {
        const int32_t *p;
        int64_t n;
    };
    const Range in[] = {{ctx_lens, d.nreq}, {new_lens, d.nreq}, {free_pages, d.free_count}, {free_head, 1}};
    const Range out[] = {{slot_map, d.max_tokens}, {cu_new, d.nreq + 1}, {kv_lens, d.nreq}, {counts, 4}};
    for (const Range &i : in)
        for (const Range &o : out)
            if (i.p < o.p + o.n && o.p < i.p + i.n) return USP_ERR_INVALID_ARG;
    const DeviceInfo *di = device_info();
    if (!di) return USP_ERR_CUDA;
    PlanArgs a{};
    a.ctx = ctx_lens; a.fresh_len = new_lens; a.free_pages = free_pages; a.free_head = free_head;
    a.table = block_table; a.slots = slot_map; a.cu = cu_new; a.kv = kv_lens; a.counts = counts;
    a.num_pages = d.num_pages; a.table_stride = d.table_stride; a.free_count = d.free_count;
    a.max_tokens = d.max_tokens;
    a.nreq = d.nreq; a.max_pages = d.max_pages; a.log_ps = log2_of(d.page_size);
    // slices of one slot per thread at least, at most two CTAs per SM (272576 slots of 256 requests: 6.0 to
    // 6.8 us, with one or four per SM the same, with eight, where the repeated scan shows, 8.1)
    const int64_t ctas = std::max<int64_t>(
        1, std::min<int64_t>((d.max_tokens + kPlanThreads - 1) / kPlanThreads, 2 * (int64_t)di->sm_count));
    a.slice = (d.max_tokens + ctas - 1) / ctas;
    return launch_overlapped(page_plan_kernel, dim3((unsigned)ctas), kPlanThreads, 0,
                             reinterpret_cast<cudaStream_t>(stream), a);
}

int usp_cache_append(const void *k, const void *v, void *k_cache, void *v_cache, const int32_t *slot_map,
                     int64_t tokens, int64_t k_stride, int64_t v_stride, usp_cache_dims d, usp_stream_t stream) {
    if (tokens < 0 || k_stride < 0 || v_stride < 0) return USP_ERR_INVALID_ARG;
    int rc = check_cache_dims(d);
    if (rc) return rc;
    const int es = elem_size(d.dtype);
    const int64_t row = (int64_t)d.hkv * d.hd;
    for (int64_t st : {k_stride, v_stride}) {
        if (st != 0 && st < row) return USP_ERR_SHAPE;
        if (st >= (int64_t(1) << 38)) return USP_ERR_UNSUPPORTED;
        if (st * es % 16 != 0) return USP_ERR_ALIGN;
    }
    if (tokens == 0 || d.num_pages == 0) return USP_OK;
    if (!k || !v || !k_cache || !v_cache || !slot_map) return USP_ERR_INVALID_ARG;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(slot_map, 4))
        return USP_ERR_ALIGN;
    const int64_t per_token = row * es / 16;
    if (tokens >= (int64_t(1) << 31) / per_token) return USP_ERR_UNSUPPORTED;
    AppendArgs a{};
    a.k = static_cast<const char *>(k); a.v = static_cast<const char *>(v);
    a.kc = static_cast<char *>(k_cache); a.vc = static_cast<char *>(v_cache);
    a.slots = slot_map;
    const int64_t dense = row * d.page_size;
    a.k_stride = (k_stride ? k_stride : row) * es;
    a.v_stride = (v_stride ? v_stride : row) * es;
    a.k_page = (d.k_page_stride ? d.k_page_stride : dense) * es;
    a.v_page = (d.v_page_stride ? d.v_page_stride : dense) * es;
    a.pieces = (uint32_t)(tokens * per_token);
    a.nslots = (uint32_t)(d.num_pages * d.page_size);
    a.log_ps = log2_of(d.page_size);
    a.log_row = log2_of((int64_t)d.hd * es / 16);
    a.per_token = FastDiv((uint32_t)per_token);
    const unsigned grid = (a.pieces + (unsigned)(kAppendThreads * kUnroll) - 1) / (kAppendThreads * kUnroll);
    return launch_overlapped(cache_append_kernel, dim3(grid), kAppendThreads, 0, reinterpret_cast<cudaStream_t>(stream), a);
}

}  // extern "C"
