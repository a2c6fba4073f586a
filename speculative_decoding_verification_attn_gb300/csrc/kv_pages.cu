// Pages of a paged cache that several rows hold: forking and releasing rows,
// and moving the accepted path of a token tree to the front.
//
// A row of the block table lists its pages, then -1.  page_refs counts the
// rows that hold a page; 0 means free, and fresh pages are the free ones of
// lowest id in the order of the pairs that ask for them, so a call's result does not depend
// on the order in which its blocks run.
//
// Fork, two launches, since every decision is taken on the state before the call:
//  * plan: blocks of kScan pages write two bits per page (free, held by one
//    row) and the number of free ones; a block per pair checks it and counts the
//    fresh pages it needs.
//  * apply: a block per pair and slice of its copy finds the pair's first
//    fresh page (pairs before it, then blocks of pages before it, then bits), shares
//    the whole pages, takes the fresh ones, and copies the rows of the page in
//    use.
// Release, one launch: a block per row (the first that lists it), eight entries of a
// thread under way together.
// All of it is launch latency, a few dependent round trips and the atomics on the counts:
// a table row of 2048 entries is 8 KB, a copy at most a page.  240 rows of 1024 to 2048
// pages released and forked again: 37 us with one entry of a thread at a time and an
// exchange for each, 25 us so.  56 beams of 64 to 512 pages: 10 us.
//
// Compaction, one launch: a block per (sequence, kv-head, tensor).  Row path[i]
// goes to place i <= path[i], so blocks of rows in ascending order may be read
// and written in turn; an e4m3 page's rows are all read first, since its scale,
// and with it the codes of every row it keeps, may change.
#include <math.h>

#include "common.cuh"
#include "places.h"

namespace specv {
namespace {

constexpr int kThreads = 256;
constexpr int kScan = 2048;  // pages of a planning block: 8 ballots a warp
constexpr float kE4m3Max = 448.f;
constexpr int kBatch = 8;    // entries of a thread whose loads and atomics are under way together

__device__ __forceinline__ int block_sum(int v, int* s_warp) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();  // s_warp may still be read from before
    if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = v;
    __syncthreads();
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) sum += s_warp[w];
    return sum;
}

// Pages of a pair: `whole` shared, then up to `total`; `part` rows of page
// `whole` are in use.
struct Span {
    int whole, total, part;
};
__device__ __forceinline__ bool pair_span(const ForkArgs& a, int ctx, Span* s) {
    const int64_t total = ((int64_t)ctx + a.room + a.P - 1) / a.P;
    if (ctx < 0 || total > a.max_pages) return false;
    s->whole = ctx / a.P;
    s->total = (int)total;
    s->part = ctx - s->whole * a.P;
    return true;
}

__global__ void __launch_bounds__(kThreads) fork_plan_kernel(const ForkArgs a) {
    __shared__ int s_warp[kThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dep_launch_dependents();
    grid_dep_wait();
    if ((int)blockIdx.x >= a.n) {  // pages
        constexpr int kWords = kScan / 32 / (kThreads / 32);
        const int64_t p0 = (int64_t)(blockIdx.x - a.n) * kScan + warp * (32 * kWords);
        int refs[kWords];
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            const int64_t p = p0 + i * 32 + lane;
            refs[i] = p < a.num_pages ? a.page_refs[p] : -1;
        }
        uint32_t none = 0, one = 0;
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            const uint32_t w0 = __ballot_sync(0xffffffffu, refs[i] == 0);
            const uint32_t w1 = __ballot_sync(0xffffffffu, refs[i] == 1);
            if (lane == i) {
                none = w0;
                one = w1;
            }
        }
        if (lane < kWords) {
            a.free_bits[p0 / 32 + lane] = none;
            a.one_bits[p0 / 32 + lane] = one;
        }
        int free = __popc(none);
        free = block_sum(free, s_warp);
        if (tid == 0) a.free_count[blockIdx.x - a.n] = free;
        return;
    }
    // a pair
    const int j = blockIdx.x, p = a.parents[j], c = a.children[j];
    int bad = 0, fresh = 0, src = -1;
    Span span = {0, 0, 0};
    if (p < 0 || p >= a.rows || c < 0 || c >= a.rows) {
        bad = SPEC_DEVERR_POOL;
    } else {
        const int32_t* from = a.block_table + (int64_t)p * a.max_pages;
        if (!pair_span(a, a.ctx_lens[p], &span)) bad = SPEC_DEVERR_CTX;
        // a child that is another pair's child or parent, or that holds pages
        for (int i = tid; i < a.n; i += kThreads)
            if ((a.children[i] == c && i < j) || (i != j && c != p && a.parents[i] == c))
                bad |= SPEC_DEVERR_POOL;
        if (c != p && a.block_table[(int64_t)c * a.max_pages] >= 0) bad |= SPEC_DEVERR_POOL;
        if (!(bad & SPEC_DEVERR_CTX)) {
#pragma unroll 8
            for (int i = tid; i < span.whole + (span.part > 0); i += kThreads) {
                const int page = __ldg(from + i);
                if (page < 0 || page >= a.num_pages) bad |= SPEC_DEVERR_PAGE;
                if (i == span.whole) src = page;
            }
            for (int i = span.whole + tid; i < span.total; i += kThreads) {
                const int page = c == p ? from[i] : -1;
                fresh += page < 0 || page >= a.num_pages || a.page_refs[page] != 1;
                if (page >= a.num_pages) bad |= SPEC_DEVERR_PAGE;
            }
        }
    }
    const int flags = (__syncthreads_or(bad & SPEC_DEVERR_PAGE) ? SPEC_DEVERR_PAGE : 0) |
                      (__syncthreads_or(bad & SPEC_DEVERR_CTX) ? SPEC_DEVERR_CTX : 0) |
                      (__syncthreads_or(bad & SPEC_DEVERR_POOL) ? SPEC_DEVERR_POOL : 0);
    fresh = block_sum(fresh, s_warp);
    if (flags && tid == 0) raise_device_error(a.dev_err, flags);
    if (tid == 0) a.need[j] = flags ? -1 : fresh;
    if (src >= 0 || (tid == 0 && span.part == 0)) a.src[j] = src;  // one thread
}

// The fresh page of rank r (the r-th lowest free one): called by a warp that is
// converged; first[b] of the block of pages that holds it comes from a scan.
__device__ __forceinline__ int select_bit(const uint32_t* words, int r) {
    // words of a block of pages: 8 per lane
    const int lane = threadIdx.x & 31;
    uint32_t w[kScan / 1024];
    int n = 0;
#pragma unroll
    for (int i = 0; i < kScan / 1024; ++i) {
        w[i] = words[lane * (kScan / 1024) + i];
        n += __popc(w[i]);
    }
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    int at = -1, left = r - (incl - n);
    if (left >= 0 && left < n) {
#pragma unroll
        for (int i = 0; i < kScan / 1024; ++i) {
            const int k = __popc(w[i]);
            if (at < 0 && left < k) at = (lane * (kScan / 1024) + i) * 32 + (int)__fns(w[i], 0, left + 1);
            left -= k;
        }
    }
    const uint32_t who = __ballot_sync(0xffffffffu, at >= 0);
    return __shfl_sync(0xffffffffu, at, who ? __ffs(who) - 1 : 0);
}

// Page of the r-th lowest free id, or -1 (warp).
__device__ __forceinline__ int fresh_page(const ForkArgs& a, int64_t r) {
    const int lane = threadIdx.x & 31;
    const int blocks = (int)(((int64_t)a.num_pages + kScan - 1) / kScan);
    int64_t before = 0;
    for (int b0 = 0; b0 < blocks; b0 += 32) {
        const int n = b0 + lane < blocks ? a.free_count[b0 + lane] : 0;
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, before + incl > r);
        if (past) {
            const int w = __ffs(past) - 1;
            const int64_t base = before + __shfl_sync(0xffffffffu, incl - n, w);
            return (b0 + w) * kScan + select_bit(a.free_bits + (int64_t)(b0 + w) * (kScan / 32),
                                                 (int)(r - base));
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
    return -1;
}

__device__ __forceinline__ bool bit_of(const uint32_t* bits, int page) {
    return (bits[page >> 5] >> (page & 31)) & 1;
}

// Copies the first `part` rows of heads [h0, h1) of page `src` to page `dst`.
__device__ __forceinline__ void copy_rows(const ForkArgs& a, int src, int dst, int part, int h0, int h1) {
    const int chunks = row_pieces(part, a.D, a.elem);  // of a head
    const int64_t head = (int64_t)a.P * a.D * a.elem / 16;
    const int all = chunks * (h1 - h0) * 2;
    for (int e = threadIdx.x; e < all; e += kThreads) {
        const int t = e & 1, r = e >> 1, h = h0 + r / chunks, i = r % chunks;
        uint4* cache = reinterpret_cast<uint4*>(t ? a.v_cache : a.k_cache);
        cache[((int64_t)dst * a.Hkv + h) * head + i] = cache[((int64_t)src * a.Hkv + h) * head + i];
    }
    if (a.cache_dtype == SPEC_DTYPE_I8) {
        for (int e = threadIdx.x; e < part * (h1 - h0) * 2; e += kThreads) {
            const int t = e & 1, r = e >> 1, h = h0 + r / part, i = r % part;
            uint16_t* sc = static_cast<uint16_t*>(t ? a.v_scale : a.k_scale);
            sc[((int64_t)dst * a.Hkv + h) * a.P + i] = sc[((int64_t)src * a.Hkv + h) * a.P + i];
        }
    } else if (a.cache_dtype == SPEC_DTYPE_E4M3) {
        for (int e = threadIdx.x; e < (h1 - h0) * 2; e += kThreads) {
            float* sc = static_cast<float*>(e & 1 ? a.v_scale : a.k_scale);
            sc[(int64_t)dst * a.Hkv + h0 + (e >> 1)] = sc[(int64_t)src * a.Hkv + h0 + (e >> 1)];
        }
    }
}

// grid (pairs, slices of the heads)
__global__ void __launch_bounds__(kThreads) fork_apply_kernel(const ForkArgs a) {
    __shared__ int s_warp[kThreads / 32];
    __shared__ int s_first;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int j = blockIdx.x;
    grid_dep_launch_dependents();
    grid_dep_wait();
    const int need = a.need[j];
    if (need < 0) return;
    // (a sum of needs may pass 32 bits: in two halves)
    int64_t before = 0;
    for (int i = tid; i < j; i += kThreads) before += max(0, a.need[i]);
    const int low = block_sum((int)(before & 0xfffff), s_warp);
    before = ((int64_t)block_sum((int)min(before >> 20, (int64_t)1 << 22), s_warp) << 20) + low;
    int free = 0;
    const int blocks = (int)(((int64_t)a.num_pages + kScan - 1) / kScan);
    for (int i = tid; i < blocks; i += kThreads) free += a.free_count[i];
    free = block_sum(free, s_warp);
    const int p = a.parents[j], c = a.children[j];
    if (need > 0 && before + need > free) {  // out of pages
        if (tid == 0 && blockIdx.y == 0) raise_device_error(a.dev_err, SPEC_DEVERR_POOL);
        return;
    }
    Span span;
    const int ctx = a.ctx_lens[p];
    pair_span(a, ctx, &span);
    const int32_t* from = a.block_table + (int64_t)p * a.max_pages;
    int32_t* to = a.block_table + (int64_t)c * a.max_pages;
    const int src = a.src[j];

    // the page in use: copied unless the row itself goes on and holds it alone
    const bool copy = span.part > 0 && span.whole < span.total &&
                      !(c == p && bit_of(a.one_bits, src));
    if (copy) {
        if (warp == 0) {
            const int page = fresh_page(a, before);  // the pair's first
            if (lane == 0) s_first = page;
        }
        __syncthreads();
        const int per = (a.Hkv + gridDim.y - 1) / gridDim.y;
        const int h0 = blockIdx.y * per, h1 = min(a.Hkv, h0 + per);
        if (h0 < h1 && s_first >= 0) copy_rows(a, src, s_first, span.part, h0, h1);
    }
    if (blockIdx.y) return;

    if (c != p) {
        for (int i0 = tid; i0 < span.whole; i0 += kThreads * kBatch) {
            int page[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                if (i0 + u * kThreads < span.whole) page[u] = __ldcg(from + i0 + u * kThreads);
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                if (i0 + u * kThreads < span.whole) {
                    to[i0 + u * kThreads] = page[u];
                    atomicAdd(&a.page_refs[page[u]], 1);
                }
        }
        for (int i = span.total + tid; i < a.max_pages; i += kThreads) to[i] = -1;
        if (tid == 0) a.ctx_lens[c] = ctx;
    }
    // fresh pages, in the order of their places: a warp each, ranks by counting
    // the places before (a row's own pages that it keeps take none)
    int taken = 0;
    for (int i0 = span.whole; i0 < span.total; i0 += kThreads / 32) {
        // whether each of this round's places needs a page
        bool want[kThreads / 32];
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            const int i = i0 + w;
            want[w] = false;
            if (i < span.total) {
                const int page = c == p ? from[i] : -1;
                want[w] = page < 0 || !bit_of(a.one_bits, page);
            }
        }
        __syncthreads();  // every warp has read the round's places
        int rank = taken, mine = -1;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w == warp && want[w]) mine = rank;
            rank += want[w];
        }
        if (mine >= 0) {
            const int page = fresh_page(a, before + mine);
            if (lane == 0 && page >= 0) {
                const int i = i0 + warp, old = c == p ? to[i] : -1;
                to[i] = page;
                a.page_refs[page] = 1;
                if (old >= 0) atomicSub(&a.page_refs[old], 1);  // another row goes on with it
            }
        }
        taken = rank;
    }
}

__global__ void __launch_bounds__(kThreads) release_kernel(const ReleaseArgs a) {
    const int tid = threadIdx.x, j = blockIdx.x;
    grid_dep_launch_dependents();
    grid_dep_wait();
    const int r = a.rows[j];
    if (r < 0 || r >= a.batch) {
        if (tid == 0) raise_device_error(a.dev_err, SPEC_DEVERR_POOL);
        return;
    }
    // a row that is listed several times keeps the least, and its first block drops the pages
    int keep = a.keep_lens ? max(0, a.keep_lens[j]) : 0;
    bool earlier = false;
    int least = keep;
    for (int i = tid; i < a.n; i += kThreads)
        if (i != j && a.rows[i] == r) {
            earlier |= i < j;
            least = min(least, a.keep_lens ? max(0, a.keep_lens[i]) : 0);
        }
    const int again = __syncthreads_or((earlier ? 1 : 0) | (least < keep ? 2 : 0));
    if (again) {  // (rare) settle both with the whole block
        if (__syncthreads_or(earlier)) return;
        __shared__ int s_least;
        if (tid == 0) s_least = keep;
        __syncthreads();
        atomicMin(&s_least, least);
        __syncthreads();
        keep = s_least;
    }
    int32_t* row = a.block_table + (int64_t)r * a.max_pages;
    if (tid == 0) a.ctx_lens[r] = min(a.ctx_lens[r], keep);
    // (no more than the table has: what follows adds to it)
    const int first = entries_kept(keep, a.P, a.max_pages);
    int bad = 0;
    for (int i0 = first + tid; i0 < a.max_pages; i0 += kThreads * kBatch) {
        int page[kBatch], old[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int i = i0 + u * kThreads;
            page[u] = i < a.max_pages ? row[i] : -1;
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            old[u] = 1;
            if (page[u] < 0) continue;
            row[i0 + u * kThreads] = -1;
            if (page[u] >= a.num_pages) bad |= SPEC_DEVERR_PAGE;
            else old[u] = atomicSub(&a.page_refs[page[u]], 1);
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (old[u] <= 0) {  // nobody held it
                atomicAdd(&a.page_refs[page[u]], 1);
                bad |= SPEC_DEVERR_POOL;
            }
    }
    if (bad) raise_device_error(a.dev_err, bad);
}

// ------------------------------------------------------------------ compaction

constexpr int kCThreads = 128;
constexpr int kChunks = 4;  // 16-byte pieces of a thread between two barriers

// A sequence's moves in one kv-head: rows of the cache ((page * Hkv + head) * P + slot) of
// the place i and of its source, -1 where nothing moves, and their pages.
struct Moves {
    int64_t dst[64], src[64];
    int dst_page[64], src_page[64];
    int n;
};

struct Place {
    int page, slot;
};
__device__ __forceinline__ Place place_of(const CompactArgs& a, int b, uint32_t pos, int* bad) {
    const uint32_t n = pos / (uint32_t)a.P;
    if (n >= (uint32_t)a.max_pages) {
        *bad |= SPEC_DEVERR_CTX;
        return {-1, 0};
    }
    const int page = a.block_table[(int64_t)b * a.max_pages + n];
    if (page < 0 || page >= a.num_pages) {
        *bad |= SPEC_DEVERR_PAGE;
        return {-1, 0};
    }
    return {page, (int)(pos - n * a.P)};
}

__device__ __forceinline__ void find_moves(const CompactArgs& a, int b, int h, Moves& mv) {
    const int tid = threadIdx.x;
    if (tid < 64) {
        const int from = tid < a.k ? a.path[(int64_t)b * a.k + tid] : -1;
        int n = a.accepted[b], bad = 0;
        const int ctx = a.ctx_lens[b];
        n = n < 0 ? 0 : n > a.k ? a.k : n;
        Place d = {-1, 0}, s = {-1, 0};
        if (tid < n) {
            if (from < tid || from >= a.k) {
                bad = SPEC_DEVERR_TREE;
            } else if (ctx < 0) {
                bad = SPEC_DEVERR_CTX;
            } else if (from != tid) {
                d = place_of(a, b, (uint32_t)ctx + tid, &bad);
                s = place_of(a, b, (uint32_t)ctx + from, &bad);
            }
        }
        if (bad) raise_device_error(a.dev_err, bad);
        const bool go = d.page >= 0 && s.page >= 0;
        mv.dst[tid] = go ? ((int64_t)d.page * a.Hkv + h) * a.P + d.slot : -1;
        mv.src[tid] = ((int64_t)s.page * a.Hkv + h) * a.P + s.slot;
        mv.dst_page[tid] = d.page;
        mv.src_page[tid] = s.page;
        if (tid == 0) mv.n = n;
    }
    __syncthreads();
}

// Rows whose bytes move as they are (fp32, bf16, INT8 with its scales).
__global__ void __launch_bounds__(kCThreads) compact_kernel(const CompactArgs a) {
    __shared__ Moves mv;
    const int tid = threadIdx.x, t = blockIdx.x & 1, h = blockIdx.x >> 1, b = blockIdx.y;
    grid_dep_launch_dependents();
    grid_dep_wait();
    find_moves(a, b, h, mv);
    const int per = a.D * a.elem / 16;  // pieces of a row
    uint4* cache = reinterpret_cast<uint4*>(t ? a.v_cache : a.k_cache);
    uint16_t* sc = static_cast<uint16_t*>(t ? a.v_scale : a.k_scale);
    uint16_t scale = 0;
    const bool with_scale = a.cache_dtype == SPEC_DTYPE_I8 && tid < mv.n && mv.dst[tid] >= 0;
    if (with_scale) scale = sc[mv.src[tid]];
    for (int e0 = 0; e0 < mv.n * per; e0 += kCThreads * kChunks) {
        uint4 x[kChunks];
#pragma unroll
        for (int u = 0; u < kChunks; ++u) {
            const int e = e0 + u * kCThreads + tid, i = e / per;
            if (i < mv.n && mv.dst[i] >= 0) x[u] = cache[mv.src[i] * per + e - i * per];
        }
        __syncthreads();  // places up to the last read are written only now
#pragma unroll
        for (int u = 0; u < kChunks; ++u) {
            const int e = e0 + u * kCThreads + tid, i = e / per;
            if (i < mv.n && mv.dst[i] >= 0) cache[mv.dst[i] * per + e - i * per] = x[u];
        }
        __syncthreads();
    }
    if (with_scale) sc[mv.dst[tid]] = scale;
}

__device__ __forceinline__ uint8_t e4m3_of(float x) {
    return (uint8_t)__nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float e4m3_value(uint8_t c) {
    __nv_fp8_e4m3 v;
    v.__x = c;
    return (float)v;
}

// e4m3: a place's page may have to take a larger scale.  The moved rows and every scale come
// in one round trip; the rest is arithmetic between barriers.
constexpr int kEThreads = 256;

__global__ void __launch_bounds__(kEThreads) compact_e4m3_kernel(const CompactArgs a) {
    __shared__ Moves mv;
    __shared__ __align__(16) uint8_t s_row[64 * 256];
    __shared__ float s_src[64];             // scale of a move's source page
    __shared__ float s_old[65], s_new[65];  // scales of the pages that hold the drafts' places
    __shared__ int s_page[65];
    const int tid = threadIdx.x, lane = tid & 31, t = blockIdx.x & 1, h = blockIdx.x >> 1, b = blockIdx.y;
    grid_dep_launch_dependents();
    grid_dep_wait();
    uint8_t* cache = static_cast<uint8_t*>(t ? a.v_cache : a.k_cache);
    float* scales = static_cast<float*>(t ? a.v_scale : a.k_scale);
    const int ctx = a.ctx_lens[b];
    const int g0 = ctx / a.P;
    const int pages = ctx < 0 ? 0 : ((uint32_t)ctx + a.k - 1) / (uint32_t)a.P - g0 + 1;  // 65 at most
    // (the last threads, while the first 64 find the moves)
    for (int g = kEThreads - 1 - tid; g < pages; g += kEThreads) {
        int page = -1;
        if (in_table(g0, g, a.max_pages)) page = a.block_table[(int64_t)b * a.max_pages + g0 + g];
        if (page >= a.num_pages) page = -1;
        s_page[g] = page;
        s_old[g] = s_new[g] = page >= 0 ? scales[(int64_t)page * a.Hkv + h] : 0.f;
    }
    find_moves(a, b, h, mv);
    if (ctx < 0) return;
    if (tid < mv.n && mv.dst[tid] >= 0) s_src[tid] = scales[(int64_t)mv.src_page[tid] * a.Hkv + h];
    const int per = a.D / 16;  // 16-byte pieces of a row
    for (int e = tid; e < mv.n * per; e += kEThreads) {
        const int i = e / per;
        if (mv.dst[i] >= 0)
            *reinterpret_cast<uint4*>(s_row + e * 16) =
                *reinterpret_cast<const uint4*>(cache + mv.src[i] * a.D + (e - i * per) * 16);
    }
    __syncthreads();
    // the scale that a row needs in another page (a warp per row)
    for (int i = tid >> 5; i < mv.n; i += kEThreads / 32) {
        if (mv.dst[i] < 0 || mv.src_page[i] == mv.dst_page[i]) continue;
        int top = 0;  // largest code without its sign: codes are ordered as their values
        for (int d = lane * 4; d < a.D; d += 128) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(s_row + i * a.D + d);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int c = (w >> (8 * u)) & 0x7f;
                top = max(top, c == 0x7f ? 0 : c);  // a NaN asks for no scale
            }
        }
        top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0) {
            const float x = __fdiv_rn(e4m3_value((uint8_t)top) * s_src[i], kE4m3Max);
            const int g = ((uint32_t)ctx + i) / (uint32_t)a.P - g0;
            // (scales are >= 0: their bits are ordered as they are)
            atomicMax(reinterpret_cast<int*>(&s_new[g]), __float_as_int(x));
        }
    }
    __syncthreads();
    // pages whose scale grew: every row of the sequence keeps its value
    for (int g = 0; g < pages; ++g) {
        if (s_page[g] < 0 || !(s_new[g] > s_old[g])) continue;
        const int64_t left = (int64_t)ctx + a.k - (int64_t)(g0 + g) * a.P;
        const int slots = (int)(left < a.P ? left : a.P);
        uint8_t* p = cache + ((int64_t)s_page[g] * a.Hkv + h) * a.P * a.D;
        for (int e = tid * 4; e < slots * a.D; e += kEThreads * 4) {
            uint32_t w = *reinterpret_cast<const uint32_t*>(p + e), o = 0;
#pragma unroll
            for (int u = 0; u < 4; ++u)
                o |= (uint32_t)e4m3_of(__fdiv_rn(e4m3_value((w >> (8 * u)) & 0xff) * s_old[g],
                                                 s_new[g])) << (8 * u);
            *reinterpret_cast<uint32_t*>(p + e) = o;
        }
        if (tid == 0) scales[(int64_t)s_page[g] * a.Hkv + h] = s_new[g];
    }
    __syncthreads();
    const int words = a.D / 4;
    for (int e = tid; e < mv.n * words; e += kEThreads) {
        const int i = e / words;
        if (mv.dst[i] < 0) continue;
        const int g = ((uint32_t)ctx + i) / (uint32_t)a.P - g0;
        const bool same = mv.src_page[i] == mv.dst_page[i] && s_new[g] == s_old[g];
        const uint32_t w = *reinterpret_cast<const uint32_t*>(s_row + e * 4);
        uint32_t o = w;
        if (!same) {
            const float s = s_src[i], to_scale = s_new[g];
            o = 0;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float x = e4m3_value((w >> (8 * u)) & 0xff) * s;
                // (a page of zeros has scale 0; a NaN stays one there too)
                const float y = to_scale > 0.f || x != x ? __fdiv_rn(x, to_scale) : 0.f;
                o |= (uint32_t)e4m3_of(y) << (8 * u);
            }
        }
        *reinterpret_cast<uint32_t*>(cache + mv.dst[i] * a.D + (e - i * words) * 4) = o;
    }
}

}  // namespace

size_t fork_workspace_bytes(int num_pages, int n) {
    const size_t blocks = ((size_t)num_pages + kScan - 1) / kScan;
    return blocks * (kScan / 32) * 8 + blocks * 4 + (size_t)n * 8;
}

cudaError_t launch_kv_fork(ForkArgs a, void* workspace, cudaStream_t stream) {
    const size_t blocks = ((size_t)a.num_pages + kScan - 1) / kScan;
    a.free_bits = static_cast<uint32_t*>(workspace);
    a.one_bits = a.free_bits + blocks * (kScan / 32);
    a.free_count = reinterpret_cast<int32_t*>(a.one_bits + blocks * (kScan / 32));
    a.need = a.free_count + blocks;
    a.src = a.need + a.n;
    cudaError_t e = launch_dependent(fork_plan_kernel, dim3((unsigned)(a.n + blocks)), dim3(kThreads),
                                     0, stream, a);
    if (e != cudaSuccess) return e;
    // a copy in slices of about 16 KB, so that large pages do not wait on one block
    const int64_t bytes = (int64_t)a.Hkv * a.P * a.D * a.elem * 2;
    const int slices = (int)(bytes / 16384 < 1 ? 1 : bytes / 16384 < a.Hkv ? bytes / 16384 : a.Hkv);
    return launch_dependent(fork_apply_kernel, dim3((unsigned)a.n, (unsigned)(slices < 65535 ? slices : 65535)),
                            dim3(kThreads), 0, stream, a);
}

cudaError_t launch_kv_release(const ReleaseArgs& a, cudaStream_t stream) {
    return launch_dependent(release_kernel, dim3((unsigned)a.n), dim3(kThreads), 0, stream, a);
}

cudaError_t launch_kv_compact(const CompactArgs& a, cudaStream_t stream) {
    const dim3 grid((unsigned)(2 * a.Hkv), (unsigned)a.B);
    return a.cache_dtype == SPEC_DTYPE_E4M3
               ? launch_dependent(compact_e4m3_kernel, grid, dim3(kEThreads), 0, stream, a)
               : launch_dependent(compact_kernel, grid, dim3(kCThreads), 0, stream, a);
}

}  // namespace specv
