// Verification attention of groups of sequences that share a prefix, on the
// tcgen05 tensor cores: bf16 q, bf16 / INT8 / e4m3 paged cache, head_dim 128, up
// to 128 query rows per kv-head.
//
// Mathematics.  For a query of sequence b in a group whose sequences hold the
// keys [0, s) in the same pages,
//   out = (e^L1 O1 + e^L2 O2) / (e^L1 + e^L2),  lse = ln(e^L1 + e^L2),
// where (O1, L1) is its normalised attention and log-sum-exp over [0, s) and
// (O2, L2) over its own keys [s, ctx + k).  O1 is one product for the group: the
// query rows of all its sequences against each prefix key once, n k G rows of a
// kv-head instead of n times k G over n copies of the same bytes.
//
// Segments.  The work is a list of segments, each the 128-key tiles of
//  * one sequence's own keys: its k G rows (from key s; the whole context where
//    nothing is shared), or
//  * a block of a group's query rows over its prefix: up to 2 NT tokens of
//    consecutive sequences (NT = 128 / G tokens fill a 128-row MMA tile),
// times the kv-heads, and a persistent grid takes equal parts of it (stream-K
// over a cost coordinate: a piece's fixed work and, for a block of more than NT
// tokens, twice the tile).  The host knows no lengths; every CTA builds the list.
//
// Two streams.  A CTA has two pipelines of a TMA producer warp, an MMA warp and a
// softmax set of eight warps, each with a slot of K and of V, a Q tile, an S and an O:
//  * narrow segments (one Q tile): each stream works on half of the CTA's range by
//    itself, so the end of one's piece (its last P V, O read and written) lies under
//    the other's tiles; nothing is merged between them.
//  * wide blocks (two Q tiles) follow: tile j lies in slot j % 2 and both streams,
//    each with a Q of its own, read it: 64 KB of L2 traffic for 16.8 MFLOP, half of
//    what narrow tiles would ask of L2.
//  * TMEM (512 columns): S of the streams [0,128), [128,256), their O [256,384),
//    [384,512); P (bf16; INT8: fp16) over the S columns it came from.
//  * Warps: 0-7 and 8-15 softmax (two for the 32 rows of a TMEM quadrant, half of the keys
//    each); 16 and 19 MMAs; 17 and 18 producers; with codes, 20-23 and 24-27 widen
//    what lands in slot 0 and slot 1.
//  * INT8 and e4m3 codes become bf16 exactly, INT8's of V fp16: a sequence's own keys in
//    place (raw bytes land in the upper half of their operand slot), and so a prefix that one
//    block reads; prefixes of several blocks by a launch before this one, once (widen_kernel).
//    Scales enter the scores and, before its rounding, P, in fp32.  So the MMAs see the stored
//    values and the only roundings are the output's and P's: to 8 bits over bf16 and e4m3
//    caches, to fp16's 11 over INT8, each as the kernels of single sequences do.
//  * Every mbarrier wait is bounded (1 s); a timeout sets the device error word
//    and an abort flag, after which every role skips its remaining work, drains
//    its copies and tensor-core operations, and returns.
//
// What bounds it (cycles of an SM): a narrow bf16 tile ~2700, which is its share of HBM
// (7.0 TB/s); a wide one ~4500 (1000 TFLOP/s), of which the tensor core is busy 1024: with the
// tensor pipe at 30 %, issue at 23 to 47 and the exponentials at 10 to 15, no unit but the latency
// of the chain S, maximum, exponents, P V of a stream; which link of it has not been timed.
// e4m3 ~3450 and ~6000, INT8 ~4000 and ~7000, with the scales in the softmax and the widening
// of narrow tiles.  And ~17 us of a call: the list ~4, first loads, the last pieces, the join
// ~4 and 2 KB of fp32 for every row.
// Measured: 32 sequences, 6000 shared and 100-900 own keys, 32/8 heads, 4 drafts, bf16 47 us
// (117 each by itself; the bytes' floor 13.7); 128 in four groups, 2-8K shared, 100-1500
// own, 64/8 heads, e4m3 242 (264; the products' floor 50); 16 trees of 16, 32K shared, 28/4
// heads, INT8 215 (485; 62).
// INT8 weights of fp16 for bf16's 8 bits: those trees 215 us for 211, 128 sequences of 1000 to
// 2500 own keys 266 for 272.  Of the references tried, the upper bound of a tile's maximum (the
// slow way for bounds 8 apart) took 224 on the trees, this one 215.
// Measured and not kept: S in two buffers of 64 keys a stream, Q K^T a buffer ahead of the
// softmax: wide blocks 13 % faster (16 trees behind 8K, bf16, 61 -> 53 us), narrow tiles 8 %
// (bf16) to 25 % (codes) slower, since a tile's softmax then takes twice the meetings and
// waits, and a K slot is free only after the second; own keys of e4m3 by the kernel that
// feeds codes to 8-bit MMAs, in a launch of its own: 252 against 258 us on the 128
// sequences, 50 against 45 and 65 against 52 on smaller calls.
//
// Every query's pieces meet in a second launch: rows of whole segments wait in
// two fp32 arrays (own keys, prefix), those of segments that a range cuts in two
// slots per range.
#include <cuda.h>
#include <math.h>

#include "common.cuh"

namespace specv {
namespace {

constexpr int D = 128;
constexpr int TN = 128;                 // keys per tile
constexpr int ROWS = 128;               // MMA M
constexpr int NVB = TN / 16;            // P V MMAs per tile (16 keys each)
constexpr int Q_HALF = ROWS * 128;      // 16 KB: 64 head-dim columns of Q
constexpr int Q_BYTES = 2 * Q_HALF;     // 32 KB
constexpr int SLOT_BYTES = TN * D * 2;  // 32 KB: one tile of K or of V
constexpr int RAW_OFF = SLOT_BYTES / 2;
constexpr int LOOKAHEAD = 6;            // tiles of block-table entries prefetched
constexpr int MAX_SEGS = 1024;
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t TM_S = 0, TM_O = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
enum { KV_BF16, KV_I8, KV_E4M3 };
// A tile's maximum (log2 units) that passes the reference of a row's weights by more moves it.
// bf16 weights have fp32's exponents.  INT8's, times V's scales, are fp16: the scores count with
// the power of two next above V's scales (the largest of 16 keys), and a reference is set to the
// greatest lower bound of their maximum, at most kFollow below the upper one.  So the largest
// product of a weight and such a scale lies in [2^-1, 2^15]; those of 2^-13 of it and more have
// all of fp16's 11 bits, the others half a step of 2^-24 of it or less.
template <int KV> constexpr float kFollow = KV == KV_I8 ? 15.f : 40.f;
// What the split over the CTAs charges, in quarters of a narrow tile's time: a tile
// of a wide block (two Q tiles), and a piece's fixed work.  A narrow piece's end lies
// under the other stream's tiles and goes with its rows (3 for 32 of them, which are
// 16 KB of fp32 to write); a wide one holds both streams.  Measured: one charge of 12 for
// all pieces left 144 sequences of 10-150 own keys behind 208 shared at 283 us against 138 then,
// 39 sequences of one group 69 against 51; one of 4 for narrow pieces of any rows left 16
// sequences of 112 rows behind 32K shared keys at 239 against 149.
constexpr int kTileCost = 4;
struct Cost {
    int wide, piece, wide_piece;
};
constexpr int kSnap = 1;  // tiles by which the two streams' parts may differ to save a cut
// Keys below which a prefix is read sequence by sequence: one tile
constexpr int kMinShared = TN;
// Rows of K (and of V) that widened prefixes may take: 1 GiB together
constexpr int64_t kMaxPrefixRows = (int64_t)1 << 21;

template <int KV> constexpr int threads() { return KV == KV_BF16 ? 20 * 32 : 28 * 32; }

constexpr uint32_t IDESC_QK = umma_idesc_bf16(ROWS, TN, 0, 0);
// B (V) MN-major.  INT8: P in fp16's 11 bits (as over an INT8 cache elsewhere), V's codes too
template <int KV>
constexpr uint32_t IDESC_PV = KV == KV_I8 ? umma_idesc_f16(ROWS, D, 0, 1) : umma_idesc_bf16(ROWS, D, 0, 1);

struct Smem {
    static constexpr int Q = 0;                         // 2 tiles
    static constexpr int KS = Q + 2 * Q_BYTES;          // 2 K slots
    static constexpr int VS = KS + 2 * SLOT_BYTES;      // 2 V slots
    static constexpr int BARS = VS + 2 * SLOT_BYTES;
    // of each slot / stream
    static constexpr int B_KFULL = 0, B_KEMPTY = 2, B_VFULL = 4, B_VEMPTY = 6, B_QFULL = 8,
                         B_SFULL = 10, B_PREADY = 12, B_SFREE = 14, B_EPI = 16, B_DRAIN = 18,
                         B_KREADY = 20, B_VREADY = 22;  // 24 in all
    static constexpr int MISC = BARS + 256;  // tmem base, abort flag, Range at +16
    static constexpr int STAT = MISC + 128;  // fp32 [maxima of 2 tiles in turn, sums][stream][half][row]
    static constexpr int PIDS = STAT + 3 * 2 * 2 * ROWS * 4;  // [2 producers][LOOKAHEAD+1][8] int
    // scales of a slot's use u at stage u % 2 of the slot, K then V.  Two stages: a
    // tile's softmax may still read its scales when its K slot is refilled.
    // e4m3: fp32 for every 16 keys, K's (with the softmax scale), V's, V's logarithm and
    // reciprocal;
    // INT8: the fp16 words as they are stored, and the least and largest of K's for
    // every 16 keys
    static constexpr int SCALE = (PIDS + 2 * (LOOKAHEAD + 1) * NVB * 4 + 15) / 16 * 16;
    static constexpr int SCRAW = SCALE + 4 * 32 * 4;
    static constexpr int SEG = SCRAW + 4 * 2 * TN * 2;    // int4 [MAX_SEGS]
    static constexpr int TPRE = SEG + MAX_SEGS * 16;
    static constexpr int CPRE = TPRE + (MAX_SEGS + 4) * 4;
    static constexpr int END = CPRE + (MAX_SEGS + 4) * 4;
};
constexpr size_t SMEM_BYTES = Smem::END + 1024;  // + alignment slack
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
static_assert(Smem::SCALE % 16 == 0 && Smem::SCRAW % 16 == 0 && Smem::SEG % 16 == 0, "alignment");

struct Params {
    AttnArgs a;
    const int32_t* group_starts;
    const int32_t* shared_lens;
    int groups;
    // codes: [groups][max_pages][Hkv][P][D] values of the prefixes' codes as the MMAs take them,
    // or null (they are widened tile by tile)
    __nv_bfloat16* k_prefix;
    __nv_bfloat16* v_prefix;
    // rows [8 C][128] of pieces of cut segments (slot_row), then [2][B k Hq] rows of whole
    // ones (own keys, prefix): values and log2-sums
    float* slot_o;
    float* slot_lse;
    int slots;         // 8 C * 128
    int G, NT;         // query heads of a kv-head, tokens that fill a Q tile
    int4* seq_block;   // [B] the group's wide blocks (first, count), its narrow one, its
                       // first token (-1: nothing shared)
    int* n_begin;      // [2 C + 1] first tile of each stream's narrow range
    int* w_begin;      // [C + 1] first tile of each CTA's wide range
    int* tile_pre;     // [segments + 1] tiles before a segment (per kv-head)
};

// First row among the slots of a cut piece: in stream s of CTA c (narrow) or the
// CTA (wide, 256 rows); `tail`: the piece's segment began before the range.
__device__ __forceinline__ int slot_row(bool wide, int c, int s, bool tail) {
    return (8 * c + (wide ? 4 + (tail ? 0 : 2) : 2 * s + (tail ? 0 : 1))) * ROWS;
}

// A segment: rows of tokens tok0 .. tok0 + ntok - 1, keys [key0, key1); a block's group.
struct Seg {
    int tok0;
    int16_t ntok, group;
    int key0, key1;
};

// V segments: the sequences' own keys, then narrow blocks, then wide ones.
struct List {
    const Seg* seg;
    const int* tpre;
    int B, Hkv, NT, V;
};

// A CTA's part: tiles [n[0], n[1]) and [n[1], n[2]) of narrow segments for its
// streams, [w[0], w[1]) of wide ones for both.
struct Range {
    int n[3], w[2];
};

// Walks tiles: segment v, kv-head, tile in the segment.  (Tiles and costs of a
// call are below 2^31: shared_supported.)
struct Cursor {
    int v, kvh, lt, nt;
    int start;  // global index of the segment's first tile
    __device__ void init(int t, const List& L) {
        int lo = 0, hi = L.V - 1;  // largest v with tpre[v] * Hkv <= t
#pragma unroll 1
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (L.tpre[mid] * L.Hkv <= t) lo = mid; else hi = mid - 1;
        }
        v = lo;
        nt = L.tpre[v + 1] - L.tpre[v];
        const int base = L.tpre[v] * L.Hkv;
        kvh = (int)((uint32_t)(t - base) / (uint32_t)nt);
        start = base + kvh * nt;
        lt = t - start;
    }
    __device__ void next_segment(const List& L) {
        lt = 0;
        start += nt;
        if (++kvh == L.Hkv) {
            kvh = 0;
            ++v;
            nt = L.tpre[v + 1] - L.tpre[v];
        }
    }
    __device__ void next(const List& L) {
        if (++lt == nt) next_segment(L);
    }
    __device__ void skip(int n, const List& L) {
#pragma unroll 1
        for (lt += n; lt >= nt;) {
            const int over = lt - nt;
            next_segment(L);
            lt = over;
        }
    }
    __device__ int key0(const List& L) const { return L.seg[v].key0 + lt * TN; }
    __device__ int valid(const List& L) const { return min(TN, L.seg[v].key1 - key0(L)); }
};

// Visible columns [c0, c0 + 64) of a 128-key tile for a query row: the context keys,
// then the drafts of the row's bits, limited to the tile's keys.
__device__ __forceinline__ uint64_t visible64(int key0, int c0, int nvalid, int ctx, uint64_t mrow) {
    const int nctx = ctx - key0 - c0;
    auto below = [](int n) { return n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1; };
    const uint64_t dbits = nctx >= 64    ? 0ull
                           : nctx >= 0   ? mrow << nctx
                           : nctx > -64  ? mrow >> -nctx
                                         : 0ull;
    return (below(nctx) | dbits) & below(nvalid - c0);
}

// A value that every lane holds, where the compiler knows it (tcgen05 operands from
// registers that it takes for different in each lane cost several times the issue).
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// First tile of CTA c's range: equal parts of the cost (a charge a segment and
// one a tile).
__device__ __forceinline__ int range_begin(const List& L, const int* cpre, Cost cost, uint32_t c,
                                           uint32_t C) {
    const uint32_t W = (uint32_t)(cpre[L.V] * L.Hkv), each_c = W / C;
    const int x = (int)(c * each_c + c * (W - each_c * C) / C);  // c W / C; C < 2^16
    if (x >= (int)W) return L.tpre[L.V] * L.Hkv;
    int lo = 0, hi = L.V - 1;
#pragma unroll 1
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cpre[mid] * L.Hkv <= x) lo = mid; else hi = mid - 1;
    }
    const bool wide = L.seg[lo].ntok > L.NT;
    const int nt = L.tpre[lo + 1] - L.tpre[lo], each = wide ? cost.wide : kTileCost;
    const int fixed = wide ? cost.wide_piece : cost.piece;
    const uint32_t off = (uint32_t)(x - cpre[lo] * L.Hkv), one = (uint32_t)(cpre[lo + 1] - cpre[lo]);
    const int h = (int)(off / one), r = (int)(off - h * one);
    const int lt = r > fixed ? (r - fixed + each - 1) / each : 0;
    return L.tpre[lo] * L.Hkv + h * nt + lt;
}

// Inclusive running maximum or sum of s[0 .. n) in place, by one warp.
template <bool MAX>
__device__ __forceinline__ void warp_scan(int* s, int n) {
    const int lane = threadIdx.x & 31, per = (n + 31) / 32, lo = lane * per, hi = min(n, lo + per);
    int run = 0;
#pragma unroll 1
    for (int i = lo; i < hi; ++i) run = MAX ? max(run, s[i]) : run + s[i];
    int incl = run;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl = MAX ? max(incl, v) : incl + v;
    }
    run = __shfl_up_sync(0xffffffffu, incl, 1);
    if (lane == 0) run = 0;
#pragma unroll 1
    for (int i = lo; i < hi; ++i) {
        run = MAX ? max(run, s[i]) : run + s[i];
        s[i] = run;
    }
    __syncwarp();
}

// Builds the list in shared memory (every thread); returns the number of
// segments.  One round trip to memory, and few barriers: a call of one tile
// waits for it.
template <int NTHREADS>
__device__ __forceinline__ int build_list(const Params& prm, Seg* seg, int* tpre, int* cpre,
                                          int* s_narrow, Cost charge, int NT) {
    const AttnArgs& a = prm.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, k = a.k, groups = prm.groups;
    const bool one = blockIdx.x == 0;
    int* starts = tpre;  // scratch until the prefixes are taken
    int* blocks = cpre;  // first each group's shared length, then its blocks
    bool bad = false;
#pragma unroll 1
    for (int g = tid; g <= groups; g += NTHREADS) {
        const int s = __ldg(prm.group_starts + g), n = g < groups ? __ldg(prm.shared_lens + g) : 0;
        bad |= s < 0 || s > a.B;
        starts[g] = s < 0 ? 0 : s > a.B ? a.B : s;
        blocks[g] = n;
    }
#pragma unroll 1
    for (int b = tid; b < a.B; b += NTHREADS) {
        int c = __ldg(a.ctx_lens + b);
        const int64_t cap = (int64_t)a.max_pages * a.P - k;
        if (c < 0 || (int64_t)c > cap) {
            raise_device_error(a.dev_err, SPEC_DEVERR_CTX);
            c = c < 0 ? 0 : (int)(cap < 0 ? 0 : cap);
        }
        seg[b] = Seg{b * k, (int16_t)k, -1, 0, c + k};
        if (one) prm.seq_block[b] = make_int4(0, 0, 0, -1);
    }
    __syncthreads();
#pragma unroll 1
    for (int g = tid; g < groups; g += NTHREADS) bad |= starts[g + 1] < starts[g];
    if (__syncthreads_or(bad)) {
        if (bad) raise_device_error(a.dev_err, SPEC_DEVERR_GROUP);
        if (warp == 0) warp_scan<true>(starts, groups + 1);  // ascending from here on
        __syncthreads();
    }
    // how many blocks each group's prefix takes, and where each sequence's own keys begin
#pragma unroll 1
    for (int g = warp; g < groups; g += NTHREADS / 32) {
        const int lo = starts[g], hi = starts[g + 1];
        int least = INT32_MAX;
#pragma unroll 1
        for (int b = lo + lane; b < hi; b += 32) least = min(least, seg[b].key1 - k);
        least = __reduce_min_sync(0xffffffffu, least);
        int s = blocks[g], n = 0;
        if (hi > lo && (s < 0 || s > least)) {
            if (lane == 0) raise_device_error(a.dev_err, SPEC_DEVERR_GROUP);
            s = s < 0 ? 0 : least;
        }
        s = hi - lo >= 2 && s >= kMinShared ? s & ~(a.P - 1) : 0;  // whole pages
        if (s > 0) {  // wide blocks, and what is left: one more of either kind
            const int tok = (hi - lo) * k, left = tok % (2 * NT);
            n = tok / (2 * NT) + (left > NT) + (left > 0 && left <= NT ? 1 << 16 : 0);
        }
        __syncwarp();
        if (lane == 0) blocks[g] = n;
#pragma unroll 1
        for (int b = lo + lane; b < hi; b += 32) seg[b].key0 = s;
    }
    __syncthreads();
    if (groups > 1) {
        if (warp == 0) warp_scan<false>(blocks, groups);
        __syncthreads();
    }
    const int all = blocks[groups - 1], narrow = a.B + (all >> 16), V = narrow + (all & 0xffff);
#pragma unroll 1
    for (int g = warp; g < groups; g += NTHREADS / 32) {
        const int before = g ? blocks[g - 1] : 0, mine = blocks[g] - before;
        if (mine == 0) continue;
        const int w0 = narrow + (before & 0xffff), nw = mine & 0xffff, n0 = a.B + (before >> 16);
        const int lo = starts[g], hi = starts[g + 1], s = seg[lo].key0, tok = (hi - lo) * k;
#pragma unroll 1
        for (int i = lane; i < nw; i += 32)
            seg[w0 + i] = Seg{lo * k + i * 2 * NT, (int16_t)min(tok - i * 2 * NT, 2 * NT), (int16_t)g, 0, s};
        if (lane == 0 && mine >> 16)
            seg[n0] = Seg{lo * k + nw * 2 * NT, (int16_t)(tok - nw * 2 * NT), (int16_t)g, 0, s};
        if (one)
#pragma unroll 1
            for (int b = lo + lane; b < hi; b += 32) prm.seq_block[b] = make_int4(w0, nw, n0, lo * k);
    }
    if (tid == 0) *s_narrow = narrow;
    __syncthreads();
    // prefixes of tiles (warp 0) and cost (warp 1), V / 32 segments a lane
    if (warp < 2) {
        int* pre = warp ? cpre : tpre;
        const int per = (V + 31) / 32, lo = min(V, lane * per), hi = min(V, lo + per);
        auto cost = [&](int v) {
            const Seg q = seg[v];
            const int nt = (q.key1 - q.key0 + TN - 1) / TN;
            return !warp ? nt : q.ntok > NT ? charge.wide_piece + nt * charge.wide : charge.piece + nt * kTileCost;
        };
        int sum = 0;
#pragma unroll 1
        for (int v = lo; v < hi; ++v) sum += cost(v);
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        int run = incl - sum;
        if (lane == 0) pre[0] = 0;
#pragma unroll 1
        for (int v = lo; v < hi; ++v) {
            run += cost(v);
            pre[v + 1] = run;
        }
    }
    __syncthreads();
    return V;
}

// Eight codes to fp16, which holds every one exactly (and a NaN as one).
template <int KV> __device__ __forceinline__ uint4 codes_to_f16(const uint2 r) {
    uint4 o;
    if constexpr (KV == KV_I8) {
        uint4 none;
        i8x16_to_f16(make_uint4(r.x, r.y, 0, 0), o, none);
    } else {
        auto two = [](uint32_t w) {
            uint32_t h;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)w));
            return h;
        };
        o = make_uint4(two(r.x), two(r.x >> 16), two(r.y), two(r.y >> 16));
    }
    return o;
}
// The same values in bf16, exactly for codes.  (e4m3 by bits, exponent and fraction moved to
// bf16's places and scaled by 2^120, is five operations a pair as this is four, and makes 480
// of a NaN: 128 sequences 250 us against 245, with a look at every word for NaN codes 286.)
__device__ __forceinline__ uint4 f16_to_bf16(const uint4 r) {
    auto two = [](uint32_t h) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        return pack_bf16x2(f.x, f.y);
    };
    return make_uint4(two(r.x), two(r.y), two(r.z), two(r.w));
}
// Eight codes as the MMAs take them: bf16, INT8's of V fp16.
template <int KV> __device__ __forceinline__ uint4 widen8(const uint2 r, bool is_v) {
    const uint4 h = codes_to_f16<KV>(r);
    return KV == KV_I8 && is_v ? h : f16_to_bf16(h);
}

// The keys' scales of a tile as its softmax reads them.
template <int KV> struct Scales {
    // of 16 keys: e4m3: K's; 8 words on V's; 16 on log2 of V's; 24 on 1 / V's
    // INT8: K's least; 8 on their largest; 16 on log2 of the power of two above V's
    const float* e4m3;
    const __half* i8;     // K, and 128 on V
};

// Exponents of N columns from c0 on (raw fp32 scores, rewritten in place): score times
// the softmax scale in log2 units (for codes: and the keys' scales), less m.  LOGV (e4m3):
// plus the logarithm of V's scale.
template <int KV, bool LOGV, int N>
__device__ __forceinline__ void exponents(uint32_t (&r)[N], float sl2, const Scales<KV>& sc, int c0,
                                          float m) {
    uint64_t neg = f2(-m, -m), s = f2(sl2, sl2);
#pragma unroll
    for (int c = 0; c < N; c += 8) {
        uint4 h;
        if (KV == KV_I8) h = *reinterpret_cast<const uint4*>(sc.i8 + c0 + c);
        if (KV == KV_E4M3 && c % 16 == 0) {
            const float x = sc.e4m3[(c0 + c) / 16];
            s = f2(x, x);
            if (LOGV) {
                const float y = sc.e4m3[16 + (c0 + c) / 16] - m;
                neg = f2(y, y);
            }
        }
        const uint32_t w[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            uint64_t v = f2(__uint_as_float(r[c + 2 * u]), __uint_as_float(r[c + 2 * u + 1]));
            if (KV == KV_I8) {
                const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w[u]));
                v = f2_mul(v, f2(x.x, x.y));
            }
            float v0, v1;
            f2_split(f2_fma(v, s, neg), v0, v1);
            r[c + 2 * u] = __float_as_uint(v0);
            r[c + 2 * u + 1] = __float_as_uint(v1);
        }
    }
}

// p = 2^v of N columns from c0 on, for codes times the keys' scales of V (LOGV: they are in
// v), packed to bf16 (INT8: fp16) pairs; adds the sum of p to l.
template <int KV, bool LOGV, int N>
__device__ __forceinline__ void weights(const uint32_t (&v)[N], const Scales<KV>& sc, int c0, float& l,
                                        uint32_t (&pk)[N / 2]) {
    uint64_t s = 0, ps[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
    auto total = [&]() {
        float a0, a1, b0, b1;
        f2_split(ps[0], a0, a1);
        f2_split(ps[1], b0, b1);
        ps[0] = ps[1] = f2(0.f, 0.f);
        return (a0 + b0) + (a1 + b1);
    };
#pragma unroll
    for (int c = 0; c < N; c += 8) {
        uint4 h;
        if (KV == KV_I8) h = *reinterpret_cast<const uint4*>(sc.i8 + TN + c0 + c);
        if (KV == KV_E4M3 && !LOGV && c % 16 == 0) {
            const float x = sc.e4m3[8 + (c0 + c) / 16];
            s = f2(x, x);
        }
        const uint32_t w[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            float e0 = fast_exp2(__uint_as_float(v[c + 2 * u]));
            float e1 = fast_exp2(__uint_as_float(v[c + 2 * u + 1]));
            const uint64_t e = f2(e0, e1);
            ps[u & 1] = f2_add(ps[u & 1], e);
            if (KV == KV_I8) {
                const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w[u]));
                s = f2(x.x, x.y);
            }
            if (KV != KV_BF16 && !LOGV) f2_split(f2_mul(e, s), e0, e1);
            pk[c / 2 + u] = KV == KV_I8 ? pack_f16x2(e0, e1) : pack_bf16x2(e0, e1);
        }
        // (the sums of 16 keys that share a scale, without it)
        if (LOGV && c % 16 == 8) l = fmaf(total(), sc.e4m3[24 + (c0 + c) / 16], l);
    }
    if (!LOGV) l += total();
}

template <int KV>
__global__ void __launch_bounds__(threads<KV>(), 1)
attn_shared_kernel(const __grid_constant__ CUtensorMap own_map,  // q: boxes of k tokens
                   const __grid_constant__ CUtensorMap block_map,  // q: boxes of NT tokens
                   const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap,
                   const __grid_constant__ CUtensorMap kwide,  // codes: prefixes as bf16
                   const __grid_constant__ CUtensorMap vwide, const Params prm) {
    constexpr int NTH = threads<KV>();
    constexpr bool CODES = KV != KV_BF16;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const AttnArgs& a = prm.a;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Smem::BARS);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + Smem::MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + Smem::MISC + 4);
    int* s_narrow = reinterpret_cast<int*>(sm + Smem::MISC + 8);
    Range* s_rng = reinterpret_cast<Range*>(sm + Smem::MISC + 16);
    Cursor* s_cur = reinterpret_cast<Cursor*>(sm + Smem::MISC + 48);  // of n[0], n[1], w[0]
    Seg* s_seg = reinterpret_cast<Seg*>(sm + Smem::SEG);
    int* s_tpre = reinterpret_cast<int*>(sm + Smem::TPRE);
    int* s_cpre = reinterpret_cast<int*>(sm + Smem::CPRE);
    float* s_scale = reinterpret_cast<float*>(sm + Smem::SCALE);  // [slot][stage][32]
    __half* s_half = reinterpret_cast<__half*>(sm + Smem::SCRAW);  // [slot][stage][2][TN]

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int k = a.k, Hkv = a.Hkv, G = prm.G, P = a.P, NT = prm.NT;

    if (tid < 2) {
        mbar_init(&bars[Smem::B_KFULL + tid], 1);
        mbar_init(&bars[Smem::B_KEMPTY + tid], 2);  // both streams, or one twice
        mbar_init(&bars[Smem::B_VFULL + tid], 1);
        mbar_init(&bars[Smem::B_VEMPTY + tid], 2);
        mbar_init(&bars[Smem::B_QFULL + tid], 1);
        mbar_init(&bars[Smem::B_SFULL + tid], 1);
        mbar_init(&bars[Smem::B_PREADY + tid], 8);  // the 8 softmax warps of the stream
        mbar_init(&bars[Smem::B_SFREE + tid], 1);
        mbar_init(&bars[Smem::B_EPI + tid], 8);
        mbar_init(&bars[Smem::B_DRAIN + tid], 1);
        mbar_init(&bars[Smem::B_KREADY + tid], 4);  // the 4 warps that widen the slot
        mbar_init(&bars[Smem::B_VREADY + tid], 4);
        *abort_flag = 0;
        fence_mbar_init();
    }
    grid_dep_launch_dependents();
    grid_dep_wait();
    if (warp == 16) {
        tmem_alloc(tmem_slot, TMEM_COLS);
        tmem_relinquish();
    }
    // (rows of a Q tile that no copy of q writes hold anything: a row of S, P or O
    // depends on its own row of Q alone, and those are not stored)
    const int opt = kTileCost * a.split_alpha;
    const Cost cost = {KV == KV_E4M3 ? 7 : 8,
                       opt >= 0 ? opt : (k * G + 31) / 32 * 3, opt >= 0 ? opt : 20};
    const int V = build_list<NTH>(prm, s_seg, s_tpre, s_cpre, s_narrow, cost, NT);
    const List L = {s_seg, s_tpre, a.B, Hkv, NT, V};
    if (warp == 0) {
        // the CTA's range [t0, t1); its narrow part in two, at a segment's end where
        // one is near (a cut costs more than the imbalance), and where they begin
        const int edge = range_begin(L, s_cpre, cost, blockIdx.x + (lane & 1), gridDim.x);
        const int t0 = __shfl_sync(0xffffffffu, edge, 0), t1 = __shfl_sync(0xffffffffu, edge, 1);
        const int border = s_tpre[*s_narrow] * Hkv, last = s_tpre[V] * Hkv - 1;
        const int n0 = min(t0, border), n2 = min(t1, border), w0 = max(t0, border);
        int mid = n0 + (n2 - n0 + 1) / 2;
        Cursor c;
        c.init(min(lane == 0 ? n0 : lane == 1 ? mid : w0, last), L);
        if (lane == 1) {
            const int back = c.lt, on = c.nt - c.lt;
            if (back <= kSnap && mid - back > n0) mid -= back;
            else if (on <= kSnap && mid + on < n2) mid += on;
            if (mid != c.start + c.lt) c.init(min(mid, last), L);
        }
        mid = __shfl_sync(0xffffffffu, mid, 1);
        if (lane < 3) s_cur[lane] = c;
        if (lane == 0) *s_rng = Range{{n0, mid, n2}, {w0, max(t1, border)}};
        // what the second launch needs to find the pieces
        if (lane < 2) prm.n_begin[2 * blockIdx.x + lane] = lane ? mid : n0;
        if (lane == 0) prm.w_begin[blockIdx.x] = w0;
        if (lane == 0 && blockIdx.x == gridDim.x - 1) {
            prm.n_begin[2 * gridDim.x] = border;
            prm.w_begin[gridDim.x] = last + 1;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(*tmem_slot);
    if (blockIdx.x == 0)
#pragma unroll 1
        for (int v = tid; v <= V; v += NTH) prm.tile_pre[v] = s_tpre[v];

    // a range without a tile can lie inside a segment: its slot counts as a piece of weight 0
    if (tid < 2 * ROWS) {
        const Range g = *s_rng;
        const int s = tid >> 7, r = tid & (ROWS - 1);
        if (g.n[s] == g.n[s + 1]) prm.slot_lse[slot_row(false, blockIdx.x, s, true) + r] = -INFINITY;
        if (g.w[0] == g.w[1]) prm.slot_lse[slot_row(true, blockIdx.x, 0, true) + tid] = -INFINITY;
    }

    // Stream s: narrow tiles, then the wide ones of the CTA.  Slot s holds tile i of
    // the stream's narrow ones as its use i, and wide tile 2 i + s as its use
    // (narrow tiles of s) + i.
    const int n_wide = uniform(s_rng->w[1] - s_rng->w[0]);
    auto narrow_tiles = [&](int s) { return uniform(s_rng->n[s + 1] - s_rng->n[s]); };

    // Registers (a thread, per warpgroup; the launch gives 96, with codes 72): softmax
    // 104 / 88, MMAs and copies 64 / 56, widening 48 (4 x 104 + 64 = 5 x 96, 4 x 88 + 56 +
    // 2 x 48 = 7 x 72; with 80 and 64 INT8 was 3 % slower)
    if (warp >= 16 && warp < 20) {
        regs_dec<CODES ? 56 : 64>();
        if (warp == 17 || warp == 18) {
            // ================= producers: slot s of K and of V =================
            // A tile is chunks of CH = min(P, 128) keys, each inside one page and one TMA
            // copy, in the layouts of the 128-key kernel without groups; block-table
            // entries come LOOKAHEAD tiles ahead.
            const int s = warp - 17;
            const int shift = 31 - __clz(P), CH = min(P, TN), NCH = TN / CH;  // P is a power of two
            int* pids = reinterpret_cast<int*>(sm + Smem::PIDS) + s * (LOOKAHEAD + 1) * NVB;
            uint8_t* kslot = sm + Smem::KS + s * SLOT_BYTES;
            uint8_t* vslot = sm + Smem::VS + s * SLOT_BYTES;
            const int n = narrow_tiles(s), total = n + (n_wide - s + 1) / 2;
            const uint64_t once = l2_policy_evict_first();
            uint64_t again;  // a prefix is read by many CTAs
            asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(again));
            if (lane == 0) {
                prefetch_tmap(&kmap);
                prefetch_tmap(&vmap);
            }
            // the tile after tile i, wherever it lies
            auto step = [&](Cursor& c, int i) {
                if (i + 1 < n) {
                    c.next(L);
                } else if (i + 1 == n) {
                    c = s_cur[2];
                    if (s && n_wide > 1) c.next(L);
                } else {
                    c.skip(2, L);
                }
            };
            Cursor cur = s_cur[n > 0 ? s : 2];
            if (n == 0 && s && n_wide > 1) cur.next(L);
            Cursor ahead = cur;
            auto fetch_pids = [&](int i) {
                if (i < total) {
                    const int key = ahead.key0(L) + lane * CH;
                    if (lane < NCH && lane * CH < ahead.valid(L)) {
                        const int row = ahead.v < L.B ? ahead.v : L.seg[ahead.v].tok0 / k;
                        cp_async_4(&pids[i % (LOOKAHEAD + 1) * NVB + lane],
                                   &a.block_table[(int64_t)row * a.max_pages + (key >> shift)]);
                    }
                    if (i + 1 < total) step(ahead, i);
                }
                cp_async_commit();
            };
            auto page_of = [&](int i, int chunk) {
                int page = pids[i % (LOOKAHEAD + 1) * NVB + chunk];
                if (page < 0 || page >= a.num_pages) {
                    raise_device_error(a.dev_err, SPEC_DEVERR_PAGE);
                    page = 0;
                }
                return page;
            };
            // e4m3: lane l < 8 the scale of K of keys [16 l, 16 l + 16) of tile i at cursor c,
            // l + 8 that of V; and into the stage of the tile's use
            auto fetch_scale = [&](const Cursor& c, int i) {
                const int j = (lane & 7) * 16;
                if (lane >= 16 || j >= c.valid(L)) return 0.f;
                const float* from = lane < 8 ? a.k_page_scale : a.v_page_scale;
                return __ldg(from + (int64_t)page_of(i, j / CH) * Hkv + c.kvh);
            };
            auto put_scale = [&](float x, int i) {
                if (lane >= 16) return;
                float* to = s_scale + (2 * s + (i & 1)) * 32 + lane;
                to[0] = lane < 8 ? x * a.scale * kLog2e : x;
                if (lane >= 8) {
                    to[8] = log2f(x);
                    to[16] = __frcp_rn(x);
                }
            };
#pragma unroll 1
            for (int i = 0; i < LOOKAHEAD; ++i) fetch_pids(i);
            bool ok = true;
            if (KV == KV_E4M3 && total > 0) {
                cp_async_wait<LOOKAHEAD - 1>();
                __syncwarp();
                put_scale(fetch_scale(cur, 0), 0);
            }
            int k_loads = 0, v_loads = 0;
#pragma unroll 1
            for (int i = 0; i < total; ++i) {
                fetch_pids(i + LOOKAHEAD);
                cp_async_wait<LOOKAHEAD - 1>();  // entries of tiles i and i + 1
                __syncwarp();
                const int nck = (cur.valid(L) + CH - 1) / CH;
                const bool wide = CODES && prm.k_prefix && cur.v >= L.B;  // values, not codes
                int row = 0, row16 = 0;
                if (lane < nck) {
                    const int key = cur.key0(L) + lane * CH;
                    row = row16 = (page_of(i, lane) * Hkv + cur.kvh) * P + (key & (P - 1));
                    if (wide)
                        row16 = ((L.seg[cur.v].group * a.max_pages + (key >> shift)) * Hkv + cur.kvh) * P +
                                (key & (P - 1));
                }
                const uint64_t pol = cur.v < L.B ? once : again;
                Cursor nx = cur;
                float scale = 0.f;  // the next tile's, stored when this one's V is on its way
                if (i + 1 < total) {
                    step(nx, i);
                    if (KV == KV_E4M3) scale = fetch_scale(nx, i + 1);
                }
                if (i > 0) ok = warp_wait(&bars[Smem::B_KEMPTY + s], (i - 1) & 1, abort_flag, a.dev_err);
                if (!ok) break;
                const uint32_t bytes = (uint32_t)(nck * CH) * (CODES && !wide ? 128u : 256u);
                __syncwarp();
                uint64_t* full = &bars[Smem::B_KFULL + s];
                if (lane == 0)
                    mbar_arrive_expect_tx(full, bytes + (KV == KV_I8 ? (uint32_t)(nck * CH) * 4 : 0u));
                __syncwarp();
                if (lane < nck) {
                    if constexpr (CODES) {
                        if (wide)
                            tma_load_4d_hint(kslot + lane * CH * 256, &kwide, full, 0, 0, 0, row16 >> 3, pol);
                        else
                            tma_load_2d(kslot + RAW_OFF + lane * CH * 128, &kmap, full, 0, row, pol);
                        if (KV == KV_I8) {
                            __half* raw = s_half + (2 * s + (i & 1)) * 2 * TN + lane * CH;
                            bulk_load(raw, a.k_scale + row, CH * 2, full);
                            bulk_load(raw + TN, a.v_scale + row, CH * 2, full);
                        }
                    } else {
                        tma_load_4d_hint(kslot + lane * CH * 256, &kmap, full, 0, 0, 0, row >> 3, pol);
                    }
                }
                k_loads = i + 1;
                __syncwarp();
                if (i > 0) ok = warp_wait(&bars[Smem::B_VEMPTY + s], (i - 1) & 1, abort_flag, a.dev_err);
                if (!ok) break;
                full = &bars[Smem::B_VFULL + s];
                if (lane == 0) mbar_arrive_expect_tx(full, bytes);
                __syncwarp();
                if (lane < nck) {
                    if (CODES && !wide)
                        tma_load_2d(vslot + RAW_OFF + lane * CH * 128, &vmap, full, 0, row, pol);
                    else
                        tma_load_4d_hint(vslot + lane * CH * 256, CODES ? &vwide : &vmap, full, 0, 0, 0,
                                         row16 >> 4, pol);
                }
                v_loads = i + 1;
                __syncwarp();
                // (the stage's last tile, i - 1, is through: its P V freed the slot of V)
                if (KV == KV_E4M3 && i + 1 < total) put_scale(scale, i + 1);
                cur = nx;
            }
            cp_async_wait<0>();
            if (!ok && lane == 0) {
                // the copies in flight land before the CTA exits
                if (k_loads) mbar_drain(&bars[Smem::B_KFULL + s], (k_loads - 1) & 1);
                if (v_loads) mbar_drain(&bars[Smem::B_VFULL + s], (v_loads - 1) & 1);
            }
        } else {
            // ================= MMAs of stream s =================
            const int s = uniform(warp == 19);
            const int n = narrow_tiles(s), other = narrow_tiles(1 - s);
            const int total = n + n_wide;
            bool ok = true;
            int q_loads = 0;
            const uint32_t sbuf = tmem + TM_S + s * TN, od = tmem + TM_O + s * D;
            const uint64_t qd = umma_sdesc_sw128(smem_u32(sm + Smem::Q) + s * Q_BYTES, 16, 1024);
            const uint64_t kd0 = umma_sdesc_sw128(smem_u32(sm + Smem::KS), 16, 2048);
            const uint64_t vd0 = umma_sdesc_sw128(smem_u32(sm + Smem::VS), 2048, 1024);
            Cursor cur = s_cur[n > 0 ? s : 2];
            int pc = 0;
            bool met = n_wide == 0;  // the streams, before the wide tiles
            // Q of the piece at cursor c
            auto load_q = [&](const Cursor& c, bool wide) {
                if (lane == 0) {
                    const bool own = c.v < L.B;
                    uint64_t* bar = &bars[Smem::B_QFULL + s];
                    mbar_arrive_expect_tx(bar, 2 * (own ? k : NT) * G * 128);
#pragma unroll 1
                    for (int h = 0; h < 2; ++h)
                        tma_load_3d(sm + Smem::Q + s * Q_BYTES + h * Q_HALF,
                                    own ? &own_map : &block_map, bar, h * 64, c.kvh * G,
                                    L.seg[c.v].tok0 + (wide && s ? NT : 0));
                }
                __syncwarp();
                ++q_loads;
            };
            if (lane == 0) {
                prefetch_tmap(&own_map);
                prefetch_tmap(&block_map);
            }
            if (total > 0) load_q(cur, n == 0);
#pragma unroll 1
            for (int t0 = 0; t0 < total && ok; ++pc) {  // a piece
                const bool wide = t0 >= n;
                if (wide && !met) {
                    // the other stream has seen every narrow tile of its slot land, so the
                    // phases of that slot are counted from there
                    named_bar_sync(9, 64);
                    met = true;
                }
                const int len = uniform(min(cur.nt - cur.lt, (wide ? total : n) - t0));
                const int keys = uniform(L.seg[cur.v].key1 - cur.key0(L));  // from its first tile on
                const bool values = CODES && prm.k_prefix && uniform(cur.v >= L.B);
                // (INT8's bounds of the scales come from the widening warps for every tile)
                const bool widened = CODES && (KV == KV_I8 || !values);
                ok = warp_wait(&bars[Smem::B_QFULL + s], (q_loads - 1) & 1, abort_flag, a.dev_err);
#pragma unroll 1
                for (int j = 0; j < len && ok; ++j) {
                    const int t = t0 + j;
                    // the tile's slot and the number of its use
                    const int slot = wide ? (t - n) & 1 : s;
                    const int use = wide ? (slot == s ? n : other) + ((t - n) >> 1) : t;
                    const int nvalid = min(TN, keys - j * TN), nvb = (nvalid + 15) / 16;
                    ok = warp_wait(&bars[(widened ? Smem::B_KREADY : Smem::B_KFULL) + slot], use & 1,
                                   abort_flag, a.dev_err);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_lane()) {
                        // S = Q K^T: k-slice kk at half kk/4 (Q: 16 KB on, K: 1 KB on in every
                        // 8-key group), 32-byte step kk%4
                        const uint64_t kd = kd0 + ((uint32_t)(slot * SLOT_BYTES) >> 4);
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            umma_ss(sbuf, qd + (kk >> 2) * (Q_HALF >> 4) + (kk & 3) * 2,
                                    kd + (kk >> 2) * (1024 >> 4) + (kk & 3) * 2, IDESC_QK, kk ? 1u : 0u);
                    }
                    __syncwarp();
                    umma_commit_w(&bars[Smem::B_SFULL + s]);
                    umma_commit_w(&bars[Smem::B_KEMPTY + slot]);
                    if (!wide) umma_commit_w(&bars[Smem::B_KEMPTY + slot]);  // for the other stream
                    ok = warp_wait(&bars[(widened ? Smem::B_VREADY : Smem::B_VFULL) + slot], use & 1,
                                   abort_flag, a.dev_err);
                    if (!ok) break;
                    if (nvalid % 16 != 0 && (!CODES || values)) {
                        // keys past the end that the last P V reads: 0 * (stale or canary) never
                        // reaches O (both streams may write the zeros of a wide tile)
                        uint8_t* vst = sm + Smem::VS + slot * SLOT_BYTES;
#pragma unroll 1
                        for (int e = lane; e < (nvb * 16 - nvalid) * 16; e += 32) {
                            const int key = nvalid + e / 16, h = (e / 8) & 1, c16 = e % 8;
                            *reinterpret_cast<uint4*>(vst + (key / 16) * 4096 + h * 2048 +
                                                      (key % 16) * 128 + c16 * 16) =
                                make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    // the previous piece's O has been read
                    if (j == 0 && pc > 0)
                        ok = warp_wait(&bars[Smem::B_EPI + s], (pc - 1) & 1, abort_flag, a.dev_err);
                    if (ok)
                        ok = warp_wait(&bars[Smem::B_PREADY + s], t & 1, abort_flag, a.dev_err);
                    if (!ok) break;
                    if (j == len - 1 && t + 1 < total) {
                        // the next piece's Q: this one's last Q K^T is done (its S was read)
                        if (t + 1 == n) cur = s_cur[2];
                        else cur.next_segment(L);
                        load_q(cur, t + 1 >= n);
                    }
                    tc_fence_after();
                    if (elect_lane()) {
                        // O (+)= P V: MMA i takes keys [16i, 16i + 16) (4 KB group i), their P
                        // at the S columns [8i, 8i + 8) (i < 4) or [64 + 8(i-4), ...)
                        const uint64_t vd = vd0 + ((uint32_t)(slot * SLOT_BYTES) >> 4);
#pragma unroll
                        for (int i = 0; i < NVB; ++i)
                            if (i < nvb)
                                umma_ts(od, sbuf + (i < 4 ? 8 * i : 64 + 8 * (i - 4)),
                                        vd + ((uint32_t)(i * 4096) >> 4), IDESC_PV<KV>,
                                        (j > 0 || i > 0) ? 1u : 0u);
                    }
                    __syncwarp();
                    umma_commit_w(&bars[Smem::B_SFREE + s]);
                    umma_commit_w(&bars[Smem::B_VEMPTY + slot]);
                    if (!wide) umma_commit_w(&bars[Smem::B_VEMPTY + slot]);
                    // S is written again (and at a piece's end Q) once P has been read
                    ok = warp_wait(&bars[Smem::B_SFREE + s], t & 1, abort_flag, a.dev_err);
                }
                t0 += len;
            }
            if (!met) named_bar_sync(9, 64);
            // a Q copy in flight lands before the CTA exits
            if (!ok && lane == 0 && q_loads > 0) mbar_drain(&bars[Smem::B_QFULL + s], (q_loads - 1) & 1);
            // every tensor-core op of this warp finishes before TMEM is released
            __syncwarp();
            umma_commit_w(&bars[Smem::B_DRAIN + s]);
            if (lane == 0) mbar_drain(&bars[Smem::B_DRAIN + s], 0);
            __syncwarp();
        }
    } else if (CODES && warp >= 20) {
        if constexpr (CODES) {
            regs_dec<48>();
            // ================= widening of slot s (warps 20-23, 24-27) =================
            // Each code exactly to bf16, in place, in the layout the MMAs read.  The raw tile
            // sits in the upper half of its slot, row r at 16 KB + 128 r; its bf16 row
            // takes the 256 bytes from 256 r on (in groups of 8 or 16 rows), so
            // ascending rows never land on unread ones.  Rows past the end
            // become zeros.  Every warp runs every tile and every barrier,
            // also after an abort.
            const int s = warp >= 24, ct = tid - (20 + 4 * s) * 32;  // 0..127
            const int n = narrow_tiles(s), total = n + (n_wide - s + 1) / 2;
            Cursor c = s_cur[n > 0 ? s : 2];
            if (n == 0 && s && n_wide > 1) c.next(L);
            bool ok = true;
#pragma unroll 1
            for (int i = 0; i < total; ++i) {
                const int nvalid = c.valid(L);
                const bool values = prm.k_prefix && c.v >= L.B;  // nothing to widen
                if (KV == KV_E4M3 && values) break;  // nor in any tile from here on
#pragma unroll 1
                for (int is_v = 0; is_v < 2; ++is_v) {
                    if (ok)
                        ok = warp_wait(&bars[(is_v ? Smem::B_VFULL : Smem::B_KFULL) + s], i & 1,
                                       abort_flag, a.dev_err);
                    uint8_t* slot = sm + (is_v ? Smem::VS : Smem::KS) + s * SLOT_BYTES;
                    if (KV == KV_I8 && !is_v && ok) {
                        // bounds of K's scales over 16 keys, the power of two above V's (of
                        // 2^-24, fp16's least, where all are zero), and no V scale past the
                        // end (a weight of 0 times whatever is stored there)
                        __half* raw = s_half + (2 * s + (i & 1)) * 2 * TN;
                        float* to = s_scale + (2 * s + (i & 1)) * 32;
                        const int j = ct;
                        const float x = __half2float(raw[j]);
                        float lo = j < nvalid ? x : INFINITY, hi = j < nvalid ? x : 0.f;
                        float v = j < nvalid ? fabsf(__half2float(raw[TN + j])) : 0.f;
#pragma unroll
                        for (int o = 8; o > 0; o >>= 1) {
                            lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
                            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
                            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
                        }
                        if (j % 16 == 0) {
                            // (with a negative scale of K they are no bounds: the slow way)
                            to[j / 16] = lo < 0.f ? -INFINITY : lo;
                            to[8 + j / 16] = lo < 0.f ? INFINITY : hi;
                            to[16 + j / 16] = (float)((__float_as_int(fmaxf(v, 0x1p-24f)) >> 23) - 126);
                        }
                        if (j >= nvalid) raw[TN + j] = __float2half(0.f);
                    }
                    // piece id: key id / 8, head dims 16 (id % 8) ..; 32 rows at a time; rows
                    // from 64 on land over raw rows that all four warps have read by then
                    const int c16 = ct & 7, h = c16 >> 2, cc = (c16 & 3) * 2, j0 = ct >> 3;
                    // chunks cc, cc + 1 of half h, swizzled by the row; lanes of half 1
                    // store their odd chunk first so that 8 consecutive lanes hit 8
                    // bank groups
                    const int o0 = ((cc + h) ^ (j0 & 7)) << 4, o1 = ((cc + 1 - h) ^ (j0 & 7)) << 4;
                    // row 32 pass + 16 u + j0: K groups of 8 rows 2 KB apart, V of 16 4 KB
                    uint8_t* to = slot + (is_v ? h * 2048 + j0 * 128
                                               : h * 1024 + (j0 >> 3) * 2048 + (j0 & 7) * 128);
                    const uint8_t* from = slot + RAW_OFF + ct * 16;
#pragma unroll 1
                    for (int pass = values ? 4 : 0; pass < 4; ++pass) {
                        uint4 raw[2];
#pragma unroll
                        for (int u = 0; u < 2; ++u)
                            raw[u] = *reinterpret_cast<const uint4*>(from + pass * 4096 + u * 2048);
                        if (pass >= 2) named_bar_sync(10 + s, 128);
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            uint4 lo, hi;
                            if (pass * 32 + u * 16 + j0 >= nvalid) raw[u] = make_uint4(0, 0, 0, 0);
                            lo = codes_to_f16<KV>(make_uint2(raw[u].x, raw[u].y));
                            hi = codes_to_f16<KV>(make_uint2(raw[u].z, raw[u].w));
                            if (KV != KV_I8 || !is_v) {
                                lo = f16_to_bf16(lo);
                                hi = f16_to_bf16(hi);
                            }
                            uint8_t* row = to + pass * 8192 + u * 4096;
                            *reinterpret_cast<uint4*>(row + o0) = h ? hi : lo;
                            *reinterpret_cast<uint4*>(row + o1) = h ? lo : hi;
                        }
                    }
                    fence_proxy_async_smem();  // generic-proxy writes -> tensor-core reads
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars[(is_v ? Smem::B_VREADY : Smem::B_KREADY) + s]);
                }
                if (i + 1 < n) {
                    c.next(L);
                } else if (i + 1 == n) {
                    c = s_cur[2];
                    if (s && n_wide > 1) c.next(L);
                } else if (i + 1 < total) {
                    c.skip(2, L);
                }
            }
        }
    } else {
        regs_inc<CODES ? 88 : 104>();
        // ================= softmax of stream s =================
        // Two warps for the 32 rows of a TMEM quadrant, each on 64 of the tile's keys and
        // 64 of O's columns; they meet at the row's maximum.
        const int s = warp >> 3, half = (warp >> 2) & 1, quad = warp & 3;
        const int r = quad * 32 + lane;            // row of this thread in its Q tile
        const float sl2 = a.scale * kLog2e;
        const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
        const uint32_t s_mine = lane_base + TM_S + s * TN + half * 64;
        const uint32_t o_mine = lane_base + TM_O + s * D + half * 64;
        float* stat = reinterpret_cast<float*>(sm + Smem::STAT) + s * 2 * ROWS + r;
        const int meet = 1 + s * 4 + quad;         // named barrier of the pair
        const int n = narrow_tiles(s), other = narrow_tiles(1 - s), total = n + n_wide;
        float m_ref = -INFINITY, l = 0.f;          // l: over this half of the keys
        uint64_t mrow = 0;
        int rows = 0, ctx = 0;  // rows of this stream's Q tile; keys that are no drafts
        Cursor cur = s_cur[n > 0 ? s : 2];
        bool ok = true, first = true;
#pragma unroll 1
        for (int t = 0; t < total; ++t) {
            const bool wide = t >= n;
            if (first) {
                const Seg q = L.seg[cur.v];
                rows = (wide ? (s ? q.ntok - NT : NT) : q.ntok) * G;
                m_ref = -INFINITY;
                l = 0.f;
                const bool own = cur.v < L.B;
                ctx = own ? q.key1 - k : q.key1;
                mrow = own ? draft_bits(a, cur.v, r < rows ? r / G : k - 1) : 0;
            }
            const bool active = quad * 32 < rows;
            if (ok) ok = warp_wait(&bars[Smem::B_SFULL + s], t & 1, abort_flag, a.dev_err);
            if (active) {  // (also after an abort: the pair meets at every tile)
                tc_fence_after();
                const int slot = wide ? (t - n) & 1 : s;
                const int use = wide ? (slot == s ? n : other) + ((t - n) >> 1) : t;
                const int stage = 2 * slot + (use & 1);
                // scales of this half: e4m3 (and INT8's bounds) 4 of 8, INT8 64 of 128
                const Scales<KV> sc = {s_scale + stage * 32 + half * 4,
                                       s_half + stage * 2 * TN + half * 64};
                const uint64_t vis =
                    visible64(cur.key0(L), half * 64, cur.valid(L), ctx, mrow);
                // the row's maximum: with the loads where all keys are visible (INT8: bounds
                // of it, by the scales of 16 keys, which do unless a reference has to follow
                // and they lie too far apart)
                float mx = -INFINITY, least = -INFINITY;
                bool slow = vis != ~0ull || a.scale < 0.f;
                if (!__any_sync(0xffffffffu, slow && r < rows)) {
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        uint32_t d[2][16];
                        float x[2];
                        tmem_ld16_max(s_mine + h * 32, d[0], x[0]);
                        tmem_ld16_max(s_mine + h * 32 + 16, d[1], x[1]);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            if (KV == KV_I8) {
                                const float lo = sc.e4m3[h * 2 + j], hi = sc.e4m3[8 + h * 2 + j];
                                const float v = sc.e4m3[16 + h * 2 + j], y = x[j] * sl2;
                                // (0 times an infinite bound: a NaN, and the slow way)
                                asm("max.NaN.f32 %0, %0, %1;" : "+f"(mx) : "f"(fmaf(y, x[j] > 0.f ? hi : lo, v)));
                                least = fmaxf(least, fmaf(y, x[j] > 0.f ? lo : hi, v));
                            } else {
                                mx = fmaxf(mx, x[j] * (KV == KV_E4M3 ? sc.e4m3[h * 2 + j] : sl2));
                                // a scale of V whose logarithm would cost weights
                                if (KV == KV_E4M3) slow |= !(sc.e4m3[8 + h * 2 + j] > 1e-18f);
                            }
                        }
                    }
                    if (KV == KV_I8)
                        slow = !(mx <= m_ref + kFollow<KV> || mx - least <= kFollow<KV>);
                }
                // (rows past the piece's hold anything: they decide nothing)
                slow = __any_sync(0xffffffffu, slow && r < rows);
                // 16 columns less m (the slow way: hidden keys to -inf, small code)
                auto some = [&](int c, float m, uint32_t (&v)[16]) {
                    tmem_ld16(s_mine + c, v);
                    tmem_wait_ld();
                    exponents<KV, false, 16>(v, sl2, sc, c, m);
                    const uint32_t bits = (uint32_t)(vis >> c);
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        v[e] = ((bits >> e) & 1u) ? v[e] : __float_as_uint(-INFINITY);
                };
                if (slow) {
                    mx = -INFINITY;
#pragma unroll 1
                    for (int c = 0; c < 64; c += 16) {
                        uint32_t v[16];
                        some(c, 0.f, v);
                        float most = -INFINITY;
#pragma unroll
                        for (int e = 0; e < 16; e += 2)
                            most = fmax3(most, __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
                        if (KV == KV_I8) most += sc.e4m3[16 + c / 16];
                        mx = fmaxf(mx, most);
                    }
                    least = mx;
                }
                {
                    float* mine = stat + (t & 1) * 4 * ROWS;
                    if (r >= rows) mx = least = 0.f;
                    mine[half * ROWS] = mx;
                    named_bar_sync(meet, 64);
                    mx = fmaxf(mx, mine[(1 - half) * ROWS]);
                }
                // the reference follows only a maximum far above it (weights and
                // sums have the exponents for that), so O is almost never rescaled
                float al = 1.f;
                const bool move = mx > m_ref + kFollow<KV>;  // also -inf -> finite
                if (KV == KV_I8 && __any_sync(0xffffffffu, move)) {  // both warps of the pair
                    float* mine = stat + 2 * 4 * ROWS;
                    mine[half * ROWS] = least;
                    named_bar_sync(meet, 64);
                    mx = fmaxf(least, mine[(1 - half) * ROWS]);
                }
                if (move) {
                    al = (m_ref == -INFINITY) ? 0.f : fast_exp2(m_ref - mx);
                    m_ref = mx;
                    l *= al;
                }
                const float m_use = m_ref == -INFINITY ? 0.f : m_ref;  // keeps -inf - m finite
                // P over the first 32 of this half's S columns, read by then.  (A branch on
                // hidden keys inside the loop cost a third of the kernel's time: the
                // compiler no longer runs the exponents under the products.)
                constexpr bool LOGV = KV == KV_E4M3;
                if (!slow) {
#pragma unroll(KV == KV_E4M3 ? 2 : 1)
                    for (int c = 0; c < 64; c += 32) {
                        uint32_t v[32], pk[16];
                        tmem_ld32(s_mine + c, v);
                        tmem_wait_ld();
                        exponents<KV, LOGV, 32>(v, sl2, sc, c, m_use);
                        weights<KV, LOGV, 32>(v, sc, c, l, pk);
                        tmem_st16(s_mine + c / 2, pk);
                    }
                } else {
#pragma unroll 1
                    for (int c = 0; c < 64; c += 16) {
                        uint32_t v[16], pk[8];
                        some(c, m_use, v);
                        weights<KV, false, 16>(v, sc, c, l, pk);
                        tmem_st8(s_mine + c / 2, pk);
                    }
                }
                if (!first && __any_sync(0xffffffffu, move)) {
                    // O holds every earlier P V of the piece (S of this tile came after them)
#pragma unroll 1
                    for (int c = 0; c < 64; c += 16) {
                        uint32_t ov[16];
                        tmem_ld16(o_mine + c, ov);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            ov[e] = __float_as_uint(__uint_as_float(ov[e]) * al);
                        tmem_st16(o_mine + c, ov);
                    }
                }
                tmem_wait_st();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[Smem::B_PREADY + s]);
            first = false;
            const bool last = t == total - 1 || t == n - 1 || cur.lt == cur.nt - 1;
            if (last) {
                // ---- the end of a piece: its last P V, then its rows
                if (ok) ok = warp_wait(&bars[Smem::B_SFREE + s], t & 1, abort_flag, a.dev_err);
                tc_fence_after();
                if (active) {
                    float* mine = stat + 2 * 4 * ROWS;  // the row's sum
                    mine[half * ROWS] = l;
                    named_bar_sync(meet, 64);
                    l += mine[(1 - half) * ROWS];
                }
                if (ok && active) {
                    const Seg q = L.seg[cur.v];
                    const int tb = wide ? s_rng->w[0] : s_rng->n[s];
                    const int te = wide ? s_rng->w[1] : s_rng->n[s + 1];
                    const bool complete = cur.start >= tb && cur.start + cur.nt <= te;
                    const bool final = complete && cur.v < L.B && q.key0 == 0;
                    // (a NaN among the keys stays one, in the row's sum too)
                    const float inv = l == 0.f ? 0.f : 1.f / l;
                    const float lse = l == 0.f ? -INFINITY : m_ref + log2f(l);
                    // this row's place: out, the arrays of whole segments, or a slot
                    const int64_t orow =
                        (int64_t)(q.tok0 + (wide && s ? NT : 0) + r / G) * a.Hq + cur.kvh * G + r % G;
                    const int64_t at =
                        complete ? prm.slots + (cur.v < L.B ? 0 : (int64_t)a.B * k * a.Hq) + orow
                                 : (int64_t)(slot_row(wide, blockIdx.x, s, cur.start < tb) +
                                             (wide && s ? ROWS : 0) + r);
                    float* po = prm.slot_o + at * D + half * 64;
                    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + orow * D + half * 64;
#pragma unroll 1
                    for (int c = 0; c < 64; c += 16) {
                        uint32_t ov[16];
                        tmem_ld16(o_mine + c, ov);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            ov[e] = __float_as_uint(__uint_as_float(ov[e]) * inv);
                        if (r >= rows) {
                        } else if (final) {
                            uint32_t w[8];
#pragma unroll
                            for (int u = 0; u < 8; ++u)
                                w[u] = pack_bf16x2(__uint_as_float(ov[2 * u]), __uint_as_float(ov[2 * u + 1]));
                            uint4* dst = reinterpret_cast<uint4*>(out + c);
                            dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
                            dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
                        } else {
                            // (whole sectors: a lane's row is 512 bytes from the next one's)
#pragma unroll
                            for (int u = 0; u < 16; u += 8)
                                asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                                                 po + c + u),
                                             "r"(ov[u]), "r"(ov[u + 1]), "r"(ov[u + 2]), "r"(ov[u + 3]),
                                             "r"(ov[u + 4]), "r"(ov[u + 5]), "r"(ov[u + 6]), "r"(ov[u + 7])
                                             : "memory");
                        }
                        __syncwarp();
                    }
                    if (r < rows && half == 0) {
                        if (!final) prm.slot_lse[at] = lse;
                        else if (a.lse) a.lse[orow] = lse * kLn2;
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[Smem::B_EPI + s]);
                first = true;
            }
            if (t + 1 < total) {
                if (t + 1 == n) cur = s_cur[2];
                else cur.next(L);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 16) tmem_dealloc(tmem, TMEM_COLS);
}

// ------------------------------------------------------------------ the pieces' sum

constexpr int kJoinWarps = 4;  // three look segments up

// A segment's pieces for one kv-head: ranges first .. first + count - 1; one alone is
// whole.  (Ranges without a tile among them have left sums of -inf.)
struct Pieces {
    int first, count, wide;
};

// Of n ranges with these first tiles, the last that starts at or before tile t0, and the
// number of them up to tile t1's; a warp.
__device__ __forceinline__ void find_ranges(const int* begin, int n, int t0, int t1, Pieces& p) {
    int c0 = 0, c1 = 0;
#pragma unroll 5
    for (int c = threadIdx.x & 31; c < n; c += 32) {
        const int t = __ldg(begin + c);
        c0 += t <= t0;
        c1 += t <= t1;
    }
    p.first = (int)__reduce_add_sync(0xffffffffu, (unsigned)c0) - 1;
    p.count = (int)__reduce_add_sync(0xffffffffu, (unsigned)c1) - 1 - p.first + 1;
}

// x / y for 0 <= x < 2^20, given 1 / y
__device__ __forceinline__ int quotient(int x, float inverse) { return (int)((x + 0.5f) * inverse); }

// A block per (sequence, kv-head) and 8 rows: its own keys' pieces and those of the (up to two)
// blocks that hold its tokens are looked up once, by a warp each; then half a
// warp per query row, its pieces' sums and values in one round trip.  The launch runs once
// through its code: short code counts more here than few instructions.  32768 rows: 16 us
// cold, 24 with a warp per row in blocks of eight.
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const Params prm, int C) {
    __shared__ Pieces s_seg[3];
    grid_dep_launch_dependents();
    grid_dep_wait();
    const AttnArgs& a = prm.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = prm.G, NT = prm.NT, kvh = blockIdx.y, b = blockIdx.x;
    const float inv_g = 1.f / G, inv_nt = 1.f / NT;
    const int4 blk = __ldg(prm.seq_block + b);
    const bool shared = blk.w >= 0;
    const int dt0 = b * a.k - blk.w, nth0 = shared ? quotient(dt0, 0.5f * inv_nt) : 0;
    if (warp < 3) {
        const int nth = nth0 + warp - 1;
        const bool wide = warp > 0 && nth < blk.y;
        const int v = warp == 0 ? b : wide ? blk.x + nth : blk.z;
        Pieces p = {0, 0, wide};
        // (where its last token lies in the first block nobody asks for the second)
        if (warp == 0 || (shared && dt0 + a.k > 2 * NT * nth)) {
            const int p0 = __ldg(prm.tile_pre + v), nt = __ldg(prm.tile_pre + v + 1) - p0;
            const int t0 = p0 * a.Hkv + kvh * nt;
            find_ranges(wide ? prm.w_begin : prm.n_begin, wide ? C : 2 * C, t0, t0 + nt - 1, p);
        }
        if (lane == 0) s_seg[warp] = p;
    }
    __syncthreads();
    // two rows per warp, 16 lanes with eight columns each
    const int l = lane & 15, R = a.k * G;
    const int row0 = (blockIdx.z * kJoinWarps + warp) * 2, row = min(row0 + (lane >> 4), R - 1);
    const Pieces own = s_seg[0];
    if ((!shared && own.count == 1) || row0 >= R) return;  // written already
    const int tok = quotient(row, inv_g), dt = dt0 + tok;
    const int nth = shared ? quotient(dt, 0.5f * inv_nt) : 0, off = dt - nth * 2 * NT;
    const int orow = (b * a.k + tok) * a.Hq + kvh * G + row - tok * G;
    const Pieces pre = shared ? s_seg[1 + nth - nth0] : Pieces{0, 0, 0};
    const int row1 = (off >= NT ? ROWS + (off - NT) * G : off * G) + row - tok * G;
    const int rows = a.B * a.k * a.Hq, slots = 8 * C * ROWS, n = own.count + pre.count;
    const int most = max(n, __shfl_xor_sync(0xffffffffu, n, 16));
    // piece i: its row among the slots, or past them among the whole rows
    auto place = [&](int i) {
        const bool p = i >= own.count;
        const Pieces q = p ? pre : own;
        if (p) i -= own.count;
        if (q.count == 1) return slots + (p ? rows : 0) + orow;
        const int c = q.first + i;
        return slot_row(q.wide, q.wide ? c : c >> 1, q.wide ? 0 : c & 1, i > 0) + (p ? row1 : row);
    };
    // (the arrays of whole segments lie behind the slots': one base for both)
    float m = -INFINITY, sum = 0.f;
    uint64_t acc[4] = {f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll 1
    for (int i0 = 0; i0 < most; i0 += 16) {  // (one round but for very long segments)
        int mine = 0;
        float z = -INFINITY;
        if (i0 + l < n) {
            mine = place(i0 + l);
            z = __ldg(prm.slot_lse + mine);
        }
        float top = z;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        top = fmaxf(top, m);
        const float back = m == -INFINITY ? 0.f : fast_exp2(m - top);
        const float w_mine = z == -INFINITY ? 0.f : fast_exp2(z - top);
        m = top;
        float part = w_mine;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
        sum = sum * back + part;
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = f2_mul(acc[e], f2(back, back));
        const int left = min(16, most - i0);
#pragma unroll 4
        for (int i = 0; i < left; ++i) {
            const int p = __shfl_sync(0xffffffffu, mine, i, 16);
            const float w = __shfl_sync(0xffffffffu, w_mine, i, 16);
            const float4* from = reinterpret_cast<const float4*>(prm.slot_o + (int64_t)p * D);
            const float4 x = __ldg(from + l), y = __ldg(from + 16 + l);
            if (w != 0.f) {  // a place that nobody wrote holds anything; a NaN counts
                const uint64_t ww = f2(w, w);
                acc[0] = f2_fma(ww, f2(x.x, x.y), acc[0]);
                acc[1] = f2_fma(ww, f2(x.z, x.w), acc[1]);
                acc[2] = f2_fma(ww, f2(y.x, y.y), acc[2]);
                acc[3] = f2_fma(ww, f2(y.z, y.w), acc[3]);
            }
        }
    }
    if (row0 + (lane >> 4) >= R) return;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint2* out = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + (int64_t)orow * D);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float x0, x1, x2, x3;
        f2_split(acc[2 * h], x0, x1);
        f2_split(acc[2 * h + 1], x2, x3);
        out[16 * h + l] = make_uint2(pack_bf16x2(x0 * inv, x1 * inv), pack_bf16x2(x2 * inv, x3 * inv));
    }
    if (l == 0 && a.lse) a.lse[orow] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
}

// ------------------------------------------------------------------ prefixes of codes

// The codes of every group's prefix as the MMAs take them: a prefix of several blocks is read by
// each of them.  grid (blocks, groups); a thread takes 8 codes of K and of V at a time, so
// that a warp's loads and stores are whole lines.  (A warp per page and kv-head found its
// place less often, and was slower, 26 us against 24 for 20000 keys of 8 kv-heads: fewer
// loads under way, and a page's id before every 16 KB.)
template <int KV>
__global__ void __launch_bounds__(256) widen_kernel(const Params prm) {
    grid_dep_launch_dependents();
    grid_dep_wait();
    const AttnArgs& a = prm.a;
    const int g = blockIdx.y, lane = threadIdx.x & 31;
    // the group's whole pages, as build_list finds them (a group that is no range of
    // sequences shares nothing there)
    int lo = max(0, min(a.B, __ldg(prm.group_starts + g)));
    for (int i = lane; i < g; i += 32) lo = max(lo, min(a.B, __ldg(prm.group_starts + i)));
    lo = (int)__reduce_max_sync(0xffffffffu, lo);
    const int hi = max(lo, min(a.B, __ldg(prm.group_starts + g + 1)));
    if (hi - lo < 2) return;
    int least = INT32_MAX;
    const int64_t cap = (int64_t)a.max_pages * a.P - a.k;
    for (int b = lo + lane; b < hi; b += 32)
        least = min(least, (int)max((int64_t)0, min(cap, (int64_t)__ldg(a.ctx_lens + b))));
    least = __reduce_min_sync(0xffffffffu, least);
    const int s = min(least, __ldg(prm.shared_lens + g));
    if (s < kMinShared) return;
    const int shift = 31 - __clz(a.P), per = a.P * D / 8;  // pieces of a (page, kv-head)
    const int64_t all = (int64_t)(s >> shift) * a.Hkv * per, step = (int64_t)gridDim.x * 256;
    const uint2* kc = static_cast<const uint2*>(a.k_cache);
    const uint2* vc = static_cast<const uint2*>(a.v_cache);
    uint4* ko = reinterpret_cast<uint4*>(prm.k_prefix);
    uint4* vo = reinterpret_cast<uint4*>(prm.v_prefix);
    for (int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x; i0 < all; i0 += 4 * step) {
        uint2 k[4], v[4];
        int64_t to[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t i = i0 + u * step;
            if (i >= all) continue;
            const int piece = (int)(i & (per - 1));
            const uint32_t block = (uint32_t)(i >> (shift + 4));  // page of the prefix, kv-head
            const uint32_t n = block / (uint32_t)a.Hkv, h = block - n * a.Hkv;
            int page = __ldg(a.block_table + (int64_t)lo * a.max_pages + n);
            if (page < 0 || page >= a.num_pages) page = 0;  // flagged by the attention kernel
            const int64_t from = ((int64_t)page * a.Hkv + h) * per + piece;
            to[u] = (((int64_t)g * a.max_pages + n) * a.Hkv + h) * per + piece;
            k[u] = __ldg(kc + from);
            v[u] = __ldg(vc + from);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (i0 + u * step >= all) continue;
            ko[to[u]] = widen8<KV>(k[u], false);
            vo[to[u]] = widen8<KV>(v[u], true);
        }
    }
}

// Bytes of the widened prefixes, K and V, or 0 where they are widened tile by tile: with one
// block a group (256 query rows of a kv-head) on average, or too large a table.
size_t prefix_bytes(const AttnArgs& a, int groups) {
    if (a.kv_dtype == SPEC_DTYPE_BF16) return 0;
    const int64_t G = a.Hq / a.Hkv, rows = (int64_t)a.B * a.k * G;
    const int64_t all = (int64_t)groups * a.max_pages * a.Hkv * a.P;  // rows of K
    if (rows < 2 * 2 * ROWS * (int64_t)groups || all >= kMaxPrefixRows) return 0;
    return (size_t)all * D * 2 * 2;
}

struct Maps {
    CUtensorMap own, block, k, v, kwide, vwide;
};

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn get_encode_fn() {
    static EncodeTiledFn fn = nullptr;
    if (!fn) {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    }
    return fn;
}

template <int KV>
cudaError_t launch_typed(const Maps& m, const Params& prm, int num_ctas, cudaStream_t stream) {
    auto kern = attn_shared_kernel<KV>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)SMEM_BYTES);
    if (e != cudaSuccess) return e;
    if constexpr (KV != KV_BF16) {
        if (prm.k_prefix) {
            const AttnArgs& a = prm.a;
            const int64_t pieces = (int64_t)a.max_pages * a.Hkv * a.P * D / 16 / 256 + 1;
            const int64_t want = (num_ctas * 8 + prm.groups - 1) / prm.groups;
            e = launch_dependent(widen_kernel<KV>,
                                 dim3((unsigned)(pieces < want ? pieces : want), (unsigned)prm.groups),
                                 dim3(256), 0, stream, prm);
            if (e != cudaSuccess) return e;
        }
    }
    return launch_dependent(kern, dim3(num_ctas), dim3(threads<KV>()), SMEM_BYTES, stream, m.own,
                            m.block, m.k, m.v, m.kwide, m.vwide, prm);
}

}  // namespace

bool shared_supported(const AttnArgs& a, int groups) {
    const int G = a.Hq / a.Hkv, R = a.k * G;
    const bool pow2 = (a.P & (a.P - 1)) == 0;
    bool kv_ok = a.kv_dtype == SPEC_DTYPE_BF16 || a.kv_dtype == SPEC_DTYPE_E4M3;
    // the scales of an INT8 cache are fetched a page chunk (>= 32 bytes) at a
    // time with bulk copies, which need 16-byte aligned sources
    if (a.kv_dtype == SPEC_DTYPE_I8)
        kv_ok = ((reinterpret_cast<uintptr_t>(a.k_scale) | reinterpret_cast<uintptr_t>(a.v_scale)) &
                 15) == 0;
    if (groups < 1 || groups > a.B || a.q_dtype != SPEC_DTYPE_BF16 || !kv_ok || a.D != D || R > ROWS ||
        !pow2 || a.P < 16 || a.P > 256 || a.window > 0 || a.B > MAX_SEGS)
        return false;
    // sequences, and blocks of 2 NT tokens (each group's last may be short)
    const int64_t tokens = (int64_t)a.B * a.k, NT = ROWS / G;
    const int64_t segs = a.B + tokens / (2 * NT) + groups;
    if (segs > MAX_SEGS) return false;
    // keys, rounded up to tiles, and tile and cost counts are 32-bit (a charge of up to 256
    // tiles a segment)
    const int64_t keys = (int64_t)a.max_pages * a.P, tiles = (keys + TN - 1) / TN + 1;
    return keys < (1LL << 31) - 2 * TN &&
           segs * (kTileCost * 256 + 2 * kTileCost * tiles) < (1LL << 31) / a.Hkv &&
           (int64_t)a.num_pages * a.Hkv * a.P < (1LL << 31) && tokens * a.Hq < (1LL << 28) &&
           a.Hkv < 65536;
}

// What this kernel saves over reading each sequence by itself is the tiles that a
// group's blocks stand for, (B - blocks) Hkv T of a table of T tiles (a wide block's
// tile takes the time of 7/4 narrow ones); what it costs is every CTA's list and the
// second launch (10-20 us), and fp32 pieces of every row, written and read (2 KB, a
// tile a CTA for some 12000 rows).  The table's width stands for lengths that the host does
// not know, equal groups for the groups: the rule is for tables that the contexts
// fill.  The kernels that read each sequence by itself differ by type.  Measured on 75
// calls (this kernel / each sequence by itself, us, at saved tiles a CTA):
//   bf16  4.8 47 / 42   10.7 30 / 28   19 33 / 52   32 29 / 59   112 68 / 169
//   e4m3  8 66 / 52   25 35 / 37   28 43 / 39   363 249 / 266   973 229 / 651
//   i8    1.7 71 / 55   3.5 37 / 41   9.1 48 / 71   22 54 / 132   682 163 / 1768
// The worst left: bf16 12 62 / 61 and 7.6 24.5 / 28.9, e4m3 25 35 / 37 (not taken).
bool shared_pays(const AttnArgs& a, int groups, int sms) {
    const int64_t T = ((int64_t)a.max_pages * a.P + TN - 1) / TN, NT = ROWS / (a.Hq / a.Hkv);
    const int64_t tok = ((int64_t)a.B * a.k + groups - 1) / groups, left = tok % (2 * NT);  // of a group
    const int64_t blocks = tok / (2 * NT) * 7 + (left > NT ? 7 : left > 0 ? 4 : 0);
    const int64_t saved = (4 * a.B - groups * blocks) * a.Hkv * T;  // quarters of a tile
    const int fixed = a.kv_dtype == SPEC_DTYPE_BF16 ? 13 : a.kv_dtype == SPEC_DTYPE_E4M3 ? 48 : 3;
    return T >= 2 && saved >= 4 * (fixed + (int64_t)a.B * a.k * a.Hq / 12000) * sms;
}

size_t shared_workspace_bytes(const AttnArgs& a, int groups, int num_ctas) {
    const size_t rows = (size_t)a.B * a.k * a.Hq, slots = (size_t)8 * num_ctas * ROWS;
    return prefix_bytes(a, groups) + (2 * rows + slots) * (D + 1) * sizeof(float) +
           ((size_t)3 * num_ctas + 2) * 4 + (size_t)(MAX_SEGS + 4) * 4 + (size_t)a.B * 16 + 64;
}

cudaError_t launch_attn_shared(const AttnArgs& a, const int32_t* group_starts,
                               const int32_t* shared_lens, int groups, int num_ctas, void* workspace,
                               cudaStream_t stream) {
    EncodeTiledFn encode = get_encode_fn();
    if (!encode) return cudaErrorNotSupported;
    const int G = a.Hq / a.Hkv;
    Params prm;
    prm.a = a;
    prm.group_starts = group_starts;
    prm.shared_lens = shared_lens;
    prm.groups = groups;
    const size_t wide = prefix_bytes(a, groups);
    prm.k_prefix = wide ? static_cast<__nv_bfloat16*>(workspace) : nullptr;
    prm.v_prefix = wide ? prm.k_prefix + wide / 4 : nullptr;
    const size_t nrows = (size_t)a.B * a.k * a.Hq, slots = (size_t)8 * num_ctas * ROWS;
    prm.slot_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + wide);
    prm.slot_lse = prm.slot_o + (slots + 2 * nrows) * D;
    prm.slots = (int)slots;
    prm.G = G;
    prm.NT = ROWS / G;
    // (the fp32 arrays together are a multiple of 16 bytes)
    prm.seq_block = reinterpret_cast<int4*>(prm.slot_lse + slots + (2 * nrows + 3) / 4 * 4);
    prm.n_begin = reinterpret_cast<int*>(prm.seq_block + a.B);
    prm.w_begin = prm.n_begin + 2 * num_ctas + 1;
    prm.tile_pre = prm.w_begin + num_ctas + 1;

    Maps m;
    const cuuint32_t es[4] = {1, 1, 1, 1};
    for (int t = 0; t < 2; ++t) {
        cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.Hq, (cuuint64_t)a.B * a.k};
        cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)a.Hq * D * 2};
        cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)(t ? ROWS / G : a.k)};
        if (encode(t ? &m.block : &m.own, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(a.q),
                   dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    // K / V rows as in the 128-key kernel: bf16 as [groups of g rows] x [2 halves]
    // x [g rows] x [64 columns], g = 8 (K) or 16 (V); codes row by row
    const cuuint32_t ch = (cuuint32_t)(a.P < TN ? a.P : TN);
    auto map16 = [&](CUtensorMap* map, const void* base, cuuint64_t rows, cuuint32_t g) {
        cuuint64_t dims[4] = {64, g, 2, rows / g};
        cuuint64_t strides[3] = {(cuuint64_t)D * 2, 128, (cuuint64_t)g * D * 2};
        cuuint32_t box[4] = {64, g, 2, ch / g};
        return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides,
                      box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    auto map8 = [&](CUtensorMap* map, const void* base, cuuint64_t rows) {
        cuuint64_t dims[2] = {(cuuint64_t)D, rows};
        cuuint64_t strides[1] = {(cuuint64_t)D};
        cuuint32_t box[2] = {(cuuint32_t)D, ch};
        return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box,
                      es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    const cuuint64_t rows = (cuuint64_t)a.num_pages * a.Hkv * a.P;
    bool ok;
    if (a.kv_dtype == SPEC_DTYPE_BF16) {
        ok = map16(&m.k, a.k_cache, rows, 8) && map16(&m.v, a.v_cache, rows, 16);
        m.kwide = m.k;
        m.vwide = m.v;
    } else {
        ok = map8(&m.k, a.k_cache, rows) && map8(&m.v, a.v_cache, rows);
        m.kwide = m.k;
        m.vwide = m.v;
        if (ok && wide) {
            const cuuint64_t n = (cuuint64_t)groups * a.max_pages * a.Hkv * a.P;
            ok = map16(&m.kwide, prm.k_prefix, n, 8) && map16(&m.vwide, prm.v_prefix, n, 16);
        }
    }
    if (!ok) return cudaErrorInvalidValue;
    const cudaError_t e = a.kv_dtype == SPEC_DTYPE_I8     ? launch_typed<KV_I8>(m, prm, num_ctas, stream)
                          : a.kv_dtype == SPEC_DTYPE_E4M3 ? launch_typed<KV_E4M3>(m, prm, num_ctas, stream)
                                                          : launch_typed<KV_BF16>(m, prm, num_ctas, stream);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)a.B, (unsigned)a.Hkv, (unsigned)((a.k * G + 2 * kJoinWarps - 1) / (2 * kJoinWarps)));
    return launch_dependent(join_kernel, grid, dim3(kJoinWarps * 32), 0, stream, prm, num_ctas);
}

}  // namespace specv
