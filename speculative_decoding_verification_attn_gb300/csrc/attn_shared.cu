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
// A narrow tile (one 128-row Q) goes to one of two softmax sets in turn, as in
// the 128-key kernel without groups.  A wide one (two Q tiles) goes to both:
// each set has a Q of its own and the K and V tile is read from shared memory
// twice but loaded once: 64 KB of L2 traffic for 33.6 MFLOP, half of what narrow
// tiles would ask of L2.
//  * TMEM (512 columns): S of set 0 [0,128), S of set 1 [128,256), O of the sets
//    [256,384), [384,512); P (bf16) over the S columns it came from.
//  * Warps: 0-3 and 8-11 the softmax sets; 4 Q loads and Q K^T; 5 and 6 TMA
//    producers of K and V; 7 P V; with codes, 12-13 (K) and 14-15 (V) widen them.
//  * INT8 and e4m3 codes become bf16 exactly, in place (raw bytes land in the
//    upper half of their operand slot); scales are fp32 and enter the scores
//    and, before its rounding to bf16, P.  So the MMAs see the stored values and
//    the only roundings are P's (8 bits) and the output's.
//  * Every mbarrier wait is bounded (1 s); a timeout sets the device error word
//    and an abort flag, after which every role skips its remaining work, drains
//    its copies and tensor-core operations, and returns.
//
// Every query's pieces meet in a second launch: rows of whole segments wait in
// two fp32 arrays (own keys, prefix), those of segments that a CTA's range cuts
// in two slots per CTA.
#include <cuda.h>
#include <math.h>

#include "attn_tile.cuh"
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
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr int kSplitAlpha = 3;  // narrow tiles' time that a piece's fixed work takes
constexpr int kWideCost = 2;    // narrow tiles' time that a wide tile takes
// Keys below which a prefix is read sequence by sequence: one tile
constexpr int kMinShared = TN;

enum { KV_BF16, KV_I8, KV_E4M3 };
template <int KV> constexpr int threads() { return KV == KV_BF16 ? 12 * 32 : 16 * 32; }

constexpr uint32_t IDESC_QK = umma_idesc_bf16(ROWS, TN, 0, 0);
constexpr uint32_t IDESC_PV = umma_idesc_bf16(ROWS, D, 0, 1);  // B (V) MN-major

struct Smem {
    static constexpr int Q = 0;                         // 2 tiles
    static constexpr int KS = Q + 2 * Q_BYTES;          // 2 K slots
    static constexpr int VS = KS + 2 * SLOT_BYTES;      // 2 V slots
    static constexpr int BARS = VS + 2 * SLOT_BYTES;
    static constexpr int B_KFULL = 0, B_KEMPTY = 2, B_VFULL = 4, B_VEMPTY = 6, B_QFULL = 8,
                         B_QFREE = 10, B_SFULL = 12, B_PREADY = 14, B_SFREE = 16,
                         B_EPI = 18, B_DRAIN = 19, B_KREADY = 21, B_VREADY = 23, NUM_BARS = 25;
    static constexpr int MISC = BARS + 256;             // tmem base, abort flag, range at +16
    static constexpr int STAT = MISC + 64;              // (m, l) of [set][row]
    static constexpr int PIDS = STAT + 2 * 2 * ROWS * 4;  // [2 producers][LOOKAHEAD+1][8] int
    // scales of tile it at stage it % 4 (K, then V): INT8 128 fp32 each, e4m3
    // one per 16 keys.  Four stages: a tile's softmax may still read its scales
    // when the K slot of its parity is refilled
    static constexpr int SCALE = (PIDS + 2 * (LOOKAHEAD + 1) * NVB * 4 + 15) / 16 * 16;
    static constexpr int SCRAW = SCALE + 4 * 2 * TN * 4;  // INT8: fp16 scales, stage it % 2
    static constexpr int SEG = SCRAW + 2 * 2 * TN * 2;    // int4 [MAX_SEGS]
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
    float* slot_o;     // [2 C][256][D]: pieces of cut segments
    float* slot_lse;   // [2 C][256]
    float* home_o;     // [2][B k Hq][D]: own keys, prefix
    float* home_lse;   // [2][B k Hq]
    int64_t* t_begin;  // [C + 1] first tile of each CTA
    int* tile_pre;     // [segments + 1] tiles before a segment (per kv-head)
    int2* seq_block;   // [B] first block of the sequence's group (-1: none), its first token
};

// A segment: rows of tokens tok0 .. tok0 + ntok - 1, keys [key0, key1).
struct Seg {
    int tok0, ntok, key0, key1;
};

struct List {
    const Seg* seg;
    const int* tpre;
    int B, Hkv, NT, V;  // V segments, the first B of them the sequences' own keys
};

// Walks a CTA's tiles: segment v, kv-head, tile in the segment.
struct Cursor {
    int v, kvh, lt, nt;
    int64_t start;  // global index of the segment's first tile
    __device__ void init(int64_t t, const List& L) {
        int lo = 0, hi = L.V - 1;  // largest v with tpre[v] * Hkv <= t
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if ((int64_t)L.tpre[mid] * L.Hkv <= t) lo = mid; else hi = mid - 1;
        }
        v = lo;
        nt = L.tpre[v + 1] - L.tpre[v];
        const int64_t off = t - (int64_t)L.tpre[v] * L.Hkv;
        kvh = (int)(off / nt);
        lt = (int)(off % nt);
        start = (int64_t)L.tpre[v] * L.Hkv + (int64_t)kvh * nt;
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
    __device__ bool wide(const List& L) const { return L.seg[v].ntok > L.NT; }
    __device__ int key0(const List& L) const { return L.seg[v].key0 + lt * TN; }
    __device__ int valid(const List& L) const { return min(TN, L.seg[v].key1 - key0(L)); }
    // row of the block table that holds the segment's pages
    __device__ int table_row(const List& L, int k) const { return L.seg[v].tok0 / k; }
};

// First tile of CTA c's range: equal parts of the cost (alpha a segment, 1 or
// kWideCost a tile).
__device__ __forceinline__ int64_t range_begin(const List& L, const int* cpre, int alpha, int64_t c,
                                               int64_t C) {
    const int64_t W = (int64_t)cpre[L.V] * L.Hkv, T = (int64_t)L.tpre[L.V] * L.Hkv;
    const int64_t x = c * W / C;
    if (x >= W) return T;
    int lo = 0, hi = L.V - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((int64_t)cpre[mid] * L.Hkv <= x) lo = mid; else hi = mid - 1;
    }
    const int nt = L.tpre[lo + 1] - L.tpre[lo], each = L.seg[lo].ntok > L.NT ? kWideCost : 1;
    const int64_t off = x - (int64_t)cpre[lo] * L.Hkv, one = cpre[lo + 1] - cpre[lo];
    const int64_t h = off / one, r = off % one;
    const int64_t lt = r > alpha ? (r - alpha + each - 1) / each : 0;
    return (int64_t)L.tpre[lo] * L.Hkv + h * nt + lt;
}

// Inclusive running maximum or sum of s[0 .. n) in place, by one warp.
template <bool MAX>
__device__ __forceinline__ void warp_scan(int* s, int n) {
    const int lane = threadIdx.x & 31, per = (n + 31) / 32, lo = lane * per, hi = min(n, lo + per);
    int run = 0;
    for (int i = lo; i < hi; ++i) run = MAX ? max(run, s[i]) : run + s[i];
    int incl = run;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl = MAX ? max(incl, v) : incl + v;
    }
    run = __shfl_up_sync(0xffffffffu, incl, 1);
    if (lane == 0) run = 0;
    for (int i = lo; i < hi; ++i) {
        run = MAX ? max(run, s[i]) : run + s[i];
        s[i] = run;
    }
    __syncwarp();
}

// Builds the list in shared memory (every thread); V in *s_count.
template <int NTHREADS>
__device__ __forceinline__ void build_list(const Params& prm, Seg* seg, int* tpre, int* cpre,
                                           int* s_count, int alpha, int NT) {
    const AttnArgs& a = prm.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, k = a.k;
    const bool one = blockIdx.x == 0;
    int* starts = tpre;  // scratch until the prefixes are taken
    int* blocks = cpre;
    for (int b = tid; b < a.B; b += NTHREADS) {
        int c = a.ctx_lens[b];
        const int64_t cap = (int64_t)a.max_pages * a.P - k;
        if (c < 0 || (int64_t)c > cap) {
            raise_device_error(a.dev_err, SPEC_DEVERR_CTX);
            c = c < 0 ? 0 : (int)(cap < 0 ? 0 : cap);
        }
        seg[b] = Seg{b * k, k, 0, c + k};
        if (one) prm.seq_block[b] = make_int2(-1, 0);
    }
    for (int g = tid; g <= prm.groups; g += NTHREADS) {
        const int s = prm.group_starts[g];
        if (s < 0 || s > a.B) raise_device_error(a.dev_err, SPEC_DEVERR_GROUP);
        starts[g] = s < 0 ? 0 : s > a.B ? a.B : s;
    }
    __syncthreads();
    for (int g = tid; g < prm.groups; g += NTHREADS)
        if (starts[g + 1] < starts[g]) raise_device_error(a.dev_err, SPEC_DEVERR_GROUP);
    __syncthreads();
    if (warp == 0) warp_scan<true>(starts, prm.groups + 1);  // ascending from here on
    __syncthreads();
    // how many blocks each group's prefix takes, and where each sequence's own keys begin
    for (int g = warp; g < prm.groups; g += NTHREADS / 32) {
        const int lo = starts[g], hi = starts[g + 1];
        int least = INT32_MAX;
        for (int b = lo + lane; b < hi; b += 32) least = min(least, seg[b].key1 - k);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
        int s = prm.shared_lens[g], n = 0;
        if (hi > lo && (s < 0 || s > least)) {
            if (lane == 0) raise_device_error(a.dev_err, SPEC_DEVERR_GROUP);
            s = s < 0 ? 0 : least;
        }
        if (hi - lo >= 2 && s >= kMinShared) {
            s = s / a.P * a.P;
            n = ((hi - lo) * k + 2 * NT - 1) / (2 * NT);
        } else {
            s = 0;
        }
        if (s == 0) n = 0;
        if (lane == 0) blocks[g] = n;
        __syncwarp();
        for (int b = lo + lane; b < hi; b += 32) seg[b].key0 = s;
    }
    __syncthreads();
    if (warp == 0) {
        warp_scan<false>(blocks, prm.groups);
        if (lane == 0) *s_count = a.B + (prm.groups > 0 ? blocks[prm.groups - 1] : 0);
    }
    __syncthreads();
    for (int g = warp; g < prm.groups; g += NTHREADS / 32) {
        const int v0 = g ? blocks[g - 1] : 0, n = blocks[g] - v0;
        if (n == 0) continue;
        const int lo = starts[g], hi = starts[g + 1], s = seg[lo].key0;
        for (int i = lane; i < n; i += 32) {
            const int tok = i * 2 * NT, left = (hi - lo) * k - tok;
            seg[a.B + v0 + i] = Seg{lo * k + tok, min(left, 2 * NT), 0, s};
        }
        if (one)
            for (int b = lo + lane; b < hi; b += 32) prm.seq_block[b] = make_int2(a.B + v0, lo * k);
    }
    __syncthreads();
    const int V = *s_count;
    for (int v = tid; v < V; v += NTHREADS) {
        const Seg q = seg[v];
        const int nt = (q.key1 - q.key0 + TN - 1) / TN;
        tpre[v + 1] = nt;
        cpre[v + 1] = alpha + nt * (q.ntok > NT ? kWideCost : 1);
    }
    if (tid == 0) tpre[0] = cpre[0] = 0;
    __syncthreads();
    if (warp == 0) warp_scan<false>(tpre, V + 1);
    if (warp == 1) warp_scan<false>(cpre, V + 1);
    __syncthreads();
}

// Widens 16 codes to bf16, exactly.
// INT8: the low seven bits under the exponent of 128, less 128 (or 256 for a
// negative code, whose low seven bits are its value + 128).
__device__ __forceinline__ uint32_t i8x2_to_bf16(uint32_t t) {  // bytes 0 and 2
    const uint32_t m = (t & 0x007f007fu) | 0x43004300u, s = (t & 0x00800080u) | 0x43004300u;
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(s));
    return r;
}
// e4m3: exponent and fraction moved to bf16's places, times 2^120 (the
// difference of the biases; subnormal codes come right with it).
__device__ __forceinline__ uint32_t e4m3x2_to_bf16(uint32_t t) {  // bytes 1 and 3
    const uint32_t m = ((t >> 4) & 0x07f007f0u) | (t & 0x80008000u);
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(0x7b807b80u));
    return r;
}
template <int KV>
__device__ __forceinline__ void widen16(const uint4 r, uint4& lo, uint4& hi) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (KV == KV_I8) {
            o[2 * i] = i8x2_to_bf16(__byte_perm(w[i], 0, 0x4140));
            o[2 * i + 1] = i8x2_to_bf16(__byte_perm(w[i], 0, 0x4342));
        } else {
            o[2 * i] = e4m3x2_to_bf16(__byte_perm(w[i], 0, 0x1404));
            o[2 * i + 1] = e4m3x2_to_bf16(__byte_perm(w[i], 0, 0x3424));
        }
    }
    lo = make_uint4(o[0], o[1], o[2], o[3]);
    hi = make_uint4(o[4], o[5], o[6], o[7]);
}

// Scores of 64 columns (raw fp32 bits) times the softmax scale in log2 units
// (for codes: and the keys' scales) with the invisible ones at -inf; returns their
// maximum.  ks: the stage's scales of K from the first of the columns.
template <int KV>
__device__ __forceinline__ float scores64(uint32_t (&r)[64], float sl2, const float* ks, uint64_t vis) {
    if (KV == KV_BF16) return scale_mask64(r, sl2, vis);
#pragma unroll
    for (int c = 0; c < 64; c += 4) {
        float4 s;
        if (KV == KV_I8) {
            s = *reinterpret_cast<const float4*>(ks + c);
        } else {
            s.x = s.y = s.z = s.w = ks[c / 16];
        }
        float v0, v1;
        f2_split(f2_mul(f2(__uint_as_float(r[c]), __uint_as_float(r[c + 1])), f2(s.x, s.y)), v0, v1);
        r[c] = __float_as_uint(v0);
        r[c + 1] = __float_as_uint(v1);
        f2_split(f2_mul(f2(__uint_as_float(r[c + 2]), __uint_as_float(r[c + 3])), f2(s.z, s.w)), v0,
                 v1);
        r[c + 2] = __float_as_uint(v0);
        r[c + 3] = __float_as_uint(v1);
    }
    return mask_max64(r, vis);
}

// p = 2^(v - m) of 64 columns, for codes times the keys' scales of V, packed to
// bf16 pairs; returns the sum of p.
template <int KV>
__device__ __forceinline__ float weights64(const uint32_t (&v)[64], float m, const float* vs,
                                           uint32_t (&pk)[32]) {
    if (KV == KV_BF16) return exp_pack64<false>(v, m, pk);
    const uint64_t neg_m = f2(-m, -m);
    uint64_t ps[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
    for (int c = 0; c < 64; c += 4) {
        float4 s;
        if (KV == KV_I8) {
            s = *reinterpret_cast<const float4*>(vs + c);
        } else {
            s.x = s.y = s.z = s.w = vs[c / 16];
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float e0, e1;
            f2_split(f2_add(f2(__uint_as_float(v[c + 2 * u]), __uint_as_float(v[c + 2 * u + 1])), neg_m),
                     e0, e1);
            const uint64_t e = f2(fast_exp2(e0), fast_exp2(e1));
            ps[u] = f2_add(ps[u], e);
            f2_split(f2_mul(e, u ? f2(s.z, s.w) : f2(s.x, s.y)), e0, e1);
            pk[c / 2 + u] = pack_bf16x2(e0, e1);
        }
    }
    float a0, a1, b0, b1;
    f2_split(ps[0], a0, a1);
    f2_split(ps[1], b0, b1);
    return (a0 + b0) + (a1 + b1);
}

template <int KV>
__global__ void __launch_bounds__(threads<KV>(), 1)
attn_shared_kernel(const __grid_constant__ CUtensorMap own_map,  // q: boxes of k tokens
                   const __grid_constant__ CUtensorMap block_map,  // q: boxes of NT tokens
                   const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap, const Params prm) {
    constexpr int NTH = threads<KV>();
    constexpr bool CODES = KV != KV_BF16;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const AttnArgs& a = prm.a;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Smem::BARS);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + Smem::MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + Smem::MISC + 4);
    int* s_count = reinterpret_cast<int*>(sm + Smem::MISC + 8);
    int64_t* s_rng = reinterpret_cast<int64_t*>(sm + Smem::MISC + 16);
    Seg* s_seg = reinterpret_cast<Seg*>(sm + Smem::SEG);
    int* s_tpre = reinterpret_cast<int*>(sm + Smem::TPRE);
    int* s_cpre = reinterpret_cast<int*>(sm + Smem::CPRE);
    float* s_scale = reinterpret_cast<float*>(sm + Smem::SCALE);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int k = a.k, Hkv = a.Hkv, G = a.Hq / a.Hkv, P = a.P, NT = ROWS / G;
    const int CH = P < TN ? P : TN, NCH = TN / CH;  // keys per page chunk, chunks per tile

    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bars[Smem::B_KFULL + s], 1);
            mbar_init(&bars[Smem::B_KEMPTY + s], 1);
            mbar_init(&bars[Smem::B_VFULL + s], 1);
            mbar_init(&bars[Smem::B_VEMPTY + s], 1);
            mbar_init(&bars[Smem::B_QFULL + s], 1);
            mbar_init(&bars[Smem::B_QFREE + s], 1);
            mbar_init(&bars[Smem::B_SFULL + s], 1);
            mbar_init(&bars[Smem::B_PREADY + s], 4);  // the 4 warps of the set
            mbar_init(&bars[Smem::B_SFREE + s], 1);
            mbar_init(&bars[Smem::B_KREADY + s], 2);  // the 2 warps widening K / V
            mbar_init(&bars[Smem::B_VREADY + s], 2);
        }
        mbar_init(&bars[Smem::B_EPI], 8);  // every softmax warp, once per piece
        mbar_init(&bars[Smem::B_DRAIN], 1);
        mbar_init(&bars[Smem::B_DRAIN + 1], 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    grid_dep_launch_dependents();
    grid_dep_wait();
    if (warp == 4) {
        tmem_alloc(tmem_slot, TMEM_COLS);
        tmem_relinquish();
    }
    {
        // rows that the copies of q never write stay zero
        uint4* q4 = reinterpret_cast<uint4*>(sm + Smem::Q);
        for (int e = tid; e < 2 * Q_BYTES / 16; e += NTH)
            if ((e % (Q_HALF / 16)) / 8 >= k * G) q4[e] = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
    }
    const int alpha = a.split_alpha >= 0 ? a.split_alpha : kSplitAlpha;
    build_list<NTH>(prm, s_seg, s_tpre, s_cpre, s_count, alpha, NT);
    const List L = {s_seg, s_tpre, a.B, Hkv, NT, *s_count};
    if (tid < 2) s_rng[tid] = range_begin(L, s_cpre, alpha, blockIdx.x + tid, gridDim.x);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int64_t t_begin = ld_shared_s64(s_rng);
    const int n_tiles = (int)(ld_shared_s64(s_rng + 1) - t_begin);
    // what the second launch needs to find the pieces
    if (tid < 2) prm.t_begin[blockIdx.x + tid] = ld_shared_s64(s_rng + tid);
    if (blockIdx.x == 0)
        for (int v = tid; v <= L.V; v += NTH) prm.tile_pre[v] = s_tpre[v];

    // INT8 / e4m3 (16 warps on 64K registers): 160 for each softmax warpgroup, 80 for
    // the issue / copy one, 112 for the widening one (2 x 160 + 80 + 112 = 4 x 128)
    if (warp >= 4 && warp < 8) {
    if constexpr (CODES) regs_dec<80>();
    if (warp == 5 || warp == 6) {
        // ================= TMA producers: warp 5 K, warp 6 V, every tile =================
        // Tile it to slot it % 2 of each ring, one copy per page chunk, as in the
        // 128-key kernel without groups; block-table entries LOOKAHEAD tiles
        // ahead.  With codes, the K producer also brings the scales of both.
        const bool is_v = warp == 6;
        int* pids = reinterpret_cast<int*>(sm + Smem::PIDS) + (is_v ? 1 : 0) * (LOOKAHEAD + 1) * NVB;
        uint64_t* full = &bars[is_v ? Smem::B_VFULL : Smem::B_KFULL];
        uint64_t* empty = &bars[is_v ? Smem::B_VEMPTY : Smem::B_KEMPTY];
        uint8_t* ring = sm + (is_v ? Smem::VS : Smem::KS);
        const CUtensorMap* map = is_v ? &vmap : &kmap;
        const int gshift = is_v ? 4 : 3;  // log2 of the rows of a group
        Cursor cur, ahead;
        if (n_tiles > 0) {
            cur.init(t_begin, L);
            ahead = cur;
        }
        const uint64_t once = l2_policy_evict_first();
        uint64_t again;  // a prefix is read by many CTAs
        asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(again));
        if (lane == 0) prefetch_tmap(map);
        auto fetch_pids = [&](int slot, const Cursor& c) {
            if (lane < NCH && lane * CH < c.valid(L))
                cp_async_4(&pids[slot * NVB + lane],
                           &a.block_table[(int64_t)c.table_row(L, k) * a.max_pages +
                                          (c.key0(L) + lane * CH) / P]);
        };
        auto page_of = [&](int slot, int chunk) {
            int page = pids[slot * NVB + chunk];
            if (page < 0 || page >= a.num_pages) {
                raise_device_error(a.dev_err, SPEC_DEVERR_PAGE);
                page = 0;
            }
            return page;
        };
        // e4m3: lane l < 8 the scale of K of keys [16 l, 16 l + 16), l + 8 that of V
        auto fetch_scale = [&](int slot, const Cursor& c) {
            const int j = (lane & 7) * 16;
            if (lane >= 16 || j >= c.valid(L)) return 0.f;
            const float* s = lane < 8 ? a.k_page_scale : a.v_page_scale;
            return __ldg(s + (int64_t)page_of(slot, j / CH) * Hkv + c.kvh);
        };
        for (int la = 0; la < LOOKAHEAD; ++la) {
            if (la < n_tiles) {
                fetch_pids(la % (LOOKAHEAD + 1), ahead);
                if (la + 1 < n_tiles) ahead.next(L);
            }
            cp_async_commit();
        }
        int n_issued = 0;
        bool ok = true;
        float scale = 0.f;
        if (KV == KV_E4M3 && !is_v && n_tiles > 0) {
            cp_async_wait<LOOKAHEAD - 1>();
            __syncwarp();
            scale = fetch_scale(0, cur);
        }
        for (int it = 0; it < n_tiles && ok; ++it) {
            if (it + LOOKAHEAD < n_tiles) {
                fetch_pids((it + LOOKAHEAD) % (LOOKAHEAD + 1), ahead);
                if (it + LOOKAHEAD + 1 < n_tiles) ahead.next(L);
            }
            cp_async_commit();
            cp_async_wait<LOOKAHEAD - 1>();  // entries of tiles `it` and it + 1
            __syncwarp();
            const int pslot = it % (LOOKAHEAD + 1);
            const int key0 = cur.key0(L), nck = (cur.valid(L) + CH - 1) / CH;
            const int s = it & 1;
            if (it >= 2) ok = warp_wait(&empty[s], ((it >> 1) - 1) & 1, abort_flag, a.dev_err);
            if (!ok) break;
            uint32_t bytes = (uint32_t)(nck * CH) * (CODES ? 128u : 256u);
            if (!is_v && KV == KV_I8) bytes += (uint32_t)(nck * CH) * 4;
            if (!is_v && KV == KV_E4M3 && lane < 16)
                s_scale[((it & 3) * 2 + (lane >> 3)) * TN + (lane & 7)] =
                    lane < 8 ? scale * a.scale * kLog2e : scale;
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(&full[s], bytes);
            __syncwarp();
            if (lane < nck) {
                const int page = page_of(pslot, lane);
                const int row = (page * Hkv + cur.kvh) * P + (key0 + lane * CH) % P;
                const uint64_t pol = cur.v >= L.B ? again : once;
                if constexpr (CODES) {
                    tma_load_2d(ring + s * SLOT_BYTES + RAW_OFF + lane * CH * 128, map, &full[s], 0,
                                row, pol);
                    if (KV == KV_I8 && !is_v) {
                        uint8_t* raw = sm + Smem::SCRAW + s * 2 * TN * 2 + lane * CH * 2;
                        bulk_load(raw, a.k_scale + row, CH * 2, &full[s]);
                        bulk_load(raw + TN * 2, a.v_scale + row, CH * 2, &full[s]);
                    }
                } else {
                    tma_load_4d_hint(ring + s * SLOT_BYTES + lane * CH * 256, map, &full[s], 0, 0,
                                     0, row >> gshift, pol);
                }
            }
            n_issued = it + 1;
            __syncwarp();
            if (it + 1 < n_tiles) {
                cur.next(L);
                if (KV == KV_E4M3 && !is_v) scale = fetch_scale((it + 1) % (LOOKAHEAD + 1), cur);
            }
        }
        cp_async_wait<0>();
        if (!ok && lane == 0) {
            // the latest copy into each slot lands before the CTA exits
            for (int sl = 0; sl < 2; ++sl) {
                const int last = (n_issued - 1) - (((n_issued - 1) - sl) & 1);
                if (last >= 0) mbar_drain(&full[sl], (last >> 1) & 1);
            }
        }
    } else if (warp == 4) {
        // ================= Q loads and Q K^T issue =================
        // A narrow piece's Q is in one of the two tiles, a wide one's in both.
        // After a narrow piece the next narrow one takes the other tile, and
        // its Q is on the way while this one is worked on.
        if (n_tiles > 0) {
            Cursor cur;
            cur.init(t_begin, L);
            int loads[2] = {0, 0};   // copies into each Q tile
            int uses[2] = {0, 0};    // S buffers handed out
            int qb = 1, next_qb = -1;  // this piece's Q tile (narrow); that of the next, on its way
            bool ok = true;
            // the Q of `half` of segment c into tile t, once its last user is done
            auto load_q = [&](int t, const Cursor& c, int half) {
                if (loads[t] > 0 &&
                    !warp_wait(&bars[Smem::B_QFREE + t], (loads[t] - 1) & 1, abort_flag, a.dev_err))
                    return false;
                const bool own = c.v < L.B;
                if (lane == 0) {
                    uint64_t* bar = &bars[Smem::B_QFULL + t];
                    mbar_arrive_expect_tx(bar, 2 * (own ? k : NT) * G * 128);
                    for (int h = 0; h < 2; ++h)
                        tma_load_3d(sm + Smem::Q + t * Q_BYTES + h * Q_HALF,
                                    own ? &own_map : &block_map, bar, h * 64, c.kvh * G,
                                    L.seg[c.v].tok0 + half * NT);
                }
                __syncwarp();
                ++loads[t];
                return true;
            };
            const uint64_t qdesc0 = umma_sdesc_sw128(smem_u32(sm + Smem::Q), 16, 1024);
            const uint64_t kdesc0 = umma_sdesc_sw128(smem_u32(sm + Smem::KS), 16, 2048);
            for (int it = 0; it < n_tiles && ok; ++it) {
                const bool first = (it == 0) || (cur.lt == 0);
                const bool last = (it == n_tiles - 1) || (cur.lt == cur.nt - 1);
                const bool wide = cur.wide(L);
                const int s = it & 1;
                if (first) {
                    if (wide) {
                        ok = load_q(0, cur, 0) && load_q(1, cur, 1);
                    } else if (next_qb >= 0) {
                        qb = next_qb;
                    } else {
                        qb ^= 1;
                        ok = load_q(qb, cur, 0);
                    }
                    if (!ok) break;
                    next_qb = -1;
                    if (!wide && cur.start + cur.nt < ld_shared_s64(s_rng + 1)) {
                        Cursor nx = cur;
                        nx.next_segment(L);
                        if (!nx.wide(L)) {
                            next_qb = qb ^ 1;
                            ok = load_q(next_qb, nx, 0);
                        }
                    }
                    for (int t = 0; t < 2 && ok; ++t)
                        if (wide || t == qb) {
                            // (the tile's last copy but one where the next piece's is under way)
                            ok = warp_wait(&bars[Smem::B_QFULL + t], (loads[t] - 1) & 1, abort_flag,
                                           a.dev_err);
                        }
                    if (!ok) break;
                }
                ok = warp_wait(&bars[(CODES ? Smem::B_KREADY : Smem::B_KFULL) + s], (it >> 1) & 1,
                               abort_flag, a.dev_err);
                for (int set = 0; set < 2 && ok; ++set) {
                    if (!wide && set != s) continue;
                    // S buffer free: P V of its last tile has read P
                    if (uses[set] > 0)
                        ok = warp_wait(&bars[Smem::B_SFREE + set], (uses[set] - 1) & 1, abort_flag,
                                       a.dev_err);
                    if (!ok) break;
                    ++uses[set];
                    __syncwarp();
                    tc_fence_after();
                    // S = Q K^T: k-slice kk at half kk/4 (Q: 16 KB on, K: 1 KB on
                    // in every 8-key group), 32-byte step kk%4
                    const uint64_t qd = qdesc0 + ((uint32_t)((wide ? set : qb) * Q_BYTES) >> 4);
                    const uint64_t kd = kdesc0 + ((uint32_t)(s * SLOT_BYTES) >> 4);
                    if (elect_lane()) {
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            umma_ss(tmem + TM_S + set * TN,
                                    qd + (kk >> 2) * (Q_HALF >> 4) + (kk & 3) * 2,
                                    kd + (kk >> 2) * (1024 >> 4) + (kk & 3) * 2, IDESC_QK,
                                    kk ? 1u : 0u);
                    }
                    __syncwarp();
                    umma_commit_w(&bars[Smem::B_SFULL + set]);
                }
                if (!ok) break;
                umma_commit_w(&bars[Smem::B_KEMPTY + s]);
                if (last) {
                    if (wide || qb == 0) umma_commit_w(&bars[Smem::B_QFREE + 0]);
                    if (wide || qb == 1) umma_commit_w(&bars[Smem::B_QFREE + 1]);
                }
                if (it + 1 < n_tiles) cur.next(L);
            }
            // Q copies in flight land before the CTA exits
            if (!ok && lane == 0)
                for (int t = 0; t < 2; ++t)
                    if (loads[t] > 0) mbar_drain(&bars[Smem::B_QFULL + t], (loads[t] - 1) & 1);
            // every tensor-core op of this warp finishes before TMEM is released
            __syncwarp();
            umma_commit_w(&bars[Smem::B_DRAIN]);
            if (lane == 0) mbar_drain(&bars[Smem::B_DRAIN], 0);
            __syncwarp();
        }
    } else if (warp == 7) {
        // ================= P V issue =================
        if (n_tiles > 0) {
            Cursor cur;
            cur.init(t_begin, L);
            int pc = -1;
            int uses[2] = {0, 0};
            bool ok = true;
            bool has[2] = {false, false};  // the set issued a P V in this piece
            const uint64_t vdesc0 = umma_sdesc_sw128(smem_u32(sm + Smem::VS), 2048, 1024);
            for (int it = 0; it < n_tiles && ok; ++it) {
                const bool first = (it == 0) || (cur.lt == 0);
                const bool wide = cur.wide(L);
                const int s = it & 1, nvalid = cur.valid(L), nvb = (nvalid + 15) / 16;
                if (first) {
                    ++pc;
                    has[0] = has[1] = false;
                    // the previous piece's epilogue has read both O
                    if (pc >= 1)
                        ok = warp_wait(&bars[Smem::B_EPI], (pc - 1) & 1, abort_flag, a.dev_err);
                }
                if (ok)
                    ok = warp_wait(&bars[(CODES ? Smem::B_VREADY : Smem::B_VFULL) + s],
                                   (it >> 1) & 1, abort_flag, a.dev_err);
                if (!ok) break;
                if (!CODES && nvalid % 16 != 0) {
                    // keys past the end that the last P V reads: 0 * (stale or canary) never reaches O
                    uint8_t* vst = sm + Smem::VS + s * SLOT_BYTES;
                    for (int e = lane; e < (nvb * 16 - nvalid) * 16; e += 32) {
                        const int t = nvalid + e / 16, h = (e / 8) & 1, c16 = e % 8;
                        *reinterpret_cast<uint4*>(vst + (t / 16) * 4096 + h * 2048 +
                                                  (t % 16) * 128 + c16 * 16) =
                            make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                for (int set = 0; set < 2 && ok; ++set) {
                    if (!wide && set != s) continue;
                    ok = warp_wait(&bars[Smem::B_PREADY + set], uses[set] & 1, abort_flag, a.dev_err);
                    if (!ok) break;
                    ++uses[set];
                    tc_fence_after();
                    // O_set += P V: MMA j takes keys [16j, 16j + 16) (4 KB group j), their
                    // P at the S columns [8j, 8j + 8) (j < 4) or [64 + 8(j-4), ...)
                    const uint64_t vd = vdesc0 + ((uint32_t)(s * SLOT_BYTES) >> 4);
                    const bool hs = set ? has[1] : has[0];
                    const uint32_t sbuf = tmem + TM_S + set * TN, od = tmem + TM_O + set * D;
                    if (elect_lane()) {
#pragma unroll
                        for (int j = 0; j < NVB; ++j)
                            if (j < nvb)
                                umma_ts(od, sbuf + (j < 4 ? 8 * j : 64 + 8 * (j - 4)),
                                        vd + ((uint32_t)(j * 4096) >> 4), IDESC_PV,
                                        (hs || j > 0) ? 1u : 0u);
                    }
                    __syncwarp();
                    umma_commit_w(&bars[Smem::B_SFREE + set]);
                    if (set) has[1] = true;
                    else has[0] = true;
                }
                if (!ok) break;
                umma_commit_w(&bars[Smem::B_VEMPTY + s]);
                if (it + 1 < n_tiles) cur.next(L);
            }
            __syncwarp();
            umma_commit_w(&bars[Smem::B_DRAIN + 1]);
            if (lane == 0) mbar_drain(&bars[Smem::B_DRAIN + 1], 0);
            __syncwarp();
        }
    }
    } else if (CODES && warp >= 12) {
        if constexpr (CODES) {
        regs_dec<112>();
        // ================= widening (warps 12-13 K, 14-15 V) =================
        // Every tile in order, each code exactly to bf16, in place, in the layout the
        // MMAs read.  The raw tile sits in the upper half of its slot: rows
        // 0..63 are written to the lower half straight away; rows 64..127 land
        // over the raw bytes, so the pair first reads all of them and meets
        // at a barrier.  Rows past the end become zeros.  Every warp runs
        // every tile and every barrier, also after an abort.
        const bool is_v = warp >= 14;
        const int ct = tid - (is_v ? 14 : 12) * 32;  // 0..63
        Cursor c;
        if (n_tiles > 0) c.init(t_begin, L);
        bool ok = true;
        for (int it = 0; it < n_tiles; ++it) {
            const int s = it & 1;
            const int nvalid = c.valid(L);
            const int nch = (nvalid + 15) / 16 * 16 * 8;  // 16-code pieces the MMAs read
            if (ok)
                ok = warp_wait(&bars[(is_v ? Smem::B_VFULL : Smem::B_KFULL) + s], (it >> 1) & 1,
                               abort_flag, a.dev_err);
            uint8_t* slot = sm + (is_v ? Smem::VS : Smem::KS) + s * SLOT_BYTES;
            // piece id: key id / 8, head dims 16 (id % 8) ..
            auto put = [&](int id, uint4 raw) {
                const int j = id >> 3, c16 = id & 7, h = c16 >> 2, sw = j & 7;
                uint4 lo, hi;
                widen16<KV>(raw, lo, hi);
                if (j >= nvalid) lo = hi = make_uint4(0, 0, 0, 0);
                // chunks cc, cc+1 of half h (swizzled by the row); lanes of half 1
                // store their odd chunk first so that 8 consecutive lanes hit 8
                // bank groups
                const int cc = (c16 & 3) * 2;
                const int o0 = ((cc + h) ^ sw) << 4, o1 = ((cc + 1 - h) ^ sw) << 4;
                uint8_t* row = is_v ? slot + (j >> 4) * 4096 + h * 2048 + (j & 15) * 128
                                    : slot + (j >> 3) * 2048 + h * 1024 + (j & 7) * 128;
                *reinterpret_cast<uint4*>(row + o0) = h ? hi : lo;
                *reinterpret_cast<uint4*>(row + o1) = h ? lo : hi;
            };
            if (KV == KV_I8 && !is_v && ok) {
                // the keys' scales to fp32 (K's with the softmax scale), 0 past the end
                const __half* raw = reinterpret_cast<const __half*>(sm + Smem::SCRAW + s * 2 * TN * 2);
                float* to = s_scale + (it & 3) * 2 * TN;
                for (int j = ct; j < TN; j += 64) {
                    to[j] = j < nvalid ? __half2float(raw[j]) * a.scale * kLog2e : 0.f;
                    to[TN + j] = j < nvalid ? __half2float(raw[TN + j]) : 0.f;
                }
            }
            // rows 0..63: raw in [16, 24) KB, output in [0, 16) KB
#pragma unroll 4
            for (int u = 0; u < 8; ++u) {
                const int id = ct + 64 * u;
                if (ok && id < nch) put(id, *reinterpret_cast<const uint4*>(slot + RAW_OFF + id * 16));
            }
            // rows 64..127: read all raw first, their output overlaps it
            uint4 raw[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int id = 512 + ct + 64 * u;
                if (ok && id < nch) raw[u] = *reinterpret_cast<const uint4*>(slot + RAW_OFF + id * 16);
            }
            named_bar_sync(is_v ? 7 : 6, 64);
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int id = 512 + ct + 64 * u;
                if (ok && id < nch) put(id, raw[u]);
            }
            fence_proxy_async_smem();  // generic-proxy writes -> tensor-core reads
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[(is_v ? Smem::B_VREADY : Smem::B_KREADY) + s]);
            if (it + 1 < n_tiles) c.next(L);
        }
        }
    } else {
        if constexpr (CODES) regs_inc<160>();
        // ================= softmax sets (0: warps 0-3, 1: 8-11) =================
        // Narrow tiles by parity, wide ones both (set = half of the block's rows).
        const int set = warp >= 8 ? 1 : 0;
        const int quad = warp & 3;                 // TMEM lane quadrant
        const int r = quad * 32 + lane;            // row of this thread in its Q tile
        const float sl2 = a.scale * kLog2e;
        const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
        const uint32_t s_mine = lane_base + TM_S + set * TN;
        const uint32_t o_mine = TM_O + set * D, o_other = TM_O + (1 - set) * D;
        float* s_stat_m = reinterpret_cast<float*>(sm + Smem::STAT);
        float* s_stat_l = s_stat_m + 2 * ROWS;
        float m_ref = -INFINITY, l = 0.f;
        bool has = false;       // this set took a tile of the current piece
        int own = 0;            // tiles this set has taken (its S / P V phase count)
        uint64_t mrow = 0;
        int rows = 0, ctx = 0;  // rows of this set's Q tile; keys that are no drafts
        bool wide = false;
        Cursor cur;
        if (n_tiles > 0) cur.init(t_begin, L);
        bool ok = true;
        for (int it = 0; it < n_tiles; ++it) {
            const bool first = (it == 0) || (cur.lt == 0);
            const bool last = (it == n_tiles - 1) || (cur.lt == cur.nt - 1);
            const int key0 = cur.key0(L), nvalid = cur.valid(L);
            if (first) {
                const Seg q = L.seg[cur.v];
                wide = q.ntok > NT;
                rows = (wide ? (set ? q.ntok - NT : NT) : q.ntok) * G;
                m_ref = -INFINITY;
                l = 0.f;
                has = false;
                if (cur.v < L.B) {
                    ctx = q.key1 - k;
                    mrow = draft_bits(a, cur.v, r < rows ? r / G : k - 1);
                } else {
                    ctx = q.key1;
                    mrow = 0;
                }
            }
            const bool active = quad * 32 < rows;
            if (wide || (it & 1) == set) {
                if (ok)
                    ok = warp_wait(&bars[Smem::B_SFULL + set], own & 1, abort_flag, a.dev_err);
                if (ok && active) {
                    tc_fence_after();
                    uint32_t v[64];
                    const float* ks = s_scale + (it & 3) * 2 * TN;
                    const float* vs = ks + TN;
                    constexpr int HALF = KV == KV_E4M3 ? 4 : 64;  // scales of 64 columns
                    const uint64_t vis0 = visible64<false>(key0, 0, nvalid, ctx, mrow, 0, 0);
                    const uint64_t vis1 = visible64<false>(key0, 64, nvalid, ctx, mrow, 0, 0);
                    // row maximum over both halves; the second half stays in v
                    load64(s_mine, v);
                    const float mx0 = scores64<KV>(v, sl2, ks, vis0);
                    load64(s_mine + 64, v);
                    const float mx1 = scores64<KV>(v, sl2, ks + HALF, vis1);
                    const float m_new = fmaxf(m_ref, fmaxf(mx0, mx1));
                    float al = 1.f;
                    const bool move = m_new > m_ref + kRescaleThreshold;  // also -inf -> finite
                    if (move) {
                        al = (m_ref == -INFINITY) ? 0.f : fast_exp2(m_ref - m_new);
                        m_ref = m_new;
                        l *= al;
                    }
                    const float m_use = m_ref == -INFINITY ? 0.f : m_ref;  // keeps -inf - m finite
                    uint32_t pk[32];
                    // P of keys 64..127 over S columns [64, 96), then keys 0..63
                    // (reloaded) over [0, 32)
                    l += weights64<KV>(v, m_use, vs + HALF, pk);
                    tmem_st32(s_mine + 64, pk);
                    load64(s_mine, v);
                    scores64<KV>(v, sl2, ks, vis0);
                    l += weights64<KV>(v, m_use, vs, pk);
                    tmem_st32(s_mine, pk);
                    tmem_wait_st();
                    if (has && __any_sync(0xffffffffu, move)) {
                        // O holds every earlier P V of this set (the S buffer of
                        // this tile was free only after the previous one read it)
#pragma unroll
                        for (int c4 = 0; c4 < D / 32; ++c4) {
                            uint32_t ov[32];
                            tmem_ld32(lane_base + o_mine + c4 * 32, ov);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                ov[e] = __float_as_uint(__uint_as_float(ov[e]) * al);
                            tmem_st32(lane_base + o_mine + c4 * 32, ov);
                        }
                        tmem_wait_st();
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[Smem::B_PREADY + set]);
                has = true;
                ++own;
            }
            if (last) {
                // ---- epilogue of the piece that ends at this tile
                if (ok && has)  // this set's last P V (tile own - 1) is done
                    ok = warp_wait(&bars[Smem::B_SFREE + set], (own - 1) & 1, abort_flag,
                                   a.dev_err);
                tc_fence_after();
                const int64_t tb = ld_shared_s64(s_rng), te = ld_shared_s64(s_rng + 1);
                const Seg q = L.seg[cur.v];
                const bool complete = cur.start >= tb && cur.start + cur.nt <= te;
                const bool final = complete && cur.v < L.B && q.key0 == 0;
                const int half = wide ? set : 0;
                // this row's place: out, the arrays of whole segments, or a slot
                const int64_t orow =
                    (int64_t)(q.tok0 + half * NT + r / G) * a.Hq + cur.kvh * G + r % G;
                const int64_t hrow = (cur.v < L.B ? 0 : (int64_t)a.B * k * a.Hq) + orow;
                const int64_t srow =
                    (int64_t)(2 * blockIdx.x + (cur.start < tb ? 0 : 1)) * (2 * ROWS) + half * ROWS + r;
                float* po = complete ? prm.home_o + hrow * D : prm.slot_o + srow * D;
                float* pl = complete ? prm.home_lse + hrow : prm.slot_lse + srow;
                // 32 columns of the row, normalised
                auto store = [&](int c4, const float (&o)[32]) {
                    if (r >= rows) return;
                    if (final) {
                        uint4* dst = reinterpret_cast<uint4*>(
                            static_cast<__nv_bfloat16*>(a.out) + orow * D + c4 * 32);
#pragma unroll
                        for (int v4 = 0; v4 < 4; ++v4) {
                            uint4 w;
                            w.x = pack_bf16x2(o[8 * v4 + 0], o[8 * v4 + 1]);
                            w.y = pack_bf16x2(o[8 * v4 + 2], o[8 * v4 + 3]);
                            w.z = pack_bf16x2(o[8 * v4 + 4], o[8 * v4 + 5]);
                            w.w = pack_bf16x2(o[8 * v4 + 6], o[8 * v4 + 7]);
                            dst[v4] = w;
                        }
                    } else {
                        float4* dst = reinterpret_cast<float4*>(po + c4 * 32);
#pragma unroll
                        for (int v4 = 0; v4 < 8; ++v4)
                            dst[v4] = make_float4(o[4 * v4 + 0], o[4 * v4 + 1], o[4 * v4 + 2],
                                                  o[4 * v4 + 3]);
                    }
                };
                auto store_lse = [&](float x) {
                    if (r >= rows) return;
                    if (!final) *pl = x;
                    else if (a.lse) a.lse[orow] = x;
                };
                if (wide) {
                    // a set's rows are its own
                    if (ok && active) {
                        const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
                        for (int c4 = 0; c4 < D / 32; ++c4) {
                            uint32_t ov[32];
                            tmem_ld32(lane_base + o_mine + c4 * 32, ov);
                            tmem_wait_ld();
                            float o[32];
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(ov[e]) * inv;
                            store(c4, o);
                        }
                        store_lse(l > 0.f ? (m_ref + log2f(l)) * kLn2 : -INFINITY);
                    }
                    tc_fence_before();
                } else {
                    // merge the two sets' (max, sum, O); each writes half of the columns
                    s_stat_m[set * ROWS + r] = has ? m_ref : -INFINITY;
                    s_stat_l[set * ROWS + r] = has ? l : 0.f;
                    tc_fence_before();
                    named_bar_sync(2 + quad, 64);  // the two sets' warps of this quadrant
                    tc_fence_after();
                    const float mo = s_stat_m[(1 - set) * ROWS + r];
                    const float lo = s_stat_l[(1 - set) * ROWS + r];
                    const float mm = has ? m_ref : -INFINITY;
                    const float mt = fmaxf(mm, mo);
                    const float w_mine = mm == -INFINITY ? 0.f : fast_exp2(mm - mt);
                    const float w_other = mo == -INFINITY ? 0.f : fast_exp2(mo - mt);
                    const float lt = w_mine * (has ? l : 0.f) + w_other * lo;
                    if (ok && active) {
                        const float inv_l = lt > 0.f ? 1.f / lt : 0.f;
                        const float wm = w_mine * inv_l, wo = w_other * inv_l;
#pragma unroll
                        for (int c4 = set * 2; c4 < set * 2 + 2; ++c4) {
                            uint32_t ov[32], ow[32];
                            tmem_ld32(lane_base + o_mine + c4 * 32, ov);
                            tmem_ld32(lane_base + o_other + c4 * 32, ow);
                            tmem_wait_ld();
                            float o[32];
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                // a set without a tile of this piece holds stale O: weight 0
                                const float a0 = wm > 0.f ? __uint_as_float(ov[e]) * wm : 0.f;
                                const float a1 = wo > 0.f ? __uint_as_float(ow[e]) * wo : 0.f;
                                o[e] = a0 + a1;
                            }
                            store(c4, o);
                        }
                        if (set == 0)
                            store_lse(lt > 0.f ? (mt + log2f(lt)) * kLn2 : -INFINITY);
                    }
                    // both sets have read both O: the next piece's P V may overwrite them
                    tc_fence_before();
                    named_bar_sync(2 + quad, 64);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[Smem::B_EPI]);
            }
            if (it + 1 < n_tiles) cur.next(L);
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 4) tmem_dealloc(tmem, TMEM_COLS);
}

// ------------------------------------------------------------------ the pieces' sum

constexpr int kJoinWarps = 8;

// A segment's pieces: the rows of one CTA (whole: the array of its kind), or
// of CTAs c0 .. c1, those with an empty range left out.
struct Pieces {
    int c0, c1;
};

__device__ __forceinline__ int cta_of(const int64_t* t_begin, int C, int64_t t) {
    // the last CTA whose range begins at or before t
    const int lane = threadIdx.x & 31;
    int n = 0;
    for (int c = lane; c < C; c += 32) n += t_begin[c] <= t;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    return n - 1;
}

// A warp per query row.
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const Params prm, int C) {
    grid_dep_launch_dependents();
    grid_dep_wait();
    const AttnArgs& a = prm.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = a.Hq / a.Hkv, NT = ROWS / G, b = blockIdx.x / a.Hkv, kvh = blockIdx.x % a.Hkv;
    const int row = blockIdx.y * kJoinWarps + warp;
    if (row >= a.k * G) return;
    const int64_t rows = (int64_t)a.B * a.k * a.Hq;
    const int token = b * a.k + row / G;
    const int64_t orow = (int64_t)token * a.Hq + kvh * G + row % G;
    const int2 blk = prm.seq_block[b];
    Pieces pc[2];
    int64_t seg0[2] = {0, 0};
    int in_slot[2] = {row, 0};
    int count[2] = {0, 0};
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        int v = b;
        if (which == 1) {
            if (blk.x < 0) continue;
            const int dt = token - blk.y, off = dt % (2 * NT);
            v = blk.x + dt / (2 * NT);
            in_slot[1] = off / NT * ROWS + off % NT * G + row % G;
        }
        const int p0 = prm.tile_pre[v], nt = prm.tile_pre[v + 1] - p0;
        seg0[which] = (int64_t)p0 * a.Hkv + (int64_t)kvh * nt;
        pc[which].c0 = cta_of(prm.t_begin, C, seg0[which]);
        pc[which].c1 = cta_of(prm.t_begin, C, seg0[which] + nt - 1);
        count[which] = pc[which].c1 - pc[which].c0 + 1;
    }
    if (blk.x < 0 && count[0] == 1) return;  // written already
    // piece i: its row among the slots, or past them among the whole rows; -1 for none
    const int64_t slots = (int64_t)2 * C * 2 * ROWS;
    auto place = [&](int i) -> int64_t {
        const int w = i >= count[0];
        if (w) i -= count[0];
        if (count[w] == 1) return slots + w * rows + orow;
        const int c = pc[w].c0 + i;
        if (prm.t_begin[c] == prm.t_begin[c + 1]) return -1;
        return (int64_t)(2 * c + (seg0[w] < prm.t_begin[c] ? 0 : 1)) * (2 * ROWS) + in_slot[w];
    };
    auto lse_at = [&](int64_t p) {
        return p < 0 ? -INFINITY : p < slots ? __ldg(prm.slot_lse + p) : __ldg(prm.home_lse + (p - slots));
    };
    const int n = count[0] + count[1];
    float m = -INFINITY;
    for (int i = lane; i < n; i += 32) m = fmaxf(m, lse_at(place(i)));
    m = warp_max(m);
    float sum = 0.f;
    for (int i = lane; i < n; i += 32) {
        const float x = lse_at(place(i));
        if (x != -INFINITY) sum += expf(x - m);
    }
    sum = warp_sum(sum);
    const float lse = sum > 0.f ? m + logf(sum) : -INFINITY;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < n; i0 += 4) {
        float w[4];
        float4 x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t p = i0 + u < n ? place(i0 + u) : -1;
            const float z = lse_at(p);
            w[u] = z == -INFINITY ? 0.f : expf(z - lse);
            if (w[u] > 0.f)
                x[u] = __ldg(reinterpret_cast<const float4*>(
                                 p < slots ? prm.slot_o + p * D : prm.home_o + (p - slots) * D) + lane);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (w[u] > 0.f) {
                acc.x = fmaf(w[u], x[u].x, acc.x);
                acc.y = fmaf(w[u], x[u].y, acc.y);
                acc.z = fmaf(w[u], x[u].z, acc.z);
                acc.w = fmaf(w[u], x[u].w, acc.w);
            }
    }
    uint2 o;
    o.x = pack_bf16x2(acc.x, acc.y);
    o.y = pack_bf16x2(acc.z, acc.w);
    reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + orow * D)[lane] = o;
    if (lane == 0 && a.lse) a.lse[orow] = lse;
}

template <int KV>
cudaError_t launch_typed(const CUtensorMap& own_map, const CUtensorMap& block_map,
                         const CUtensorMap& kmap, const CUtensorMap& vmap, const Params& prm,
                         int num_ctas, cudaStream_t stream) {
    auto kern = attn_shared_kernel<KV>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)SMEM_BYTES);
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, dim3(num_ctas), dim3(threads<KV>()), SMEM_BYTES, stream, own_map,
                            block_map, kmap, vmap, prm);
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
    if (a.B + tokens / (2 * NT) + groups > MAX_SEGS) return false;
    // tile and cost counts are 32-bit
    const int64_t tiles = ((int64_t)a.max_pages * a.P + TN - 1) / TN + 1;
    return tiles < (1LL << 31) / ((kWideCost + 1) * MAX_SEGS) &&
           (int64_t)a.num_pages * a.Hkv * a.P < (1LL << 31);
}

size_t shared_workspace_bytes(const AttnArgs& a, int num_ctas) {
    const size_t rows = (size_t)a.B * a.k * a.Hq, slots = (size_t)2 * num_ctas * 2 * ROWS;
    return (2 * rows + slots) * (D + 1) * sizeof(float) + ((size_t)num_ctas + 1) * 8 +
           (size_t)(MAX_SEGS + 4) * 4 + (size_t)a.B * 8 + 64;
}

cudaError_t launch_attn_shared(const AttnArgs& a, const int32_t* group_starts,
                               const int32_t* shared_lens, int groups, int num_ctas, void* workspace,
                               cudaStream_t stream) {
    EncodeTiledFn encode = get_encode_fn();
    if (!encode) return cudaErrorNotSupported;
    const int G = a.Hq / a.Hkv;
    CUtensorMap qmap[2], kmap, vmap;
    for (int t = 0; t < 2; ++t) {
        cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.Hq, (cuuint64_t)a.B * a.k};
        cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)a.Hq * D * 2};
        cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)(t ? ROWS / G : a.k)};
        cuuint32_t es[3] = {1, 1, 1};
        if (encode(&qmap[t], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(a.q), dims,
                   strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    // K / V rows as in the 128-key kernel: bf16 as [groups of g rows] x [2 halves]
    // x [g rows] x [64 columns], g = 8 (K) or 16 (V); codes row by row
    const cuuint64_t rows = (cuuint64_t)a.num_pages * a.Hkv * a.P;
    const cuuint32_t ch = (cuuint32_t)(a.P < TN ? a.P : TN);
    const bool codes = a.kv_dtype != SPEC_DTYPE_BF16;
    for (int t = 0; t < 2; ++t) {
        void* cache = const_cast<void*>(t == 0 ? a.k_cache : a.v_cache);
        CUresult res;
        if (codes) {
            cuuint64_t dims[2] = {(cuuint64_t)D, rows};
            cuuint64_t strides[1] = {(cuuint64_t)D};
            cuuint32_t box[2] = {(cuuint32_t)D, ch};
            cuuint32_t es[2] = {1, 1};
            res = encode(t == 0 ? &kmap : &vmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, cache, dims,
                         strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        } else {
            const cuuint32_t g = t == 0 ? 8 : 16;
            cuuint64_t dims[4] = {64, g, 2, rows / g};
            cuuint64_t strides[3] = {(cuuint64_t)D * 2, 128, (cuuint64_t)g * D * 2};
            cuuint32_t box[4] = {64, g, 2, ch / g};
            cuuint32_t es[4] = {1, 1, 1, 1};
            res = encode(t == 0 ? &kmap : &vmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, cache, dims,
                         strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        }
        if (res != CUDA_SUCCESS) return cudaErrorInvalidValue;
    }
    Params prm;
    prm.a = a;
    prm.group_starts = group_starts;
    prm.shared_lens = shared_lens;
    prm.groups = groups;
    const size_t nrows = (size_t)a.B * a.k * a.Hq, slots = (size_t)2 * num_ctas * 2 * ROWS;
    prm.slot_o = static_cast<float*>(workspace);
    prm.home_o = prm.slot_o + slots * D;
    prm.slot_lse = prm.home_o + 2 * nrows * D;
    prm.home_lse = prm.slot_lse + slots;
    // (the fp32 arrays together hold an even number of words)
    prm.t_begin = reinterpret_cast<int64_t*>(prm.home_lse + 2 * nrows);
    prm.seq_block = reinterpret_cast<int2*>(prm.t_begin + num_ctas + 1);
    prm.tile_pre = reinterpret_cast<int*>(prm.seq_block + a.B);
    const cudaError_t e =
        a.kv_dtype == SPEC_DTYPE_I8
            ? launch_typed<KV_I8>(qmap[0], qmap[1], kmap, vmap, prm, num_ctas, stream)
        : a.kv_dtype == SPEC_DTYPE_E4M3
            ? launch_typed<KV_E4M3>(qmap[0], qmap[1], kmap, vmap, prm, num_ctas, stream)
            : launch_typed<KV_BF16>(qmap[0], qmap[1], kmap, vmap, prm, num_ctas, stream);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(a.B * a.Hkv), (unsigned)((a.k * G + kJoinWarps - 1) / kJoinWarps));
    return launch_dependent(join_kernel, grid, dim3(kJoinWarps * 32), 0, stream, prm, num_ctas);
}

}  // namespace specv
