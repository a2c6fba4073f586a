// Verification attention over an e4m3 paged cache (one fp32 scale per page and
// kv-head) on the tcgen05 tensor cores, the codes fed to them as they are
// stored.  bf16 q, head_dim 128, up to 128 query rows per kv-head; causal
// chain, token tree, sliding window with sinks.
//
// Mathematics.  Key j of page g has K_j = sk_g c_j, V_j = sv_g d_j with e4m3
// codes c, d.  For a query row q (times the softmax scale):
//   s_j = sk_g <q, c_j>,   out = sum_j p_j sv_g d_j / sum_j p_j,  p_j = 2^(s_j - m)
// in log2 units, for any reference m.  Both products take 8-bit operands:
//  * q = 2^e (hi + lo): hi is q 2^-e rounded to e4m3 and lo the rest rounded
//    to e4m3, with 2^e chosen per row so that the largest element lies in
//    [128, 256).  A bf16 has 8 significant bits and each part holds 4, so
//    hi + lo is q itself down to 2^-10 of the row's largest element, and off
//    by at most 2^-18 of that element below.  S = hi C^T + lo C^T: two MMAs of
//    K = 32 into one fp32 accumulator, as many as a bf16 product would take.
//  * P: in each row and block of 32 keys, w_j = p_j sv_g is scaled by the power
//    of two that puts the block's largest in [128, 256) and split into hi + lo
//    in the same way (8 significant bits, as a bf16 P would have).  The
//    block-scaled MMA applies the power back per row and block, so keys far
//    below the row's maximum keep their precision: a first key that holds
//    most of the weight does not flush the thousands of light ones behind it,
//    which a P in e4m3 under one scale per row would.  sv_g enters as
//    log2(sv_g) in the exponent; the row sum takes each 16-key group's sum of w
//    back by 1 / sv_g, in fp32.  And since the block scales carry the distance
//    to the reference, m need not be the running maximum: it is a whole number
//    near the first tile's largest, moved only when a tile exceeds it by 2^40
//    (the blocks' maxima come with the load of their scores).
//
// What bounds it: the bytes of the cache (32 KB per 128 keys and kv-head), with
// the tensor pipe close behind: 8 + 8 MMAs of M128 N128 K32 per 128-key tile
// issue in ~1030 cycles (measured, one CTA), the HBM share of an SM brings a
// tile in ~1400.  So nothing may stand between the copy and the MMAs: no
// widening pass, and the softmax below a tile's time on every SMSP.
//
// Measured (one call among others, combine included; the bytes' floor at 6768
// GB/s): 32 sequences of 1 to 8K keys, 32/8 heads, 4 drafts 63 to 65 us (4.85 to
// 4.69 TB/s, floor 45.1); 32 x 2048 keys, 64/8 heads, 8 drafts 45 us (21.2); 4 x 32K
// keys, 28/4 heads, 16-node trees 51 us (20.0).  A tile takes ~1500, ~1700 and ~2600
// cycles there (16, 64 and 112 rows): the softmax of the rows is what is left
// above the HBM share, of which half is its arithmetic (the exponentials and
// the conversions to e4m3 share one pipe, 4 cycles per warp instruction each:
// 16 per pair of weights) and the rest its waits, loads and hand-overs.
// The combine costs 5 us of a call, a piece's end ~1.
//
// Layout.  Persistent grid, the tile list split as in the 128-key bf16 kernel
// (TileSplit, partials merged by the combine kernel).
//  * TMEM: three S buffers [0,384), one O [384,512).  P goes over S columns
//    [64,128) of its tile (p_col), the scale bytes of P and of V (all one) over
//    [0,4) / [4,8).  Three tiles are in flight: the chain of one tile (Q K^T,
//    softmax, P V, ~3100 cycles) is longer than two tiles' share of HBM.  That
//    both softmax sets add into one O is what frees the third buffer.
//  * Warps: 0-3 and 8-11 two softmax sets; 4 Q K^T issue; 5 and 6 TMA of K and of
//    V; 7 P V issue; 12-14 turn the q rows of the next piece into hi / lo; 7 and
//    12-14, one per TMEM lane quadrant, write a finished piece out while the
//    softmax is at the next one (by the softmax warps themselves a piece's end
//    cost 3.7 us, and the 16-row step above 3.9 us more); 15 looks up pages and
//    their scales.  16 warps share the block's 64K registers (setmaxnreg: 160,
//    96, 160, 96).
//  * Softmax: both sets take every tile, half of a lane's keys each, and meet once
//    per tile to agree on the reference.  Alternate tiles instead (the
//    reference handed on from set to set) left each tile twice as long in the
//    softmax, and three tiles in flight did not cover that: 49.4, 53.0 us at 64
//    and 112 rows against 45.2, 50.4 (at 16 rows, where a set's work per tile
//    is small against its waits, 60.8 against 63.3).
//  * Rows: R = k * G query rows are the M side of one MMA.  R <= 64 (REP 2) and
//    R <= 32 (REP 4): the rows stand REP times and copy c takes the 32-key
//    blocks of its own, with P zero elsewhere, so that every softmax thread
//    has work and a tile costs it 1 / REP of the exponentials; the copies'
//    (max, sum, O) merge through shared memory once per piece.
//  * Every wait is bounded (role_wait); after a timeout every role skips its
//    work, drains its copies and tensor-core operations and returns.
#include <cuda.h>
#include <math.h>

#include "common.cuh"

namespace specv {
namespace {

constexpr int D = 128;
constexpr int TN = 128;                // keys per tile
constexpr int ROWS = 128;              // MMA M
constexpr int THREADS = 16 * 32;
constexpr int Q_PART = ROWS * D;       // 16 KB: hi or lo of one piece's rows
constexpr int SLOT_BYTES = TN * D;     // 16 KB: one tile of K or of V
constexpr int KSLOTS = 5, VSLOTS = 4;  // a K slot is refilled one P V earlier than V's
constexpr int MAX_CHUNKS = TN / 16;    // page chunks per tile
// The page warp takes two tiles at a time (16 lanes each): block-table entries
// PAGE_PAIRS + 2 pairs ahead, scales PAGE_PAIRS ahead; the copies' first rows go
// to the producers with the latter.
constexpr int PAGE_PAIRS = 2;
constexpr int RAW_STAGES = 4;          // pairs of tiles
constexpr int ROW_STAGES = 16;         // pairs of tiles
constexpr int SCALE_STAGES = 16;       // tiles
// row exponents: the q rows of piece j are converted after piece j - 2 is written
// out, so no stage before j - 1's is still to be read
constexpr int EXP_STAGES = 4;
constexpr int MAX_BATCH = 1024;
constexpr uint32_t TMEM_COLS = 512;
constexpr int NS = 3;                   // S buffers
constexpr uint32_t TM_O = NS * TN;
constexpr uint32_t SF_P = 0, SF_V = 4;  // columns of the scale bytes inside an S buffer
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// the reference moves when a block's largest w exceeds it by more than this
// (log2 units): the block scales carry any distance below, fp32 sums this one
constexpr float kMoveThreshold = 40.f;
// tiles charged per segment in the split (1, 2, 3 and 4: 63.9, 63.3, 64.1, 64.5 us
// on the ragged 16-row step, 44.8, 44.8, 44.5, 45.3 at 64 rows, 37.8, 37.7, 37.3,
// 37.3 with a 1024-key window)
constexpr int kSplitAlpha = 3;

// Tiles' time that cutting a segment costs (whole_segments).  Whole against cut, us:
// 8 segments of 2, 4, 6, 8, 12 tiles 7.5 / 10.9, 8.9 / 11.7, 10.3 / 12.6, 11.8 / 13.3,
// 14.6 / 14.0; 64 segments 8.4 / 12.7, 9.8 / 14.1, 11.3 / 14.8, 12.8 / 15.5, 15.8 / 17.5;
// 152 segments of 12 18.3 / 19.8
constexpr int kCutTiles = 8;
// With more segments than CTAs, ranges that end with segments against cut ones, us:
// 192 segments of 3, 4, 6, 10 tiles 16.1 / 17.5, 17.8 / 18.3, 21.1 / 21.1, 27.2 / 25.3; 512
// of 3, 6, 7, 10 25.7 / 27.9, 35.3 / 36.8, 39.4 / 40.1, 47.8 / 46.9; 1280 of 4, 7, 11, 15,
// 19 56.2 / 60.4, 75.8 / 83.3, 103.5 / 109.3, 126.5 / 127.8, 160.5 / 157.2
constexpr int kRoundedBase = 3, kRoundedMore = 5;

struct Smem {
    static constexpr int Q = 0;                          // 2 buffers of [hi | lo]
    static constexpr int KS = Q + 4 * Q_PART;
    static constexpr int VS = KS + KSLOTS * SLOT_BYTES;
    static constexpr int SFP = VS + VSLOTS * SLOT_BYTES;   // scale bytes of P, per S buffer
    static constexpr int SFV = SFP + NS * 512;             // scale bytes of V: all 1.0
    static constexpr int BARS = SFV + 512;
    static constexpr int B_KFULL = 0, B_KEMPTY = B_KFULL + KSLOTS,
                         B_VFULL = B_KEMPTY + KSLOTS, B_VEMPTY = B_VFULL + VSLOTS,
                         B_QFULL = B_VEMPTY + VSLOTS, B_SFULL = B_QFULL + 2,
                         B_PREADY = B_SFULL + NS, B_SFREE = B_PREADY + NS, B_STAT = B_SFREE + NS,
                         B_STFREE = B_STAT + 2, B_DRAIN = B_STFREE + 2,
                         B_EXP = B_DRAIN + 2, B_SCALE = B_EXP + EXP_STAGES,
                         B_SCFREE = B_SCALE + SCALE_STAGES / 2,
                         B_ROWS = B_SCFREE + SCALE_STAGES / 2,
                         NUM_BARS = B_ROWS + ROW_STAGES;
    // tmem base, abort flag, the CTA's tile range at +16
    static constexpr int MISC = BARS + (NUM_BARS + 1) / 2 * 16;
    static constexpr int FIRST = MISC + 32;           // the CTA's first cursor
    static constexpr int MOST = FIRST + 48;           // largest w of [tile & 1][set][lane]
    // page warp: [stage][2 tiles][8] block-table entries, [stage][2 tiles][k, v][8]
    // scales, and for the producers [stage][2 tiles][8] cache rows (-1: no copy)
    static constexpr int PIDS = MOST + 2 * 2 * ROWS * 4;
    static constexpr int TROWS = PIDS + RAW_STAGES * 2 * MAX_CHUNKS * 4;
    static constexpr int RAW = TROWS + ROW_STAGES * 2 * MAX_CHUNKS * 4;
    static constexpr int EXPS = RAW + RAW_STAGES * 4 * MAX_CHUNKS * 4;  // [stage][row] int8
    static constexpr int SCALE = EXPS + EXP_STAGES * ROWS;  // [stage][8] {sk, log2 sv, 1/sv, on}
    static constexpr int CTX = SCALE + SCALE_STAGES * MAX_CHUNKS * 16;
    static constexpr int PRE = CTX + MAX_BATCH * 4;
    // (m, l) of [piece & 1][set][lane]: over the tile prefix, which only the start reads
    static constexpr int STAT = PRE;
    static constexpr int END = PRE + (MAX_BATCH + 1) * 4;
    static_assert(2 * 2 * ROWS * 8 <= END - PRE, "the statistics' place");
};
static_assert(Smem::MISC % 16 == 0 && Smem::SCALE % 16 == 0 && Smem::SFP % 16 == 0 &&
              Smem::STAT % 8 == 0, "alignment");
constexpr size_t SMEM_BYTES = Smem::END + 1024;  // + alignment slack
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");

struct F8Params {
    AttnArgs a;
    float* part_o;    // [2*C][ROWS][D]
    float* part_lse;  // [2*C][ROWS]
    int4* seg_rec;    // [C][2]
    int* seg_pre;     // [B+1]
    int whole;        // whole_segments: kCut, or how none is cut
};

// warp_wait in fewer instructions.  Roles of different code share each SM's
// instruction caches, so what the hot loops hold counts: the same softmax beside
// 8 KB more code in other roles ran up to 15 % slower.
__device__ __forceinline__ bool role_wait(uint64_t* bar, uint32_t parity,
                                          volatile int* abort_flag, int* dev_err) {
    constexpr uint32_t kAll = 0xffffffffu;
    if (__all_sync(kAll, mbar_try_wait(bar, parity))) return true;
    const uint64_t t0 = globaltimer_ns();
    bool late;
    do {
        if (__all_sync(kAll, mbar_try_wait(bar, parity))) return true;
        late = globaltimer_ns() - t0 > kWaitLimitNs;
    } while (!__any_sync(kAll, late || *abort_flag != 0));
    if (late) {
        *abort_flag = 1;
        raise_device_error(dev_err, SPEC_DEVERR_TIMEOUT);
    }
    __syncwarp();
    return false;
}

// Keys [k0, k0 + 32) that a query row sees: the context (with a window: the
// sinks and the keys from `low` on), then the drafts of the row's bits, up to
// key `end`.
template <bool WIN>
__device__ __forceinline__ uint32_t visible32(int k0, int end, int ctx, uint64_t mrow, int low,
                                              int sinks) {
    auto below = [](int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1; };
    const int nctx = ctx - k0;
    uint32_t c = below(nctx);
    if (WIN) c &= below(sinks - k0) | ~below(low - k0);
    const uint32_t d = nctx >= 32    ? 0u
                       : nctx >= 0   ? (uint32_t)(mrow << nctx)
                       : nctx > -64  ? (uint32_t)(mrow >> -nctx)
                                     : 0u;
    return (c | d) & below(end - k0);
}

// Two values as e4m3 hi + lo (8 significant bits together): the rest after hi is
// exact in fp16, which holds the values with 11 bits.
__device__ __forceinline__ void split_e4m3x2(float a, float b, uint16_t& hi, uint16_t& lo) {
    uint32_t h, back, rest;
    h = pack_f16x2(a, b);
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(hi) : "r"(h));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(hi));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(rest) : "r"(h), "r"(back));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(lo) : "r"(rest));
}

// w = 2^(raw mult + bias) of a 16-key group as hi / lo words (4 codes each);
// returns the sum of w.
__device__ __forceinline__ float group_weights(const uint32_t (&r)[16], float mult, float bias,
                                               bool on, uint32_t* hi, uint32_t* lo) {
    const uint64_t mm = f2(mult, mult), bb = f2(bias, bias);
    uint64_t sum[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
    for (int c = 0; c < 16; c += 4) {
        uint16_t h[2], l[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float x0, x1;
            f2_split(f2_fma(f2(__uint_as_float(r[c + 2 * e]), __uint_as_float(r[c + 2 * e + 1])),
                            mm, bb),
                     x0, x1);
            x0 = fast_exp2(x0);
            x1 = fast_exp2(x1);
            sum[e] = f2_add(sum[e], f2(x0, x1));
            split_e4m3x2(x0, x1, h[e], l[e]);
        }
        hi[c / 4] = (uint32_t)h[0] | ((uint32_t)h[1] << 16);
        lo[c / 4] = (uint32_t)l[0] | ((uint32_t)l[1] << 16);
    }
    if (!on) {  // a page of zero scale: its keys count, its values do not
#pragma unroll
        for (int c = 0; c < 4; ++c) hi[c] = lo[c] = 0;
    }
    float a0, a1, b0, b1;
    f2_split(sum[0], a0, a1);
    f2_split(sum[1], b0, b1);
    return (a0 + b0) + (a1 + b1);
}

// 2^-d for a whole d >= 0 (0 from 2^-127 on).
__device__ __forceinline__ float pow2_neg(int d) {
    return d > 126 ? 0.f : __uint_as_float((uint32_t)(127 - d) << 23);
}

// P of 32-key block b (16 columns: hi, lo) inside the S buffer: over the raw
// scores of a block that comes before it (blocks are taken from 3 down to 0).
__device__ __forceinline__ uint32_t p_col(int b) { return 64 + (b >> 1) * 32 + (b & 1 ? 0 : 16); }

template <int REP, bool WIN>
__global__ void __launch_bounds__(THREADS, 1)
attn_f8_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
               const F8Params prm) {
    using Cursor = SegCursor<TN, WIN>;
    static_assert(sizeof(Cursor) <= 48, "the first cursor's place");
    constexpr int NBLK = REP == 1 ? 2 : 1;   // 32-key blocks of a softmax thread
    constexpr int GROUPS = REP == 4 ? 1 : 2;  // 16-key groups of a block that it takes
    constexpr int COPY = ROWS / REP;     // lanes of one copy of the rows
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const AttnArgs& a = prm.a;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Smem::BARS);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + Smem::MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + Smem::MISC + 4);
    int64_t* s_rng = reinterpret_cast<int64_t*>(sm + Smem::MISC + 16);
    int* s_ctx = reinterpret_cast<int*>(sm + Smem::CTX);
    int* s_pre = reinterpret_cast<int*>(sm + Smem::PRE);
    Cursor* s_first = reinterpret_cast<Cursor*>(sm + Smem::FIRST);  // of tile t_begin
    float4* s_scale = reinterpret_cast<float4*>(sm + Smem::SCALE);
    int8_t* s_exp = reinterpret_cast<int8_t*>(sm + Smem::EXPS);
    float2* s_stat = reinterpret_cast<float2*>(sm + Smem::STAT);

    // (shuffled: the roles' branches and operands stay in uniform registers)
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int B = a.B, k = a.k, Hkv = a.Hkv, G = a.Hq / a.Hkv, R = k * G, P = a.P;
    const int CH = P < TN ? P : TN;      // keys per page chunk
    const int lgP = 31 - __clz(P), lgCH = 31 - __clz(CH);  // both powers of two

    if (tid == 0) {
        for (int s = 0; s < KSLOTS; ++s) {
            mbar_init(&bars[Smem::B_KFULL + s], 1);
            mbar_init(&bars[Smem::B_KEMPTY + s], 1);
        }
        for (int s = 0; s < VSLOTS; ++s) {
            mbar_init(&bars[Smem::B_VFULL + s], 1);
            mbar_init(&bars[Smem::B_VEMPTY + s], 1);
        }
        for (int s = 0; s < ROW_STAGES; ++s) mbar_init(&bars[Smem::B_ROWS + s], 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bars[Smem::B_QFULL + s], 3);   // the 3 converting warps
            mbar_init(&bars[Smem::B_STAT + s], 8);    // every softmax warp, at a piece's end
            mbar_init(&bars[Smem::B_STFREE + s], 4);  // the epilogue's warps
            mbar_init(&bars[Smem::B_DRAIN + s], 1);
        }
        for (int s = 0; s < NS; ++s) {
            mbar_init(&bars[Smem::B_SFULL + s], 1);
            mbar_init(&bars[Smem::B_PREADY + s], 8);  // every softmax warp
            mbar_init(&bars[Smem::B_SFREE + s], 1);
        }
        for (int s = 0; s < EXP_STAGES; ++s) mbar_init(&bars[Smem::B_EXP + s], 3);
        for (int s = 0; s < SCALE_STAGES / 2; ++s) {  // per pair of tiles
            mbar_init(&bars[Smem::B_SCALE + s], 1);
            mbar_init(&bars[Smem::B_SCFREE + s], 8);  // every softmax warp
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    {
        // q rows that no piece writes are zero at first; the scale bytes of V, and
        // of P blocks that no lane of a row writes, are 1.0.  (The epilogue's
        // scratch lies over the q rows, so from a CTA's third piece on rows >= R
        // hold any bytes.  A row of the MMAs reads no other, the softmax takes
        // such a lane's scores times 2^-126, and nothing of it is stored.)
        uint4* q4 = reinterpret_cast<uint4*>(sm + Smem::Q);
        for (int e = tid; e < 4 * Q_PART / 16; e += THREADS)
            if ((e % (Q_PART / 16)) / 8 % COPY >= R) q4[e] = make_uint4(0, 0, 0, 0);
        static_assert(NS * 128 + 128 <= THREADS && Smem::SFV == Smem::SFP + NS * 512, "one pass");
        if (tid < NS * 128 + 128) reinterpret_cast<uint32_t*>(sm + Smem::SFP)[tid] = 0x7f7f7f7fu;
        fence_proxy_async_smem();
    }
    // the grids before this one have finished with every buffer this call
    // touches (and with the tensor memory of this SM)
    grid_dep_launch_dependents();
    grid_dep_wait();
    if (warp == 4) {
        tmem_alloc(tmem_slot, TMEM_COLS);
        tmem_relinquish();
    }
    if (warp == 5) {
        const int per = (B + 31) / 32, lo = min(B, lane * per), hi = min(B, lo + per);
        int sum = 0;
        for (int b = lo; b < hi; ++b) {
            int c = a.ctx_lens[b];
            const int64_t cap = (int64_t)a.max_pages * P - k;
            if (c < 0 || (int64_t)c > cap) {
                raise_device_error(a.dev_err, SPEC_DEVERR_CTX);
                c = c < 0 ? 0 : (int)(cap < 0 ? 0 : cap);
            }
            s_ctx[b] = c;
            sum += Cursor::tiles(a, c);
        }
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        int run = incl - sum;
        for (int b = lo; b < hi; ++b) {
            s_pre[b] = run;
            run += Cursor::tiles(a, s_ctx[b]);
        }
        if (lane == 31) s_pre[B] = incl;
        __syncwarp();  // the prefix above, written by this warp's lanes
        if (lane < 2) {
            TileSplit split;
            split.init(s_pre, B, Hkv, a.split_alpha >= 0 ? a.split_alpha : kSplitAlpha, gridDim.x);
            const int c = blockIdx.x + lane;
            const int64_t t = prm.whole
                                  ? whole_begin<Cursor>(prm.whole, split, s_pre, s_ctx, a, c)
                                  : split.begin(c);
            s_rng[lane] = t;
            if (lane == 0 && t < (int64_t)s_pre[B] * Hkv) s_first->init(t, s_pre, s_ctx, a);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    const int64_t T = (int64_t)s_pre[B] * Hkv;
    const int64_t t_begin = ld_shared_s64(s_rng);
    const int n_tiles = (int)(ld_shared_s64(s_rng + 1) - t_begin);
    if (tid == 0) {
        // the segment holding tile t_begin and t_begin itself, for the combine
        int4 r0 = make_int4(0, 0, -1, 0);
        if (t_begin < T) r0 = make_int4(s_first->b, s_first->kvh, s_first->lt, s_first->nb);
        prm.seg_rec[2 * blockIdx.x] = r0;
        prm.seg_rec[2 * blockIdx.x + 1] =
            make_int4((int)(t_begin & 0xffffffff), (int)(t_begin >> 32), 0, 0);
    }
    if (blockIdx.x == 0 && warp < 4)  // (before the first statistics, barrier 1 between)
        for (int b = tid; b <= B; b += 128) prm.seg_pre[b] = s_pre[b];

    auto start_at = [&](Cursor& c) { c = *s_first; };
    // query row r of a (sequence, kv-head) in q and out, from its row 0 on: row
    // r % G of draft r / G (exact: r + 1/2 over G is 1 / 256 at least from a
    // whole number, and a division costs what a row's whole sum does)
    const float inv_g = 1.f / (float)G;
    auto row_at = [&](int r) { return (int)(((float)r + 0.5f) * inv_g) * (a.Hq - G) + r; };
    // the page chunk `l` of a tile holds a key that some query sees
    auto chunk_used = [&](const Cursor& c, int l) {
        const int k0 = c.key0() + (l << lgCH), end = s_ctx[c.b] + k;
        if ((l << lgCH) >= TN || k0 >= end) return false;
        return !WIN || k0 < a.sinks || k0 + CH > window_low(a, s_ctx[c.b]);
    };

    // ================= q rows to hi / lo =================
    // The q rows of piece j (cursor c), two rows per warp and step, from row
    // 2 w on: 16 lanes per row, 8 elements each, into buffer j & 1, the rows'
    // exponents into stage j % 4; a negative softmax scale is folded into q's
    // sign.  The first piece, which everything waits for, by the softmax warps
    // too; the others by warps 12-14.
    auto convert = [&](const Cursor& c, int j, int w, int step) {
        const int half = lane >> 4, c16 = lane & 15;
        const float sign = a.scale < 0.f ? -1.f : 1.f;
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) +
                                 ((int64_t)c.b * k * a.Hq + c.kvh * G) * D;
        uint8_t* buf = sm + Smem::Q + (j & 1) * 2 * Q_PART;
        auto q_chunk = [&](int r) {  // this lane's 16 bytes of row r
            uint4 v = make_uint4(0, 0, 0, 0);
            if (r < R)
                v = __ldg(reinterpret_cast<const uint4*>(q + (int64_t)row_at(r) * D) + c16);
            return v;
        };
        uint4 ahead = q_chunk(w * 2 + half);
#pragma unroll 1
        for (int r0 = w * 2; r0 < R; r0 += step) {
            const int r = r0 + half;
            const uint4 v = ahead;
            ahead = q_chunk(r + step);
            float x[8];
            const uint32_t pair[4] = {v.x, v.y, v.z, v.w};
            float top = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[2 * e] = __uint_as_float(pair[e] << 16);
                x[2 * e + 1] = __uint_as_float(pair[e] & 0xffff0000u);
                top = fmaxf(top, fmaxf(fabsf(x[2 * e]), fabsf(x[2 * e + 1])));
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1)
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            // 2^-ex takes the row's largest element into [128, 256)
            const int ex = max((int)(__float_as_uint(top) >> 23) - 127 - 7, -120);
            const float mul = sign * __uint_as_float((uint32_t)(127 - ex) << 23);
            uint32_t hw[2], lw[2];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint16_t h, l;
                split_e4m3x2(x[2 * e] * mul, x[2 * e + 1] * mul, h, l);
                if (e & 1) {
                    hw[e >> 1] |= (uint32_t)h << 16;
                    lw[e >> 1] |= (uint32_t)l << 16;
                } else {
                    hw[e >> 1] = h;
                    lw[e >> 1] = l;
                }
            }
            if (r < R) {
                if (c16 == 0) s_exp[(j % EXP_STAGES) * ROWS + r] = (int8_t)ex;
#pragma unroll
                for (int cp = 0; cp < REP; ++cp) {
                    const int row = r + cp * COPY;
                    const int off = row * D + (((c16 >> 1) ^ (row & 7)) << 4) + (c16 & 1) * 8;
                    *reinterpret_cast<uint2*>(buf + off) = make_uint2(hw[0], hw[1]);
                    *reinterpret_cast<uint2*>(buf + Q_PART + off) = make_uint2(lw[0], lw[1]);
                }
            }
        }
        fence_proxy_async_smem();  // generic-proxy writes -> tensor-core reads
    };

    if (warp & 4) {
    regs_dec<96>();
    if (warp == 5 || warp == 6) {
        // ================= TMA producers: warp 5 K, warp 6 V =================
        // Tile it goes to slot it % SLOTS of its ring; each page chunk (CH
        // keys of 128 bytes, swizzled by the copy) is one copy, its first row
        // of the cache from the page warp.  One warp's latency per iteration is
        // what a tile can cost here (the copies alone ~50 cycles each), so the
        // loop does no more.
        const bool is_v = warp == 6;
        const int* rows = reinterpret_cast<const int*>(sm + Smem::TROWS) + (lane & 7);
        const int slots = is_v ? VSLOTS : KSLOTS;
        uint64_t* full = &bars[is_v ? Smem::B_VFULL : Smem::B_KFULL];
        uint64_t* empty = &bars[is_v ? Smem::B_VEMPTY : Smem::B_KEMPTY];
        uint8_t* ring = sm + (is_v ? Smem::VS : Smem::KS) + ((lane << lgCH) * D);
        const CUtensorMap* map = is_v ? &vmap : &kmap;
        const uint64_t pol = l2_policy_evict_first();
        if (lane == 0) prefetch_tmap(map);
        int n_issued = 0, s = 0, round = 0;
        bool ok = true;
        for (int it = 0; it < n_tiles && ok; ++it) {
            const int p = it >> 1, stage = p % ROW_STAGES;
            if (!(it & 1))
                ok = role_wait(&bars[Smem::B_ROWS + stage], (p / ROW_STAGES) & 1, abort_flag,
                               a.dev_err);
            const int row = lane < MAX_CHUNKS ? rows[(2 * stage + (it & 1)) * MAX_CHUNKS] : -1;
            const int nck = __popc(__ballot_sync(0xffffffffu, row >= 0));
            if (ok && round > 0)
                ok = role_wait(&empty[s], (round - 1) & 1, abort_flag, a.dev_err);
            if (ok && lane == 0) mbar_arrive_expect_tx(&full[s], (uint32_t)((nck << lgCH) * D));
            __syncwarp();
            if (!ok) break;
            if (row >= 0) tma_load_2d(ring + s * SLOT_BYTES, map, &full[s], 0, row, pol);
            n_issued = it + 1;
            if (++s == slots) {
                s = 0;
                ++round;
            }
            __syncwarp();
        }
        if (!ok && lane == 0) {
            // the latest copy into each slot lands before the CTA exits
            for (int j = max(0, n_issued - slots); j < n_issued; ++j)
                mbar_drain(&full[j % slots], (j / slots) & 1);
        }
    } else if (warp == 4) {
        // ================= Q K^T issue =================
        if (n_tiles > 0) {
            Cursor cur;
            start_at(cur);
            int pc = -1;  // piece of the current tile
            bool ok = true;
            const uint64_t qdesc0 = umma_sdesc_sw128(smem_u32(sm + Smem::Q), 16, 1024);
            const uint64_t kdesc0 = umma_sdesc_sw128(smem_u32(sm + Smem::KS), 16, 1024);
            for (int it = 0; it < n_tiles && ok; ++it) {
                const bool first = (it == 0) || (cur.lt == 0);
                const int s = it % NS, slot = it % KSLOTS;
                if (first) {
                    ++pc;
                    ok = role_wait(&bars[Smem::B_QFULL + (pc & 1)], (pc >> 1) & 1, abort_flag,
                                   a.dev_err);
                    if (!ok) break;
                }
                // K of tile it landed; S buffer s free (P V of tile it - NS done)
                ok = role_wait(&bars[Smem::B_KFULL + slot], (it / KSLOTS) & 1, abort_flag,
                               a.dev_err);
                if (ok && it >= NS)
                    ok = role_wait(&bars[Smem::B_SFREE + s], (it / NS - 1) & 1, abort_flag,
                                   a.dev_err);
                if (!ok) break;
                tc_fence_after();
                const uint64_t qd = qdesc0 + ((uint32_t)((pc & 1) * 2 * Q_PART) >> 4);
                const uint64_t kd = kdesc0 + ((uint32_t)(slot * SLOT_BYTES) >> 4);
                if (elect_lane()) {
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)  // hi, then lo, in 32-byte steps
                        umma_f8_ss(tmem + s * TN, qd + (kk >> 2) * (Q_PART >> 4) + (kk & 3) * 2,
                                   kd + (kk & 3) * 2, umma_idesc_e4m3(ROWS, TN), kk ? 1u : 0u);
                }
                __syncwarp();
                umma_commit_w(&bars[Smem::B_SFULL + s]);
                umma_commit_w(&bars[Smem::B_KEMPTY + slot]);
                if (it + 1 < n_tiles) cur.next(s_ctx, a);
            }
            // every tensor-core op of this warp finishes before TMEM is released
            __syncwarp();
            umma_commit_w(&bars[Smem::B_DRAIN]);
            if (lane == 0) mbar_drain(&bars[Smem::B_DRAIN], 0);
            __syncwarp();
        }
    } else if (warp == 15) {
        // ================= pages: rows of the copies, scales =================
        // Two tiles per iteration, 16 lanes each (8 chunks of K, 8 of V).  Rows
        // of pair p to stage p % ROW_STAGES, {sk, log2 sv, 1 / sv, on} of tile
        // it to stage it % SCALE_STAGES once its softmax set has freed that;
        // by then the producers are past the rows ROW_STAGES pairs back.
        int* pids = reinterpret_cast<int*>(sm + Smem::PIDS);
        int* rows = reinterpret_cast<int*>(sm + Smem::TROWS);
        float* raw = reinterpret_cast<float*>(sm + Smem::RAW);
        const int half = lane >> 4, l = lane & 7;
        const bool is_v = lane & 8;
        const float* src = is_v ? a.v_page_scale : a.k_page_scale;
        const int pairs = (n_tiles + 1) / 2;
        Cursor c_pid, c_sc;  // of this half's tile, as the two loads advance
        int t_pid = half, t_sc = half;
        if (half < n_tiles) {
            start_at(c_pid);
            if (half) c_pid.next(s_ctx, a);
            c_sc = c_pid;
        }
        auto advance = [&](Cursor& c, int& t) {
            for (int e = 0; e < 2; ++e)
                if (++t < n_tiles) c.next(s_ctx, a);
        };
        auto fetch_pids = [&](int p) {  // pair p
            if (p >= pairs) return;
            if (t_pid < n_tiles && !is_v && chunk_used(c_pid, l))
                cp_async_4(&pids[((p % RAW_STAGES) * 2 + half) * MAX_CHUNKS + l],
                           &a.block_table[(int64_t)c_pid.b * a.max_pages +
                                          ((c_pid.key0() + (l << lgCH)) >> lgP)]);
            advance(c_pid, t_pid);
        };
        auto fetch_scales = [&](int p) {  // and the rows (entries of pair p landed)
            if (p >= pairs) return;
            int row = -1;
            if (t_sc < n_tiles) {
                float* dst = raw + (p % RAW_STAGES) * 32 + lane;
                if (chunk_used(c_sc, l)) {
                    int page = pids[((p % RAW_STAGES) * 2 + half) * MAX_CHUNKS + l];
                    if (page < 0 || page >= a.num_pages) {
                        raise_device_error(a.dev_err, SPEC_DEVERR_PAGE);
                        page = 0;
                    }
                    row = page * Hkv + c_sc.kvh;
                    cp_async_4(dst, src + row);
                    row = (row << lgP) + ((c_sc.key0() + (l << lgCH)) & (P - 1));
                } else {
                    *dst = 1.f;
                }
            }
            if (!is_v) rows[((p % ROW_STAGES) * 2 + half) * MAX_CHUNKS + l] = row;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[Smem::B_ROWS + p % ROW_STAGES]);
            advance(c_sc, t_sc);
        };
        // groups: the entries of pairs 0 and 1, then scales p with entries p + 2
        fetch_pids(0);
        fetch_pids(1);
        cp_async_commit();
        cp_async_wait<0>();
        __syncwarp();
        for (int p = 0; p < PAGE_PAIRS; ++p) {
            fetch_scales(p);
            fetch_pids(p + 2);
            cp_async_commit();
        }
        bool ok = true;
        for (int p = 0; p < pairs && ok; ++p) {
            cp_async_wait<PAGE_PAIRS - 1>();  // scales p, entries p + 2
            __syncwarp();
            fetch_scales(p + PAGE_PAIRS);
            fetch_pids(p + PAGE_PAIRS + 2);
            cp_async_commit();
            constexpr int PAIRS = SCALE_STAGES / 2;
            if (p >= PAIRS)
                ok = role_wait(&bars[Smem::B_SCFREE + p % PAIRS], (p / PAIRS - 1) & 1, abort_flag,
                               a.dev_err);
            if (!ok) break;
            const int t = 2 * p + half;
            if (!is_v && t < n_tiles) {
                const float* r = raw + (p % RAW_STAGES) * 32 + lane;
                const float sv = r[8];
                const bool on = sv > 1e-30f;
                s_scale[(t % SCALE_STAGES) * MAX_CHUNKS + l] =
                    make_float4(r[0], on ? __log2f(sv) : 0.f, on ? __fdividef(1.f, sv) : 1.f,
                                on ? 1.f : 0.f);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[Smem::B_SCALE + p % PAIRS]);
        }
        cp_async_wait<0>();
    } else {
        // ================= P V issue (warp 7) and epilogue (7, 12-14) =================
        // Piece by piece: warps 12-14 convert the q rows of piece j (the buffer
        // is the one that piece j - 2 was written out from) while warp 7 issues
        // the P V of piece j - 1, then the four, one per TMEM lane quadrant,
        // write piece j - 1 out; the softmax warps are at the next one by then.
        const bool pv = warp == 7;
        Cursor cur, prev;     // of pieces j and j - 1
        bool more = n_tiles > 0, ok = true;
        int it0 = 0;          // first tile of piece j - 1
        if (more) start_at(cur);
        for (int j = 0;; ++j) {
            if (more && !pv) {
                convert(cur, j, j > 0 ? warp - 12 : warp - 4, j > 0 ? 6 : 22);
                if (j == 0)
                    named_bar_sync(1, 11 * 32);
                else
                    __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bars[Smem::B_EXP + j % EXP_STAGES]);
                    mbar_arrive(&bars[Smem::B_QFULL + (j & 1)]);
                }
            }
            if (j > 0) {
                const int nt = min(prev.nb - prev.lt, n_tiles - it0);
                if (pv) {
                    // V of 32 keys: MN-major, 8-key groups 1 KB apart
                    const uint64_t vdesc0 =
                        umma_sdesc_sw128(smem_u32(sm + Smem::VS), 1024, 1024);
                    const uint64_t sfp0 = umma_sdesc_plain(smem_u32(sm + Smem::SFP), 128);
                    const uint64_t sfv = umma_sdesc_plain(smem_u32(sm + Smem::SFV), 128);
                    const int ctx = s_ctx[prev.b];
                    for (int it = it0; it < it0 + nt && ok; ++it, ++prev.lt) {
                        const int s = it % NS, slot = it % VSLOTS;
                        const int key0 = prev.key0();
                        const int nvalid = min(TN, ctx + k - key0), nkb = (nvalid + 31) / 32;
                        ok = role_wait(&bars[Smem::B_VFULL + slot], (it / VSLOTS) & 1, abort_flag,
                                       a.dev_err);
                        if (!ok) break;
                        // rows that no query sees and a P V reads: zero, so that
                        // 0 * (stale or a NaN code) never reaches O
                        auto clear = [&](int r0, int r1) {
                            uint4* v4 =
                                reinterpret_cast<uint4*>(sm + Smem::VS + slot * SLOT_BYTES);
                            for (int e = r0 * 8 + lane; e < r1 * 8; e += 32)
                                v4[e] = make_uint4(0, 0, 0, 0);
                        };
                        bool cleared = nvalid % 32 != 0;
                        if (cleared) clear(nvalid, nkb * 32);
                        if (WIN) {
                            const int low = window_low(a, ctx);
                            const int g0 = max(0, a.sinks >= low ? nvalid : a.sinks - key0);
                            const int g1 = min(nvalid, low - key0);
                            if (g0 < g1) {
                                clear(g0, g1);
                                cleared = true;
                            }
                        }
                        if (cleared) {
                            fence_proxy_async_smem();
                            __syncwarp();
                        }
                        ok = role_wait(&bars[Smem::B_PREADY + s], (it / NS) & 1, abort_flag,
                                       a.dev_err);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t vd = vdesc0 + ((uint32_t)(slot * SLOT_BYTES) >> 4);
                        const uint32_t sbuf = tmem + s * TN, od = tmem + TM_O;
                        tmem_cp_scales_w(sbuf + SF_P, sfp0 + ((uint32_t)(s * 512) >> 4));
                        tmem_cp_scales_w(sbuf + SF_V, sfv);
                        if (elect_lane()) {
#pragma unroll 1
                            for (int kb = 0; kb < nkb; ++kb) {
                                const uint64_t vk = vd + ((uint32_t)(kb * 4096) >> 4);
                                const uint32_t id = umma_idesc_mx_e4m3(ROWS, D, kb);
                                umma_mx_ts(od, sbuf + p_col(kb), vk, id, sbuf + SF_P, sbuf + SF_V,
                                           (it > it0 || kb > 0) ? 1u : 0u);
                                umma_mx_ts(od, sbuf + p_col(kb) + 8, vk, id, sbuf + SF_P,
                                           sbuf + SF_V, 1u);
                            }
                        }
                        __syncwarp();
                        umma_commit_w(&bars[Smem::B_VEMPTY + slot]);
                        umma_commit_w(&bars[Smem::B_SFREE + s]);
                    }
                }
                // ---- epilogue: both sets' row sums and the copies' (reference, O)
                // merge.  64 columns at a time: every lane's share to the piece's
                // q buffer (its Q K^T are done), 4-column groups swizzled by the
                // row; then 16 threads sum the copies of a row and write 128
                // contiguous bytes.  Once the second half is in shared memory
                // warp 7 goes on to the next piece's P V, which overwrites O.
                const int jp = (j - 1) & 1, end = it0 + nt - 1;
                if (ok)
                    ok = role_wait(&bars[Smem::B_STAT + jp], ((j - 1) >> 1) & 1, abort_flag,
                                   a.dev_err);
                if (ok)  // the piece's last P V is done
                    ok = role_wait(&bars[Smem::B_SFREE + end % NS], (end / NS) & 1, abort_flag,
                                   a.dev_err);
                tc_fence_after();
                const int64_t tb = ld_shared_s64(s_rng), te = ld_shared_s64(s_rng + 1);
                const bool complete = prev.seg_start >= tb && prev.seg_start + prev.nb <= te;
                const int slot = 2 * blockIdx.x + (prev.seg_start < tb ? 0 : 1);
                const int ln = (warp & 3) * 32 + lane, r = ln % COPY;
                const float2* stat = s_stat + jp * 2 * ROWS;
                float mt = -INFINITY, lt = 0.f;
#pragma unroll
                for (int c = 0; c < REP; ++c) mt = fmaxf(mt, stat[c * COPY + r].x);
                const float mt_use = mt == -INFINITY ? 0.f : mt;
#pragma unroll
                for (int c = 0; c < REP; ++c) {
                    const float2 x = stat[c * COPY + r];
                    lt += fast_exp2(x.x - mt_use) * (x.y + stat[ROWS + c * COPY + r].y);
                }
                // (a lane that saw no key has reference -inf: weight 0)
                const float wgt = lt > 0.f ? fast_exp2(stat[ln].x - mt_use) / lt : 0.f;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[Smem::B_STFREE + jp]);
                const int64_t row0 = (int64_t)prev.b * k * a.Hq + prev.kvh * G;
                if (ok && ln < R && ln < COPY) {
                    const float lse = lt > 0.f ? (mt + log2f(lt)) * kLn2 : -INFINITY;
                    if (!complete)
                        prm.part_lse[(int64_t)slot * ROWS + r] = lse;
                    else if (a.lse)
                        a.lse[row0 + row_at(r)] = lse;
                }
                float* red = reinterpret_cast<float*>(sm + Smem::Q + jp * 2 * Q_PART);
                const int t = (pv ? 96 : (warp - 12) * 32) + lane, cg = lane & 15;
                __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + row0 * D + cg * 4;
                float* part = prm.part_o + (int64_t)slot * ROWS * D + cg * 4;
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 64) {
                    if (ok && ((warp & 3) * 32) % COPY < R) {
                        float4* dst = reinterpret_cast<float4*>(red + ln * 64);
#pragma unroll 2
                        for (int h = 0; h < 4; ++h) {
                            uint32_t ov[16];
                            tmem_ld16(tmem + ((uint32_t)((warp & 3) * 32) << 16) + TM_O + c0 +
                                          16 * h,
                                      ov);
                            tmem_wait_ld();
#pragma unroll
                            for (int v4 = 0; v4 < 4; ++v4)
                                dst[(4 * h + v4) ^ (lane & 7)] =
                                    make_float4(__uint_as_float(ov[4 * v4]) * wgt,
                                                __uint_as_float(ov[4 * v4 + 1]) * wgt,
                                                __uint_as_float(ov[4 * v4 + 2]) * wgt,
                                                __uint_as_float(ov[4 * v4 + 3]) * wgt);
                        }
                    }
                    tc_fence_before();
                    named_bar_sync(2, 128);
                    tc_fence_after();
                    if (pv && c0) break;
#pragma unroll 2
                    for (int row = t >> 4; row < (ok ? R : 0); row += c0 ? 6 : 8) {
                        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                        for (int c = 0; c < REP; ++c) {
                            const float4 x = reinterpret_cast<const float4*>(
                                red + (c * COPY + row) * 64)[cg ^ (row & 7)];
                            acc.x += x.x;
                            acc.y += x.y;
                            acc.z += x.z;
                            acc.w += x.w;
                        }
                        if (complete)
                            *reinterpret_cast<uint2*>(out + (int64_t)row_at(row) * D + c0) =
                                make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
                        else
                            *reinterpret_cast<float4*>(part + row * D + c0) = acc;
                    }
                    // the shares are read: the second half's may follow, the next
                    // but one piece's q rows after those
                    if (c0)
                        named_bar_sync(4, 96);
                    else
                        named_bar_sync(3, 128);
                }
                it0 += nt;
            }
            if (!more) break;
            prev = cur;
            more = cur.seg_start + cur.nb < ld_shared_s64(s_rng + 1);
            if (more) cur.next_segment(s_ctx, a);
        }
        if (pv && n_tiles > 0) {
            __syncwarp();
            umma_commit_w(&bars[Smem::B_DRAIN + 1]);
            if (lane == 0) mbar_drain(&bars[Smem::B_DRAIN + 1], 0);
            __syncwarp();
        }
    }
    } else {
        if (n_tiles > 0) {
            Cursor first_piece;
            start_at(first_piece);
            convert(first_piece, 0, warp < 4 ? warp : warp - 4, 22);
            named_bar_sync(1, 11 * 32);
        }
        regs_inc<160>();
        // ================= softmax sets (0: warps 0-3; 1: 8-11) =================
        // Both take every tile, and of a lane's blocks half each: blocks set and
        // set + 2 (REP 1), block 2 copy + set (REP 2), 16 keys of block copy
        // (REP 4).  The two warps of a lane quadrant meet once per tile, where
        // they agree on the reference; every raw score that is not in registers by
        // then lies in columns [0, 64), and P goes to [64, 128).
        const int set = warp >= 8 ? 1 : 0;
        const int quad = warp & 3;            // TMEM lane quadrant
        const int ln = quad * 32 + lane;      // TMEM lane of this thread
        const int copy = ln / COPY, r = ln % COPY;
        const bool row_valid = r < R;
        const bool quad_active = (quad * 32) % COPY < R;
        const int i_row = row_valid ? r / G : k - 1;
        const int blk0 = REP == 1 ? set : REP == 2 ? 2 * copy + set : copy;
        const int col0 = REP == 4 ? 16 * set : 0;  // this thread's first key of a block
        const float sl2 = fabsf(a.scale) * kLog2e;
        const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
        float* s_most = reinterpret_cast<float*>(sm + Smem::MOST);
        float m = -INFINITY, l = 0.f;  // reference of the lane, and the row sum to it
        Cursor cur;
        if (n_tiles > 0) start_at(cur);
        bool ok = true;
        int it = 0, sb = 0, phase = 0;  // tile, its S buffer, that buffer's phase
        for (int pc = 0; it < n_tiles; ++pc) {
        // ---- a piece
        const int ctx = s_ctx[cur.b], it0 = it;
        const int it1 = min(n_tiles, it + cur.nb - cur.lt);
        m = -INFINITY;
        l = 0.f;
        const uint64_t bits = draft_bits(a, cur.b, i_row);
        const uint64_t mrow = WIN ? window_bits(a, bits, i_row, ctx) : bits;
        // first key of this row's window
        const int low = WIN ? window_low(a, ctx + draft_depth(bits)) : 0;
        if (ok)
            ok = role_wait(&bars[Smem::B_EXP + pc % EXP_STAGES], (pc / EXP_STAGES) & 1,
                           abort_flag, a.dev_err);
        // accumulator units to log2 units, before the page's scale
        const float qm =
            ok && row_valid ? ldexpf(sl2, (int)s_exp[(pc % EXP_STAGES) * ROWS + r]) : 0.f;
#pragma unroll 1
        for (; it < it1; ++it, ++cur.lt) {
            const int key0 = cur.key0();
            if (ok && !(it & 1))
                ok = role_wait(&bars[Smem::B_SCALE + (it % SCALE_STAGES) / 2],
                               (it / SCALE_STAGES) & 1, abort_flag, a.dev_err);
            if (ok) ok = role_wait(&bars[Smem::B_SFULL + sb], phase, abort_flag, a.dev_err);
            if (quad_active) {  // (after an abort: of no consequence, but the barrier is met)
                tc_fence_after();
                const uint32_t s_mine = lane_base + sb * TN;
                const float4* sc = s_scale + (it % SCALE_STAGES) * MAX_CHUNKS;
                // a tile's edge: invisible keys' scores become -inf where they are
                const bool full = key0 + TN <= ctx &&
                                  (!WIN || key0 >= low || key0 + TN <= a.sinks);
                if (__any_sync(0xffffffffu, !full)) {
#pragma unroll 1
                    for (int blk = blk0; blk < blk0 + 2 * NBLK; blk += 2) {
                        const uint32_t vis = visible32<WIN>(key0 + blk * 32, ctx + k, ctx, mrow,
                                                            low, a.sinks) >> col0;
#pragma unroll 1
                        for (int g = 0; g < GROUPS; ++g) {
                            uint32_t raw[16];
                            tmem_ld16(s_mine + blk * 32 + col0 + 16 * g, raw);
                            tmem_wait_ld();
#pragma unroll
                            for (int c = 0; c < 16; ++c)
                                if (!((vis >> (16 * g + c)) & 1u))
                                    raw[c] = __float_as_uint(-INFINITY);
                            tmem_st16(s_mine + blk * 32 + col0 + 16 * g, raw);
                        }
                    }
                    tmem_wait_st();
                }
                // scores of a block with the whole power of two of its largest w
                // (-inf: no visible key); mult is not 0, so that -inf stays -inf
                uint32_t raw[GROUPS][16];
                float4 s[GROUPS];
                auto load_block = [&](int blk) {
                    float x[GROUPS], top = -INFINITY;
#pragma unroll
                    for (int g = 0; g < GROUPS; ++g) {
                        tmem_ld16_max(s_mine + blk * 32 + col0 + 16 * g, raw[g], x[g]);
                        s[g] = sc[(blk * 32 + col0 + 16 * g) >> lgCH];
                        s[g].x = fmaxf(qm * s[g].x, 1.2e-38f);
                    }
                    tmem_wait_ld();
#pragma unroll
                    for (int g = 0; g < GROUPS; ++g) top = fmaxf(top, fmaf(x[g], s[g].x, s[g].y));
                    return floorf(top);
                };
                float most = -INFINITY;
                if (NBLK > 1) most = load_block(blk0);
                float top = load_block(blk0 + 2 * (NBLK - 1));
                most = fmaxf(most, top);
                // both warps' largest w; the reference follows when that exceeds it
                // by far (also -inf -> finite)
                float* mine = s_most + (it & 1) * 2 * ROWS + set * ROWS + ln;
                *mine = most;
                tc_fence_before();
                named_bar_sync(5 + quad, 64);
                tc_fence_after();
                most = fmaxf(most, mine[set ? -ROWS : ROWS]);
                if (REP == 4) top = most;  // one block, half of it each
                const bool move = most > m + kMoveThreshold;
                if (__any_sync(0xffffffffu, move)) {
                    const float alpha = !move             ? 1.f
                                        : m == -INFINITY ? 0.f
                                                          : pow2_neg((int)fminf(most - m, 255.f));
                    l *= alpha;
                    if (move) m = most;
                    if (it > it0) {
                        // O (all of the piece so far, once P V of the tile before
                        // is done) shrinks with it
                        if (ok)
                            ok = role_wait(&bars[Smem::B_SFREE + (it - 1) % NS],
                                           ((it - 1) / NS) & 1, abort_flag, a.dev_err);
                        tc_fence_after();
#pragma unroll 1
                        for (int c4 = set * 4; c4 < set * 4 + 4; ++c4) {
                            uint32_t ov[16];
                            tmem_ld16(lane_base + TM_O + c4 * 16, ov);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
                            tmem_st16(lane_base + TM_O + c4 * 16, ov);
                        }
                    }
                }
                uint8_t* sfp = sm + Smem::SFP + sb * 512 + lane * 16 + quad * 4;
#pragma unroll 1
                for (int blk = blk0 + 2 * (NBLK - 1); blk >= blk0; blk -= 2) {
                    uint32_t pw[GROUPS * 8];
                    if (NBLK > 1 && blk == blk0) top = load_block(blk);
                    const float n = fmaxf(top - m, -110.f);  // (NaN without a key: -110)
                    const uint32_t sf = (uint32_t)(120 + (int)n);  // byte of 2^(n - 7)
                    const float base = top == -INFINITY ? 0.f : 7.f - (m + n);
                    float w = 0.f;
#pragma unroll
                    for (int g = 0; g < GROUPS; ++g)
                        w += group_weights(raw[g], s[g].x, base + s[g].y, s[g].w != 0.f,
                                           pw + 4 * g, pw + 4 * (GROUPS + g)) *
                             s[g].z;
                    l += w * __uint_as_float(sf << 23);
                    if (REP < 4 || set == 0) sfp[blk] = (uint8_t)sf;
                    if constexpr (REP < 4) {
                        tmem_st16(s_mine + p_col(blk), pw);
                    } else {
                        tmem_st4(s_mine + p_col(blk) + 4 * set, pw);
                        tmem_st4(s_mine + p_col(blk) + 8 + 4 * set, pw + 4);
                    }
                }
                if (REP > 1) {  // the blocks of the other copies
                    const uint32_t zero[16] = {};
                    if (REP == 2) tmem_st16(s_mine + p_col(blk0 ^ 2), zero);
                    if (REP == 4)
#pragma unroll 1
                        for (int e = 1; e < 4; ++e)
                            tmem_st8(s_mine + p_col((copy + e) & 3) + 8 * set, zero);
                }
                fence_proxy_async_smem();
                tmem_wait_st();
            }
            // P of this tile stored (every warp arrives, active or not)
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bars[Smem::B_PREADY + sb]);
                if (it & 1) mbar_arrive(&bars[Smem::B_SCFREE + (it % SCALE_STAGES) / 2]);
            }
            if (++sb == NS) {
                sb = 0;
                phase ^= 1;
            }
        }
        // this set's reference and row sum to the epilogue (which has read
        // those of the piece before the last)
        if (ok && pc >= 2)
            ok = role_wait(&bars[Smem::B_STFREE + (pc & 1)], ((pc >> 1) - 1) & 1, abort_flag,
                           a.dev_err);
        s_stat[((pc & 1) * 2 + set) * ROWS + ln] = make_float2(m, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[Smem::B_STAT + (pc & 1)]);
        if (it < n_tiles) cur.next_segment(s_ctx, a);
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 4) tmem_dealloc(tmem, TMEM_COLS);
}

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

template <int REP, bool WIN>
cudaError_t launch_typed(const CUtensorMap& kmap, const CUtensorMap& vmap, const F8Params& prm,
                         int num_ctas, cudaStream_t stream) {
    auto kern = attn_f8_kernel<REP, WIN>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)SMEM_BYTES);
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, dim3(num_ctas), dim3(THREADS), SMEM_BYTES, stream, kmap, vmap,
                            prm);
}

}  // namespace

bool f8_supported(const AttnArgs& a) {
    const int G = a.Hq / a.Hkv;
    const bool pow2 = (a.P & (a.P - 1)) == 0;
    return a.q_dtype == SPEC_DTYPE_BF16 && a.kv_dtype == SPEC_DTYPE_E4M3 && a.D == D &&
           a.k * G <= ROWS && pow2 && a.P >= 16 && a.P <= 256 && a.B <= MAX_BATCH &&
           (int64_t)a.num_pages * a.Hkv * a.P < (1LL << 31);
}

cudaError_t launch_attn_f8(const AttnArgs& a, int num_ctas, void* workspace, cudaStream_t stream) {
    if (a.B == 0) return cudaSuccess;
    EncodeTiledFn encode = get_encode_fn();
    if (!encode) return cudaErrorNotSupported;
    const int R = a.k * (a.Hq / a.Hkv);
    // K / V as rows of 128 bytes; a box is CH = min(P, 128) rows of one page
    CUtensorMap kmap, vmap;
    for (int t = 0; t < 2; ++t) {
        cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)a.num_pages * a.Hkv * a.P};
        cuuint64_t strides[1] = {(cuuint64_t)D};
        cuuint32_t box[2] = {(cuuint32_t)D, (cuuint32_t)(a.P < TN ? a.P : TN)};
        cuuint32_t es[2] = {1, 1};
        if (encode(t == 0 ? &kmap : &vmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
                   const_cast<void*>(t == 0 ? a.k_cache : a.v_cache), dims, strides, box, es,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    F8Params prm;
    prm.a = a;
    prm.part_o = static_cast<float*>(workspace);
    prm.part_lse = prm.part_o + (size_t)2 * num_ctas * ROWS * D;
    prm.seg_rec = reinterpret_cast<int4*>(prm.part_lse + (size_t)2 * num_ctas * ROWS);
    prm.seg_pre = reinterpret_cast<int*>(prm.seg_rec + 2 * (size_t)num_ctas);
    prm.whole = whole_segments(a, num_ctas, TN, kCutTiles, kRoundedBase, kRoundedMore);
    if (prm.whole == kOwnCta) num_ctas = a.B * a.Hkv;
    const int rep = R <= 32 ? 4 : R <= 64 ? 2 : 1;
    const bool win = a.window > 0;
    const cudaError_t e =
        rep == 4   ? (win ? launch_typed<4, true>(kmap, vmap, prm, num_ctas, stream)
                          : launch_typed<4, false>(kmap, vmap, prm, num_ctas, stream))
        : rep == 2 ? (win ? launch_typed<2, true>(kmap, vmap, prm, num_ctas, stream)
                          : launch_typed<2, false>(kmap, vmap, prm, num_ctas, stream))
                   : (win ? launch_typed<1, true>(kmap, vmap, prm, num_ctas, stream)
                          : launch_typed<1, false>(kmap, vmap, prm, num_ctas, stream));
    if (e != cudaSuccess || prm.whole || max_units(a, TN) <= 1) return e;  // none is cut
    return launch_combine_stream_k(a, num_ctas, a.split_alpha >= 0 ? a.split_alpha : kSplitAlpha,
                                   prm.part_o, prm.part_lse, prm.seg_rec, prm.seg_pre, stream);
}

}  // namespace specv
