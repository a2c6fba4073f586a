// Rotary positions fused with the append to the paged cache.
//
// Mathematics.  Token t of sequence b stands at position p = ctx_b + t (or
// positions[b, t]: a tree's nodes stand at ctx_b + depth).  Pair j of the
// first `rot` elements of a q or k row, (x, y) = (2j, 2j + 1) interleaved or
// (j, j + rot/2) in halves, turns by the angle p f_j and is multiplied by the
// amplitude:
//   x' = x c - y s,  y' = x s + y c,  (c, s) = amp (cos, sin)(p f_j).
// The table holds f_j / 2 pi as a 64-bit binary fraction of a turn, so that
// p * table[j] modulo 2^64 is the angle reduced exactly, however far the
// position: one integer product instead of a 64-bit floating reduction.  Its
// upper 32 bits go to sincospif, and what their rounding to fp32 leaves out (up
// to 2^-25 turns) back by the first-order terms of the angle sum.
//
// The cache rows: f32 / bf16 as they are (bf16 rounded once, to nearest
// even); i8 as in kv_append.cu; e4m3 with one scale per (page, kv-head):
//   s' = max(s if the page keeps rows, max |x| of the new rows / 448)
//   new codes e4m3(x / s'); kept codes e4m3((c s) / s') when s' > s
// every step in fp32 with IEEE division and rounding to nearest even, the
// rotated value unrounded before it.  The scale of a page only grows while it
// is being filled (rows of rejected drafts included) and starts afresh when
// its first slot is written.
//
// Layout.  It is bound by memory (every row is read and written once), so
// lanes hold 8 consecutive elements each (16-byte loads of bf16) and the
// partner of a half-layout pair comes from another lane's registers by
// shuffles.  Two kinds of CTAs share one launch:
//  * row CTAs: a warp takes one token and a run of its heads (q, and k / v of
//    the caches whose rows are independent), the token's cosines and sines in
//    registers for all of them;
//  * page CTAs (e4m3): two warps take one (page, kv-head) of k or of v, whose
//    rows share a scale, half of the rows each, four heads at a time and, in calls
//    of many pages, several such groups in turn; the CTA's warps share the
//    cosines and sines of its 16 tokens in shared memory.  Up to 16 rows stay in
//    registers between the maximum and the codes; a longer page is read twice
//    (the second time from L1 / L2).
#include <cuda_fp8.h>

#include "common.cuh"

namespace specv {
namespace {

constexpr int kWarps = 8;
constexpr int kRowBlock = 16;  // tokens of a page CTA's table (at most)
constexpr int kPageHeads = kWarps / 2;  // heads of a page CTA
constexpr int kMaxPairs = 128;
// what the row CTAs write besides q; e4m3: page CTAs of one group of heads, of many
enum { kF32, kBf16, kI8, kPages, kPagesMany };

struct RopeParams {
    RopeAppendArgs a;
    int lr_log2;        // log2 of the lanes that hold one row (8 elements each)
    int heads;          // heads of a token's row items (q, then k, then v)
    int heads_per_warp; // heads of one row item
    int groups;         // row items of a token
    int64_t row_blocks; // CTAs of the row kind
    int pages;          // pages a sequence's append can touch
    int head_parts;     // page CTAs per (sequence, page, tensor)
};

// 8 consecutive source elements as fp32
template <typename T> struct Chunk;
template <> struct Chunk<__nv_bfloat16> {
    uint4 r;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        r = *reinterpret_cast<const uint4*>(p);  // (q_out may be q: no read-only path)
    }
    __device__ __forceinline__ void zero() { r = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[2 * e] = __uint_as_float(w[e] << 16);
            x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ Chunk from_lane(int src) const {
        Chunk o;
        o.r.x = __shfl_sync(0xffffffffu, r.x, src);
        o.r.y = __shfl_sync(0xffffffffu, r.y, src);
        o.r.z = __shfl_sync(0xffffffffu, r.z, src);
        o.r.w = __shfl_sync(0xffffffffu, r.w, src);
        return o;
    }
    __device__ __forceinline__ void flip(bool neg) {  // the signs when neg
        const uint32_t m = neg ? 0x80008000u : 0u;
        r.x ^= m; r.y ^= m; r.z ^= m; r.w ^= m;
    }
};
template <> struct Chunk<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = reinterpret_cast<const float4*>(p)[0];
        b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
    __device__ __forceinline__ Chunk from_lane(int src) const {
        constexpr uint32_t kAll = 0xffffffffu;
        Chunk o;
        o.a.x = __shfl_sync(kAll, a.x, src); o.a.y = __shfl_sync(kAll, a.y, src);
        o.a.z = __shfl_sync(kAll, a.z, src); o.a.w = __shfl_sync(kAll, a.w, src);
        o.b.x = __shfl_sync(kAll, b.x, src); o.b.y = __shfl_sync(kAll, b.y, src);
        o.b.z = __shfl_sync(kAll, b.z, src); o.b.w = __shfl_sync(kAll, b.w, src);
        return o;
    }
    __device__ __forceinline__ void flip(bool neg) {
        const float m = neg ? -1.f : 1.f;
        a.x *= m; a.y *= m; a.z *= m; a.w *= m;
        b.x *= m; b.y *= m; b.z *= m; b.w *= m;
    }
};

__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                   pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// 8 values to e4m3 codes (to nearest even, saturating), lowest byte first
__device__ __forceinline__ uint2 e4m3x8(const float (&x)[8]) {
    uint32_t h[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        h[e] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * e], x[2 * e + 1]), __NV_SATFINITE,
                                        __NV_E4M3);
    return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}
__device__ __forceinline__ void e4m3x8_to_f32(uint2 w, float (&x)[8]) {
    const uint32_t h[2] = {w.x, w.y};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(
            (__nv_fp8x2_storage_t)(h[e >> 1] >> (16 * (e & 1))), __NV_E4M3);
        const float2 f = __half22float2(__half2(r));
        x[2 * e] = f.x;
        x[2 * e + 1] = f.y;
    }
}

// (cos, sin) of the angle p * freq (64-bit fraction of a turn), times amplitude
__device__ __forceinline__ float2 turn(int64_t p, uint64_t freq, float amplitude) {
    const int32_t t = (int32_t)(((uint64_t)p * freq) >> 32);
    const float x = __int2float_rz(t);  // at most 2^31 - 128: back to an int exactly
    const float rest = (float)(t - (int32_t)x) * (0x1p-31f * 3.14159265358979f);
    float s, c;
    sincospif(x * 0x1p-31f, &s, &c);
    return make_float2((c - s * rest) * amplitude, (s + c * rest) * amplitude);
}

// The first pair of the 8 elements from e0 on, in the layout's order (halves:
// 8 pairs, interleaved: 4), or -1 when they are not rotated
template <bool INTER> __device__ __forceinline__ int first_pair(const RopeAppendArgs& a, int e0) {
    if (e0 >= a.rot) return -1;
    return INTER ? e0 / 2 : e0 < a.rot / 2 ? e0 : e0 - a.rot / 2;
}

// Rotates a lane's 8 elements (from e0 on) in place.  `other` holds the
// partner's 8 elements (halves); cs the pairs' (cos, sin), in the lower half
// of a half layout (cos, -sin).
template <bool INTER, int N>
__device__ __forceinline__ void rotate8(const RopeAppendArgs& a, int e0, float (&x)[8],
                                        const float (&other)[8], const float2 (&cs)[N]) {
    if (e0 >= a.rot) return;
    if constexpr (INTER) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float u = x[2 * e], v = x[2 * e + 1];
            x[2 * e] = u * cs[e].x - v * cs[e].y;
            x[2 * e + 1] = u * cs[e].y + v * cs[e].x;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * cs[e].x + other[e] * cs[e].y;
    }
}

// lane that holds the partner of a half-layout chunk (8 elements per lane)
__device__ __forceinline__ int partner_lane(const RopeAppendArgs& a, int lane, int e0) {
    if (e0 >= a.rot) return lane;
    return e0 < a.rot / 2 ? lane + a.rot / 16 : lane - a.rot / 16;
}

// Page and slot of position pos of sequence b; page < 0 when it is outside the
// table or the pool (flagged).
__device__ __forceinline__ int find_page(const RopeAppendArgs& a, int b, int64_t pos, bool flag) {
    if (pos < 0 || pos / a.P >= a.max_pages) {
        if (flag) raise_device_error(a.dev_err, SPEC_DEVERR_CTX);
        return -1;
    }
    const int page = __ldg(a.block_table + (int64_t)b * a.max_pages + pos / a.P);
    if (page < 0 || page >= a.num_pages) {
        if (flag) raise_device_error(a.dev_err, SPEC_DEVERR_PAGE);
        return -1;
    }
    return page;
}

// tokens sequence b appends
__device__ __forceinline__ int new_len(const RopeAppendArgs& a, int b) {
    if (!a.new_lens) return a.n;
    return max(0, min(a.n, __ldg(a.new_lens + b)));
}

// x / s for a fixed positive s, to nearest: with r = 1 / s rounded to nearest,
// q = x r and the exact remainder x - q s, q + r (x - q s) is the correctly
// rounded quotient (Markstein's theorem), three instructions per element where
// a division takes three times as many.  The remainder, exact, is rounded down:
// a zero one is then -0, which leaves the sign of a zero q as it is (+0 would turn
// -0 / s, a code of its own in e4m3, into +0).  Outside the range where no step
// underflows the division itself.
struct Divide {
    float s, r;
    bool plain;
    __device__ __forceinline__ explicit Divide(float by) : s(by) {
        plain = !(by > 0x1p-96f && by < 0x1p96f);
        r = plain ? 0.f : __frcp_rn(by);
    }
    __device__ __forceinline__ void operator()(float (&x)[8]) const {
        if (plain) {
#pragma unroll 1
            for (int e = 0; e < 8; ++e) {  // (rotated: no dynamic index)
                const float q = s > 0.f ? __fdiv_rn(x[0], s) : 0.f;
#pragma unroll
                for (int k = 0; k < 7; ++k) x[k] = x[k + 1];
                x[7] = q;
            }
            return;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float q = x[e] * r;
            x[e] = fmaf(__fmaf_rd(-q, s, x[e]), r, q);
        }
    }
};

// ---------------------------------------------------------------- row CTAs
// The rows of one kind (q, k or v) of a token's heads [h0, h1): U of a lane's
// rows in flight, rotated, and stored `head_stride` elements apart.
template <typename T, typename TD, bool INTER, bool I8, int N>
__device__ __forceinline__ void token_rows(const RopeAppendArgs& a, int lr_log2, const T* src,
                                           TD* dst, int64_t head_stride, uint16_t* scale, int h0,
                                           int h1, bool spin, const float2 (&cs)[N]) {
    const int lane = threadIdx.x & 31;
    const int lr = 1 << lr_log2, rows = 32 >> lr_log2;  // lanes of a row, rows at a time
    const int e0 = (lane & (lr - 1)) * 8;
    const bool in_row = e0 < a.D;
    const int from = in_row ? partner_lane(a, lane, e0) : lane;
    constexpr int U = 4;
    for (int hb = h0; hb < h1; hb += rows * U) {
        Chunk<T> c[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = hb + u * rows + (lane >> lr_log2);
            c[u].zero();
            if (h < h1 && in_row) c[u].load(src + h * a.D + e0);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (hb + u * rows >= h1) break;  // uniform over the warp
            const int h = hb + u * rows + (lane >> lr_log2);
            const bool mine = h < h1 && in_row;
            float x[8];
            c[u].get(x);
            if (spin) {
                float o[8];
                if constexpr (!INTER) c[u].from_lane(from).get(o);
                rotate8<INTER>(a, e0, x, o, cs);
            }
            if constexpr (!I8) {
                if (mine) store8(dst + h * head_stride + e0, x);
            } else {
                // one scale per (token, kv-head) row
                float amax = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(x[e]));
                if (!in_row) amax = 0.f;
                for (int off = lr / 2; off > 0; off >>= 1)
                    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
                const __half s16 = __float2half_rn(__fdiv_rn(amax, 127.0f));
                const float s = __half2float(s16);
                const Divide by(s);
                by(x);
                uint32_t w[2] = {0, 0};
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float v = fminf(fmaxf(rintf(x[e]), -127.f), 127.f);
                    w[e >> 2] |= (uint32_t)(uint8_t)(int8_t)v << (8 * (e & 3));
                }
                if (mine) {
                    *reinterpret_cast<uint2*>(dst + h * head_stride + e0) = make_uint2(w[0], w[1]);
                    if (e0 == 0) scale[(int64_t)h * a.P] = __half_as_ushort(s16);
                }
            }
        }
    }
}

template <typename T, bool INTER, int MODE>
__device__ __forceinline__ void row_cta(const RopeParams& p, float2* turns, int64_t block) {
    const RopeAppendArgs& a = p.a;
    const int lane = threadIdx.x & 31;
    const int64_t item = block * kWarps + (threadIdx.x >> 5);
    const int64_t token = item / p.groups;
    const int group = (int)(item % p.groups);
    if (token >= (int64_t)a.B * a.n) return;
    const int b = (int)(token / a.n), t = (int)(token % a.n);
    const int64_t ctx = __ldg(a.ctx_lens + b), pos = ctx + t;
    if (t >= new_len(a, b)) return;
    const int e0 = (lane & ((1 << p.lr_log2) - 1)) * 8;
    const int h_begin = group * p.heads_per_warp;
    const int h_end = min(p.heads, h_begin + p.heads_per_warp);
    // the cache row of a warp that holds k or v heads (none of a sequence whose
    // context is negative, also where ctx + t is a position again)
    int page = -1;
    if (MODE != kPages && h_end > a.Hq) page = find_page(a, b, ctx < 0 ? ctx : pos, lane == 0);
    constexpr int N = INTER ? 4 : 8;
    float2 cs[N];
    const int j0 = e0 < a.D ? first_pair<INTER>(a, e0) : -1;
    const bool spin = a.rot > 0 && h_begin < a.Hq + a.Hkv;
    if (spin) {
        const int64_t at = a.positions ? (int64_t)__ldg(a.positions + token) : pos;
        if constexpr (INTER) {
            if (j0 >= 0)
#pragma unroll
                for (int e = 0; e < N; ++e) cs[e] = turn(at, __ldg(a.table + j0 + e), a.amplitude);
        } else {
            // the warp computes each angle once and shares it: a lane needs eight, the
            // same ones as the lane of the other half (32 x 64 tokens 16.0 -> 14.7 us;
            // pairs side by side take four, and lost by it: 52.0 -> 53.4 on prompts)
            turns += (threadIdx.x >> 5) * kMaxPairs;
            for (int j = lane; j < a.rot / 2; j += 32)
                turns[j] = turn(at, __ldg(a.table + j), a.amplitude);
            __syncwarp();
            if (j0 >= 0)
#pragma unroll
                for (int e = 0; e < N; e += 2) {
                    const float4 two = *reinterpret_cast<const float4*>(turns + j0 + e);
                    const float sign = e0 < a.rot / 2 ? -1.f : 1.f;
                    cs[e] = make_float2(two.x, two.y * sign);
                    cs[e + 1] = make_float2(two.z, two.w * sign);
                }
        }
    }
    if (h_begin < a.Hq)
        token_rows<T, T, INTER, false>(
            a, p.lr_log2, static_cast<const T*>(a.q) + token * a.q_stride,
            static_cast<T*>(a.q_out) + token * a.q_out_stride, a.D, nullptr, h_begin,
            min(h_end, a.Hq), spin, cs);
    if (MODE == kPages || page < 0) return;
    const int64_t row = (int64_t)page * a.Hkv * a.P + pos % a.P;
#pragma unroll 1
    for (int is_v = 0; is_v < 2; ++is_v) {
        const int first = a.Hq + is_v * a.Hkv;
        const int h0 = max(0, h_begin - first), h1 = min(h_end - first, a.Hkv);
        if (h0 >= h1) continue;
        const T* src = is_v ? static_cast<const T*>(a.v_new) + token * a.v_stride
                            : static_cast<const T*>(a.k_new) + token * a.k_stride;
        void* cache = is_v ? a.v_cache : a.k_cache;
        const int64_t hs = (int64_t)a.P * a.D;
        if constexpr (MODE == kI8)
            token_rows<T, int8_t, INTER, true>(
                a, p.lr_log2, src, static_cast<int8_t*>(cache) + row * a.D, hs,
                static_cast<uint16_t*>(is_v ? a.v_scale : a.k_scale) + row, h0, h1,
                spin && !is_v, cs);
        else if constexpr (MODE == kBf16)
            token_rows<T, __nv_bfloat16, INTER, false>(
                a, p.lr_log2, src, static_cast<__nv_bfloat16*>(cache) + row * a.D, hs, nullptr, h0,
                h1, spin && !is_v, cs);
        else
            token_rows<T, float, INTER, false>(a, p.lr_log2, src,
                                               static_cast<float*>(cache) + row * a.D, hs, nullptr,
                                               h0, h1, spin && !is_v, cs);
    }
}

// ---------------------------------------------------------------- page CTAs (e4m3)
template <typename T, bool INTER, bool MANY>
__device__ __forceinline__ void page_cta(const RopeParams& p, float2 (*tab)[kMaxPairs],
                                         float (*s_max)[kWarps], int64_t item) {
    const RopeAppendArgs& a = p.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int part0 = (int)(item % p.head_parts);
    item /= p.head_parts;
    const bool is_v = item & 1;
    item >>= 1;
    const int pg = (int)(item % p.pages), b = (int)(item / p.pages);
    const int64_t ctx = __ldg(a.ctx_lens + b);
    const int count = new_len(a, b);
    const bool spin = !is_v && a.rot > 0;
    const int pairs = a.rot / 2;
    // When the pairs divide the CTA a thread computes one pair of every few rows
    // (its frequency loaded beside the context length, not after it).
    const bool even = spin && (kWarps * 32) % pairs == 0;
    const uint64_t freq = even ? __ldg(a.table + threadIdx.x % pairs) : 0;
    if (ctx < 0) {
        if (threadIdx.x == 0) raise_device_error(a.dev_err, SPEC_DEVERR_CTX);
        return;
    }
    // the page's slots [first, last) receive tokens t0 ..
    const int64_t page_start = (ctx / a.P + pg) * a.P;
    const int first = (int)max((int64_t)0, ctx - page_start);
    const int last = (int)min((int64_t)a.P, ctx + count - page_start);
    if (first >= last) return;
    const int t0 = (int)(page_start + first - ctx), nr = last - first;
    // two warps per head, each half of the rows of a block; the CTA's heads in
    // groups of kPageHeads, every head_parts-th its own
    const int pair = warp >> 1, part = warp & 1;
    const int lr = 1 << p.lr_log2, rows = 32 >> p.lr_log2;
    const int e0 = (lane & (lr - 1)) * 8, sub = lane >> p.lr_log2;
    const bool in_row = e0 < a.D;
    const int j0 = in_row ? first_pair<INTER>(a, e0) : -1;
    const int from = in_row ? partner_lane(a, lane, e0) : lane;
    const int64_t stride = is_v ? a.v_stride : a.k_stride;
    const T* src0 = static_cast<const T*>(is_v ? a.v_new : a.k_new) +
                    ((int64_t)b * a.n + t0) * stride + e0;
    constexpr int N = INTER ? 4 : 8;                   // pairs of a lane's 8 elements
    constexpr int U = 4;                               // rows in flight per lane
    const int half = min(kRowBlock / 2, U * rows);     // rows of a block per warp
    const int rb = 2 * half;                           // rows of a block: one table
    // row of the block (its first row `base`) that this lane holds at u, or -1
    auto row_of = [&](int base, int u) {
        const int in = u * rows + sub, r = part * half + in;
        return in < half && base + r < nr ? r : -1;
    };
    Chunk<T> c[U];
    float x[U][8];
    auto load_rows = [&](int g, int base) {
        const T* src = src0 + (int64_t)g * a.D;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = row_of(base, u);
            c[u].zero();
            if (r >= 0 && in_row && g < a.Hkv) c[u].load(src + (base + r) * stride);
        }
    };
    // The table of a block: pair j of a row in the order that its readers take,
    // two pairs of a lane side by side (j / N of the lanes, j % N in it).
    auto slot_of = [&](int j) {
        const int e = j % N;
        return ((e >> 1) * (pairs / N) + j / N) * 2 + (e & 1);
    };
    auto put_angle = [&](int base, int r, int j, uint64_t f) {
        const int64_t at = a.positions
                               ? (int64_t)__ldg(a.positions + (int64_t)b * a.n + t0 + base + r)
                               : page_start + first + base + r;
        tab[r][slot_of(j)] = turn(at, f, a.amplitude);
    };
    auto fill_table = [&](int base) {
        if (!spin) return;
        __syncthreads();  // the table's readers are done
        const int n = min(rb, nr - base);
        if (even) {
            const int j = threadIdx.x % pairs, step = kWarps * 32 / pairs;
            for (int r = threadIdx.x / pairs; r < n; r += step) put_angle(base, r, j, freq);
        } else {
            for (int e = threadIdx.x; e < n * pairs; e += kWarps * 32)
                put_angle(base, e / pairs, e % pairs, __ldg(a.table + e % pairs));
        }
        __syncthreads();
    };
    auto rotate_rows = [&](int base) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            c[u].get(x[u]);
            if (!spin) continue;
            float o[8];
            float2 cs[N];
            if constexpr (!INTER) {
                Chunk<T> other = c[u].from_lane(from);
                other.flip(e0 < a.rot / 2);  // x cos - y sin in the lower half
                other.get(o);
            }
            const int r = row_of(base, u);
            if (j0 >= 0 && r >= 0) {
                const float4* row = reinterpret_cast<const float4*>(tab[r]) + j0 / N;
#pragma unroll
                for (int e = 0; e < N; e += 2) {
                    const float4 two = row[(e >> 1) * (pairs / N)];
                    cs[e] = make_float2(two.x, two.y);
                    cs[e + 1] = make_float2(two.z, two.w);
                }
                rotate8<INTER>(a, e0, x[u], o, cs);
            }
        }
    };
    auto largest = [&](float amax) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(x[u][e]));  // (no row: zeros)
        return amax;
    };
    // the first rows are on their way while the page is looked up, its scale while
    // the angles are computed
    int g = part0 * kPageHeads + pair;
    load_rows(g, 0);
    const int page = find_page(a, b, page_start, threadIdx.x == 0);
    if (page < 0) return;
    float* scales = static_cast<float*>(is_v ? a.v_scale : a.k_scale) + (int64_t)page * a.Hkv;
    float old = g < a.Hkv && first > 0 ? scales[g] : 0.f;
    fill_table(0);
    const bool one_block = nr <= rb;
#pragma unroll 1
    for (int it = 0;; ++it) {
        const int next = g + p.head_parts * kPageHeads;
        const bool active = g < a.Hkv && in_row;
        uint8_t* codes = static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) +
                         ((int64_t)page * a.Hkv + g) * a.P * a.D + e0;
        float amax = 0.f;
        if (one_block) {
            // the rows stay in registers (the next group's are loaded after them: read
            // ahead they spill, 78 -> 84 us on 16.4K prompt tokens)
            rotate_rows(0);
            amax = largest(0.f);
        } else {
#pragma unroll 1
            for (int base = 0; base < nr; base += rb) {
                load_rows(g, base);
                fill_table(base);
                rotate_rows(base);
                amax = largest(amax);
            }
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
        float* mx = s_max[it & 1];
        if (lane == 0) mx[warp] = amax;
        named_bar_sync(1 + pair, 64);  // (both warps have read the old scale, too)
        float s = __fdiv_rn(fmaxf(amax, mx[warp ^ 1]), 448.0f);
        if (first > 0 && old >= s) s = old;
        const Divide by(s);
        if (g < a.Hkv && part == 0 && lane == 0) scales[g] = s;
        if (first > 0 && s > old) {
            // the kept rows' codes in the new scale
            for (int r = part * rows + sub; r < first; r += 2 * rows) {
                if (!active) continue;
                uint2* at = reinterpret_cast<uint2*>(codes + (int64_t)r * a.D);
                float v[8];
                e4m3x8_to_f32(*at, v);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = __fmul_rn(v[e], old);
                by(v);
                *at = e4m3x8(v);
            }
        }
#pragma unroll 1
        for (int base = 0; base < nr; base += rb) {
            if (!one_block) {  // more rows than the registers held
                load_rows(g, base);
                fill_table(base);
                rotate_rows(base);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = row_of(base, u);
                if (r < 0 || !active) continue;
                by(x[u]);
                *reinterpret_cast<uint2*>(codes + (int64_t)(first + base + r) * a.D) =
                    e4m3x8(x[u]);
            }
        }
        if (!MANY || next - pair >= a.Hkv) break;  // (next - pair: the CTA's group)
        g = next;
        load_rows(g, 0);
        old = g < a.Hkv && first > 0 ? scales[g] : 0.f;
    }
}

// CTAs per SM.  Row kernels whose registers allow a fourth gain by it (12.3K prompt
// tokens in pairs side by side 53.8 -> 52.0 us, 16.4K in halves into i8 82.5 -> 78.5);
// halves into bf16 spill (71.7 -> 74.3).
template <typename T, bool INTER, int MODE> constexpr int resident() {
    return sizeof(T) == 2 && MODE < kPages && (INTER || MODE == kI8) ? 4 : 3;
}

// Measured: 12.3K prompt tokens of 32 + 8 heads into bf16 52.0 us (0.89 of the copy
// rate), 16.4K into e4m3 76 us (0.72:
// the page CTAs' arithmetic; 89 with a CTA, and its own angles, per group of
// heads), 32 x 4 drafts into e4m3 4.8 us.
template <typename T, bool INTER, int MODE>
__global__ void __launch_bounds__(kWarps * 32, (resident<T, INTER, MODE>()))
rope_append_kernel(const RopeParams p) {
    grid_dep_launch_dependents();
    grid_dep_wait();
    // of a page CTA's rows, or of each warp's token
    __shared__ __align__(16) float2 tab[MODE < kPages ? kWarps : kRowBlock][kMaxPairs];
    if constexpr (MODE < kPages) {
        row_cta<T, INTER, MODE>(p, tab[0], blockIdx.x);
    } else {
        // the page CTAs, whose chain of loads is longer, start first
        const int64_t pages = gridDim.x - p.row_blocks;
        if (blockIdx.x >= pages) {
            row_cta<T, INTER, kPages>(p, tab[0], blockIdx.x - pages);
        } else {
            __shared__ float s_max[2][kWarps];
            page_cta<T, INTER, MODE == kPagesMany>(p, tab, s_max, blockIdx.x);
        }
    }
}

template <typename T, bool INTER>
cudaError_t launch_typed(const RopeParams& p, unsigned blocks, cudaStream_t stream) {
    auto go = [&](auto kern) {
        return launch_dependent(kern, dim3(blocks), dim3(kWarps * 32), 0, stream, p);
    };
    switch (p.a.cache_dtype) {
    case SPEC_DTYPE_F32: return go(rope_append_kernel<T, INTER, kF32>);
    case SPEC_DTYPE_BF16: return go(rope_append_kernel<T, INTER, kBf16>);
    case SPEC_DTYPE_I8: return go(rope_append_kernel<T, INTER, kI8>);
    case SPEC_DTYPE_E4M3:
        return p.head_parts * kPageHeads < p.a.Hkv ? go(rope_append_kernel<T, INTER, kPagesMany>)
                                                   : go(rope_append_kernel<T, INTER, kPages>);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_rope_append(const RopeAppendArgs& a, int num_sms, cudaStream_t stream) {
    RopeParams p;
    p.a = a;
    p.lr_log2 = 2;
    while ((8 << p.lr_log2) < a.D) ++p.lr_log2;
    const bool paged = a.cache_dtype == SPEC_DTYPE_E4M3;
    const int64_t tokens = (int64_t)a.B * a.n;
    p.heads = a.Hq + (paged ? 0 : 2 * a.Hkv);
    // heads of a warp: all of a token's, halved while the launch would leave
    // most of the SMs' warp slots empty (a call of few tokens is one latency
    // chain per warp; the angles are then computed by more warps)
    const int step = 32 >> p.lr_log2;
    int per = p.heads > 0 ? p.heads : 1;
    while (per > step && tokens * ((p.heads + per - 1) / per) < (int64_t)num_sms * 32)
        per = (per + 1) / 2;
    p.heads_per_warp = (per + step - 1) / step * step;
    p.groups = p.heads > 0 ? (p.heads + p.heads_per_warp - 1) / p.heads_per_warp : 0;
    p.row_blocks = (tokens * p.groups + kWarps - 1) / kWarps;
    p.pages = paged ? (int)(((int64_t)a.n + a.P - 2) / a.P + 1) : 0;
    // page CTAs take several groups of heads (the angles are theirs in common)
    // while that leaves enough of them to fill the SMs a few times
    p.head_parts = (a.Hkv + kPageHeads - 1) / kPageHeads;
    const int64_t page_ctas = (int64_t)a.B * p.pages * 2;
    while (p.head_parts > 1 && page_ctas * ((p.head_parts + 1) / 2) >= (int64_t)num_sms * 12)
        p.head_parts = (p.head_parts + 1) / 2;
    const int64_t blocks = p.row_blocks + page_ctas * p.head_parts;
    if (blocks == 0) return cudaSuccess;
    if (blocks >= (1LL << 31)) return cudaErrorInvalidConfiguration;
    const unsigned n = (unsigned)blocks;
    if (a.src_dtype == SPEC_DTYPE_F32)
        return a.interleaved ? launch_typed<float, true>(p, n, stream)
                             : launch_typed<float, false>(p, n, stream);
    return a.interleaved ? launch_typed<__nv_bfloat16, true>(p, n, stream)
                         : launch_typed<__nv_bfloat16, false>(p, n, stream);
}

}  // namespace specv
