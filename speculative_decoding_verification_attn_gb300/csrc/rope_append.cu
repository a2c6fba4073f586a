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
// upper 32 bits go to sincospif (angle error below 2^-24 turns of rounding).
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
//  * page CTAs (e4m3): a warp takes one (page, kv-head) of k or of v, whose
//    rows share a scale; the CTA's warps share the cosines and sines of its
//    16 tokens in shared memory.  Up to 16 rows stay in registers between the
//    maximum and the codes; a longer page is read twice (the second time from
//    L1 / L2).
#include <cuda_fp8.h>

#include "common.cuh"

namespace specv {
namespace {

constexpr int kWarps = 8;
constexpr int kRowBlock = 16;  // tokens of a page CTA's table (at most)
constexpr int kMaxPairs = 128;

struct RopeParams {
    RopeAppendArgs a;
    int lr_log2;        // log2 of the lanes that hold one row (8 elements each)
    int heads;          // heads of a token's row items (q, then k, then v)
    int heads_per_warp; // heads of one row item
    int groups;         // row items of a token
    int64_t row_blocks; // CTAs of the row kind
    int pages;          // pages a sequence's append can touch
    int head_groups;    // page CTAs per (sequence, page, tensor)
};

// 8 consecutive source elements as fp32
template <typename T> struct Chunk;
template <> struct Chunk<__nv_bfloat16> {
    uint4 r;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        r = __ldg(reinterpret_cast<const uint4*>(p));
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
};
template <> struct Chunk<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = __ldg(reinterpret_cast<const float4*>(p));
        b = __ldg(reinterpret_cast<const float4*>(p) + 1);
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

// (cos, sin) of pair j at position p, times the amplitude
__device__ __forceinline__ float2 turn(const RopeAppendArgs& a, int64_t p, int j) {
    const uint64_t t = (uint64_t)p * (uint64_t)__ldg(a.table + j);
    float s, c;
    sincospif((float)(int32_t)(t >> 32) * 0x1p-31f, &s, &c);
    return make_float2(c * a.amplitude, s * a.amplitude);
}

// The first pair of the 8 elements from e0 on, in the layout's order (halves:
// 8 pairs, interleaved: 4), or -1 when they are not rotated
__device__ __forceinline__ int first_pair(const RopeAppendArgs& a, int e0) {
    if (e0 >= a.rot) return -1;
    return a.interleaved ? e0 / 2 : e0 % (a.rot / 2);
}

// Rotates a lane's 8 elements (from e0 on) in place.  `other` holds the
// partner's 8 elements (halves); cs the pairs' (cos, sin).
__device__ __forceinline__ void rotate8(const RopeAppendArgs& a, int e0, float (&x)[8],
                                        const float (&other)[8], const float2 (&cs)[8]) {
    if (e0 >= a.rot) return;
    if (a.interleaved) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float u = x[2 * e], v = x[2 * e + 1];
            x[2 * e] = u * cs[e].x - v * cs[e].y;
            x[2 * e + 1] = u * cs[e].y + v * cs[e].x;
        }
    } else {
        const float sign = e0 < a.rot / 2 ? -1.f : 1.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * cs[e].x + sign * other[e] * cs[e].y;
    }
}

// lane offset (in 8-element chunks) of the partner of a half-layout chunk
__device__ __forceinline__ int partner_lane(const RopeAppendArgs& a, int lane, int e0) {
    if (a.interleaved || e0 >= a.rot) return lane;
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

// ---------------------------------------------------------------- row CTAs
template <typename T>
__device__ __forceinline__ void row_cta(const RopeParams& p) {
    const RopeAppendArgs& a = p.a;
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int64_t token = item / p.groups;
    const int group = (int)(item % p.groups);
    if (token >= (int64_t)a.B * a.n) return;
    const int b = (int)(token / a.n), t = (int)(token % a.n);
    if (t >= new_len(a, b)) return;
    const int lr = 1 << p.lr_log2, rows = 32 >> p.lr_log2;  // lanes of a row, rows at a time
    const int e0 = (lane & (lr - 1)) * 8;
    const bool in_row = e0 < a.D;
    const int h_begin = group * p.heads_per_warp;
    const int h_end = min(p.heads, h_begin + p.heads_per_warp);
    const int64_t pos = (int64_t)__ldg(a.ctx_lens + b) + t;
    // the cache row of a warp that holds k or v heads
    int page = -1;
    if (h_end > a.Hq) page = find_page(a, b, pos, lane == 0);
    float2 cs[8];
    const int j0 = in_row ? first_pair(a, e0) : -1;
    if (j0 >= 0 && h_begin < a.Hq + a.Hkv) {
        const int64_t at = a.positions ? (int64_t)__ldg(a.positions + token) : pos;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < 4 || !a.interleaved) cs[e] = turn(a, at, j0 + e);
    }
    constexpr int U = 4;  // rows in flight per lane
    for (int h0 = h_begin; h0 < h_end; h0 += rows * U) {
        Chunk<T> c[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + u * rows + (lane >> p.lr_log2);
            c[u].zero();
            if (h < h_end && in_row) {
                const T* src =
                    h < a.Hq ? static_cast<const T*>(a.q) + token * a.q_stride + (int64_t)h * a.D
                    : h < a.Hq + a.Hkv
                        ? static_cast<const T*>(a.k_new) + token * a.k_stride +
                              (int64_t)(h - a.Hq) * a.D
                        : static_cast<const T*>(a.v_new) + token * a.v_stride +
                              (int64_t)(h - a.Hq - a.Hkv) * a.D;
                c[u].load(src + e0);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (h0 + u * rows >= h_end) continue;  // uniform over the warp
            const int h = h0 + u * rows + (lane >> p.lr_log2);
            const bool mine = h < h_end && in_row;
            float x[8], o[8];
            c[u].get(x);
            if (!a.interleaved && a.rot > 0)
                c[u].from_lane(in_row ? partner_lane(a, lane, e0) : lane).get(o);
            if (mine && h < a.Hq + a.Hkv) rotate8(a, e0, x, o, cs);
            if (mine && h < a.Hq)
                store8(static_cast<T*>(a.q_out) + token * a.q_out_stride + (int64_t)h * a.D + e0, x);
            if (h0 + (u + 1) * rows <= a.Hq || p.heads == a.Hq) continue;  // q alone; uniform
            // k / v rows (q rows may stand beside them in the warp)
            const bool is_v = h >= a.Hq + a.Hkv;
            const int g = is_v ? h - a.Hq - a.Hkv : h - a.Hq;
            const bool put = mine && h >= a.Hq && page >= 0;
            const int64_t row = ((int64_t)page * a.Hkv + g) * a.P + pos % a.P;
            void* cache = is_v ? a.v_cache : a.k_cache;
            if (a.cache_dtype == SPEC_DTYPE_BF16) {
                if (put) store8(static_cast<__nv_bfloat16*>(cache) + row * a.D + e0, x);
            } else if (a.cache_dtype == SPEC_DTYPE_F32) {
                if (put) store8(static_cast<float*>(cache) + row * a.D + e0, x);
            } else {
                // i8: one scale per (token, kv-head) row
                float amax = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(x[e]));
                if (!mine) amax = 0.f;
                for (int off = lr / 2; off > 0; off >>= 1)
                    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
                const __half s16 = __float2half_rn(__fdiv_rn(amax, 127.0f));
                const float s = __half2float(s16);
                uint32_t w[2] = {0, 0};
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float v = 0.f;
                    if (s > 0.f) v = fminf(fmaxf(rintf(__fdiv_rn(x[e], s)), -127.f), 127.f);
                    w[e >> 2] |= (uint32_t)(uint8_t)(int8_t)v << (8 * (e & 3));
                }
                if (put) {
                    *reinterpret_cast<uint2*>(static_cast<int8_t*>(cache) + row * a.D + e0) =
                        make_uint2(w[0], w[1]);
                    if (e0 == 0)
                        static_cast<uint16_t*>(is_v ? a.v_scale : a.k_scale)[row] =
                            __half_as_ushort(s16);
                }
            }
        }
    }
}

// ---------------------------------------------------------------- page CTAs (e4m3)
template <typename T>
__device__ __forceinline__ void page_cta(const RopeParams& p, float2 (*tab)[kMaxPairs]) {
    const RopeAppendArgs& a = p.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t item = (int64_t)blockIdx.x - p.row_blocks;
    const int hg = (int)(item % p.head_groups);
    item /= p.head_groups;
    const bool is_v = item & 1;
    item >>= 1;
    const int pg = (int)(item % p.pages), b = (int)(item / p.pages);
    const int64_t ctx = __ldg(a.ctx_lens + b);
    const int count = new_len(a, b);
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
    const int page = find_page(a, b, page_start, threadIdx.x == 0);
    if (page < 0) return;
    const int g = hg * kWarps + warp;
    const bool active = g < a.Hkv;
    const bool spin = !is_v && a.rot > 0;
    const int lr = 1 << p.lr_log2, rows = 32 >> p.lr_log2;
    const int e0 = (lane & (lr - 1)) * 8, sub = lane >> p.lr_log2;
    const bool in_row = e0 < a.D;
    const int j0 = in_row ? first_pair(a, e0) : -1;
    const int pairs = a.rot / 2;
    const T* src = static_cast<const T*>(is_v ? a.v_new : a.k_new) +
                   ((int64_t)b * a.n + t0) * (is_v ? a.v_stride : a.k_stride) + (int64_t)g * a.D + e0;
    const int64_t stride = is_v ? a.v_stride : a.k_stride;
    uint8_t* codes = static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) +
                     ((int64_t)page * a.Hkv + g) * a.P * a.D + e0;
    float* scale = static_cast<float*>(is_v ? a.v_scale : a.k_scale) + (int64_t)page * a.Hkv + g;

    constexpr int U = 8;                     // rows in flight per lane
    const int rb = min(kRowBlock, U * rows);  // rows of a block: one table, the registers
    const bool keep = nr <= rb;
    Chunk<T> c[U];
    float amax = 0.f, s = 0.f;
    // rows [base, base + rb) of the append: load them
    auto load_rows = [&](int base) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = base + u * rows + sub;
            c[u].zero();
            if (u * rows + sub < rb && r < nr && active && in_row)
                c[u].load(src + r * stride);
        }
    };
    auto fill_table = [&](int base) {
        __syncthreads();  // the table's readers are done
        if (spin)
            for (int e = threadIdx.x; e < min(rb, nr - base) * pairs; e += kWarps * 32) {
                const int r = base + e / pairs;
                const int64_t at = a.positions
                                       ? (int64_t)__ldg(a.positions + (int64_t)b * a.n + t0 + r)
                                       : page_start + first + r;
                tab[e / pairs][e % pairs] = turn(a, at, e % pairs);
            }
        __syncthreads();
    };
    auto value = [&](int base, int u, float (&x)[8]) {
        c[u].get(x);
        if (!spin) return;
        float o[8];
        float2 cs[8];
        if (!a.interleaved) c[u].from_lane(in_row ? partner_lane(a, lane, e0) : lane).get(o);
        const int r = u * rows + sub;
        if (j0 >= 0 && base + r < nr && r < rb) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < 4 || !a.interleaved) cs[e] = tab[r][j0 + e];
            rotate8(a, e0, x, o, cs);
        }
    };
    auto maximum = [&](int base) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (u * rows >= rb || base + u * rows >= nr) continue;  // uniform
            float x[8];
            value(base, u, x);  // rows past the last are zero
#pragma unroll
            for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(x[e]));
        }
    };
    auto store = [&](int base) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (u * rows >= rb || base + u * rows >= nr) continue;  // uniform
            float x[8];
            value(base, u, x);
            const int r = base + u * rows + sub;
            if (u * rows + sub < rb && r < nr && active && in_row) {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = s > 0.f ? __fdiv_rn(x[e], s) : 0.f;
                *reinterpret_cast<uint2*>(codes + (int64_t)(first + r) * a.D) = e4m3x8(x);
            }
        }
    };
    for (int base = 0; base < nr; base += rb) {
        load_rows(base);
        fill_table(base);
        maximum(base);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    s = __fdiv_rn(amax, 448.0f);
    if (active && first > 0) {
        const float old = *scale;
        if (old >= s) {
            s = old;
        } else {
            // the kept rows' codes in the new scale
            for (int r = sub; r < first; r += rows) {
                if (!in_row) continue;
                uint2* at = reinterpret_cast<uint2*>(codes + (int64_t)r * a.D);
                float x[8];
                e4m3x8_to_f32(*at, x);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = __fdiv_rn(__fmul_rn(x[e], old), s);
                *at = e4m3x8(x);
            }
        }
    }
    __syncwarp();  // every lane has read the old scale
    if (active && lane == 0) *scale = s;
    if (keep) {
        store(0);
        return;
    }
    for (int base = 0; base < nr; base += rb) {
        load_rows(base);
        fill_table(base);
        store(base);
    }
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) rope_append_kernel(const RopeParams p) {
    __shared__ float2 tab[kRowBlock][kMaxPairs];
    grid_dep_launch_dependents();
    grid_dep_wait();
    if (blockIdx.x < p.row_blocks)
        row_cta<T>(p);
    else
        page_cta<T>(p, tab);
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
    p.head_groups = (a.Hkv + kWarps - 1) / kWarps;
    const int64_t blocks = p.row_blocks + (int64_t)a.B * p.pages * 2 * p.head_groups;
    if (blocks == 0) return cudaSuccess;
    if (blocks >= (1LL << 31)) return cudaErrorInvalidConfiguration;
    auto kern = a.src_dtype == SPEC_DTYPE_F32 ? rope_append_kernel<float>
                                              : rope_append_kernel<__nv_bfloat16>;
    return launch_dependent(kern, dim3((unsigned)blocks), dim3(kWarps * 32), 0, stream, p);
}

}  // namespace specv
