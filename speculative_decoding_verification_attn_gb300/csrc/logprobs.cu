// Log probabilities of given tokens, the entropy of their rows and the top
// alternatives, in one pass over the logits.
//
// With z = x / T of a row's V logits, m their maximum and y = (x - m) log2(e) / T:
//   l = sum 2^y,  a = sum 2^y y,   lse = m / T + ln l,
//   logprob = z_token - lse,       entropy = ln l - ln 2 * a / l
// (the entropy as a difference of two terms of its own size, not of lse and a
// mean of z).  x - m comes before the product, so an exponent near zero is
// exact; l and a are held in fp32 per thread over a few hundred terms and
// merged by their maxima.
//
// What bounds it: the logits are read once.  An element costs ~5 issue slots
// (widen, subtract, scale, clamp, 2^y, two sums), about half of what an SM has
// while the memory delivers its bf16 elements.
//
// A row goes to S CTAs (one where there are rows enough), each over a
// contiguous part in rounds of its threads x 64 bytes, the next round's loads
// in flight.  With S > 1 the CTA that takes the row's last ticket merges the
// parts; no CTA waits on another.
//
// Top alternatives, K <= 32.  In a part's first round the K-th largest of the maxima of
// 64 groups of threads is a bound that K elements reach: only those at or above it go to
// a list in shared memory, about K + a few for values in no order, and later rounds append
// what exceeds it.  After 1, 2, 4 rounds and then every kCheck the threads meet; a list past
// K + kSlack entries is ranked (each entry counts the better ones) and cut to K, whose last
// is the bound from then on: a thread that appends costs its warp half a round.  Where the
// list overflowed meanwhile (many equal or rising values) the rounds since are read once
// more, each with a bound over the 256 threads' maxima by value and index, which at most
// (K - 1) * 32 + 1 elements of a round reach, whatever they are.
// The rare parts are rolled loops, in line: unrolled, the kernel had 78 KB of code; as
// function calls they made the compiler wait for the next round's loads at every call.
//
// Rows that a warp can hold (1024 elements) go to a kernel of their own, a warp each; many
// rows to CTAs of 128 or, of up to 8192 elements, 64 threads.
//
// Measured, bf16: 2048 rows of 152064 with 5 alternatives 121 us (5.1 TB/s; the bytes' floor
// 92), without any 103; 32 sequences of up to 5 rows of 128256 with 20 alternatives 18.5,
// without 9.7; 5 fp32 rows of 1000 3.5.  What is left of the alternatives is the appends (12
// and 4 us of those), the meetings and, in parts, the merge.  Alternatives: meeting in
// every round 1.5 times as long (rows of 152064), no cut before the end 22 us more, cuts at
// 2 K + 16 entries 3, the round's maximum over widened values 2.
#include <float.h>
#include <limits.h>
#include <math.h>

#include "common.cuh"

namespace specv {
namespace {

constexpr int kVecs = 4;          // 16-byte loads of a thread per round
constexpr int kSlack = 8;         // entries beyond K that cut the list to K
constexpr int kCheck = 4;         // most rounds between two looks at the list
constexpr int kMaxParts = 32;
constexpr float kFarBelow = -1000.f;  // 2^y is +0 there; keeps -inf out of products

template <typename T> constexpr int per_vec() { return 16 / (int)sizeof(T); }

// Larger value, or the same at a lower index.
__device__ __forceinline__ bool better(float v, int i, float bv, int bi) {
    return v > bv || (v == bv && i < bi);
}

// maximum that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

struct Stats {
    float m = -INFINITY, l = 0.f, a = 0.f;
    // sums rebased to maximum `to` >= m
    __device__ void rebase(float to, float c) {
        if (l != 0.f) {
            const float d = max_nan((m - to) * c, kFarBelow), s = fast_exp2(d);
            a = s * fmaf(l, d, a);
            l *= s;
        }
        m = to;
    }
};

// The sums of a warp's lanes, in every lane.
__device__ __forceinline__ Stats warp_total(Stats v, float c) {
    const float to = warp_max(v.m);
    if (v.m < to) v.rebase(to, c);
    v.m = to;
    v.l = warp_sum(v.l);
    v.a = warp_sum(v.a);
    return v;
}

template <typename T> __device__ __forceinline__ void widen(const uint4& r, float (&x)[per_vec<T>()]);
template <> __device__ __forceinline__ void widen<float>(const uint4& r, float (&x)[4]) {
    x[0] = __uint_as_float(r.x);
    x[1] = __uint_as_float(r.y);
    x[2] = __uint_as_float(r.z);
    x[3] = __uint_as_float(r.w);
}
template <> __device__ __forceinline__ void widen<__nv_bfloat16>(const uint4& r, float (&x)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// Largest element of N vectors.  (bf16: in pairs as they lie, so that the values need not be
// widened for it)
template <typename T, int N> __device__ __forceinline__ float max_of(const uint4 (&r)[N]) {
    auto two = [](uint32_t a, uint32_t b) {
        uint32_t m;
        if constexpr (sizeof(T) == 4) m = __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
        else asm("max.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
        return m;
    };
    uint32_t m = two(two(r[0].x, r[0].y), two(r[0].z, r[0].w));
#pragma unroll
    for (int u = 1; u < N; ++u) m = two(m, two(two(r[u].x, r[u].y), two(r[u].z, r[u].w)));
    return sizeof(T) == 4 ? __uint_as_float(m)
                          : fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
}

// Vectors v0 + u step of a row: elements v EPV - off .. of [0, V), -inf outside and for
// v >= end.  The vectors lie on the 16-byte grid of memory; one at a row's edge is read whole
// and then masked, but for the tensor's last, of which the tensor has `left` elements from
// the row's first on.
template <typename T, int N>
__device__ __forceinline__ void load_edge(uint4 (&r)[N], const T* row, int V, int64_t left, int off,
                                          int v0, int step, int end) {
    constexpr int EPV = per_vec<T>(), EPW = EPV / 4;
    constexpr uint32_t kNone = EPW == 1 ? 0xff800000u : 0xff80ff80u;  // -inf
#pragma unroll
    for (int u = 0; u < N; ++u) {
        const int v = v0 + u * step;
        const int64_t e = (int64_t)v * EPV - off;
        r[u] = make_uint4(kNone, kNone, kNone, kNone);
        if (v < end && e + EPV <= left) r[u] = __ldg(reinterpret_cast<const uint4*>(row + e));
    }
#pragma unroll
    for (int u = 0; u < N; ++u) {
        const int v = v0 + u * step;
        const int64_t e = (int64_t)v * EPV - off;
        if (v >= end || (e >= 0 && e + EPV <= V)) continue;
        uint32_t w[4] = {r[u].x, r[u].y, r[u].z, r[u].w};
        const bool last = e + EPV > left;  // nothing was read
#pragma unroll 1
        for (int i = 0; i < EPV; ++i) {
            const bool in = e + i >= 0 && e + i < V;
            if (in && !last) continue;
            uint32_t bits = EPW == 1 ? 0xff800000u : 0xff80u;
            if (in) {
                if constexpr (EPW == 1) bits = __float_as_uint(row[e + i]);
                else bits = __bfloat16_as_ushort(row[e + i]);
            }
            const uint32_t keep = EPW == 1 ? 0u : 0xffff0000u >> (16 * (i & 1));
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j == i / EPW) w[j] = (w[j] & keep) | bits << (EPW == 1 ? 0 : 16 * (i & 1));
        }
        r[u] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <int TH> struct Shared {
    // list entries: a round's second look leaves (K - 1) kVecs EPV + 1 at most, after K +
    // kSlack from before
    static constexpr int kCap = TH == 256 ? 2048 : 1056;
    float v[kCap];
    int i[kCap];
    alignas(16) float tv[TH];  // maxima of the groups or threads
    int ti[TH];
    float best_v[32];
    int best_i[32];
    float4 stats[TH / 32];
    float bound_v;
    int bound_i;
    int count, last;
};

// Ranks the first `count` entries of the list and leaves its K best, sorted, at
// the front (every thread calls it; the list is complete and visible).
template <int TH> __device__ __forceinline__ int cut(Shared<TH>& s, int count, int K) {
    const int tid = threadIdx.x;
#pragma unroll 1
    for (int e = tid; e < count; e += TH) {
        const float v = s.v[e];
        const int i = s.i[e];
        int rank = 0;
#pragma unroll 4
        for (int o = 0; o < count; ++o) rank += better(s.v[o], s.i[o], v, i);
        if (rank < K) {
            s.best_v[rank] = v;
            s.best_i[rank] = i;
        }
    }
    __syncthreads();
    const int kept = count < K ? count : K;
    if (tid < kept) {
        s.v[tid] = s.best_v[tid];
        s.i[tid] = s.best_i[tid];
    }
    if (tid == 0) s.count = kept;
    __syncthreads();
    return kept;
}

// Appends the elements of a thread's round (vectors cur, elements from `first` on) that
// exceed `above` (ABOVE), reach bv (REACH), or both, an equal of bv at index bx at the
// latest (BOTH).  Most calls find one element: a vector whose maximum is too small is not
// looked into.
enum { ABOVE, REACH, BOTH };
template <typename T, int HOW, int TH>
__device__ __forceinline__ void append(Shared<TH>& s, const uint4 (&cur)[kVecs], int first, float above,
                                       float bv, int bx) {
    constexpr int EPV = per_vec<T>(), EPW = EPV / 4;  // elements of a vector, of a word
    const float least = HOW == ABOVE ? above : bv;
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
        const uint4 one[1] = {cur[u]};
        const float vm = max_of<T>(one);
        if (HOW == ABOVE ? !(vm > least) : !(vm >= least)) continue;
        float e[EPV];
        widen<T>(cur[u], e);
        const int at = first + u * TH * EPV;
        uint32_t bits = 0;
#pragma unroll
        for (int j = 0; j < EPV; ++j)
            bits |= (uint32_t)(HOW == ABOVE   ? e[j] > above
                               : HOW == REACH ? e[j] >= bv
                                              : e[j] > above && !better(bv, bx, e[j], at + j))
                    << j;
#pragma unroll 1
        for (; bits; bits &= bits - 1) {
            const int j = __ffs(bits) - 1, q = j / EPW;
            const uint32_t w = q == 0 ? cur[u].x : q == 1 ? cur[u].y : q == 2 ? cur[u].z : cur[u].w;
            const int place = atomicAdd(&s.count, 1);
            if (place < s.kCap) {
                s.v[place] = __uint_as_float(EPW == 1 ? w : j & 1 ? w & 0xffff0000u : w << 16);
                s.i[place] = at + j;
            }
        }
    }
}

// Index of the first element of a thread's round that equals v.
template <typename T, int TH>
__device__ __forceinline__ int index_of(uint4 c0, uint4 c1, uint4 c2, uint4 c3, int first, float v) {
    constexpr int EPV = per_vec<T>(), EPW = EPV / 4;
#pragma unroll 1
    for (int e = 0; e < kVecs * EPV; ++e) {
        const int u = e / EPV, j = e % EPV / EPW, h = e % EPW;
        const uint4 r = u == 0 ? c0 : u == 1 ? c1 : u == 2 ? c2 : c3;
        const uint32_t w = j == 0 ? r.x : j == 1 ? r.y : j == 2 ? r.z : r.w;
        if (__uint_as_float(EPW == 1 ? w : h ? w & 0xffff0000u : w << 16) == v)
            return first + u * TH * EPV + e % EPV;
    }
    return INT_MAX;
}

// What is written for a row, by a warp: stats complete, the sorted alternatives in v, id.
// (fp32: on this GPU a 64-bit logarithm by every warp took longer than the row.)
__device__ __forceinline__ void write_row(const LogprobArgs& a, const float* v, const int* id,
                                          const Stats& st, int64_t row, float token, int found) {
    const int lane = threadIdx.x & 31;
    const bool none = st.l == 0.f;  // every logit is -inf
    const float lnl = logf(st.l);
    // z - lse = (x - m) / T - ln l, from the difference on
    auto lp = [&](float x) { return none ? -INFINITY : (x - st.m) * a.inv_t - lnl; };
    if (lane == 0) {
        a.logprob[row] = lp(token);
        if (a.entropy) a.entropy[row] = none ? 0.f : lnl - 0.69314718055994530942f * (st.a / st.l);
    }
    if (lane < a.K) {
        const bool have = lane < found;
        if (a.top_ids) a.top_ids[row * a.K + lane] = have ? id[lane] : -1;
        if (a.top_logprobs) a.top_logprobs[row * a.K + lane] = have ? lp(v[lane]) : -INFINITY;
    }
}

// The given token's logit (lane 0), -inf and a flag for one that is none.
template <typename T> __device__ __forceinline__ float token_logit(const LogprobArgs& a, const T* x, int tok) {
    if (tok >= 0 && tok < (int)a.V) return Elem<T>::to_f32(x[tok]);
    raise_device_error(a.dev_err, SPEC_DEVERR_TOKEN);
    return -INFINITY;
}

// Adds a vector's weights to the sums l2 and a2 (in halves), relative to m.
template <typename T>
__device__ __forceinline__ void add_weights(const uint4& r, float m, float c, uint64_t& l2, uint64_t& a2) {
    constexpr int EPV = per_vec<T>();
    const uint64_t neg = f2(-m, -m), cc = f2(c, c);
    float e[EPV];
    widen<T>(r, e);
#pragma unroll
    for (int j = 0; j < EPV; j += 2) {
        float y0, y1;
        f2_split(f2_mul(f2_add(f2(e[j], e[j + 1]), neg), cc), y0, y1);
        y0 = max_nan(y0, kFarBelow);
        y1 = max_nan(y1, kFarBelow);
        const uint64_t w = f2(fast_exp2(y0), fast_exp2(y1));
        l2 = f2_add(l2, w);
        a2 = f2_fma(w, f2(y0, y1), a2);
    }
}

// Short rows (kSmall elements, those before it in its first vector among them): a warp
// holds a row in registers.  The bound is the K-th largest of 64 maxima (each lane's first
// and second halves of its vectors); what reaches it goes to the warp's list by a running
// sum of the lanes' counts and is ranked there.  Against a CTA per row: 51480 rows of 466 with
// 32 alternatives 85 us, 2172; 32768 of 1000 with 5 57, 479, without 16, 425; 5 of them 4.0, 5.3.
constexpr int kSmall = 1024;
constexpr int kSmallWarps = 4;

template <typename T, bool TOP>
__global__ void __launch_bounds__(kSmallWarps * 32) logprob_small_kernel(const LogprobArgs a) {
    constexpr int EPV = per_vec<T>(), U = kSmall / 32 / EPV;
    __shared__ float s_list[TOP ? kSmallWarps : 1][TOP ? kSmall : 1];
    __shared__ int s_id[TOP ? kSmallWarps : 1][TOP ? kSmall : 1];
    __shared__ __align__(16) float s_max[kSmallWarps][64];
    __shared__ float s_best[kSmallWarps][33];  // and the bound
    __shared__ int s_best_id[kSmallWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, K = a.K;
    grid_dep_launch_dependents();
    grid_dep_wait();
    const int row = blockIdx.x * kSmallWarps + warp;
    if (row >= a.B * a.n) return;
    if (a.lens) {
        const int b = (uint32_t)row / (uint32_t)a.n;
        if (row - b * a.n >= __ldg(a.lens + b)) return;
    }
    const T* x = static_cast<const T*>(a.logits) + (int64_t)row * a.V;
    const int V = (int)a.V, off = (int)(((uint64_t)row * (uint64_t)a.V) % EPV);
    const int64_t left = ((int64_t)a.B * a.n - row) * a.V;
    const int vecs = (V + off + EPV - 1) / EPV;
    const int tok = lane == 0 ? __ldg(a.tokens + row) : 0;
    uint4 r[U];
    load_edge<T>(r, x, V, left, off, lane, 32, vecs);
    const float token = lane == 0 ? token_logit<T>(a, x, tok) : 0.f;
    Stats st;
    st.m = warp_max(max_of<T>(r));
    uint64_t l2 = f2(0.f, 0.f), a2 = l2;
#pragma unroll
    for (int u = 0; u < U; ++u) add_weights<T>(r[u], st.m == -INFINITY ? 0.f : st.m, a.c, l2, a2);
    float p, q;
    f2_split(l2, p, q);
    st.l = warp_sum(p + q);
    f2_split(a2, p, q);
    st.a = warp_sum(p + q);
    int found = 0;
    if constexpr (TOP) {
        float* list = s_list[warp];
        int* id = s_id[warp];
        float* most = s_max[warp];
        float half[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float e[EPV];
            widen<T>(r[u], e);
#pragma unroll
            for (int j = 0; j < EPV; ++j) half[j * 2 / EPV] = fmaxf(half[j * 2 / EPV], e[j]);
        }
        most[lane] = half[0];
        most[32 + lane] = half[1];
        if (lane == 0) s_best[warp][32] = -INFINITY;
        __syncwarp();
        int rank[2] = {0, 0};
#pragma unroll 4
        for (int o = 0; o < 64; ++o) {
            const float w = most[o];
            rank[0] += better(w, o, half[0], lane);
            rank[1] += better(w, o, half[1], 32 + lane);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (rank[h] == K - 1) s_best[warp][32] = half[h];
        __syncwarp();
        const float bound = fmaxf(s_best[warp][32], -FLT_MAX);  // (-inf is no alternative)
        int mine = 0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float e[EPV];
            widen<T>(r[u], e);
#pragma unroll
            for (int j = 0; j < EPV; ++j) mine += e[j] >= bound;
        }
        int at = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int w = __shfl_up_sync(0xffffffffu, at, o);
            if (lane >= o) at += w;
        }
        int n = __shfl_sync(0xffffffffu, at, 31);
        at -= mine;
        if (n <= 128) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float e[EPV];
                widen<T>(r[u], e);
#pragma unroll
                for (int j = 0; j < EPV; ++j)
                    if (e[j] >= bound) {
                        list[at] = e[j];
                        id[at++] = (u * 32 + lane) * EPV - off + j;
                    }
            }
        } else {
            // many equal values: of those at the bound the K of lowest index will do.  The
            // vectors in turn, so that running counts are in the order of the indexes; what
            // lies above the bound is (K - 1) * 16 elements at most.
            int equal = 0;
            n = 0;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float e[EPV];
                widen<T>(r[u], e);
                int counts = 0;
#pragma unroll
                for (int j = 0; j < EPV; ++j) counts += e[j] > bound ? 1 : e[j] == bound ? 1 << 16 : 0;
                int upto = counts;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int w = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += w;
                }
                int above = n + ((upto - counts) & 0xffff), level = equal + ((upto - counts) >> 16);
#pragma unroll
                for (int j = 0; j < EPV; ++j) {
                    const int i = (u * 32 + lane) * EPV - off + j;
                    if (e[j] > bound) {
                        list[above] = e[j];
                        id[above++] = i;
                    } else if (e[j] == bound) {
                        if (level < K) s_best_id[warp][level] = i;
                        ++level;
                    }
                }
                const int total = __shfl_sync(0xffffffffu, upto, 31);
                n += total & 0xffff;
                equal += total >> 16;
            }
            __syncwarp();
            equal = min(equal, K);
            if (lane < equal) {
                list[n + lane] = bound;
                id[n + lane] = s_best_id[warp][lane];
            }
            n += equal;
        }
        __syncwarp();
#pragma unroll 1
        for (int e = lane; e < n; e += 32) {
            const float v = list[e];
            const int i = id[e];
            int place = 0;
#pragma unroll 4
            for (int o = 0; o < n; ++o) place += better(list[o], id[o], v, i);
            if (place < K) {
                s_best[warp][place] = v;
                s_best_id[warp][place] = i;
            }
        }
        __syncwarp();
        found = min(n, K);
    }
    write_row(a, s_best[warp], s_best_id[warp], st, row, token, found);
}

// The K-th largest of the maxima of 64 groups of threads (bm: a thread's), which K
// elements reach; -inf if there are fewer.
template <int TH> __device__ __forceinline__ float bound_of_groups(Shared<TH>& s, float bm, int K) {
    const int tid = threadIdx.x;
    constexpr int EACH = TH / 64;  // threads of a group
    float g = bm;
#pragma unroll
    for (int o = 1; o < EACH; o <<= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
    if (tid % EACH == 0) s.tv[tid / EACH] = g;
    __syncthreads();
    if (tid < 64) {
        const float mine = s.tv[tid];
        int rank = 0;
#pragma unroll 4
        for (int o = 0; o < 64; o += 4) {
            const float4 q = *reinterpret_cast<const float4*>(&s.tv[o]);
            rank += (q.x > mine || (q.x == mine && o < tid)) + (q.y > mine || (q.y == mine && o + 1 < tid)) +
                    (q.z > mine || (q.z == mine && o + 2 < tid)) +
                    (q.w > mine || (q.w == mine && o + 3 < tid));
        }
        if (rank == K - 1) s.bound_v = mine;
    }
    __syncthreads();
    return s.bound_v;
}

template <typename T, bool TOP, int CTAS, int TH>
__global__ void __launch_bounds__(TH, CTAS) logprob_kernel(const LogprobArgs a) {
    constexpr int EPV = per_vec<T>();
    __shared__ Shared<TH> s;
    const int tid = threadIdx.x, S = a.parts, K = a.K;
    const int row = blockIdx.x / (uint32_t)S, part = blockIdx.x - row * S;
    if (tid == 0) {
        s.count = 0;
        s.bound_v = -INFINITY;
    }
    grid_dep_launch_dependents();
    grid_dep_wait();
    if (a.lens) {
        const int b = (uint32_t)row / (uint32_t)a.n;
        if (row - b * a.n >= __ldg(a.lens + b)) return;
    }

    const T* x = static_cast<const T*>(a.logits) + (int64_t)row * a.V;
    // vectors of 16 bytes on memory's grid (indexes inside a row are 32-bit)
    const int V = (int)a.V, off = (int)(((uint64_t)row * (uint64_t)a.V) % EPV);
    const int64_t left = ((int64_t)a.B * a.n - row) * a.V;
    constexpr int kRound = kVecs * TH;
    const int vecs = (int)(((int64_t)V + off + EPV - 1) / EPV);
    const int per = S == 1 ? vecs : a.part_rounds * kRound;
    const int v0 = part * per, v1 = part == S - 1 ? vecs : v0 + per;
    const float c = a.c;
    uint64_t l2 = f2(0.f, 0.f), a2 = l2;
    float m = -INFINITY;
    // what an element has to exceed: K elements of the rounds before reach it
    float tau = -INFINITY;
    int checked = v0;  // first vector of the rounds since the list was looked at

    uint4 cur[kVecs], nxt[kVecs];
    // (of a round that lies whole inside the row no vector is looked at singly)
    auto fetch = [&](uint4 (&r)[kVecs], int v) {
        if (v + kVecs * TH <= v1 && (v > 0 || off == 0) && (int64_t)(v + kVecs * TH) * EPV - off <= V) {
            const uint4* p = reinterpret_cast<const uint4*>(x - off) + v + tid;
#pragma unroll
            for (int u = 0; u < kVecs; ++u)
                asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(r[u].x), "=r"(r[u].y), "=r"(r[u].z), "=r"(r[u].w)
                             : "l"(p + u * TH));
        } else {
            load_edge<T>(r, x, V, left, off, v + tid, TH, v1);
        }
    };
    // the given token and, once it is known, its logit (thread 0)
    const int tok = tid == 0 ? __ldg(a.tokens + row) : 0;
    float token = -INFINITY;
    fetch(cur, v0);
#pragma unroll 1
    for (int v = v0; v < v1; v += kVecs * TH) {
        if (v + kVecs * TH < v1) fetch(nxt, v + kVecs * TH);
        const float bm = max_of<T>(cur);
        if (bm > m) {
            float p, q;
            Stats old;
            old.m = m;
            f2_split(l2, p, q);
            old.l = p + q;
            f2_split(a2, p, q);
            old.a = p + q;
            old.rebase(bm, c);
            m = bm;
            l2 = f2(old.l, 0.f);
            a2 = f2(old.a, 0.f);
        }
#pragma unroll
        for (int u = 0; u < kVecs; ++u) add_weights<T>(cur[u], m == -INFINITY ? 0.f : m, c, l2, a2);
        if (v == v0 && tid == 0) token = token_logit<T>(a, x, tok);
        if (TOP) {
            const int at = (v + tid) * EPV - off;
            if (v == v0) {
                const float bv = bound_of_groups(s, bm, K);
                // (-inf is no alternative)
                if (bm >= bv) append<T, REACH>(s, cur, at, -INFINITY, fmaxf(bv, -FLT_MAX), INT_MAX);
                tau = bv;
            } else if (bm > tau) {
                append<T, ABOVE>(s, cur, at, tau, -INFINITY, INT_MAX);
            }
            const bool end = v + kRound >= v1;
            if (end || v == v0 || v + kRound - checked >= min(kCheck * kRound, checked - v0)) {
                __syncthreads();
                int count = s.count;
                if (count > s.kCap) {
                    // entries from before (at most K + kSlack) stand in front
                    const int before =
                        v == v0 ? 0 : __syncthreads_count(tid < K + kSlack && s.i[tid] < checked * EPV - off);
                    if (v == v0) tau = -INFINITY;
                    __syncthreads();
                    if (tid == 0) s.count = before;
#pragma unroll 1
                    for (int w = checked; w <= v; w += kRound) {
                        fetch(cur, w);
                        const int first = (w + tid) * EPV - off;
                        const float top = max_of<T>(cur);
                        const int bi = index_of<T, TH>(cur[0], cur[1], cur[2], cur[3], first, top);
                        s.tv[tid] = top;
                        s.ti[tid] = bi;
                        if (tid == 0) {
                            s.bound_v = -INFINITY;
                            s.bound_i = INT_MAX;
                        }
                        __syncthreads();
                        int rank = 0;
#pragma unroll 1
                        for (int o = 0; o < TH; ++o) rank += better(s.tv[o], s.ti[o], top, bi);
                        if (rank == K - 1 && top > -INFINITY) {
                            s.bound_v = top;
                            s.bound_i = bi;
                        }
                        __syncthreads();
                        append<T, BOTH>(s, cur, first, tau, s.bound_v, s.bound_i);
                        __syncthreads();
                        count = s.count;
                        cut(s, count, K);
                        if (count >= K) tau = s.v[K - 1];
                        __syncthreads();
                    }
                } else if (count > K + kSlack && !end) {
                    cut(s, count, K);
                    tau = s.v[K - 1];
                    __syncthreads();  // before the next round appends
                } else if (!end) {
                    // every thread has read the count before the next round appends: else a
                    // slower warp could read another one and take another branch, and its
                    // barriers, than the rest
                    __syncthreads();
                }
                checked = v + kRound;
            }
        }
#pragma unroll
        for (int u = 0; u < kVecs; ++u) cur[u] = nxt[u];
    }
    Stats st;
    st.m = m;
    {
        float p, q;
        f2_split(l2, p, q);
        st.l = p + q;
        f2_split(a2, p, q);
        st.a = p + q;
    }
    // the CTA's sums
    st = warp_total(st, c);
    if ((tid & 31) == 0) s.stats[tid >> 5] = make_float4(st.m, st.l, st.a, 0.f);
    __syncthreads();
    // sums in `from` of n parts (a warp: all that is needed further on)
    auto gather = [&](const float4* from, int n) {
        Stats sum;
        if ((tid & 31) < n) {
            const float4 r = __ldcg(from + (tid & 31));
            sum.m = r.x;
            sum.l = r.y;
            sum.a = r.z;
        }
        return warp_total(sum, c);
    };
    if (tid < 32) {
        const float4 r = tid < TH / 32 ? s.stats[tid] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
        st.m = r.x;
        st.l = r.y;
        st.a = r.z;
        st = warp_total(st, c);
    }
    int found = 0;
    if (TOP) found = cut(s, s.count, K);
    if (TH == 256 && S > 1) {
        // ---- parts: leave this one's record; the last CTA of the row merges them
        const int64_t rec = (int64_t)row * S + part;
        if (TOP && tid < K) {
            a.part_v[rec * K + tid] = tid < found ? s.v[tid] : -INFINITY;
            a.part_i[rec * K + tid] = tid < found ? s.i[tid] : -1;
        }
        if (tid == 0) reinterpret_cast<float4*>(a.part_stats)[rec] = make_float4(st.m, st.l, st.a, 0.f);
        __threadfence();
        __syncthreads();
        if (tid == 0) {
            s.last = atomicAdd(&a.tickets[row], 1) == S - 1;
            s.count = 0;
        }
        __syncthreads();
        if (!s.last) return;
        __threadfence();
        if (tid == 0) a.tickets[row] = 0;
        // the parts' alternatives, up to four a thread, through a bound of their own
        constexpr int kMine = kMaxParts * 32 / TH;
        float w[kMine], bm = -INFINITY;
        int id[kMine];
        if (TOP) {
#pragma unroll
            for (int u = 0; u < kMine; ++u) {
                const int e = u * TH + tid;
                w[u] = -INFINITY;
                if (e < S * K) {
                    w[u] = __ldcg(a.part_v + (int64_t)row * S * K + e);
                    id[u] = __ldcg(a.part_i + (int64_t)row * S * K + e);
                }
                bm = fmaxf(bm, w[u]);
            }
        }
        if (tid < 32) st = gather(reinterpret_cast<const float4*>(a.part_stats) + (int64_t)row * S, S);
        if (TOP) {
            if (tid == 0) s.bound_v = -INFINITY;
            const float bv = bound_of_groups(s, bm, K);
#pragma unroll
            for (int u = 0; u < kMine; ++u)
                if (w[u] >= bv && w[u] > -INFINITY) {
                    const int place = atomicAdd(&s.count, 1);
                    s.v[place] = w[u];
                    s.i[place] = id[u];
                }
            __syncthreads();
            found = cut(s, s.count, K);
        }
    }
    if (tid < 32) write_row(a, s.v, s.i, st, row, token, found);
}

}  // namespace

static bool small_rows(const LogprobArgs& a) {
    return a.V <= kSmall - (a.dtype == SPEC_DTYPE_F32 ? 3 : 7);
}

// Rounds that a row takes at least (one more where it begins inside a vector).
static int64_t rounds_of(const LogprobArgs& a) {
    const int64_t round = 256 * kVecs * (a.dtype == SPEC_DTYPE_F32 ? 4 : 8);
    return (a.V + round - 1) / round;
}

// Parts of a row: four CTAs an SM where the rows alone are fewer, each of whole rounds and
// as many as the others but for the last.
int logprob_parts(const LogprobArgs& a, int num_sms, int max_tickets) {
    const int64_t rows = (int64_t)a.B * a.n, most = rounds_of(a);
    const int64_t want = (4 * (int64_t)num_sms + rows - 1) / rows;
    if (rows > max_tickets) return 1;
    int64_t s = want < most ? want : most;
    if (s > kMaxParts) s = kMaxParts;
    const int64_t rounds = (most + s - 1) / s;
    return (int)((most + rounds - 1) / rounds);
}

size_t logprob_workspace_bytes(const LogprobArgs& a) {
    return a.parts > 1 ? (size_t)a.B * a.n * a.parts * (16 + 8 * (size_t)a.K) : 0;
}

cudaError_t launch_logprobs(LogprobArgs a, int num_sms, void* workspace, cudaStream_t stream) {
    const int64_t rows = (int64_t)a.B * a.n;
    if (small_rows(a)) {
        auto* kern = a.dtype == SPEC_DTYPE_F32 ? (a.K ? logprob_small_kernel<float, true>
                                                      : logprob_small_kernel<float, false>)
                     : a.K                     ? logprob_small_kernel<__nv_bfloat16, true>
                                               : logprob_small_kernel<__nv_bfloat16, false>;
        return launch_dependent(kern, dim3((unsigned)((rows + kSmallWarps - 1) / kSmallWarps)),
                                dim3(kSmallWarps * 32), 0, stream, a);
    }
    // Smaller CTAs, more of an SM, where rows are many (eight an SM): a row's start and end hide
    // behind more others, and fewer warps meet.  64 threads / 256, on 152 SMs: 32768 rows of
    // 1500, 4000 with 20 alternatives 113, 181 us / 277, 293; 8192 of 8000 75 / 85, 2048 26 / 23.
    // 128 / 256: 8192 rows of 32000 with 0, 5, 20 80, 130, 175 / 91, 153, 198; 2048 rows of
    // 152064 106, 121, 144 / 102, 124, 149; 1200 58, 74, 88 / 58, 75, 90; 700 55, 71, 84 / 47,
    // 55, 66.
    const int threads = a.parts > 1 || rows < 8 * (int64_t)num_sms     ? 256
                        : a.V <= 4096 || (a.V <= 8192 && rows >= 4096) ? 64
                                                                       : 128;
    // (parts - 1) part_rounds < rounds_of(a): no part is empty
    a.part_rounds = (int)((rounds_of(a) + a.parts - 1) / a.parts);
    a.part_stats = static_cast<float*>(workspace);
    a.part_v = a.part_stats + rows * a.parts * 4;
    a.part_i = reinterpret_cast<int32_t*>(a.part_v + rows * a.parts * a.K);
    const dim3 grid((unsigned)(rows * a.parts)), block(threads);
    // CTAs of an SM: 1024 threads of 64 registers hide more of the loads.  Rows in parts
    // with alternatives are faster with three CTAs of 256: fewer of the given rows may be in
    // use, and four of those on one SM are what the others wait for.  2048 rows of 152064, 5
    // alternatives, 256 threads: 132 us with four, 143 with three; 32 x up to 5 rows of 128256,
    // 20 alternatives: 23.2, 20.4.
    const bool f32 = a.dtype == SPEC_DTYPE_F32, three = a.K && !f32 && a.parts > 1;
    using B16 = __nv_bfloat16;
    auto* kern =
        threads == 64    ? (f32 ? (a.K ? logprob_kernel<float, true, 16, 64> : logprob_kernel<float, false, 16, 64>)
                                : (a.K ? logprob_kernel<B16, true, 16, 64> : logprob_kernel<B16, false, 16, 64>))
        : threads == 128 ? (f32 ? (a.K ? logprob_kernel<float, true, 8, 128> : logprob_kernel<float, false, 8, 128>)
                                : (a.K ? logprob_kernel<B16, true, 8, 128> : logprob_kernel<B16, false, 8, 128>))
        : f32            ? (a.K ? logprob_kernel<float, true, 4, 256> : logprob_kernel<float, false, 4, 256>)
        : three          ? logprob_kernel<B16, true, 3, 256>
        : a.K            ? logprob_kernel<B16, true, 4, 256>
                         : logprob_kernel<B16, false, 4, 256>;
    return launch_dependent(kern, grid, block, 0, stream, a);
}

}  // namespace specv
